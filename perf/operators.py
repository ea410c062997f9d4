"""The expert-grouped QLoRA linear, its backward, and adapter dropout, as cases to measure.

Notation: E experts, each an NF4 weight W_e [N, K] with adapters A_e [K, r] and B_e [r, N]; T token rows sorted by expert,
expert e's being offsets[e] .. offsets[e+1] - 1; s = alpha / r; D the dropout with keep probability 1 - p, whose mask is a
function of (seed, offset, element) and is never stored.

  forward   Y_e  = X_e W'_e^T + s (D(X_e) A_e) B_e          (XA = D(X) A is saved for the backward)
  backward  G_e  = s dY_e B_e^T
            dX_e = dY_e W'_e + D'(G_e A_e^T)                 (D' : the same mask and factor)
            dA_e = D(X_e)^T G_e,   dB_e = s XA_e^T dY_e

W'_e is the 16-bit weight that the framework's dequantization gives: round16(level[code] * t8[q] * S). One expert with no
offsets is the dense linear. The packed codes, constants and scales of the experts lie one after another, as one weight
[E N, K] quantized in one call has them.
"""
import math

import numpy as np
import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


# ------------------------------------------------------------------ cases --
def listed():
    def case(name, op, E, T, N, K, r, p=0.0, dtype="bf16", pad=0, skew=0.5):
        return dict(name=name, op=op, E=E, T=T, N=N, K=K, r=r, p=p, dtype=dtype, pad=pad, skew=skew)

    return [
        # decoding one token that is routed to two of eight small experts: nothing but latency
        case("fwd-2rows-1024", "fwd", 8, 2, 1024, 1024, 8),
        # decoding a batch of 16 sequences, two experts each, through the gate of a 7B-shaped expert
        case("fwd-decode-7b-gate", "fwd", 8, 32, 11008, 4096, 64),
        # a prefill of odd length in fp16 over uneven experts, with padding rows behind the last one
        case("fwd-ragged-f16", "fwd", 12, 777, 4096, 4096, 16, dtype="f16", pad=55, skew=1.0),
        # a training step's forward with adapter dropout
        case("fwd-train-7b-gate", "fwd", 8, 8192, 11008, 4096, 64, p=0.05),
        # the smallest backward
        case("bwd-33rows-1024", "bwd", 4, 33, 1024, 1024, 8),
        # backward of the ragged prefill
        case("bwd-ragged-f16", "bwd", 12, 777, 4096, 4096, 16, dtype="f16", pad=55, skew=1.0),
        # a training step's backward through the down projection, with adapter dropout
        case("bwd-train-7b-down", "bwd", 8, 8192, 4096, 11008, 64, p=0.05),
        # the dense linear of the 7B set with adapter dropout, both directions
        case("fwd-dense-dropout-7b-q", "fwd", 1, 2048, 4096, 4096, 64, p=0.1),
        case("bwd-dense-dropout-7b-gate", "bwd", 1, 2048, 11008, 4096, 64, p=0.1),
        # dropout of a tensor by itself: the 16 tokens of the single linear, and a 7B set's tokens in and out of the ffn
        case("dropout-16x1024", "dropout", 1, 16, 0, 1024, 0, p=0.05),
        case("dropout-2047x4099-f32", "dropout", 1, 2047, 0, 4099, 0, p=0.5, dtype="f32"),
        case("dropout-8192x11008", "dropout", 1, 8192, 0, 11008, 0, p=0.1),
    ]


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["fwd", "fwd", "bwd", "bwd", "dropout"])
    dtype = rng.choice(["bf16", "bf16", "f16"])
    if op == "dropout":
        return dict(op=op, E=1, T=log(1, 8192), N=0, K=log(64, 11008), r=0, p=rng.choice([0.05, 0.1, 0.25, 0.5]),
                    dtype=rng.choice(["bf16", "f16", "f32"]), pad=0, skew=0.0)
    N, K = 64 * log(4, 172), 64 * log(4, 172)
    E = log(1, 32)
    while E > 1 and E * N * K > 8 * 11008 * 4096:
        E -= 1
    T = log(1, 8192)
    while T > 1 and T * N * K > 8192 * 11008 * 4096:
        T //= 2
    pad = rng.choice([0, 0, rng.randrange(1, 100)]) if E > 1 else 0
    return dict(op=op, E=E, T=T, N=N, K=K, r=rng.choice([8, 16, 24, 32, 64, 64, 128]), p=rng.choice([0.0, 0.05, 0.1, 0.5]),
                dtype=dtype, pad=pad, skew=rng.choice([0.0, 0.5, 1.0]))


def work(case):
    T, N, K, r, E = case["T"], case["N"], case["K"], case["r"], case["E"]
    size = 4 if case["dtype"] == "f32" else 2
    if case["op"] == "dropout":
        return {"bytes": 2 * size * T * K, "flops": T * K}
    hit = E * (1.0 - (1.0 - 1.0 / E) ** T) if E > 1 else 1.0  # experts that have a token, for even routing
    weight = hit * (N * K * (0.5 + 1.0 / 64) + N * K / 4096.0 + 2 * r * (N + K))
    if case["op"] == "fwd":
        return {"bytes": weight + 2 * T * (N + K + r), "flops": 2.0 * T * N * K + 2.0 * T * r * (N + K)}
    return {"bytes": weight + 2 * T * (N + 2 * K + r) + 2 * E * r * (N + K), "flops": 2.0 * T * N * K + 6.0 * T * r * (N + K)}


# ----------------------------------------------------------------- inputs --
def _levels():
    """The 16 NF4 levels and the 256 levels of the 8-bit constants, in fp32."""
    delta = 0.5 * ((1 - 1 / 30) + (1 - 1 / 32))
    quant = torch.special.ndtri(torch.cat([torch.linspace(delta, 0.5, 9, dtype=torch.float64)[:-1],
                                           torch.linspace(delta, 0.5, 8, dtype=torch.float64)[:-1]]))
    pos, neg = quant[:8], -quant[8:]
    nf4 = torch.cat([neg, torch.zeros(1, dtype=torch.float64), pos.flip(0)]) / quant[0]
    return nf4.float().numpy(), (torch.arange(256, dtype=torch.float64) / 255).float().numpy()


def prepare(case, seed):
    T, N, K, r, E, p = case["T"], case["N"], case["K"], case["r"], case["E"], case["p"]
    dt, dev = TYPES[case["dtype"]], "cuda"
    g = torch.Generator(device=dev).manual_seed(seed * 7919 + 17)
    hg = torch.Generator().manual_seed(seed * 104729 + 3)
    rnd = lambda *shape, std=1.0: (torch.randn(*shape, device=dev, generator=g) * std).to(dt)  # noqa: E731
    st = dict(case)
    st["seed"], st["offset"] = (seed * 0x9E3779B97F4A7C15 + 12345) % 2**64, (seed * 1000003) % 2**40
    if case["op"] == "dropout":
        st["X"], st["Y"] = rnd(T, K), torch.empty(T, K, dtype=dt, device=dev)
        return st
    rows = T + case["pad"]
    # token rows of each expert: a router's counts, uneven by `skew`
    prob = torch.softmax(torch.randn(E, generator=hg) * case["skew"], 0)
    counts = torch.bincount(torch.multinomial(prob, T, replacement=True, generator=hg), minlength=E)
    offsets = torch.zeros(E + 1, dtype=torch.int32)
    offsets[1:] = counts.cumsum(0)
    st["offsets"], st["largest"] = offsets.to(dev), int(counts.max())
    # codes of normal weights are spread evenly over the levels by construction; the block constants are maxima of 64
    # normals of deviation 0.02, the second-level scale the largest of 256 of them
    st["packed"] = torch.randint(0, 256, (E * N * K // 2,), dtype=torch.uint8, device=dev, generator=g)
    nb = E * N * K // 64
    ng = -(-nb // 256)
    absmax = (0.02 * (2.4 + 0.42 * torch.randn(nb, device=dev, generator=g))).clamp_(0.02, 0.1)
    st["scale2"] = torch.nn.functional.pad(absmax, (0, ng * 256 - nb)).view(ng, 256).amax(1)
    st["q"] = (absmax / st["scale2"].repeat_interleave(256)[:nb] * 255).round_().to(torch.uint8)
    st["X"], st["A"], st["B"] = rnd(rows, K), rnd(E, K, r, std=0.01), rnd(E, r, N, std=0.01)
    st["alpha"] = 16.0
    st["levels"] = [torch.from_numpy(t).to(dev) for t in _levels()]
    # buffers that a program keeps: rows that no expert owns stay as they are
    if case["op"] == "fwd":
        st["Y"] = torch.zeros(rows, N, dtype=dt, device=dev)
        st["XA"] = torch.zeros(rows, r, dtype=dt, device=dev)
    else:
        st["dY"], st["XA"] = rnd(rows, N), rnd(rows, r, std=0.01 * math.sqrt(K))
        st["dX"] = torch.zeros(rows, K, dtype=dt, device=dev)
        st["dA"], st["dB"] = torch.empty_like(st["A"]), torch.empty_like(st["B"])
    return st


# ------------------------------------------------------------- plain form --
def _keep(n, p, seed, offset, dev):
    """Keep mask of n elements: Philox4x32-10 (Salmon et al., SC'11) of counter offset + i // 8 under key `seed` gives four
    words; element i takes 16-bit half i % 8 of them, low halves first, and is kept where that is at least p 2^16."""
    low = 0xFFFFFFFF
    ctr = torch.arange(-(-n // 8), dtype=torch.int64, device=dev) + offset
    c0, c1, c2, c3 = ctr & low, (ctr >> 32) & low, torch.zeros_like(ctr), torch.zeros_like(ctr)
    k0, k1 = seed & low, (seed >> 32) & low
    for _ in range(10):
        a, b = c0 * 0xD2511F53, c2 * 0xCD9E8D57  # 64-bit products; the high words by an arithmetic shift and a mask
        c0, c1, c2, c3 = ((b >> 32) & low) ^ c1 ^ k0, b & low, ((a >> 32) & low) ^ c3 ^ k1, a & low
        k0, k1 = (k0 + 0x9E3779B9) & low, (k1 + 0xBB67AE85) & low
    words = torch.stack([c0, c1, c2, c3], 1)
    halves = torch.stack([words & 0xFFFF, words >> 16], 2).view(-1)[:n]
    return halves >= int(math.floor(p * 65536 + 0.5))


def _factor(p):
    return 65536.0 / (65536.0 - math.floor(p * 65536 + 0.5))


def _dropped(st, x):
    """D(x) in fp32."""
    x = x.float()
    if st["p"] == 0.0:
        return x
    keep = _keep(x.numel(), st["p"], st["seed"], st["offset"], x.device).view_as(x)
    return torch.where(keep, x * _factor(st["p"]), 0.0)


def _weights(st):
    """W' [E, N, K] in fp32, its values rounded to the 16-bit type."""
    nf4, t8 = st["levels"]
    codes = torch.stack([st["packed"] & 15, st["packed"] >> 4], 1).view(-1, 64)
    scale = t8[st["q"].int()] * st["scale2"].repeat_interleave(256)[: st["q"].numel()]
    w = nf4[codes.int()] * scale[:, None]
    return w.to(TYPES[st["dtype"]]).float().view(st["E"], st["N"], st["K"])


def _plain(st):
    if st["op"] == "dropout":
        return _dropped(st, st["X"]).to(TYPES[st["dtype"]])
    dt, s = TYPES[st["dtype"]], st["alpha"] / st["r"]
    rows = st["X"].shape[0]
    off = st["offsets"].long()
    # every expert's rows, padded to the largest expert's count; padding takes and gives the extra row behind the last
    at = off[:-1, None] + torch.arange(st["largest"], device=off.device)
    at = torch.where(at < off[1:, None], at, rows)

    def take(x):  # [rows, c] -> [E, largest, c]
        return torch.cat([x.float(), x.new_zeros(1, x.shape[1], dtype=torch.float32)])[at]

    def give(y):  # [E, largest, c] -> [rows, c]
        out = y.new_zeros(rows + 1, y.shape[2])
        out[at.view(-1)] = y.view(-1, y.shape[2])
        return out[:rows].to(dt)

    A, B, W = st["A"].float(), st["B"].float(), _weights(st)
    if st["op"] == "fwd":
        xa = take(_dropped(st, st["X"])) @ A
        return {"Y": give(take(st["X"]) @ W.mT + s * (xa @ B)), "XA": give(xa)}
    dy = take(st["dY"])
    G = s * (dy @ B.mT)
    low = G @ A.mT
    if st["p"] > 0.0:
        keep = _keep(st["X"].numel(), st["p"], st["seed"], st["offset"], off.device).view_as(st["X"])
        low = low * take(keep) * _factor(st["p"])
    return {"dX": give(dy @ W + low), "dA": (take(_dropped(st, st["X"])).mT @ G).to(dt),
            "dB": (s * (take(st["XA"]).mT @ dy)).to(dt)}


def _own(st):
    from bit_quantized_lora_blockwise_b200 import binding

    drop = binding.Dropout(st["p"], st["seed"], st["offset"]) if st["p"] > 0.0 else None
    if st["op"] == "dropout":
        return binding.dropout(st["X"], drop, out=st["Y"])
    N, K, dense = st["N"], st["K"], st["E"] == 1 and st["pad"] == 0
    weight = (st["packed"], st["q"], st["scale2"])
    if "workspace" not in st:  # kept from the first pass on, as a training or decoding loop keeps it
        need = binding.grouped_workspace_bytes(st["E"], st["X"].shape[0], N, K, st["r"], drop is not None)
        st["workspace"] = torch.empty(need, dtype=torch.uint8, device="cuda")
    ws = st["workspace"]
    if st["op"] == "fwd":
        if dense:
            Y = binding.linear_fwd(*weight, st["X"], st["A"][0], st["B"][0], st["alpha"], N, K, Y=st["Y"], XA_out=st["XA"],
                                   workspace=ws, dropout=drop)
        else:
            Y = binding.grouped_linear_fwd(*weight, st["X"], st["offsets"], st["A"], st["B"], st["alpha"], N, K, Y=st["Y"],
                                           XA_out=st["XA"], workspace=ws, dropout=drop)
        return {"Y": Y, "XA": st["XA"]}
    if dense:
        dX, _, _ = binding.linear_bwd(*weight, st["X"], st["dY"], st["A"][0], st["B"][0], st["alpha"], N, K, XA=st["XA"],
                                      dX=st["dX"], dA=st["dA"][0], dB=st["dB"][0], workspace=ws, dropout=drop)
    else:
        dX, _, _ = binding.grouped_linear_bwd(*weight, st["X"], st["dY"], st["offsets"], st["A"], st["B"], st["alpha"], N, K,
                                              XA=st["XA"], dX=st["dX"], dA=st["dA"], dB=st["dB"], workspace=ws, dropout=drop)
    return {"dX": dX, "dA": st["dA"], "dB": st["dB"]}


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------- 64-bit reference --
def exact(case, seed):
    st = prepare(case, seed)
    T, N, K, E, r, p = st["X"].shape[0], st["N"], st["K"], st["E"], st["r"], st["p"]
    cut = int(p * 65536 + 0.5)
    D = st["X"].double()
    mask = None
    if cut:
        n = T * K
        with np.errstate(over="ignore"):
            counter = np.arange((n + 7) // 8, dtype=np.uint64) + np.uint64(st["offset"])
            v = [counter & np.uint64(0xFFFFFFFF), counter >> np.uint64(32)] + [np.zeros_like(counter)] * 2
            key = [st["seed"] % 2**32, st["seed"] // 2**32]
            for _ in range(10):
                m0, m1 = v[0] * np.uint64(0xD2511F53), v[2] * np.uint64(0xCD9E8D57)
                v = [(m1 >> np.uint64(32)) ^ v[1] ^ np.uint64(key[0]), m1 & np.uint64(0xFFFFFFFF),
                     (m0 >> np.uint64(32)) ^ v[3] ^ np.uint64(key[1]), m0 & np.uint64(0xFFFFFFFF)]
                key = [(key[0] + 0x9E3779B9) % 2**32, (key[1] + 0xBB67AE85) % 2**32]
        bits = np.stack(v, 1).astype("<u4").view("<u2").reshape(-1)[:n].reshape(T, K)
        mask = torch.from_numpy((bits >= cut).astype(np.float64) * 65536 / (65536 - cut)).cuda()
        D = D * mask
    if st["op"] == "dropout":
        return D
    nf4, t8 = (t.cpu().numpy() for t in st["levels"])
    s, ends = st["alpha"] / r, st["offsets"].tolist()
    A, B, X = st["A"].double(), st["B"].double(), st["X"].double()
    pair = torch.from_numpy(np.stack([nf4[np.arange(256) % 16], nf4[np.arange(256) // 16]], 1)).cuda()
    const = torch.from_numpy(t8).cuda()

    def weight(e):
        blocks = torch.arange(e * N * K // 64, (e + 1) * N * K // 64, device="cuda")
        c = const[st["q"][blocks].long()] * st["scale2"][blocks // 256]
        w = pair[st["packed"][e * N * K // 2:(e + 1) * N * K // 2].long()].view(-1, 64) * c[:, None]
        return w.to(TYPES[st["dtype"]]).double().view(N, K)

    if st["op"] == "fwd":
        Y, XA = X.new_zeros(T, N), X.new_zeros(T, r)
        for e in range(E):
            rows = slice(ends[e], ends[e + 1])
            XA[rows] = D[rows] @ A[e]
            Y[rows] = X[rows] @ weight(e).T + s * XA[rows] @ B[e]
        return {"Y": Y, "XA": XA}
    dY, XA = st["dY"].double(), st["XA"].double()
    dX, dA, dB = X.new_zeros(T, K), torch.zeros_like(A), torch.zeros_like(B)
    for e in range(E):
        rows = slice(ends[e], ends[e + 1])
        G = s * dY[rows] @ B[e].T
        low = G @ A[e].T
        dX[rows] = dY[rows] @ weight(e) + (low if mask is None else low * mask[rows])
        dA[e], dB[e] = D[rows].T @ G, s * XA[rows].T @ dY[rows]
    return {"dX": dX, "dA": dA, "dB": dB}

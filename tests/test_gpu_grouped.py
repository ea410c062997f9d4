"""The expert-grouped linear and the dense linear with adapter dropout, on the
GPU, against the 64-bit oracle on the same 16-bit inputs and the same
dequantized weight.

Tolerances, elementwise, from the roundings that the calls make (u = half a
step of the 16-bit type, relative; a product's result below the smallest
normal number adds at most half the smallest subnormal, t):
  * every output is rounded once: u |out| + t;
  * s XA and G are rounded to 16 bits before their rank-r product: u times
    the product of magnitudes (and t times the other factor);
  * sums are fp32 in the tensor core, which adds 16 products per step and may
    truncate: each of the k / 16 steps (plus one joining each of at most 8
    parts of a split sum) is off by at most 2^-22 of the sum of magnitudes;
  * scales (s, the dropout factor) and the joining of the two sums are a few
    fp32 operations: 2^-21 of the magnitudes.
"""
import numpy as np
import pytest
import torch

import oracle
from bit_quantized_lora_blockwise_b200 import binding
from oracle import grouped as og

pytestmark = pytest.mark.gpu
BF, HF = torch.bfloat16, torch.float16


def f64(t):
    return t.detach().cpu().double().numpy()


class Layer:
    """E experts with random quantized weights and adapters, and T token rows."""

    def __init__(self, counts, N, K, r, dt=BF, seed=0, lead=0, trail=0, alpha=16.0, std=0.05):
        E = len(counts)
        self.E, self.N, self.K, self.r, self.dt, self.alpha = E, N, K, r, dt, alpha
        self.off = [lead + int(c) for c in np.concatenate([[0], np.cumsum(counts)])]
        self.T = self.off[-1] + trail
        g = torch.Generator().manual_seed(seed)
        rnd = lambda *s, std=1.0: (torch.randn(*s, generator=g) * std).to(dt).cuda()  # noqa: E731
        W = (torch.randn(E * N, K, generator=g) * 0.05).bfloat16().cuda()
        self.packed, am = binding.quantize_nf4(W)
        self.q, self.scale2 = binding.double_quant(am)
        self.W = f64(binding.dequant(self.packed, self.q, self.scale2, E * N, K, dtype=dt)).reshape(E, N, K)
        self.X, self.dY = rnd(self.T, K), rnd(self.T, N)
        self.A, self.B = rnd(E, K, r, std=std), rnd(E, r, N, std=std)
        self.offsets = torch.tensor(self.off, dtype=torch.int32, device="cuda")

    @property
    def weight(self):
        return self.packed, self.q, self.scale2

    def fwd(self, drop=None, **kw):
        XA = torch.full((self.T, self.r), 7.0, dtype=self.dt, device="cuda")
        Y = torch.full((self.T, self.N), 7.0, dtype=self.dt, device="cuda")
        binding.grouped_linear_fwd(*self.weight, self.X, self.offsets, self.A, self.B, self.alpha, self.N, self.K, Y=Y,
                                   XA_out=XA, dropout=drop, **kw)
        return Y, XA

    def bwd(self, XA, drop=None, **kw):
        dX = torch.full((self.T, self.K), 7.0, dtype=self.dt, device="cuda")
        _, dA, dB = binding.grouped_linear_bwd(*self.weight, self.X, self.dY, self.offsets, self.A, self.B, self.alpha,
                                               self.N, self.K, XA=XA, dX=dX, dropout=drop, **kw)
        return dX, dA, dB


def steps(k):
    return (k / 16 + 8) * 2.0**-22


def close(got, want, tol, name):
    got, bad = f64(got), None
    err = np.abs(got - want)
    bad = ~(err <= tol)
    assert not bad.any(), f"{name}: {bad.sum()} of {bad.size} off, first at {np.argwhere(bad)[0]}: " \
                          f"{got[bad][0]} for {want[bad][0]} +- {tol[bad][0]}"


def check(L, drop=None, save_xa=True):
    """Forward and backward against the oracle, rows of no expert untouched, error word clear."""
    d = None if drop is None else (drop.p, drop.seed, drop.offset)
    u = torch.finfo(L.dt).eps / 2
    t = 2.0**-25 if L.dt == HF else 0.0
    X, A, B, dY, off, s = f64(L.X), f64(L.A), f64(L.B), f64(L.dY), L.off, L.alpha / L.r
    D = X if d is None else og.dropout(X, *d)
    mask = np.ones_like(X) if d is None else og.dropout(np.ones_like(X), *d)
    Y, XA = L.fwd(drop)
    wantY, wantXA = og.grouped_fwd(X, L.W, off, A, B, L.alpha, d)
    owned = slice(off[0], off[-1])
    magXA, tolXA, tolY = np.zeros_like(wantXA), np.zeros_like(wantXA), np.zeros_like(wantY)
    fp = 2.0**-21
    for e in range(L.E):
        rows = slice(off[e], off[e + 1])
        a, b = np.abs(A[e]), np.abs(B[e])
        magXA[rows] = np.abs(D[rows]) @ a
        tolXA[rows] = u * np.abs(wantXA[rows]) + t + (steps(L.K) + fp) * magXA[rows]
        xas = s * np.abs(wantXA[rows])
        tolY[rows] = (u * np.abs(wantY[rows]) + t + (u * xas + t + s * (steps(L.K) + fp) * magXA[rows]) @ b +
                      (steps(L.K + L.r) + fp) * (np.abs(X[rows]) @ np.abs(L.W[e]).T + s * magXA[rows] @ b))
    close(XA[owned], wantXA[owned], tolXA[owned], "XA")
    close(Y[owned], wantY[owned], tolY[owned], "Y")
    dX, dA, dB = L.bwd(XA if save_xa else None, drop)
    # the backward is handed (or recomputes) the rounded XA: dB is compared for the one it used
    xa16 = np.nan_to_num(f64(XA))
    wantdX, wantdA, wantdB = og.grouped_bwd(X, dY, L.W, off, A, B, L.alpha, xa16, d)
    for e in range(L.E):
        rows = slice(off[e], off[e + 1])
        n = off[e + 1] - off[e]
        a, b, dy, w = np.abs(A[e]), np.abs(B[e]), np.abs(dY[rows]), np.abs(L.W[e])
        magG = s * (dy @ b.T)
        errG = u * np.abs(s * (dY[rows] @ B[e].T)) + t + (steps(L.N) + fp) * magG
        tol = (u * np.abs(wantdX[rows]) + t + mask[rows] * (errG @ a.T) +
               (steps(L.N + L.r) + fp) * (dy @ w + mask[rows] * (magG @ a.T)))
        close(dX[rows], wantdX[rows], tol, f"dX of expert {e}")
        tol = u * np.abs(wantdA[e]) + t + np.abs(D[rows]).T @ errG + (steps(n) + fp) * (np.abs(D[rows]).T @ magG)
        close(dA[e], wantdA[e], tol, f"dA of expert {e}")
        # a recomputed XA may round the other way: one more rounding of each of its elements
        dxa = 0.0 if save_xa else tolXA[rows] + u * np.abs(wantXA[rows])
        tol = u * np.abs(wantdB[e]) + t + s * ((np.abs(xa16[rows]) * (steps(n) + fp) + dxa).T @ dy)
        close(dB[e], wantdB[e], tol, f"dB of expert {e}")
    for out in (Y, XA, dX):
        assert (out[:off[0]] == 7).all() and (out[off[-1]:] == 7).all(), "rows of no expert were written"
    assert binding.device_error() == 0
    return Y, XA, dX, dA, dB


# counts per expert, on both sides of the average that picks one or two 256-token sub-tiles; each with experts without
# tokens, ragged tails and uneven experts
COUNTS = [[1], [0, 1], [2, 0, 0, 3], [8, 9, 16, 17, 0, 33], [0, 0, 64], [32, 65, 0, 1], [25], [100, 0, 64, 63], [256, 257],
          [300, 1, 0, 129], [384], [512, 513], [1025, 0, 700], [1, 1400]]


@pytest.mark.parametrize("counts", COUNTS, ids=lambda c: "-".join(map(str, c)))
@pytest.mark.parametrize("N,K,r", [(192, 320, 8), (320, 192, 24)])
def test_counts(counts, N, K, r):
    check(Layer(counts, N, K, r, seed=len(counts), lead=3, trail=5))


@pytest.mark.parametrize("dt", [BF, HF])
@pytest.mark.parametrize("p", [0.05, 0.5])
@pytest.mark.parametrize("counts", [[3, 0, 2], [70, 30, 129], [600, 500]], ids=str)
def test_dropout(dt, p, counts):
    check(Layer(counts, 256, 448, 16, dt, seed=5, lead=1, trail=2), binding.Dropout(p, 2**63 + 11, 2**40 + 3))


@pytest.mark.parametrize("dt", [BF, HF])
@pytest.mark.parametrize("r", [8, 64, 72, 128, 136, 256])
@pytest.mark.parametrize("counts", [[5, 4], [80, 70], [500, 400]], ids=str)
def test_ranks_and_types(dt, r, counts):
    check(Layer(counts, 128, 192, r, dt, seed=r, std=0.02), None if r % 16 else binding.Dropout(0.1, r), save_xa=r != 64)


@pytest.mark.parametrize("N,K", [(64, 64), (64, 1088), (1088, 64), (704, 2048), (2048, 704)])
@pytest.mark.parametrize("counts", [[4, 0, 7], [40, 50], [900]], ids=str)
def test_shapes(N, K, counts):
    check(Layer(counts, N, K, 16, seed=N + K, trail=1))


def test_large_adapters():
    """The adapter term is far above the base term, so it is what is compared."""
    for counts in ([3, 4], [90, 33], [700, 300]):
        check(Layer(counts, 192, 256, 32, seed=2, std=3.0), binding.Dropout(0.3, 4))
        check(Layer(counts, 192, 256, 32, seed=2, std=3.0))


def test_many_experts():
    rng = np.random.default_rng(1)
    counts = np.bincount(rng.integers(0, 1024, 300), minlength=1024)
    L = Layer(counts, 64, 64, 8, seed=9)
    check(L)
    check(Layer(np.bincount(rng.integers(0, 40, 2500), minlength=40), 128, 128, 8, seed=10))


@pytest.mark.parametrize("r,dt,p", [(8, BF, 0.0), (64, HF, 0.1), (72, BF, 0.5), (128, BF, 0.0), (136, HF, 0.0),
                                    (256, BF, 0.1)])
def test_more_tiles_than_resident_ctas(r, dt, p):
    """Enough experts and rows that the adapter gradients run over persistent CTAs, several units each: empty experts,
    whole and ragged 64-token blocks, experts that start anywhere."""
    counts = [0, 1, 64, 130, 0, 63, 65, 200, 5, 128, 0, 17] * 3
    drop = binding.Dropout(p, 9, 1) if p else None
    L = Layer(counts, 704, 576, r, dt, seed=r, lead=5, trail=9, std=0.02)  # 36 x (5 + 6) = 396 tiles of 128 rows
    first = check(L, drop)
    again = L.bwd(first[1], drop)
    assert all(torch.equal(x, y) for x, y in zip(first[2:], again))


@pytest.mark.parametrize("drop", [None, binding.Dropout(0.2, 3)])
@pytest.mark.parametrize("T", [1, 20, 33, 300, 1100])
def test_one_expert_without_offsets_is_the_dense_linear(T, drop):
    L = Layer([T], 256, 320, 16, seed=T)
    Y, XA = L.fwd(drop)
    dX, dA, dB = L.bwd(XA, drop)
    L.offsets = None
    Y2, XA2 = L.fwd(drop)
    for a, b in zip((Y, XA, dX, dA, dB), (Y2, XA2, *L.bwd(XA2, drop))):
        assert torch.equal(a, b)
    if drop is not None:
        XA3 = torch.empty_like(XA)
        Y3 = binding.linear_fwd(*L.weight, L.X, L.A[0], L.B[0], L.alpha, L.N, L.K, XA_out=XA3, dropout=drop)
        got = binding.linear_bwd(*L.weight, L.X, L.dY, L.A[0], L.B[0], L.alpha, L.N, L.K, XA=XA3, dropout=drop)
        for a, b in zip((Y, XA, dX, dA[0], dB[0]), (Y3, XA3, *got)):
            assert torch.equal(a, b)
    else:  # the dense calls compute the same sums, in an order of their own: their bounds are the same
        u = torch.finfo(BF).eps
        Yd = binding.linear_fwd(*L.weight, L.X, L.A[0], L.B[0], L.alpha, L.N, L.K)
        lim = u * (np.abs(f64(Y)) + L.alpha / L.r * np.abs(f64(XA)) @ np.abs(f64(L.B[0]))) + \
            4 * steps(L.K + L.r) * (np.abs(f64(L.X)) @ np.abs(L.W[0]).T)
        assert (np.abs(f64(Y) - f64(Yd)) <= lim).all()


def test_repeats_are_identical():
    for counts in ([2, 3], [30, 200, 61], [900, 800]):
        L = Layer(counts, 320, 512, 16, seed=7)
        d = binding.Dropout(0.1, 1)
        first = L.fwd(d)
        grads = L.bwd(first[1], d)
        for _ in range(3):
            again = L.fwd(d)
            assert all(torch.equal(a, b) for a, b in zip(first, again))
            assert all(torch.equal(a, b) for a, b in zip(grads, L.bwd(again[1], d)))


@pytest.mark.parametrize("counts", [[5, 6, 4], [40, 70, 33], [530, 397, 600]], ids=str)
def test_experts_are_isolated(counts):
    """NaN and infinities in one expert's rows and adapters, and in rows of no expert, reach no other expert."""
    L = Layer(counts, 192, 256, 24, seed=3, trail=70)
    for drop in (None, binding.Dropout(0.5, 1)):
        Y, XA = L.fwd(drop)
        clean = (Y, *L.bwd(XA, drop))
        keep = [x.clone() for x in (L.X, L.dY, L.A, L.B)]
        mid, bad = slice(L.off[1], L.off[2]), [float("nan"), float("inf")]
        for t in (L.X, L.dY):
            t[mid] = bad[0]
            t[L.off[2] - 1] = bad[1]
            t[L.off[-1]:] = bad[0]
        for t in (L.A, L.B):
            t[1] = bad[0]
        Y, XA2 = L.fwd(drop)
        XA2[L.off[-1]:] = bad[0]
        got = (Y, *L.bwd(XA2, drop))
        for e in (0, 2):
            rows = slice(L.off[e], L.off[e + 1])
            for i in (0, 1):
                assert torch.equal(got[i][rows], clean[i][rows])
            for i in (2, 3):
                assert torch.equal(got[i][e], clean[i][e])
        for t, k in zip((L.X, L.dY, L.A, L.B), keep):
            t.copy_(k)


@pytest.mark.parametrize("drop", [None, binding.Dropout(0.1, 1)])
def test_no_tokens(drop):
    L = Layer([0, 0, 0], 128, 64, 8)
    check(L, drop)  # offsets all 0, T = 0
    assert not L.bwd(None, drop)[1].any() and not L.bwd(None, drop)[2].any()
    M = Layer([0, 0], 128, 64, 8, lead=40, trail=30)  # rows, but no expert owns one
    check(M, drop)


@pytest.mark.parametrize("T", [40, 900])
def test_offsets_out_of_order_are_contained(T):
    """Descending or out-of-range offsets set bit 1 of the error word; no access leaves the buffers (guard bands), and
    the groups are those of the clamped, raised sequence."""
    L = Layer([T // 2, T - T // 2, 0], 128, 192, 8, seed=1)
    guard = lambda rows, cols: torch.full((rows + 200, cols), 7.0, dtype=BF, device="cuda")  # noqa: E731
    for off, fixed in (([0, T + 50, 5, T], [0, T, T, T]), ([-7, 9, 4, T], [0, 9, 9, T]), ([T, 0, 0, 0], [T, T, T, T])):
        outs = []
        for o in (off, fixed):
            L.offsets = torch.tensor(o, dtype=torch.int32, device="cuda")
            Y, XA, dX = guard(T, L.N), guard(T, L.r), guard(T, L.K)
            binding.grouped_linear_fwd(*L.weight, L.X, L.offsets, L.A, L.B, 16.0, L.N, L.K, Y=Y[100:100 + T],
                                       XA_out=XA[100:100 + T])
            _, dA, dB = binding.grouped_linear_bwd(*L.weight, L.X, L.dY, L.offsets, L.A, L.B, 16.0, L.N, L.K,
                                                   XA=XA[100:100 + T], dX=dX[100:100 + T])
            torch.cuda.synchronize()
            assert binding.device_error(clear=True) == (2 if o is off else 0)
            for b in (Y, XA, dX):
                assert (b[:100] == 7).all() and (b[100 + T:] == 7).all()
            outs.append((Y, XA, dX, dA, dB))
        assert all(torch.equal(a, b) for a, b in zip(*outs))


def test_workspace_and_output_guard_bands():
    for counts, drop in (([3, 5], None), ([60, 41], binding.Dropout(0.2, 1)), ([700, 400], None)):
        L = Layer(counts, 192, 320, 8, seed=4)
        need = binding.grouped_workspace_bytes(L.E, L.T, L.N, L.K, L.r, drop is not None)
        raw = torch.full((need + 8192,), 0xA5, dtype=torch.uint8, device="cuda")
        ws = raw[4096:4096 + need]
        Y, XA = L.fwd(drop, workspace=ws)
        grads = L.bwd(XA, drop, workspace=ws)
        torch.cuda.synchronize()
        assert (raw[:4096] == 0xA5).all() and (raw[-4096:] == 0xA5).all()
        assert all(torch.equal(a, b) for a, b in zip((Y, XA, *grads), (*L.fwd(drop), *L.bwd(XA, drop))))
        with pytest.raises(binding.QLoRAError, match="WORKSPACE"):
            L.bwd(XA, drop, workspace=raw[:256])


@pytest.mark.parametrize("counts", [[4, 0, 3], [90, 0, 60], [600, 424, 0]], ids=str)
def test_graph_replay_with_other_offsets(counts):
    """A captured forward + backward follows the offsets that the device holds at replay."""
    L = Layer(counts, 192, 256, 16, seed=6)
    d = binding.Dropout(0.1, 5)
    XA = torch.zeros(L.T, L.r, dtype=BF, device="cuda")
    Y, dX = torch.zeros(L.T, L.N, dtype=BF, device="cuda"), torch.zeros(L.T, L.K, dtype=BF, device="cuda")
    dA, dB = torch.empty_like(L.A), torch.empty_like(L.B)
    ws = torch.empty(binding.grouped_workspace_bytes(L.E, L.T, L.N, L.K, L.r, True), dtype=torch.uint8, device="cuda")

    def step():
        binding.grouped_linear_fwd(*L.weight, L.X, L.offsets, L.A, L.B, L.alpha, L.N, L.K, Y=Y, XA_out=XA, workspace=ws,
                                   dropout=d)
        binding.grouped_linear_bwd(*L.weight, L.X, L.dY, L.offsets, L.A, L.B, L.alpha, L.N, L.K, XA=XA, dX=dX, dA=dA,
                                   dB=dB, workspace=ws, dropout=d)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for off in (L.off, [0, 1, L.T // 3, L.T], [0, L.T, L.T, L.T], [0, 0, 0, L.T]):
        L.offsets.copy_(torch.tensor(off, dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        L.off = off
        got = [t.clone() for t in (Y, XA, dX, dA, dB)]
        Y1, XA1 = L.fwd(d)
        assert all(torch.equal(a, b) for a, b in zip(got, (Y1, XA1, *L.bwd(XA1, d))))
    assert binding.device_error() == 0


@pytest.mark.parametrize("drop", [None, binding.Dropout(0.3, 11)])
def test_graph_replay_with_many_tiles(drop):
    """The same with more adapter-gradient tiles than resident CTAs: uneven, one expert, none, and the first ones again."""
    E, T = 36, 700
    L = Layer([T // E] * E, 704, 576, 8, seed=12, trail=T - T // E * E, std=0.02)
    dX = torch.zeros(T, L.K, dtype=BF, device="cuda")
    dA, dB = torch.empty_like(L.A), torch.empty_like(L.B)
    ws = torch.empty(binding.grouped_workspace_bytes(E, T, L.N, L.K, L.r, drop is not None), dtype=torch.uint8,
                     device="cuda")

    def step():
        binding.grouped_linear_bwd(*L.weight, L.X, L.dY, L.offsets, L.A, L.B, L.alpha, L.N, L.K, XA=None, dX=dX, dA=dA,
                                   dB=dB, workspace=ws, dropout=drop)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    rng = np.random.default_rng(3)
    uneven = [0, *sorted(rng.integers(0, T + 1, E - 1).tolist()), T]
    for off in (uneven, [0] * 20 + [T] * (E - 19), [5] * (E + 1), L.off, uneven):
        L.offsets.copy_(torch.tensor(off, dtype=torch.int32))
        L.off = off
        dX.fill_(7)
        dA.fill_(7)
        dB.fill_(7)
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (dX, dA, dB)]
        for e in range(E):
            if off[e] == off[e + 1]:
                assert not got[1][e].any() and not got[2][e].any()
        assert all(torch.equal(a, b) for a, b in zip(got, L.bwd(None, drop)))
        check(L, drop, save_xa=False)
    assert binding.device_error() == 0


def test_two_streams_at_once():
    """Two calls in flight, a workspace each, on side streams."""
    Ls = [Layer(c, 448, 512, 16, seed=i) for i, c in enumerate(([300, 410, 77], [6, 8, 2]))]
    want = []
    for L in Ls:
        Y, XA = L.fwd()
        want.append((Y, XA, *L.bwd(XA)))
    streams = [torch.cuda.Stream() for _ in Ls]
    torch.cuda.synchronize()
    got = [None] * len(Ls)
    for _ in range(5):
        for i, (L, s) in enumerate(zip(Ls, streams)):
            with torch.cuda.stream(s):
                Y, XA = L.fwd()
                got[i] = (Y, XA, *L.bwd(XA))
    torch.cuda.synchronize()
    for a, b in zip(want, got):
        assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_indices_past_32_bits():
    """Outputs of more than 2^31 elements: the last expert's rows, compared alone."""
    N, K, T, r = 8256, 64, 262144, 8
    L = Layer([0, 0], N, K, r, seed=1)
    L.T, L.off = T, [0, T - 300, T]
    L.offsets = torch.tensor(L.off, dtype=torch.int32, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(1)
    L.X = torch.randn(T, K, generator=g, device="cuda").bfloat16()
    d = binding.Dropout(0.25, 3)
    Y = torch.empty(T, N, dtype=BF, device="cuda")
    XA = torch.empty(T, r, dtype=BF, device="cuda")
    binding.grouped_linear_fwd(*L.weight, L.X, L.offsets, L.A, L.B, L.alpha, N, K, Y=Y, XA_out=XA, dropout=d)
    rows = slice(T - 300, T)
    X = f64(L.X[rows])
    keep = og.keep_mask(300 * K, 0.25, 3, 0, first=(T - 300) * K).reshape(300, K)
    xa = np.where(keep, X * og.factor(0.25), 0.0) @ f64(L.A[1])
    want = X @ L.W[1].T + L.alpha / r * xa @ f64(L.B[1])
    u, mag = torch.finfo(BF).eps / 2, np.abs(X) @ np.abs(L.W[1]).T
    lim = u * np.abs(want) + u * L.alpha / r * np.abs(xa) @ np.abs(f64(L.B[1])) + steps(4 * K) * (mag + 1)
    assert (np.abs(f64(Y[rows]) - want) <= lim).all()
    # and the backward's dX over a token operand of more than 2^31 elements
    dY = Y
    dX, dA, dB = binding.grouped_linear_bwd(*L.weight, L.X, dY, L.offsets, L.A, L.B, L.alpha, N, K, XA=XA, dropout=d)
    dy = f64(Y[rows])
    G = L.alpha / r * dy @ f64(L.B[1]).T
    M = np.where(keep, og.factor(0.25), 0.0)
    want = dy @ L.W[1] + M * (G @ f64(L.A[1]).T)
    lim = (u * np.abs(want) + M * (2 * u * np.abs(G) @ np.abs(f64(L.A[1])).T) +
           2 * steps(N) * (np.abs(dy) @ np.abs(L.W[1]) + 1))
    assert (np.abs(f64(dX[rows]) - want) <= lim).all()
    assert binding.device_error() == 0


@pytest.mark.parametrize("T,E", [(24, 4), (700, 4)])
def test_expert_mlp_training_step(T, E):
    """The calls as a mixture-of-experts block uses them: gate, up and down over the same routed rows with adapter
    dropout, forward, backward and an optimizer step on the experts' adapters; every call against the oracle on the
    inputs that it got, and the loss's gradient of one adapter against a difference."""
    rng = np.random.default_rng(T)
    counts = np.bincount(rng.integers(0, E, T), minlength=E)
    gate, up, down = Layer(counts, 320, 192, 8, seed=1), Layer(counts, 320, 192, 8, seed=2), Layer(counts, 192, 320, 8, seed=3)
    up.X = gate.X
    drops = [binding.Dropout(0.1, 42, i << 32) for i in range(3)]
    Yg, XAg, *_ = check(gate, drops[0])
    Yu, XAu, *_ = check(up, drops[1])
    down.X = (torch.nn.functional.silu(Yg.float()) * Yu.float()).to(BF)
    Yd, XAd, dh, dAd, dBd = check(down, drops[2])
    dh = dh.float()
    sg = torch.sigmoid(Yg.float())
    gate.dY = (dh * Yu.float() * (sg * (1 + Yg.float() * (1 - sg)))).to(BF)
    up.dY = (dh * Yg.float() * sg).to(BF)
    _, _, dXg, dAg, dBg = check(gate, drops[0])
    _, _, dXu, dAu, dBu = check(up, drops[1])
    assert torch.isfinite((dXg.float() + dXu.float())).all()
    params = [gate.A, gate.B, up.A, up.B, down.A, down.B]
    before = [p.clone() for p in params]
    opt = binding.PagedAdamW(params, lr=1e-2)
    opt.step([dAg, dBg, dAu, dBu, dAd, dBd])
    torch.cuda.synchronize()
    assert all((p != b).any() for p, b in zip(params, before))
    opt.close()
    # loss = sum(Yd * down.dY) along down.B: linear in B, so the difference quotient is exact up to roundings
    s, u = down.alpha / down.r, torch.finfo(BF).eps / 2
    down.A, down.B = before[4], before[5].clone()
    e = int(np.argmax(counts))
    rows = slice(down.off[e], down.off[e + 1])
    base = f64(down.fwd(drops[2])[0][rows])
    down.B[e, 3] += 1.0
    step = f64(down.B[e, 3]) - f64(before[5][e, 3])
    moved = f64(down.fwd(drops[2])[0][rows])
    dy = f64(down.dY[rows])
    quotient = ((moved - base) * dy).sum()
    want = (f64(dBd[e, 3]) * step).sum()
    tol = (u * (np.abs(moved) + np.abs(base)) * np.abs(dy)).sum() + 2 * u * np.abs(f64(dBd[e, 3]) * step).sum() + \
        2 * u * (s * np.abs(f64(XAd[rows, 3]))[:, None] * np.abs(step) * np.abs(dy)).sum()
    assert abs(quotient - want) <= tol

"""The backward of many experts (adapter gradients over persistent CTAs, with
dropout through the keep bits that dX leaves): experts isolated from one
another's NaN and infinities, two calls in flight, infinities kept."""
import pytest
import torch

from bit_quantized_lora_blockwise_b200 import binding
from test_gpu_grouped import Layer

pytestmark = pytest.mark.gpu
COUNTS = [3, 1, 64, 130, 0, 63, 65, 200, 5, 128, 0, 17] * 3  # with 704 x 576: 396 tiles of 128 rows


@pytest.mark.parametrize("p", [0.0, 0.5])
@pytest.mark.parametrize("r", [8, 72, 136])
def test_experts_are_isolated(r, p):
    """NaN and infinities in every other expert with rows, and in rows of no expert: the others' bits do not change."""
    L = Layer(COUNTS, 704, 576, r, seed=r, lead=5, trail=40, std=0.02)
    drop = binding.Dropout(p, 3) if p else None
    XA = L.fwd(drop)[1]
    clean = L.bwd(XA, drop)
    busy = [e for e in range(L.E) if L.off[e] < L.off[e + 1]]
    for i, e in enumerate(busy[::2]):
        rows = slice(L.off[e], L.off[e + 1])
        bad = (float("nan"), float("inf"))[i % 2]
        for t in (L.X, L.dY, XA):
            t[rows] = bad
        L.A[e] = L.B[e] = bad
    for rows in (slice(0, L.off[0]), slice(L.off[-1], None)):
        for t in (L.X, L.dY, XA):
            t[rows] = float("nan")
    got = L.bwd(XA, drop)
    for e in busy[1::2]:
        rows = slice(L.off[e], L.off[e + 1])
        assert torch.equal(got[0][rows], clean[0][rows])
        assert torch.equal(got[1][e], clean[1][e]) and torch.equal(got[2][e], clean[2][e])
    assert binding.device_error() == 0


@pytest.mark.parametrize("counts", [COUNTS, [40, 30]], ids=["many", "few"])
def test_an_infinite_activation_makes_its_row_of_dA_infinite(counts):
    """X[t, k] = inf: dA[k] is the sign of G[t] times infinity (the second part of G, which may be 0, adds no NaN)."""
    L = Layer(counts, 704, 576, 16, torch.float16, seed=2, std=0.1)
    XA = L.fwd()[1]
    e = 0
    t, k = L.off[e] + 2, 131
    G = L.alpha / L.r * L.dY[t].float() @ L.B[e].float().T
    L.X[t, k] = float("inf")
    dA = L.bwd(XA)[1]
    assert G.abs().min() > 1e-4
    assert torch.equal(dA[e, k].float(), torch.sign(G) * float("inf"))
    assert torch.isfinite(dA[e, :k]).all() and torch.isfinite(dA[e, k + 1:]).all() and torch.isfinite(dA[e + 1:]).all()


def test_two_streams_at_once():
    """Two backward calls in flight, a workspace and unit counter each."""
    Ls = [Layer(c, 704, 576, r, seed=i, std=0.02) for i, (c, r) in enumerate(((COUNTS, 8), (COUNTS[::-1], 72)))]
    drops = [binding.Dropout(0.3, 1), None]
    XAs = [L.fwd(d)[1] for L, d in zip(Ls, drops)]
    want = [L.bwd(XA, d) for L, XA, d in zip(Ls, XAs, drops)]
    streams = [torch.cuda.Stream() for _ in Ls]
    torch.cuda.synchronize()
    for _ in range(5):
        got = []
        for L, XA, d, s in zip(Ls, XAs, drops, streams):
            with torch.cuda.stream(s):
                got.append(L.bwd(XA, d))
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for g, w in zip(got, want) for a, b in zip(g, w))
    assert binding.device_error() == 0

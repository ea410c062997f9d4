"""The adapter branch of the backward at both ends of fp16's range: G = s dY B^T
within it although the dropout factor times G is not, and G below its normal
numbers although dA is not; with few adapter-gradient tiles and with many, and
one and two token sub-tiles a tile. Bounds as in test_gpu_grouped.py."""
import numpy as np
import pytest
import torch

from bit_quantized_lora_blockwise_b200 import binding
from oracle import grouped as og
from test_gpu_grouped import Layer, check, close, f64, steps

pytestmark = pytest.mark.gpu
HF = torch.float16
MANY = [0, 1, 64, 130, 0, 63, 65, 200, 5, 128, 0, 17] * 3  # with 704 x 576: more 128-row tiles than resident CTAs


@pytest.mark.parametrize("counts,N,K,r", [([60, 0, 40], 192, 256, 8), ([600, 500], 192, 256, 72), (MANY, 704, 576, 8),
                                          (MANY, 704, 576, 136)], ids=lambda c: str(c)[:20])
def test_factor_times_g_past_fp16(counts, N, K, r):
    """p = 0.97: G is some thousands, 33 G is past 65504; every output is in range."""
    L = Layer(counts, N, K, r, HF, seed=3, lead=2, trail=3, alpha=2.0 * r)
    L.X *= 0.01
    L.A.mul_(0.04)
    L.dY *= 100
    L.B.mul_(20.0 * (192 / N) ** 0.5)  # A 0.002, B 1 (std 0.05 as made)
    drop = binding.Dropout(0.97, 11, 5)
    G = 2.0 * L.dY.float() @ L.B[1].float().T
    assert 65504 / 33.3 < G.abs().max() < 65504
    for out in check(L, drop):
        assert torch.isfinite(out[L.off[0]:L.off[-1]] if out.shape[0] == L.T else out).all()


def tight_dA(L, drop, dA):
    """dA against the oracle with G's own error bounded by its two 16-bit parts: the second holds what the first rounds
    away, scaled by c (2^11 for fp16, 2^8 for bf16) so that it is no smaller in magnitude than the first's rounding unit
    allows. |G - parts| <= u (u |G| + t) + t / c, and the fp32 sum that G is; the rest as for every sum."""
    u, t, c = torch.finfo(L.dt).eps / 2, 2.0**-25 if L.dt == HF else 0.0, 2.0**11 if L.dt == HF else 2.0**8
    s, fp = L.alpha / L.r, 2.0**-21
    X, dY, B = f64(L.X), f64(L.dY), f64(L.B)
    D = X if drop is None else og.dropout(X, *drop)
    for e in range(L.E):
        rows = slice(L.off[e], L.off[e + 1])
        G, mag = s * dY[rows] @ B[e].T, s * np.abs(dY[rows]) @ np.abs(B[e]).T
        err = u * (u * np.abs(G) + t) + t / c + (steps(L.N) + fp) * mag
        want, d = D[rows].T @ G, np.abs(D[rows]).T
        close(dA[e], want, u * np.abs(want) + t + d @ err + (steps(len(G)) + fp) * (d @ mag), f"dA of expert {e}")


SHAPES = [([60, 0, 41], 192, 256, 8), ([600, 500], 192, 256, 72), ([700], 256, 320, 136), (MANY, 704, 576, 8),
          (MANY, 704, 576, 72), (MANY, 704, 576, 200)]


@pytest.mark.parametrize("counts,N,K,r", SHAPES, ids=lambda c: str(c)[:20])
@pytest.mark.parametrize("p", [0.0, 0.3])
def test_g_below_fp16s_normal_numbers(counts, N, K, r, p):
    """The first steps of a training run, whose B is next to zero: most of G rounds to 0 or a few units of 2^-24 in
    fp16, and dA, a sum over the tokens, is in its range."""
    L = Layer(counts, N, K, r, HF, seed=4, lead=2, trail=3, alpha=0.25 * r)
    L.X *= 100
    L.dY *= 1e-3
    L.B *= 2e-5
    drop = binding.Dropout(p, 13, 9) if p else None
    assert (0.25 * L.dY.float() @ L.B[0].float().T).abs().max() < 2.0**-20
    _, _, _, dA, _ = check(L, drop)
    tight_dA(L, drop, dA)


@pytest.mark.parametrize("counts,N,K,r", SHAPES, ids=lambda c: str(c)[:20])
@pytest.mark.parametrize("dt", [torch.bfloat16, HF])
def test_dA_is_rounded_once(dt, counts, N, K, r):
    """At ordinary magnitudes too dA carries its own rounding and none of G's."""
    L = Layer(counts, N, K, r, dt, seed=6, lead=1, trail=2, std=0.02)
    for drop in (None, binding.Dropout(0.1, 2)):
        tight_dA(L, drop, check(L, drop)[3])


def test_infinite_g_stays_in_its_column():
    """G past fp16's range is infinite, as in one part: dA of that rank and expert is not finite, every other one is
    unchanged."""
    L = Layer([70, 90], 192, 256, 16, HF, seed=7)
    XA = L.fwd()[1]
    clean = L.bwd(XA)[1].clone()
    L.B[1, 3] = 6e4
    L.dY[L.off[1]:] = 100
    dA = L.bwd(XA)[1]
    assert torch.equal(dA[0], clean[0]) and not torch.isfinite(dA[1, :, 3]).any()
    assert torch.isfinite(dA[1, :, 4:]).all() and torch.isfinite(dA[1, :, :3]).all()

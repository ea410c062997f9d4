"""The adapter branch of the backward at both ends of fp16's range: G = s dY B^T
within it although the dropout factor times G is not, with few adapter-gradient
tiles and with many, and one and two token sub-tiles a tile."""
import pytest
import torch

from bit_quantized_lora_blockwise_b200 import binding
from test_gpu_grouped import Layer, check

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

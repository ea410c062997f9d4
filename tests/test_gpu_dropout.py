"""Counter-based dropout on the GPU against the 64-bit oracle: the mask is
exact (a kept element is one rounding of x * factor, half a step of its type;
a dropped one is +0 whatever it held)."""
import numpy as np
import pytest
import torch

from bit_quantized_lora_blockwise_b200 import binding
from oracle import grouped as og

pytestmark = pytest.mark.gpu
TYPES = [torch.bfloat16, torch.float16, torch.float32]


def _expect(x, p, seed, offset):
    """The rounded product, element by element: fp32 x * fp32 factor rounded to x's type. One 64-bit product rounded to
    fp32 is the fp32 product, so the comparison is exact."""
    keep = torch.from_numpy(og.keep_mask(x.numel(), p, seed, offset)).view(x.shape)
    f = np.float32(og.factor(p))
    y = (x.cpu().double() * float(f)).float().to(x.dtype)
    return torch.where(keep, y, torch.zeros((), dtype=x.dtype))


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("n", [1, 7, 8, 9, 255, 2048, 2049, 300007])
def test_matches_oracle(dt, n):
    x = (torch.randn(n, generator=torch.Generator().manual_seed(n)) * 3).to(dt)
    for p, seed, offset in ((0.1, 2**63 + 5, 7), (0.5, 0, 2**64 - 3), (0.97, 2**64 - 1, 0)):
        y = binding.dropout(x.cuda(), binding.Dropout(p, seed, offset))
        assert torch.equal(y.cpu(), _expect(x, p, seed, offset))
        assert not torch.signbit(y.cpu()[~torch.from_numpy(og.keep_mask(n, p, seed, offset))]).any()


@pytest.mark.parametrize("dt", TYPES)
def test_special_values_and_in_place(dt):
    x = torch.tensor([float("nan"), float("inf"), -float("inf"), -0.0, 1.0, -2.0, 3.0, 65504.0] * 500).to(dt)
    d = binding.Dropout(0.5, 3, 4)
    keep = torch.from_numpy(og.keep_mask(x.numel(), 0.5, 3, 4))
    y = binding.dropout(x.cuda(), d).cpu()
    assert (y[~keep] == 0).all() and torch.isnan(y[keep & torch.isnan(x)]).all()
    want = _expect(x, 0.5, 3, 4)
    assert torch.equal(y.nan_to_num(1234.0), want.nan_to_num(1234.0))
    z = x.cuda()
    assert binding.dropout(z, d, out=z) is z
    assert torch.equal(z.cpu().nan_to_num(1234.0), want.nan_to_num(1234.0))


def test_p_zero_is_the_identity_and_gradient_is_the_same_map():
    x = torch.randn(1000, 37, device="cuda")
    assert torch.equal(binding.dropout(x, binding.Dropout(0.0, 9)), x)
    assert torch.equal(binding.dropout(x, binding.Dropout(2.0**-18, 9)), x)  # rounds to a threshold of 0
    d = binding.Dropout(0.3, 5, 1)
    # y = D(x) is linear in x: its gradient is D(dy), and differences of D see the same factors (both exact: a power of
    # two step on values that are small integers)
    xi = torch.randint(-8, 8, (4096,), device="cuda").float()
    ones = binding.dropout(torch.ones_like(xi), d)
    assert torch.equal(binding.dropout(xi + 1, d) - binding.dropout(xi, d) != 0, ones != 0)
    keep = torch.from_numpy(og.keep_mask(4096, 0.3, 5, 1)).cuda()
    assert torch.equal(ones, torch.where(keep, torch.tensor(np.float32(og.factor(0.3)), device="cuda"), 0.0))


def test_empty_and_guard_bands():
    assert binding.dropout(torch.empty(0, 5, device="cuda"), binding.Dropout(0.5, 1)).shape == (0, 5)
    raw = torch.full((64 + 999 + 64,), 7.0, device="cuda")
    out = raw[64:64 + 999]
    binding.dropout(torch.randn(999, device="cuda"), binding.Dropout(0.5, 1), out=out)
    assert (raw[:64] == 7).all() and (raw[-64:] == 7).all()
    with pytest.raises(binding.QLoRAError):  # 4-byte aligned only
        binding.dropout(raw[1:], binding.Dropout(0.5, 1))


def test_graph_replay_and_side_stream():
    x = torch.randn(5000, device="cuda").bfloat16()
    d = binding.Dropout(0.2, 8, 100)
    want = binding.dropout(x, d)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = binding.dropout(x, d)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got, want)
    out = torch.empty_like(x)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        binding.dropout(x, d, out=out)
    x.copy_(torch.randn(5000, device="cuda").bfloat16())
    g.replay()
    assert torch.equal(out, binding.dropout(x, d))


def test_indices_past_32_bits():
    n = 2**32 + 41
    x = torch.ones(n, dtype=torch.bfloat16, device="cuda")
    d = binding.Dropout(0.25, 77, 5)
    binding.dropout(x, d, out=x)
    for first in (0, 2**31 - 64, 2**32 - 64, 2**32):
        keep = og.keep_mask(min(n - first, 1000), 0.25, 77, 5, first=first)
        assert np.array_equal(x[first:first + keep.size].float().cpu().numpy() != 0, keep)

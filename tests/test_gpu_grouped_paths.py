"""The grouped calls on the paths that the device picks from the routing: a last
round of tiles cut by token sub-tile (tiles with one sub-tile among them), and
tiles cut over K, with and without adapter dropout. Which cut a case takes is
checked on the CPU with the kernel's own plan function, so the cases cannot
drift off their path."""
import os
import subprocess

import pytest
import torch

from bit_quantized_lora_blockwise_b200 import binding
from bit_quantized_lora_blockwise_b200.build import ARCH, CSRC, ROOT, nvcc
from test_gpu_grouped import Layer, check

BF, HF = torch.bfloat16, torch.float16
PAIRS = 74  # CTA pairs of a 148-SM part

# name: counts, N, K, r, p, type, cut of the forward and of dX
CASES = {
    # 80 tiles, one of them with a single sub-tile, in rounds of 74
    "subtiles": ([512 * 79, 100], 64, 64, 72, 0.0, BF, "subtiles", "subtiles"),
    "subtiles-drop": ([512 * 79, 100], 64, 64, 72, 0.3, BF, "subtiles", "subtiles"),
    # the same with adapter gradients over persistent CTAs, which read the keep bits that dX leaves
    "subtiles-keep": ([0, 300, 0, 512 * 101] + [0] * 155 + [100], 64, 64, 8, 0.25, HF, "subtiles", "subtiles"),
    # three row tiles, the last half empty: the last round starts inside an expert
    "subtiles-rows": ([2561, 0, 10240, 300], 64, 640, 136, 0.1, BF, "split", "subtiles"),
    "subtiles-rows-fwd": ([2561, 0, 10240, 300], 640, 64, 24, 0.5, HF, "subtiles", "split"),
    # two sub-tiles and one sub-tile a tile, cut over K
    "split-2": ([600, 500], 1024, 256, 72, 0.2, BF, "whole", "split"),
    "split-2-fwd": ([600, 500], 256, 1024, 8, 0.2, HF, "split", "whole"),
    "split-1": ([40, 50, 0], 1024, 192, 136, 0.4, BF, "whole", "split"),
}


def cuts(counts, N, K):
    """(tiles, pairs, K blocks, sub-tiles) of the forward and of dX."""
    ntt = 2 if sum(counts) // len(counts) >= 320 else 1
    tokens = sum(-(-c // (256 * ntt)) for c in counts)
    return [(-(-rows // 256) * tokens, PAIRS, kdim // 64, ntt) for rows, kdim in ((N, K), (K, N))]


def test_the_cases_take_their_paths(tmp_path):
    exe = tmp_path / "grouped_plan_print"
    subprocess.check_call([nvcc(), *ARCH, "-O1", "-std=c++17", "-I", os.path.join(ROOT, "include"), "-I", CSRC, "-o",
                           str(exe), os.path.join(ROOT, "tests", "host", "grouped_plan_print.cu")], timeout=600)
    for name, (counts, N, K, _, _, _, *want) in CASES.items():
        args = [str(v) for cut in cuts(counts, N, K) for v in cut]
        lines = subprocess.check_output([str(exe), *args], text=True, timeout=60).split("\n")[:2]
        for line, w in zip(lines, want):
            units, full, splits, subtiles = map(int, line.split())
            got = "split" if splits > 1 else "subtiles" if subtiles > 1 else "whole"
            assert got == w, (name, line)
            assert got != "subtiles" or full == PAIRS * (full // PAIRS) > 0


@pytest.mark.gpu
@pytest.mark.parametrize("name", CASES)
def test_paths(name):
    counts, N, K, r, p, dt, *_ = CASES[name]
    assert torch.cuda.get_device_properties(0).multi_processor_count == 2 * PAIRS
    drop = binding.Dropout(p, 2**40 + 7, 3) if p else None
    L = Layer(counts, N, K, r, dt, seed=len(name), lead=3, trail=70)
    first = check(L, drop)
    for _ in range(2):  # and again, bit for bit
        Y, XA = L.fwd(drop)
        assert all(torch.equal(a, b) for a, b in zip(first, (Y, XA, *L.bwd(XA, drop))))

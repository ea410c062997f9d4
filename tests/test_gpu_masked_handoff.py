"""Adapter dropout in dX: the low-rank sums that the peer CTA's warps mask in its
TMEM, handed to the MMAs that the leader CTA issues."""
import os
import re

import pytest

from bit_quantized_lora_blockwise_b200 import binding
from bit_quantized_lora_blockwise_b200.build import CSRC
from test_gpu_grouped import Layer, check


def test_masked_sums_cross_the_pair_at_cluster_scope():
    """In dX with dropout the peer's warps rewrite the low-rank sums in their TMEM and the leader's MMAs accumulate on
    them: the arrival that hands them over releases at cluster scope, and the leader's wait acquires at it."""
    src = open(os.path.join(CSRC, "gemm.cuh")).read()
    uses = [m.group(0) for m in re.finditer(r"\w+\((?:map_cluster\()?masked\(acc\)", src)]
    assert sorted(uses) == ["mbar_arrive_cluster(map_cluster(masked(acc)", "mbar_wait_cluster(masked(acc)"]
    ptx = open(os.path.join(CSRC, "ptx.cuh")).read()
    body = lambda name: ptx[ptx.index(f"{name}("):].split("\n}\n")[0]  # noqa: E731
    assert "mbarrier.arrive.release.cluster.shared::cluster" in body("void mbar_arrive_cluster")
    assert "mbarrier.try_wait.parity.acquire.cluster" in body("bool mbar_wait_cluster")


@pytest.mark.gpu
@pytest.mark.parametrize("counts,N,K", [([700, 900, 400], 64, 1024), ([60, 200, 129], 64, 1024)], ids=str)
def test_masked_sums_are_exact_in_both_ctas(counts, N, K):
    """Adapter terms far above the base term, many tiles a pair: whatever one CTA of the pair masked too late would
    show in its 128 rows."""
    L = Layer(counts * 4, N, K, 64, seed=1, std=3.0)
    for p in (0.5, 0.9):
        check(L, binding.Dropout(p, 5))

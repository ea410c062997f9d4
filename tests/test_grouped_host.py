"""Expert-grouped linear and dropout, host side (CPU only): the argument
checks return the documented status before anything touches a GPU, the
binding refuses wrong shapes, types and devices, and the work plan that the
kernels derive from the tile count covers every tile once within the
workspace's bound (a host program compiled against the kernel's header)."""
import ctypes
import math
import os
import subprocess

import pytest
import torch

from bit_quantized_lora_blockwise_b200 import binding
from bit_quantized_lora_blockwise_b200.build import ARCH, CSRC, ROOT, build, nvcc


@pytest.fixture(scope="module")
def lib():
    build()
    return binding.load()


def _fake(addr=0x10000):
    return ctypes.c_void_p(addr)


S = ctypes.c_void_p(0)
OK_SHAPE = dict(E=4, T=16, N=128, K=128, r=8, alpha=16.0)


def _drop(p):
    return binding.Dropout(p, 1, 2)._desc()


def _fwd(lib, ptr={}, dtype=0, ws=_fake(), wsb=1 << 40, drop=None, tables=None, **kw):
    a = {**OK_SHAPE, **kw}
    tb = tables or binding._tables(None, None)
    g = lambda k: ptr.get(k, _fake())  # noqa: E731
    return lib.qlora_grouped_linear_fwd(g("packed"), g("q"), g("scale2"), tb.nf4, tb.t8, dtype, a["E"], a["T"], a["N"],
                                        a["K"], g("offsets"), g("X"), g("A"), g("B"), a["r"], a["alpha"], drop, g("Y"),
                                        ptr.get("XA"), ws, wsb, S)


def _bwd(lib, ptr={}, dtype=0, ws=_fake(), wsb=1 << 40, drop=None, tables=None, **kw):
    a = {**OK_SHAPE, **kw}
    tb = tables or binding._tables(None, None)
    g = lambda k: ptr.get(k, _fake())  # noqa: E731
    return lib.qlora_grouped_linear_bwd(g("packed"), g("q"), g("scale2"), tb.nf4, tb.t8, dtype, a["E"], a["T"], a["N"],
                                        a["K"], g("offsets"), g("X"), g("dY"), g("A"), g("B"), ptr.get("XA"), a["r"],
                                        a["alpha"], drop, g("dX"), g("dA"), g("dB"), ws, wsb, S)


@pytest.mark.parametrize("call,ptrs", [(_fwd, ("packed", "q", "scale2", "offsets", "X", "A", "B", "Y")),
                                       (_bwd, ("packed", "q", "scale2", "offsets", "X", "dY", "A", "B", "dX", "dA", "dB"))])
def test_grouped_argument_checks(lib, call, ptrs):
    for p in ptrs:
        assert call(lib, {p: None}) == 1, p
        if p != "offsets":
            assert call(lib, {p: _fake(0x10008)}) == 3, p
    assert call(lib, {"offsets": _fake(0x10002)}) == 3
    assert call(lib, {"XA": _fake(0x10008)}) == 3
    assert call(lib, ws=_fake(0x10008)) == 3
    for bad in (dict(E=0), dict(E=1025), dict(E=-1), dict(T=-1), dict(N=96), dict(N=32), dict(K=100), dict(K=0),
                dict(E=1024, N=1 << 21), dict(E=1024, K=1 << 21), dict(T=1 << 31)):
        assert call(lib, **bad) == 2, bad
    for bad in (dict(r=0), dict(r=264), dict(r=12), dict(alpha=math.inf), dict(alpha=math.nan), dict(dtype=2),
                dict(dtype=-1)):
        assert call(lib, **bad) == 4, bad
    for p in (-0.1, 1.0, 1.5, math.nan, math.inf, 0.999999):
        assert call(lib, drop=_drop(p)) == 4, p
    wrong = binding._HostTables([*range(16)], None)
    wrong.nf4[3] = -5.0
    assert call(lib, tables=wrong) == 8
    # no tokens: the token pointers may be NULL (what is left to check needs a device)
    none = {p: None for p in ("X", "Y", "dY", "dX")}
    assert call(lib, none) == 1 and call(lib, none, T=0) in (0, 5, 6)
    # NULL offsets are for one expert
    assert call(lib, {"offsets": None}, E=2) == 1


def test_dropout_argument_checks(lib):
    f, d = lib.qlora_dropout, _drop(0.5)
    assert f(None, _fake(), 8, 0, d, S) == 1 and f(_fake(), None, 8, 0, d, S) == 1 and f(_fake(), _fake(), 8, 0, None, S) == 1
    assert f(_fake(), _fake(), -1, 0, d, S) == 2
    assert f(_fake(0x10008), _fake(), 8, 0, d, S) == 3 and f(_fake(), _fake(0x10004), 8, 0, d, S) == 3
    for t in (-1, 3):
        assert f(_fake(), _fake(), 8, t, d, S) == 4
    for p in (-1e-9, 1.0, math.nan, 1 - 2.0**-18):
        assert f(_fake(), _fake(), 8, 0, _drop(p), S) == 4


def test_workspace_query(lib):
    ws = binding.grouped_workspace_bytes
    assert ws(4, 16, 96, 128, 8) == 0 and ws(0, 16, 128, 128, 8) == 0 and ws(4, -1, 128, 128, 8) == 0
    assert ws(4, 16, 128, 128, 12) == 0 and ws(1025, 16, 128, 128, 8) == 0
    assert ws(4, 0, 128, 128, 8) > 0
    plain = ws(4, 1000, 1024, 2048, 8)
    assert plain >= 2 * 1000 * 8 * 2
    # no call keeps the mask and X is never copied: with few tiles dropout needs no scratch of its own
    assert ws(4, 1000, 1024, 2048, 8, True) == plain
    # many rows and experts: a bit for each element, from dX to dA
    assert ws(8, 1000, 4096, 11008, 8, True) == ws(8, 1000, 4096, 11008, 8) + 1000 * 11008 // 8


def test_binding_refusals(lib):
    """Types, shapes and devices are checked before the library is called."""
    E, T, N, K, r = 2, 8, 64, 64, 8
    bf = torch.bfloat16
    good = dict(packed=torch.zeros(E * N * K // 2, dtype=torch.uint8), q=torch.zeros(E * N * K // 64, dtype=torch.uint8),
                scale2=torch.zeros(1), X=torch.zeros(T, K, dtype=bf), offsets=torch.zeros(E + 1, dtype=torch.int32),
                A=torch.zeros(E, K, r, dtype=bf), B=torch.zeros(E, r, N, dtype=bf), alpha=1.0, N=N, K=K)
    with pytest.raises(ValueError, match="CUDA"):
        binding.grouped_linear_fwd(**good)
    with pytest.raises(TypeError):
        binding.grouped_linear_fwd(**{**good, "X": torch.zeros(T, K)})
    with pytest.raises(ValueError, match="shape"):
        binding.grouped_linear_fwd(**{**good, "A": torch.zeros(K, r, dtype=bf)})
    with pytest.raises(ValueError, match="shape"):
        binding.linear_fwd(good["packed"], good["q"], good["scale2"], good["X"], good["A"], good["B"], 1.0, N, K,
                           dropout=binding.Dropout(0.1, 0))
    with pytest.raises(TypeError):
        binding.dropout(torch.zeros(8, dtype=torch.float64), binding.Dropout(0.1, 0))
    with pytest.raises(ValueError, match="CUDA"):
        binding.dropout(torch.zeros(8), binding.Dropout(0.1, 0))
    # any Python integers are taken mod 2^64
    d = binding.Dropout(0.25, -1, 2**64 + 5)._desc()
    assert (d.p, d.seed, d.offset) == (0.25, 2**64 - 1, 5)


def test_grouped_plan_covers_every_tile(tmp_path):
    exe = tmp_path / "grouped_plan_check"
    src = os.path.join(ROOT, "tests", "host", "grouped_plan_check.cu")
    subprocess.check_call([nvcc(), *ARCH, "-O1", "-std=c++17", "-I", os.path.join(ROOT, "include"), "-I", CSRC,
                           "-o", str(exe), src], timeout=600)
    p = subprocess.run([str(exe)], capture_output=True, text=True, timeout=600)
    assert p.returncode == 0 and p.stdout.strip() == "ok", p.stdout + p.stderr

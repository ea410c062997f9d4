"""Pins of the grouped/dropout oracle (CPU): Philox against the published
known answers, the mask's frequency and independence of the tensor's size, and
the backward formulas against central differences of the forward."""
import numpy as np
import pytest

from oracle import grouped as og


def _block(ctr, key):
    return [int(v) for v in og._rounds([np.array([c], np.uint64) for c in ctr], *key)[0]]


def test_philox_known_answers():
    # the known-answer vectors published with the generator (philox 4x32, 10 rounds)
    assert _block([0, 0, 0, 0], (0, 0)) == [0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8]
    f = 0xFFFFFFFF
    assert _block([f, f, f, f], (f, f)) == [0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD]
    assert _block([0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344], (0xA4093822, 0x299F31D0)) == \
        [0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1]


@pytest.mark.parametrize("p", [0.0, 0.05, 0.1, 0.5, 0.999])
def test_keep_frequency(p):
    n = 1 << 20
    keep = og.keep_mask(n, p, seed=1234567890123, offset=77)
    q = 1.0 - og.threshold(p) / 65536.0
    # five standard deviations of a binomial share
    assert abs(keep.mean() - q) <= 5 * np.sqrt(q * (1 - q) / n) + 1e-12
    assert abs(og.factor(p) * q - 1.0) < 1e-15


def test_mask_is_a_function_of_the_element():
    a = og.keep_mask(4096, 0.3, 5, 9)
    assert np.array_equal(a[:1001], og.keep_mask(1001, 0.3, 5, 9))
    assert np.array_equal(a[1024:], og.keep_mask(4096 - 1024, 0.3, 5, 9, first=1024))
    assert np.array_equal(a[8 * 10:], og.keep_mask(4096 - 80, 0.3, 5, 19))
    assert not np.array_equal(a, og.keep_mask(4096, 0.3, 6, 9))
    # the counter wraps mod 2^64
    w = og.keep_mask(64, 0.5, 5, 2**64 - 4)
    assert np.array_equal(w[32:], og.keep_mask(32, 0.5, 5, 0))


@pytest.mark.parametrize("drop", [None, (0.25, 11, 3)])
def test_backward_formulas_against_differences(drop):
    rng = np.random.default_rng(0)
    off, E, N, K, r, alpha = [1, 4, 4, 9], 3, 5, 8, 2, 3.0
    X, W = rng.normal(size=(10, K)), rng.normal(size=(E, N, K))
    A, B, dY = rng.normal(size=(E, K, r)), rng.normal(size=(E, r, N)), rng.normal(size=(10, N))

    def loss(X, A, B):
        Y, _ = og.grouped_fwd(X, W, off, A, B, alpha, drop)
        return float(np.nansum(Y * dY))

    dX, dA, dB = og.grouped_bwd(X, dY, W, off, A, B, alpha, None, drop)
    assert np.isnan(dX[0]).all() and np.isnan(dX[9]).all()
    assert not dA[1].any() and not dB[1].any()  # the expert without rows
    h = 1e-6
    for args, grad, i in (((X, A, B), dX, 0), ((X, A, B), dA, 1), ((X, A, B), dB, 2)):
        for _ in range(12):
            at = tuple(rng.integers(0, n) for n in grad.shape)
            plus, minus = [a.copy() for a in args], [a.copy() for a in args]
            plus[i][at] += h
            minus[i][at] -= h
            want = 0.0 if np.isnan(grad[at]) else grad[at]
            assert abs((loss(*plus) - loss(*minus)) / (2 * h) - want) <= 1e-6 * (1 + abs(want))

"""Pins of the oracle's 8-bit cache functions: worked examples, closed forms
and invariants (no GPU)."""
import math

import numpy as np
import pytest

from oracle import flashsvd_oracle as oracle


@pytest.mark.parametrize("fmt,lim", [("int8", 127.0), ("e4m3", 448.0)])
def test_exponent_is_the_least_that_fits(fmt, lim):
    for amax in (1e-20, 0.3, 1.0, lim / 4, lim, lim * 1.0001, 3e38):
        e = oracle.kv8_exponent(amax, fmt)
        assert amax <= lim * 2.0 ** e
        assert amax > lim * 2.0 ** (e - 1)
    assert oracle.kv8_exponent(0.0, fmt) == -100
    assert oracle.kv8_exponent(lim, fmt) == 0


def test_int8_codes_worked():
    rows = np.zeros((64, 64))
    rows[0, :6] = [127.0, 0.5, 1.5, 2.5, -0.5, -1.5]
    codes, s = oracle.kv8_block(rows, "int8")
    assert s == 1.0
    assert codes[0, :6].tolist() == [127.0, 0.0, 2.0, 2.0, 0.0, -2.0]


def test_e4m3_codes_worked():
    # 448 = 1.75 * 2^8; spacing 32 there, 1/8 in [1, 2), 2^-9 below 2^-6
    y = np.array([448.0, 431.9, 1.0625, 1.1875, 2.0 ** -9, 2.0 ** -10, 3 * 2.0 ** -10, 0.0])
    assert oracle.kv8_round(y, "e4m3").tolist() == [448.0, 416.0, 1.0, 1.25, 2.0 ** -9, 0.0, 2.0 ** -8, 0.0]


def test_e4m3_codes_match_the_format():
    """Every number of the format is a fixed point, and every midpoint of two
    neighbours goes to the one with an even last bit."""
    vals = sorted({(m / 8 + (e > 0)) * 2.0 ** (max(e, 1) - 7) for e in range(16) for m in range(8)} - {480.0})
    vals = np.array(vals)
    assert np.array_equal(oracle.kv8_round(vals, "e4m3"), vals)
    mid = (vals[:-1] + vals[1:]) / 2
    even = np.where(np.arange(len(mid)) % 2 == 0, vals[:-1], vals[1:])
    assert np.array_equal(oracle.kv8_round(mid, "e4m3"), even)


@pytest.mark.parametrize("fmt,step", [("int8", 0.5), ("e4m3", 16.0)])
def test_rows_within_half_a_step_and_bf16(fmt, step):
    rng = np.random.default_rng(3)
    rows = rng.standard_normal((150, 64)).astype(np.float32)
    rows = (rows.view(np.uint32) & 0xFFFF0000).view(np.float32).astype(np.float64)
    got = oracle.kv8_rows(rows, fmt)
    assert np.array_equal(got[128:], rows[128:])          # the newest block as it is
    for b in range(2):
        sl = slice(64 * b, 64 * b + 64)
        s = 2.0 ** oracle.kv8_exponent(np.abs(rows[sl]).max(), fmt)
        assert np.max(np.abs(got[sl] - rows[sl])) <= step * s
    bits = got.astype(np.float32).view(np.uint32)
    assert not np.any(bits & 0xFFFF)                      # values are bf16 numbers
    assert np.array_equal(oracle.kv8_rows(got, fmt), got)  # and fixed points
    # 64 tokens: one block, and it is the newest
    assert np.array_equal(oracle.kv8_rows(rows[:64], fmt), rows[:64])


def test_non_finite_block():
    rows = np.ones((64, 64))
    rows[5, 5] = np.inf
    codes, s = oracle.kv8_block(rows, "int8")
    assert math.isnan(s) and not codes.any()


def test_weight_sums_closed_forms():
    n, D = 7, 4
    q = np.zeros((n, 2, D))                                # equal scores: query i gives 1/(i+1)
    k = np.random.default_rng(0).standard_normal((n, D))
    w = oracle.attn_weight_sums(q, k, n, 1.0)
    want = [2 * sum(1.0 / (i + 1) for i in range(j, n)) for j in range(n)]
    assert np.allclose(w, want, atol=1e-12)
    assert math.isclose(w.sum(), 2 * n)                    # every query hands out one
    w = oracle.attn_weight_sums(q, k, 1, 1.0)
    assert np.allclose(w, 2.0 / n, atol=1e-12)
    # one key takes everything
    q = np.ones((n, 1, D))
    k = np.zeros((n, D))
    k[2] = 1000.0
    w = oracle.attn_weight_sums(q, k, 3, 1.0)
    assert np.allclose(w, [0, 0, 3, 0, 0, 0, 0], atol=1e-12)


def test_evict_kept_worked():
    w = [0.5, 2.0, 2.0, math.nan, 0.0, 2.0, 9.0, 1.0]
    assert oracle.evict_kept(w, 8, 2).tolist() == list(range(8))
    assert oracle.evict_kept(w, 4, 2).tolist() == [1, 2, 6, 7]
    assert oracle.evict_kept(w, 4, 0).tolist() == [1, 2, 5, 6]
    assert oracle.evict_kept(w, 3, 3).tolist() == [5, 6, 7]
    assert oracle.evict_kept(w, 7, 1).tolist() == [0, 1, 2, 4, 5, 6, 7]  # NaN goes first
    assert oracle.evict_kept([0.0, -0.0, 0.0, -1.0, 1.0], 3, 1).tolist() == [0, 1, 4]

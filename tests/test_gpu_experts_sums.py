"""The rows products keep fp32 sums, whatever the operands and whichever kernel a shape selects.

Where large products cancel, what stands beside them has to remain: pairs of 448 * 448 of opposite sign are planted
next to each other among small whole numbers.  Scales are 2^-1..2^1, so every value is a multiple of 2^-2 and a pair's
products are at most 448 * 448 * 2^2 < 2^20: with at most four pairs under way at a time every partial sum is a
multiple of 2^-2 below 2^22, exact in fp32 in any order, and the results are compared bit for bit.

Real values are compared under K * 2^-23 of the sum of magnitudes (K additions in fp32, each off by at most a step
whichever way the adder rounds) plus half a bf16 step, 2^-8, for the one rounding of the result.
"""
import numpy as np
import pytest

import oracle.experts_oracle as X
from gpu_common import say
from test_gpu_experts import BF16_STEP, F32_ADD, gemm_values, operands, run_gemm, to_bf16

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

# 16-row and 32-row tiles, 128-row and 256-row ones, last rounds shared by two workgroups
SHAPES = [([3, 0, 14], 72, 264), ([200, 0, 40, 3, 16, 17, 32, 33, 64], 520, 264), ([300, 0, 40, 3, 500], 1544, 392),
          ([700, 0, 300, 211], 8200, 392), ([2600, 300], 6152, 264)]


def zero(a):
    return np.where(a == 0x8000, 0, a)


@pytest.mark.parametrize("loads,N,K", SHAPES)
def test_what_stands_beside_cancelling_products_remains(loads, N, K):
    say(f"cancelling products loads={loads} N={N} K={K}")
    rng = np.random.default_rng([N, K, 77])
    seg, q, qs, w, ws = operands(rng, loads, N, K, whole=True)
    big, minus = X.to_e4m3(np.array([448.0, -448.0]))
    for k in (0, 43, 126, K - 2):   # both of a pair in one block, so under one scale
        q[:, k], q[:, k + 1] = big, minus
        w[:, :, k] = w[:, :, k + 1] = big
    got = run_gemm(seg, q, qs, w, ws, N, K)
    want, _ = to_bf16(X.expert_gemm(*gemm_values(seg, q, qs, w, ws), seg.off) + 0.0)
    assert np.array_equal(zero(got[:seg.rows]), zero(want))
    assert (got[seg.rows:] == 0x7FC1).all()


@pytest.mark.parametrize("loads,N,K", SHAPES)
def test_real_values_with_missing_weights_a_nan_and_a_cut(loads, N, K):
    say(f"real values loads={loads} N={N} K={K}")
    rng = np.random.default_rng([N, K, 78])
    seg, q, qs, w, ws = operands(rng, loads, N, K, whole=False)
    nan, cap, hole = 1, seg.rows - 3, len(loads) - 1
    q[nan, K - 1] = 0x7F
    got = run_gemm(seg, q, qs, w, ws, N, K, cap=cap, holes=(hole,))
    q[nan, K - 1] = 0
    x, wv = gemm_values(seg, q, qs, w, ws)
    want = X.expert_gemm(x, wv, seg.off)[:cap]
    mag = X.expert_gemm(np.abs(x), [np.abs(v) for v in wv], seg.off)[:cap]
    val = (got.astype(np.uint32) << 16).view(np.float32).astype(np.float64)
    slack = K * F32_ADD * mag
    ok = np.abs(val - want) <= slack + BF16_STEP * (np.abs(want) + slack)
    ok[nan] = np.isnan(val[nan])
    ok[seg.off[hole]:] = got[seg.off[hole]:] == 0x7FC1
    assert ok.all()


@pytest.mark.parametrize("loads,N", [([3, 0, 14], 72), ([300, 0, 40, 3, 500], 1544), ([700, 0, 300, 211], 8200)])
def test_scale_bytes_behind_the_last_block_are_not_used(loads, N):
    """K = 264 has three scales a row and a byte of padding, here the one that stands for no number."""
    K = 264
    rng = np.random.default_rng([N, 79])
    seg, q, qs, w, ws = operands(rng, loads, N, K, whole=True)
    want, _ = to_bf16(X.expert_gemm(*gemm_values(seg, q, qs, w, ws), seg.off) + 0.0)
    qs[:, 3:], ws[:, :, 3:] = 255, 255
    got = run_gemm(seg, q, qs, w, ws, N, K)
    assert np.array_equal(zero(got[:seg.rows]), zero(want))


@pytest.mark.parametrize("rows_at,weights_at", [(1, 230), (245, 20)])
@pytest.mark.parametrize("loads,N,K", SHAPES[:4])
def test_scales_at_the_ends_of_their_range(loads, N, K, rows_at, weights_at):
    """Values of 2^-126 to 2^120: still bf16 numbers of the normal range, so the whole numbers' results stay exact."""
    rng = np.random.default_rng([N, K, rows_at])
    seg, q, qs, w, ws = operands(rng, loads, N, K, whole=True)
    qs[:], ws[:] = qs - 126 + rows_at, ws - 126 + weights_at
    got = run_gemm(seg, q, qs, w, ws, N, K)
    want, _ = to_bf16(X.expert_gemm(*gemm_values(seg, q, qs, w, ws), seg.off) + 0.0)
    assert np.array_equal(zero(got[:seg.rows]), zero(want))

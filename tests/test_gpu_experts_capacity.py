"""Buffers for many more rows than came, and more experts than a wave has lanes, on every kind of tile.

The number of rows is known on the device only, so a program that does not wait for it passes what could come at most.
Small whole numbers: every sum is exact in fp32, so results are compared bit for bit whatever the kernel."""
import numpy as np
import pytest

import moe_expert_load_ultraep_amd as U
import oracle.experts_oracle as X
from gpu_common import say
from test_gpu_experts import DEV, SENT, Segment, bytes_like, columns, dev, gemm_values, operands, run_gemm, same_bytes, special_rows, to_bf16

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


def zero(a):
    return np.where(a == 0x8000, 0, a)


def check_gemm(loads, N, K, cap):
    rng = np.random.default_rng([N, K, sum(loads), cap])
    seg, q, qs, w, ws = operands(rng, loads, N, K, whole=True)
    got = run_gemm(seg, q, qs, w, ws, N, K, cap=cap)
    want, _ = to_bf16(X.expert_gemm(*gemm_values(seg, q, qs, w, ws), seg.off) + 0.0)
    n = min(cap, seg.rows)
    assert np.array_equal(zero(got[:n]), zero(want[:n]))
    assert (got[n:] == 0x7FC1).all()


@pytest.mark.parametrize("cap", [24, 700, 5000, 40000])
@pytest.mark.parametrize("loads,N,K", [([3, 0, 14, 1], 1544, 264), ([0, 0, 0, 1], 264, 136), ([140, 0, 0, 300, 5], 1288, 392)])
def test_expert_gemm_with_a_loose_capacity(loads, N, K, cap):
    say(f"loose capacity loads={loads} N={N} K={K} cap={cap}")
    check_gemm(loads, N, K, cap)


# 128-row tiles, whole ones and ragged ones, and with more than 64 experts; 256-row tiles of them too
@pytest.mark.parametrize("loads,N,K", [([256, 128, 128], 2056, 264), ([7, 0, 130, 40] * 20, 1544, 136), ([1] * 70 + [900] + [3] * 9, 1800, 264),
                                       ([0, 60, 257] * 25, 4104, 136)])
def test_expert_gemm_of_many_experts(loads, N, K):
    say(f"many experts={len(loads)} rows={sum(loads)} N={N} K={K}")
    check_gemm(loads, N, K, sum(loads) + 2)


@pytest.mark.parametrize("cap", [50, 3000])
def test_quantisers_and_weight_gradients_with_a_loose_capacity(cap):
    loads, N, K = [17, 0, 30], 136, 72
    rng = np.random.default_rng(cap)
    seg = Segment(loads, p0=1)
    blocks = U.quant_blocks(cap, seg.ne)
    src, val = special_rows(rng, cap, K)
    q, qs = bytes_like((cap, U.quant_pitch(K))), bytes_like((cap, U.quant_scale_pitch(K)))
    qt, qts = bytes_like((blocks, K, 128)), bytes_like((blocks, K))
    U.ultraep_permute_quant(seg.ctx, seg.plan, None, 1, dev(src), seg.p0, seg.p1, q, qs, qt, qts)
    torch.cuda.synchronize()
    wq, wqs = X.quant_rows(val[:seg.rows])
    wqt, wqts = X.quant_cols(val[:seg.rows], seg.off, blocks, fill=SENT)
    same_bytes(q.cpu().numpy()[:seg.rows], wq)
    same_bytes(qt.cpu().numpy(), wqt)
    assert np.array_equal(qs.cpu().numpy()[:seg.rows], wqs) and np.array_equal(qts.cpu().numpy(), wqts)
    assert bool((q[seg.rows:] == SENT).all()) and bool((qs[seg.rows:] == SENT).all())

    seg.blocks = blocks                                 # blocks of nobody hold NaN and scales of 200
    dyt, dys = columns(rng, seg, N, True)
    xt, xs = columns(rng, seg, K, True)
    g = torch.full((seg.ne, N, K), 3.0, device=DEV)
    U.ultraep_expert_wgrad(seg.ctx, seg.plan, dev(dyt), dev(dys), N, dev(xt), dev(xs), K, seg.p0, seg.p1, cap, U.pointer_table(list(g)))
    torch.cuda.synchronize()
    for p, want in enumerate(X.expert_wgrad(dyt, dys, xt, xs, seg.off)):
        assert np.array_equal(g[p].cpu().numpy().astype(np.float64), want)


def test_weight_gradients_of_more_experts_than_lanes():
    rng = np.random.default_rng(70)
    seg = Segment([5, 0, 129, 40] * 20, p0=1)
    N, K = 264, 136
    dyt, dys = columns(rng, seg, N, True)
    xt, xs = columns(rng, seg, K, True)
    g = torch.full((seg.ne, N, K), 3.0, device=DEV)
    U.ultraep_expert_wgrad(seg.ctx, seg.plan, dev(dyt), dev(dys), N, dev(xt), dev(xs), K, seg.p0, seg.p1, seg.rows, U.pointer_table(list(g)))
    torch.cuda.synchronize()
    for p, want in enumerate(X.expert_wgrad(dyt, dys, xt, xs, seg.off)):
        assert np.array_equal(g[p].cpu().numpy().astype(np.float64), want), p

"""A rank that got no rows: exact-size buffers, some of which have no elements, and buffers for rows that did not come.

Nothing is written but the weight gradients, which are zeros."""
import pytest

import moe_expert_load_ultraep_amd as U
from gpu_common import say
from test_gpu_experts import DEV, SENT, Segment, bytes_like

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

N, K = 136, 264


def untouched(*tensors):
    return all(bool((t == SENT).all()) for t in tensors)


@pytest.mark.parametrize("loads", [[0, 0, 0], [0]], ids=len)
@pytest.mark.parametrize("cap", [0, 1, 40, 700])
def test_no_rows(cap, loads):
    say(f"no rows: cap={cap} experts={len(loads)}")
    seg = Segment(loads, p0=1)
    blocks = U.quant_blocks(cap, seg.ne)
    q, qs = bytes_like((cap, U.quant_pitch(K))), bytes_like((cap, U.quant_scale_pitch(K)))
    qt, qts = bytes_like((blocks, K, 128)), bytes_like((blocks, K))
    for tokens in (0, 5):
        hidden = torch.ones(tokens, K, dtype=torch.bfloat16, device=DEV)
        for inv in (None, torch.zeros(0, dtype=torch.int32, device=DEV), torch.zeros(9, dtype=torch.int32, device=DEV)):
            args = (seg.ctx, seg.plan, inv, 2, hidden, seg.p0, seg.p1)
            U.ultraep_permute_quant(*args, q, qs)
            U.ultraep_permute_quant(*args, q, qs, qt, qts)
            U.ultraep_permute_quant(*args, qt=qt, qt_scale=qts, rows=cap)
    w = torch.zeros(seg.ne, N, U.quant_pitch(K), dtype=torch.uint8, device=DEV)
    ws = torch.full((seg.ne, 2, U.quant_scale_pitch(K)), 127, dtype=torch.uint8, device=DEV)
    out = torch.full((cap, N), SENT, dtype=torch.int16, device=DEV)
    U.ultraep_expert_gemm(seg.ctx, seg.plan, q, qs, K, U.pointer_table(list(w)), U.pointer_table(list(ws)), N, seg.p0, seg.p1, out)
    dyt, dyts = bytes_like((blocks, N, 128)), bytes_like((blocks, N))
    grads = torch.full((seg.ne, N, K), 3.0, device=DEV)
    table = U.pointer_table(list(grads))
    U.ultraep_expert_wgrad(seg.ctx, seg.plan, dyt, dyts, N, qt, qts, K, seg.p0, seg.p1, cap, table, accumulate=True)
    torch.cuda.synchronize()
    assert untouched(q, qs, qt, qts, out) and bool((grads == 3.0).all())
    U.ultraep_expert_wgrad(seg.ctx, seg.plan, dyt, dyts, N, qt, qts, K, seg.p0, seg.p1, cap, table)
    torch.cuda.synchronize()
    assert bool((grads == 0.0).all())


def test_no_experts():
    seg = Segment([3, 4], p0=1)
    none = torch.zeros(0, dtype=torch.int64, device=DEV)
    at = (seg.p0, seg.p0)
    hidden = torch.ones(2, K, dtype=torch.bfloat16, device=DEV)
    qt, qts = bytes_like((0, K, 128)), bytes_like((0, K))
    dyt, dyts = bytes_like((0, N, 128)), bytes_like((0, N))
    q, qs = bytes_like((9, U.quant_pitch(K))), bytes_like((9, U.quant_scale_pitch(K)))
    out = torch.full((9, N), SENT, dtype=torch.int16, device=DEV)
    U.ultraep_permute_quant(seg.ctx, seg.plan, None, 1, hidden, *at, q, qs, qt, qts)
    U.ultraep_expert_gemm(seg.ctx, seg.plan, q, qs, K, none, none, N, *at, out)
    U.ultraep_expert_wgrad(seg.ctx, seg.plan, dyt, dyts, N, qt, qts, K, *at, 9, none)
    wq, wqs = bytes_like((0, N, U.quant_pitch(K))), bytes_like((0, 2, U.quant_scale_pitch(K)))
    U.ultraep_weight_quant(seg.ctx, none, 0, N, K, wq, wqs)
    torch.cuda.synchronize()
    assert untouched(q, qs, out)


def test_no_source_rows():
    """Rows whose tokens are elsewhere: zeros, with no source at all."""
    seg = Segment([130, 7], p0=1)
    hidden = torch.ones(0, K, dtype=torch.bfloat16, device=DEV)
    inv = torch.arange(200, dtype=torch.int32, device=DEV)
    blocks = U.quant_blocks(seg.rows, seg.ne)
    for i in (None, inv):
        q, qs = bytes_like((seg.rows, U.quant_pitch(K))), bytes_like((seg.rows, U.quant_scale_pitch(K)))
        q2, qs2 = bytes_like(q.shape), bytes_like(qs.shape)
        qt, qts = bytes_like((blocks, K, 128)), bytes_like((blocks, K))
        U.ultraep_permute_quant(seg.ctx, seg.plan, i, 3, hidden, seg.p0, seg.p1, q, qs)
        U.ultraep_permute_quant(seg.ctx, seg.plan, i, 3, hidden, seg.p0, seg.p1, q2, qs2, qt, qts)
        torch.cuda.synchronize()
        assert bool((q == 0).all()) and bool((qs == 127).all()) and bool((q2 == 0).all()) and bool((qs2 == 127).all())
        # 130 rows in blocks 0 and 1, 7 rows in block 130 // 128 + 1
        assert blocks == 3 and bool((qt == 0).all()) and bool((qts == 127).all())

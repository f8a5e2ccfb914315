"""Calls over nothing (no GPU): a rank that got no rows, an empty range, no weights.

An array of no elements often has no address, so its pointer may be NULL; the same NULL is refused where the
array has elements."""
import os

import pytest

import moe_expert_load_ultraep_amd as U

pytestmark = pytest.mark.skipif(not os.path.exists(U.LIB_PATH), reason="libultraep.so not built")

F = 1 << 20   # never dereferenced


@pytest.fixture(scope="module")
def ctx():
    yield U.ultraep_create(8, 4, 1, 4)


def test_permute_quant_of_no_rows(ctx):
    def call(hid=F, n=10, p1=3, q=None, qs=None, qt=None, qts=None, cap=0, blocks=0, inv=None, k=0, H=16):
        return U.lib().ultraep_permute_quant(ctx.handle, F, inv, k, hid, n, H, 0, p1, q, qs, qt, qts, cap, blocks, None)

    assert call() == 0                                  # the rows form's buffers have no rows
    assert call(hid=None, n=0) == 0                     # nor has the source
    assert call(qt=F, qts=F, blocks=3) == 0             # the columns form keeps a block an expert
    assert call(p1=0, cap=100) == 0                     # no experts: no blocks below 128 rows
    assert call(p1=0, cap=100, hid=None, n=0) == 0
    for bad in (dict(hid=None), dict(cap=1), dict(cap=1, q=F), dict(cap=1, qs=F), dict(H=0), dict(n=-1), dict(p1=13),
                dict(qt=F, qts=F, blocks=2), dict(inv=F, k=0)):
        assert call(**bad) == -1, bad


def test_weight_quant_of_no_experts(ctx):
    call = lambda n, q=None: U.lib().ultraep_weight_quant(ctx.handle, None, n, 16, 24, q, q, None, None, None)  # noqa: E731
    assert call(0) == 0 and call(0, F) == 0
    assert call(1) == -1


def test_expert_gemm_of_no_rows(ctx):
    def call(q=None, qs=None, w=F, ws=F, out=None, p1=3, cap=0, N=16, K=64):
        return U.lib().ultraep_expert_gemm(ctx.handle, F, q, qs, K, w, ws, N, 0, p1, out, cap, None)

    assert call() == 0
    assert call(q=F, qs=F, out=F, w=None, ws=None, p1=0, cap=10) == 0
    full = dict(q=F, qs=F, out=F, cap=10)
    for name in ("q", "qs", "w", "ws", "out"):
        assert call(**{**full, name: None}) == -1, name
    assert call(N=0) == -1 and call(K=0) == -1 and call(p1=13) == -1 and call(N=12) == -2


def test_expert_wgrad_of_no_experts(ctx):
    def call(a=None, g=None, p1=0, cap=0, acc=0):
        return U.lib().ultraep_expert_wgrad(ctx.handle, F, a, a, 16, a, a, 24, 0, p1, cap, g, acc, None)

    assert call() == 0 and call(cap=100) == 0
    assert call(p1=3, g=F) == -1 and call(p1=3, a=F) == -1 and call(acc=2) == -1 and call(cap=-1) == -1

"""The steps around the experts on the host (no GPU): symbols and refusals.

Every call fails its argument check, or has nothing to do, before anything is
launched."""
import ctypes
import os
import re

import pytest

import moe_expert_load_ultraep_amd as U

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "ultraep_layer.h")
torch = pytest.importorskip("torch")
pytestmark = pytest.mark.skipif(not os.path.exists(U.LIB_PATH), reason="libultraep.so not built")

F = 1 << 20   # never dereferenced
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def ctx():
    c = U.ultraep_create(8, 4, 1, 4)   # 12 physical experts
    yield c


def test_library_exports_the_header():
    src = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = set(re.findall(r"\b(ultraep_[a-z_]+)\s*\(", src))
    assert names == set(U._LAYER_SIGNATURES)
    lib = ctypes.CDLL(U.LIB_PATH)
    for n in names:
        assert hasattr(lib, n), n


def test_header_constants():
    text = open(HEADER).read()
    for name, value in (("ROUTE_SOFTMAX", U.ROUTE_SOFTMAX), ("ROUTE_SIGMOID", U.ROUTE_SIGMOID), ("GLU_SILU", U.GLU_SILU),
                        ("GLU_GELU", U.GLU_GELU), ("MAX_ROUTE_GROUPS", U.MAX_ROUTE_GROUPS), ("MAX_NORM_WIDTH", U.MAX_NORM_WIDTH)):
        assert int(re.search(rf"ULTRAEP_{name} (\d+)", text).group(1)) == value


def test_route_refusals(ctx):
    def call(l=F, t=0, n=10, k=2, s=0, b=F, g=2, tg=1, top=2, r=1, sc=1.0, i=F, w=F, c=ctx.handle):
        return U.lib().ultraep_route(c, l, t, n, k, s, b, g, tg, top, r, sc, i, w, None)

    for bad in (dict(c=None), dict(l=None), dict(i=None), dict(w=None), dict(t=2), dict(t=-1), dict(n=-1), dict(k=0), dict(k=9),
                dict(s=2), dict(g=0), dict(g=3), dict(tg=0), dict(tg=3), dict(top=0), dict(top=3), dict(r=2), dict(sc=NAN), dict(sc=INF)):
        assert call(**bad) == -1, bad
    for bad in (dict(l=F + 2), dict(l=F + 1, t=1), dict(b=F + 2), dict(i=F + 2), dict(w=F + 1), dict(n=1 << 31)):
        assert call(**bad) == -2, bad
    assert call(n=0, l=None, i=None, w=None) == 0 and call(n=0, b=None) == 0
    wide = U.ultraep_create(128, 128, 0, 1)
    assert call(c=wide.handle, g=128, n=0) == -2 and call(c=wide.handle, k=65, n=0) == -1


def test_route_backward_refusals(ctx):
    def call(l=F, t=0, n=10, k=2, s=0, r=1, sc=1.0, i=F, w=F, o=F, c=ctx.handle):
        return U.lib().ultraep_route_backward(c, l, t, n, k, s, r, sc, i, w, o, None)

    for bad in (dict(c=None), dict(l=None), dict(i=None), dict(w=None), dict(o=None), dict(t=2), dict(n=-1), dict(k=0), dict(k=9),
                dict(s=-1), dict(r=2), dict(sc=NAN)):
        assert call(**bad) == -1, bad
    for bad in (dict(l=F + 2), dict(o=F + 2), dict(o=F + 1, t=1), dict(i=F + 2), dict(w=F + 1), dict(n=1 << 31)):
        assert call(**bad) == -2, bad
    assert call(n=0, l=None, i=None, w=None, o=None) == 0


def test_residual_norm_refusals(ctx):
    def call(x=F, r=F, rt=1, w=F, wt=0, e=1e-6, n=10, H=64, h=F, y=F, q=F, qs=F, v=F, c=ctx.handle):
        return U.lib().ultraep_residual_norm(c, x, r, rt, w, wt, e, n, H, h, y, q, qs, v, None)

    for bad in (dict(c=None), dict(x=None), dict(w=None), dict(r=None), dict(q=None), dict(qs=None), dict(rt=2), dict(wt=-1), dict(n=-1),
                dict(H=0), dict(e=-1e-6), dict(e=NAN), dict(e=INF), dict(h=None, y=None, q=None, qs=None, v=None)):
        assert call(**bad) == -1, bad
    for bad in (dict(H=12), dict(H=16392), dict(n=1 << 31), dict(x=F + 8), dict(r=F + 8), dict(w=F + 8), dict(h=F + 8), dict(y=F + 8),
                dict(q=F + 8), dict(qs=F + 2), dict(v=F + 2)):
        assert call(**bad) == -2, bad
    assert call(n=0, x=None, r=None, w=None, h=None, y=None, q=None, qs=None, v=None) == 0


def test_residual_norm_backward_refusals(ctx):
    size = ctypes.c_size_t()
    assert U.lib().ultraep_residual_norm_workspace_bytes(10, 64, ctypes.byref(size)) == 0
    need = size.value

    def call(g=F, h=F, ht=0, w=F, wt=0, v=F, gi=F, n=10, H=64, gh=F, gx=F, gw=F, acc=0, ws=F, b=need, c=ctx.handle):
        return U.lib().ultraep_residual_norm_backward(c, g, h, ht, w, wt, v, gi, n, H, gh, gx, gw, acc, ws, b, None)

    for bad in (dict(c=None), dict(g=None), dict(h=None), dict(w=None), dict(v=None), dict(gh=None), dict(ws=None), dict(ht=1), dict(ht=2),
                dict(wt=2), dict(n=-1), dict(H=-8), dict(acc=2)):
        assert call(**bad) == -1, bad
    for bad in (dict(H=12), dict(H=16392), dict(n=1 << 31), dict(g=F + 8), dict(h=F + 8), dict(w=F + 8), dict(v=F + 2), dict(gi=F + 8),
                dict(gh=F + 8), dict(gx=F + 8), dict(gw=F + 8), dict(ws=F + 8)):
        assert call(**bad) == -2, bad
    assert call(b=need - 1) == -4
    assert call(n=0, g=None, h=None, w=None, v=None, gi=None, gh=None, gx=None, gw=None, ws=None) == 0
    for n, H, status in ((-1, 64, -1), (1, 0, -1), (1, 12, -2), (1, 16392, -2), (1 << 31, 64, -2)):
        assert U.lib().ultraep_residual_norm_workspace_bytes(n, H, ctypes.byref(size)) == status
    assert U.lib().ultraep_residual_norm_workspace_bytes(1, 64, None) == -1
    assert U.residual_norm_workspace_bytes(10, 64) == need
    with pytest.raises(U.UltraEPError):
        U.residual_norm_workspace_bytes(-1, 64)


def test_glu_refusals(ctx):
    def call(plan=F, h=F, w=64, act=0, p0=0, p1=3, q=F, qs=F, qt=F, qts=F, cap=300, blocks=5, c=ctx.handle):
        return U.lib().ultraep_glu_quant(c, plan, h, w, act, p0, p1, q, qs, qt, qts, cap, blocks, None)

    def back(plan=F, h=F, g=F, w=64, act=0, p0=0, p1=3, q=F, qs=F, qt=F, qts=F, cap=300, blocks=5, c=ctx.handle):
        return U.lib().ultraep_glu_quant_backward(c, plan, h, g, w, act, p0, p1, q, qs, qt, qts, cap, blocks, None)

    for f in (call, back):
        for bad in (dict(c=None), dict(plan=None), dict(h=None), dict(q=None), dict(qs=None), dict(qt=None), dict(qts=None),
                    dict(q=None, qs=None, qt=None, qts=None), dict(w=0), dict(act=2), dict(cap=-1), dict(p0=-1), dict(p0=4), dict(p1=13),
                    dict(blocks=4)):
            assert f(**bad) == -1, bad
        for bad in (dict(w=12), dict(w=(1 << 22) + 8), dict(h=F + 8), dict(q=F + 8), dict(qs=F + 2), dict(qt=F + 8), dict(plan=F + 2),
                    dict(cap=1 << 31, blocks=1 << 40)):
            assert f(**bad) == -2, bad
        assert f(cap=0, h=None, q=None, qs=None, qt=None, qts=None) == 0 and f(p1=0, blocks=2) == 0
    assert back(g=None) == -1 and back(g=F + 8) == -2 and back(g=None, cap=0) == 0


def test_binding_refuses_host_tensors_and_wrong_types(ctx):
    plan = torch.zeros(ctx.plan_words, dtype=torch.int32)
    l, i, w = torch.zeros(4, 8), torch.zeros(4, 2, dtype=torch.int32), torch.zeros(4, 2)
    x, one = torch.zeros(4, 64, dtype=torch.bfloat16), torch.zeros(64)
    q, s = torch.zeros(4, 128, dtype=torch.uint8), torch.zeros(4, 4, dtype=torch.uint8)
    for f in (lambda: U.ultraep_route(ctx, l, 2, i, w), lambda: U.ultraep_route(ctx, l.double(), 2, i, w),
              lambda: U.ultraep_route(ctx, None, 2, i, w), lambda: U.ultraep_route_backward(ctx, l, 2, i, w, l),
              lambda: U.ultraep_residual_norm(ctx, x, one, 1e-6, y=x), lambda: U.ultraep_residual_norm(ctx, x, one.half(), 1e-6, y=x),
              lambda: U.ultraep_residual_norm(ctx, x, one, 1e-6, q=q), lambda: U.ultraep_residual_norm(ctx, None, one, 1e-6, y=x),
              lambda: U.ultraep_residual_norm_backward(ctx, x, x, one, one[:4], x),
              lambda: U.ultraep_residual_norm_backward(ctx, x, None, one, one[:4], x),
              lambda: U.ultraep_glu_quant(ctx, plan, x, 0, 3, q, s), lambda: U.ultraep_glu_quant(ctx, plan, x, 0, 3, q),
              lambda: U.ultraep_glu_quant(ctx, plan, None, 0, 3, q, s), lambda: U.ultraep_glu_quant(ctx, plan, x, 0, 3, q, s, rows=5),
              lambda: U.ultraep_glu_quant_backward(ctx, plan, x, x, 0, 3, q, s)):
        with pytest.raises(U.UltraEPError) as ei:
            f()
        assert ei.value.status == -1

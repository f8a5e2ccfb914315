"""The experts' entry points on the host (no GPU): symbols and refusals.

Every call fails its argument check, or has nothing to do, before anything is
launched."""
import ctypes
import os
import re

import pytest

import moe_expert_load_ultraep_amd as U

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "ultraep_experts.h")
torch = pytest.importorskip("torch")
pytestmark = pytest.mark.skipif(not os.path.exists(U.LIB_PATH), reason="libultraep.so not built")

F = 1 << 20   # never dereferenced


@pytest.fixture(scope="module")
def ctx():
    c = U.ultraep_create(8, 4, 1, 4)   # 12 physical experts
    yield c


def test_library_exports_the_header():
    src = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = set(re.findall(r"\b(ultraep_[a-z_]+)\s*\(", src))
    assert names == set(U._EXPERT_SIGNATURES)
    lib = ctypes.CDLL(U.LIB_PATH)
    for n in names:
        assert hasattr(lib, n), n


def test_header_constants():
    text = open(HEADER).read()
    for name, value in (("QUANT_BLOCK", U.QUANT_BLOCK), ("MAX_GRAD_TENSORS", U.MAX_GRAD_TENSORS),
                        ("GRAD_WORKSPACE_BYTES", U.GRAD_WORKSPACE_BYTES)):
        assert int(re.search(rf"ULTRAEP_{name} (\d+)", text).group(1)) == value
    assert U.quant_pitch(129) == 256 and U.quant_scale_pitch(128) == 4 and U.quant_scale_pitch(513) == 8
    assert U.quant_blocks(0, 3) == 3 and U.quant_blocks(256, 3) == 5


def test_permute_quant_refusals(ctx):
    def call(plan=F, inv=F, k=2, hid=F, n=10, H=16, p0=0, p1=3, q=F, qs=F, qt=F, qts=F, cap=300, blocks=5, c=ctx.handle):
        return U.lib().ultraep_permute_quant(c, plan, inv, k, hid, n, H, p0, p1, q, qs, qt, qts, cap, blocks, None)

    for bad in (dict(c=None), dict(plan=None), dict(hid=None), dict(qs=None), dict(q=None), dict(qt=None), dict(qts=None),
                dict(q=None, qs=None, qt=None, qts=None), dict(H=0), dict(n=-1), dict(cap=-1), dict(p0=-1), dict(p0=4),
                dict(p1=13), dict(k=0), dict(k=65), dict(blocks=4)):
        assert call(**bad) == -1, bad
    for bad in (dict(H=12), dict(H=(1 << 24) + 8), dict(hid=F + 8), dict(q=F + 4), dict(qs=F + 2), dict(qt=F + 8),
                dict(inv=F + 1), dict(plan=F + 2), dict(cap=1 << 31, blocks=1 << 40)):
        assert call(**bad) == -2, bad
    assert call(cap=0) == 0 and call(p1=0) == 0 and call(inv=None, k=0, cap=0) == 0


def test_weight_quant_refusals(ctx):
    def call(w=F, n=2, N=16, K=24, q=F, qs=F, qt=F, qts=F, c=ctx.handle):
        return U.lib().ultraep_weight_quant(c, w, n, N, K, q, qs, qt, qts, None)

    for bad in (dict(c=None), dict(w=None), dict(n=-1), dict(N=0), dict(K=0), dict(qs=None), dict(qt=None),
                dict(q=None, qs=None, qt=None, qts=None)):
        assert call(**bad) == -1, bad
    for bad in (dict(N=12), dict(K=12), dict(N=(1 << 20) + 8), dict(n=1025), dict(w=F + 4), dict(q=F + 8), dict(qts=F + 2)):
        assert call(**bad) == -2, bad
    assert call(n=0, w=None) == 0


def test_expert_gemm_refusals(ctx):
    def call(plan=F, q=F, qs=F, K=64, w=F, ws=F, N=16, p0=0, p1=3, out=F, cap=10, c=ctx.handle):
        return U.lib().ultraep_expert_gemm(c, plan, q, qs, K, w, ws, N, p0, p1, out, cap, None)

    for bad in (dict(c=None), dict(plan=None), dict(q=None), dict(qs=None), dict(w=None), dict(ws=None), dict(out=None),
                dict(K=0), dict(N=0), dict(cap=-1), dict(p0=-1), dict(p0=4), dict(p1=13)):
        assert call(**bad) == -1, bad
    for bad in (dict(N=12), dict(K=(1 << 20) + 8), dict(q=F + 8), dict(qs=F + 1), dict(w=F + 4), dict(ws=F + 4),
                dict(out=F + 8), dict(cap=1 << 31), dict(cap=1 << 30, N=1 << 20)):
        assert call(**bad) == -2, bad
    assert call(cap=0) == 0 and call(p0=2, p1=2) == 0


def test_expert_wgrad_refusals(ctx):
    def call(plan=F, dy=F, dys=F, N=16, x=F, xs=F, K=24, p0=0, p1=3, cap=10, g=F, acc=0, c=ctx.handle):
        return U.lib().ultraep_expert_wgrad(c, plan, dy, dys, N, x, xs, K, p0, p1, cap, g, acc, None)

    for bad in (dict(c=None), dict(plan=None), dict(dy=None), dict(dys=None), dict(x=None), dict(xs=None), dict(g=None),
                dict(N=0), dict(K=0), dict(cap=-1), dict(p1=13), dict(p0=4), dict(acc=2)):
        assert call(**bad) == -1, bad
    for bad in (dict(N=12), dict(K=12), dict(dy=F + 8), dict(x=F + 8), dict(g=F + 4),
                dict(cap=1 << 31), dict(K=(1 << 20) + 8), dict(N=1 << 20, K=1 << 20)):
        assert call(**bad) == -2, bad
    assert call(p0=2, p1=2) == 0


def test_grad_refusals(ctx):
    def norm(t=F, m=F, n=3, dt=0, s=F, acc=0, ws=F, b=16384, c=ctx.handle):
        return U.lib().ultraep_grad_sumsq(c, t, m, n, dt, s, acc, ws, b, None)

    for bad in (dict(c=None), dict(t=None), dict(m=None), dict(n=-1), dict(dt=2), dict(s=None), dict(acc=2), dict(ws=None)):
        assert norm(**bad) == -1, bad
    for bad in (dict(n=4097), dict(t=F + 4), dict(m=F + 4), dict(s=F + 4), dict(ws=F + 4)):
        assert norm(**bad) == -2, bad
    assert norm(b=16383) == -4

    def clip(t=F, m=F, n=3, dt=0, s=F, mx=1.0, nrm=F, out=None, c=ctx.handle):
        return U.lib().ultraep_grad_clip(c, t, m, n, dt, s, mx, nrm, out, None)

    for bad in (dict(c=None), dict(t=None), dict(m=None), dict(n=-1), dict(dt=-1), dict(s=None), dict(mx=-1.0),
                dict(mx=float("nan"))):
        assert clip(**bad) == -1, bad
    for bad in (dict(n=4097), dict(t=F + 4), dict(s=F + 4), dict(nrm=F + 2), dict(out=F + 4)):
        assert clip(**bad) == -2, bad


def test_binding_refuses_host_tensors_and_wrong_types(ctx):
    plan = torch.zeros(ctx.plan_words, dtype=torch.int32)
    hid = torch.zeros(4, 64, dtype=torch.bfloat16)
    q, s = torch.zeros(4, 128, dtype=torch.uint8), torch.zeros(4, 4, dtype=torch.uint8)
    table = torch.zeros(3, dtype=torch.int64)
    for f in (lambda: U.ultraep_permute_quant(ctx, plan, None, 1, hid, 0, 3, q, s),
              lambda: U.ultraep_permute_quant(ctx, plan, None, 1, hid, 0, 3, q),
              lambda: U.ultraep_weight_quant(ctx, table, 3, 64, 64, q, s),
              lambda: U.ultraep_expert_gemm(ctx, plan, q, s, 64, table, table, 64, 0, 3, hid),
              lambda: U.ultraep_expert_wgrad(ctx, plan, q, s, 64, q, s, 64, 0, 3, 4, table),
              lambda: U.ultraep_grad_sumsq(ctx, table, table, 3, torch.float16, q, q),
              lambda: U.ultraep_grad_clip(ctx, table, table, 3, torch.float32, q, 1.0)):
        with pytest.raises(U.UltraEPError) as ei:
            f()
        assert ei.value.status == -1


def test_binding_refuses_missing_buffers(ctx):
    table = torch.zeros(3, dtype=torch.int64)
    for f in (lambda: U.ultraep_permute_quant(ctx, table, None, 1, None, 0, 3, table, table),
              lambda: U.ultraep_permute_quant(ctx, None, None, 1, torch.zeros(4, 64), 0, 3, table, table),
              lambda: U.ultraep_weight_quant(ctx, None, 3, 64, 64, table, table),
              lambda: U.ultraep_expert_gemm(ctx, None, table, table, 64, table, table, 64, 0, 3, table),
              lambda: U.ultraep_expert_wgrad(ctx, None, table, table, 64, table, table, 64, 0, 3, 4, table),
              lambda: U.ultraep_grad_sumsq(ctx, None, table, 3, torch.float32, table, table),
              lambda: U.ultraep_grad_clip(ctx, None, table, 3, torch.float32, table, 1.0)):
        with pytest.raises(U.UltraEPError) as ei:
            f()
        assert ei.value.status == -1

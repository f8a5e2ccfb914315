"""Passes longer than the caches, which take kernels of their own (streaming ones), against the short ones and the
64-bit oracle.

The norm's rows and the activation's do not depend on the others, so a long call's rows are those of short calls, bit
for bit; the short calls' kernels are compared with the oracle here and elsewhere."""
import numpy as np
import pytest

import moe_expert_load_ultraep_amd as U
import oracle.experts_oracle as X
import oracle.layer_oracle as Y
from gpu_common import say
from test_gpu_experts import SENT, Segment, bytes_like
from test_gpu_layer import (BF16_STEP, F32_STEP, check_cols_form, check_rows_form, ctx_of, host, norm_blocks_slack,
                            norm_slack)

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
DEV = "cuda"
MIB = 1 << 20


def normal(gen, *shape, dtype=torch.bfloat16, std=1.0, spread=False):
    x = torch.empty(shape, dtype=dtype, device=DEV).normal_(0, std, generator=gen)
    return x.mul_(torch.empty(shape[-1], device=DEV).normal_(generator=gen).exp_().to(dtype)) if spread else x


def same(a, b):
    return torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))


STREAMS = [None, torch.bfloat16, torch.float32]
SIZES = {None: 0, torch.bfloat16: 4, torch.float32: 8}


@pytest.mark.parametrize("H", [64, 520, 1032, 2048, 4096, 7168, 16384])
@pytest.mark.parametrize("dtype", STREAMS)
@pytest.mark.parametrize("quant", [False, True])
def test_norm_of_a_long_pass(H, dtype, quant):
    rows = 256 * MIB // (H * (4 + SIZES[dtype] + quant)) + 77
    say(f"norm: {rows} x {H} {dtype} quant {quant}")
    gen = torch.Generator(DEV).manual_seed(H)
    x, w = normal(gen, rows, H), torch.empty(H, device=DEV).normal_(1, 0.2, generator=gen)
    r = None if dtype is None else normal(gen, rows, H, dtype=dtype, spread=True)

    def call(part):
        n = len(range(rows)[part])
        out = dict(y=torch.empty(n, H, dtype=torch.bfloat16, device=DEV), rstd=torch.empty(n, device=DEV))
        if dtype is not None:
            out["h"] = torch.empty(n, H, dtype=dtype, device=DEV)
        if quant:
            out["q"], out["q_scale"] = bytes_like((n, U.quant_pitch(H))), bytes_like((n, U.quant_scale_pitch(H)))
        U.ultraep_residual_norm(ctx_of(8), x[part], w, 1e-6, residual=None if r is None else r[part], **out)
        return out

    whole = call(slice(None))
    for at in range(0, rows, -(-rows // 3)):
        part = slice(at, min(rows, at + -(-rows // 3)))
        for name, t in call(part).items():
            assert same(whole[name][part], t), (name, at)
    tail = slice(rows - 20, rows)
    h = host(x[tail]) if r is None else host((r[tail].double() + x[tail].double()).to(dtype))
    v, y = Y.residual_norm(h, host(w), float(np.float32(1e-6)))
    if r is not None:
        assert np.array_equal(host(whole["h"][tail]), h)
    rel = (norm_slack(H) + 3 * F32_STEP) * np.abs(y)
    assert (np.abs(host(whole["rstd"][tail]) - v) <= norm_slack(H) * v).all()
    assert (np.abs(host(whole["y"][tail]) - y) <= rel + BF16_STEP * (np.abs(y) + rel)).all()
    if quant:
        check_rows_form(host(whole["q"][tail]), host(whole["q_scale"][tail]), y, rel, H)


@pytest.mark.parametrize("H", [64, 520, 1032, 2048, 4096, 7168, 16384])
@pytest.mark.parametrize("dtype", STREAMS[1:])
@pytest.mark.parametrize("with_in", [False, True])
def test_norm_gradients_of_a_long_pass(H, dtype, with_in):
    rows = 256 * MIB // (H * (14 if dtype == torch.float32 else 8)) + 77
    say(f"norm gradients: {rows} x {H} {dtype} grad_in {with_in}")
    gen = torch.Generator(DEV).manual_seed(H)
    g, w = normal(gen, rows, H, std=0.1), torch.empty(H, device=DEV).normal_(1, 0.2, generator=gen)
    h = normal(gen, rows, H, dtype=dtype, spread=True)
    v = (h.double().square().mean(1) + 1e-6).rsqrt().float()
    back = normal(gen, rows, H, dtype=dtype, std=0.1) if with_in else None

    def call(part):
        n = len(range(rows)[part])
        out = dict(grad_weight=torch.full((H,), 3.0, device=DEV))
        grad_h = torch.empty(n, H, dtype=dtype, device=DEV)
        if dtype == torch.float32:
            out["grad_x"] = torch.empty(n, H, dtype=torch.bfloat16, device=DEV)
        U.ultraep_residual_norm_backward(ctx_of(8), g[part], h[part], w, v[part], grad_h, grad_in=None if back is None else back[part],
                                         workspace=bytes_like((U.residual_norm_workspace_bytes(n, H),)), accumulate=with_in, **out)
        return dict(out, grad_h=grad_h)

    whole = call(slice(None))
    for at in range(0, rows, -(-rows // 3)):
        part = slice(at, min(rows, at + -(-rows // 3)))
        for name, t in call(part).items():
            if name != "grad_weight":
                assert same(whole[name][part], t), (name, at)
    tail = slice(rows - 20, rows)
    want, mag, _, _ = Y.residual_norm_backward(host(g[tail]), host(h[tail]), host(w), host(v[tail]), None if back is None else host(back[tail]))
    slack = (2 * norm_slack(H) + 6 * F32_STEP) * mag
    step = BF16_STEP if dtype == torch.bfloat16 else F32_STEP
    assert (np.abs(host(whole["grad_h"][tail]) - want) <= slack + step * (np.abs(want) + slack)).all()
    if "grad_x" in whole:
        assert same(whole["grad_x"], whole["grad_h"].bfloat16())
    total, total_mag = torch.zeros(H, dtype=torch.float64, device=DEV), torch.zeros(H, dtype=torch.float64, device=DEV)
    for a, b, c in zip(g.split(20000), h.split(20000), v.split(20000)):
        t = a.double() * (b.double() * c.double()[:, None])
        total += t.sum(0)
        total_mag += t.abs().sum(0)
    total += 3.0 if with_in else 0.0
    err = (whole["grad_weight"].double() - total).abs()
    assert (err <= norm_blocks_slack(rows) * total_mag + F32_STEP * total.abs()).all()


@pytest.mark.parametrize("F", [128, 1000, 2048, 2880])
@pytest.mark.parametrize("back", [False, True])
@pytest.mark.parametrize("gelu", [False, True])
def test_activation_of_a_long_pass(F, back, gelu):
    """Both forms, and either alone, of one call over three experts, against a call each."""
    W = 2 * F if back else F
    rows = 128 * MIB // (F * ((6 if back else 4) + (2 if back else 1))) + 333   # long in one form too
    say(f"activation: {rows} x {F} gradients {back} gelu {gelu}")
    loads = [rows // 3 + 5, 0, rows // 5, rows - rows // 3 - 5 - rows // 5]
    seg = Segment(loads)
    gen = torch.Generator(DEV).manual_seed(F)
    h = normal(gen, rows, 2 * F, spread=True)
    args = (normal(gen, rows, F, std=0.01),) if back else ()
    f = U.ultraep_glu_quant_backward if back else U.ultraep_glu_quant

    def call(p0, p1, forms):
        part = slice(seg.off[p0], seg.off[p1])
        n = seg.off[p1] - seg.off[p0]
        blocks = U.quant_blocks(n, p1 - p0)
        out = {}
        if "q" in forms:
            out.update(q=bytes_like((n, U.quant_pitch(W))), q_scale=bytes_like((n, U.quant_scale_pitch(W))))
        if "t" in forms:
            out.update(qt=bytes_like((blocks, W, 128)), qt_scale=bytes_like((blocks, W)))
        f(seg.ctx, seg.plan, h[part], *[a[part] for a in args], p0, p1, activation=int(gelu), **out)
        return out

    whole = call(0, seg.ne, "qt")
    for forms in ("q", "t"):
        for name, t in call(0, seg.ne, forms).items():
            assert same(whole[name], t), (forms, name)
    first = X.first_blocks(seg.off)
    for p in range(seg.ne):
        if loads[p] == 0:
            continue
        part, used = call(p, p + 1, "qt"), -(-loads[p] // 128)
        for name in ("q", "q_scale"):
            assert same(whole[name][seg.off[p]:seg.off[p + 1]], part[name]), (name, p)
        for name in ("qt", "qt_scale"):
            assert same(whole[name][first[p]:first[p] + used], part[name][:used]), (name, p)
            assert (whole[name][first[p] + used:first[p + 1]] == SENT).all()
    tail = loads[3] % 128 + 128                         # the last block and the one before it
    values = host(h[rows - tail:])
    if back:
        want, mag = Y.glu_backward(values, host(args[0][rows - tail:]), gelu)
    else:
        want = Y.glu(values, gelu)
        mag = np.abs(want)
    check_rows_form(host(whole["q"][rows - tail:]), host(whole["q_scale"][rows - tail:]), want, 2.0 ** -14 * mag, W)
    at = first[3] + loads[3] // 128 - 1
    check_cols_form(host(whole["qt"][at:at + 2]), host(whole["qt_scale"][at:at + 2]), want, 2.0 ** -14 * mag, [0, tail], 2)

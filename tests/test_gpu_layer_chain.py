"""The steps around the experts together with the experts' own, as a program uses them: a layer's
training step with padded tokens, every stage checked on the inputs it was given; differences;
graphs; streams; offsets beyond 32 bits; choices that fp32 cannot tell apart."""
import numpy as np
import pytest

import moe_expert_load_ultraep_amd as U
import oracle.experts_oracle as X
import oracle.layer_oracle as Y
from gpu_common import say
from test_gpu_experts import Segment, bytes_like, dev, to_bf16
from test_gpu_layer import (BF16_STEP, F32_STEP, check_cols_form, check_rows_form, ctx_of, host, logits_of, norm_slack,
                            weight_slack)

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
DEV = "cuda"


def empty(*shape, dtype=torch.uint8):
    return torch.empty(shape, dtype=dtype, device=DEV)


class Forms:
    """Buffers of the rows form and the columns form of W columns."""

    def __init__(self, rows, W, blocks):
        self.W = W
        self.q, self.s = bytes_like((rows, U.quant_pitch(W))), bytes_like((rows, U.quant_scale_pitch(W)))
        self.qt, self.st = bytes_like((blocks, W, 128)), bytes_like((blocks, W))

    @property
    def all(self):
        return self.q, self.s, self.qt, self.st


def test_a_layer_with_padded_tokens():
    """norm -> logits -> route -> balance -> permute, products and activation -> combine -> norm, and back."""
    E, R, S, T, k, H, F = 16, 4, 1, 70, 3, 264, 128
    rng = np.random.default_rng(1)
    bf16 = lambda *shape, std=1.0: dev(to_bf16(rng.standard_normal(shape) * std)[0]).view(torch.bfloat16)  # noqa: E731
    tokens, padded = R * T, 33
    ctx = U.ultraep_create(E, R, S, R)
    x, stream = bf16(tokens, H), torch.from_numpy(rng.standard_normal((tokens, H)).astype(np.float32)).to(DEV)
    norm_w = torch.from_numpy((1 + 0.1 * rng.standard_normal(H)).astype(np.float32)).to(DEV)
    say("layer: norm, routing")
    h, y, rstd = torch.empty_like(stream), torch.empty_like(x), empty(tokens, dtype=torch.float32)
    U.ultraep_residual_norm(ctx, x, norm_w, 1e-6, residual=stream, h=h, y=y, rstd=rstd)
    assert torch.equal(h, stream + x.float())
    v, yn = Y.residual_norm(host(h), host(norm_w), float(np.float32(1e-6)))
    slack = (norm_slack(H) + 3 * F32_STEP) * np.abs(yn)
    assert (np.abs(host(y) - yn) <= slack + BF16_STEP * (np.abs(yn) + slack)).all()
    router, bias = bf16(E, H, std=0.1), torch.from_numpy((rng.standard_normal(E) * 0.1).astype(np.float32)).to(DEV)
    logits = y.float() @ router.float().t()
    logits[tokens - padded:] = -float("inf")
    idx, w = empty(tokens, k, dtype=torch.int32), empty(tokens, k, dtype=torch.float32)
    how = dict(score=U.ROUTE_SIGMOID, renormalize=True, scale=2.5)
    U.ultraep_route(ctx, logits, k, idx, w, bias=bias, groups=4, topk_groups=2, group_top=2, **how)
    want_i, want_w = Y.route(host(logits), k, True, host(bias), 4, 2, 2, True, 2.5)
    assert np.array_equal(host(idx), want_i) and (want_i[tokens - padded:] == -1).all() and (want_i[:tokens - padded] >= 0).all()
    assert (np.abs(host(w) - want_w) <= weight_slack(host(logits), want_i, 1, True)[:, None] * want_w).all()
    say("layer: balance, experts")
    buf = U.Buffers(ctx, 1, T, k, DEV)
    U.ultraep_balance(ctx, idx, T, k, buf.workspace, buf.plans, buf.phys_idx, buf.pos, topk_w=w, inv=buf.inv, w_perm=buf.w_perm, L=1)
    plan, pos, inv = buf.plans[0], buf.pos[0], buf.inv[0]
    got = ctx.decode_plan(plan.cpu().numpy())
    assert got["dropped"] == padded * k and got["total"] == (tokens - padded) * k
    rows, off = got["total"], got["phys_off"].astype(int).tolist()
    blocks = U.quant_blocks(rows, ctx.P)
    assert off[-1] == rows
    of = np.zeros(ctx.P, dtype=int)
    for e in range(E):
        of[got["inst_phys"][got["inst_ptr"][e]:got["inst_ptr"][e + 1]]] = e

    def weights(N, K):
        src = bf16(E, N, K, std=0.2)
        out = [empty(*s) for a, b in ((N, K), (K, N)) for s in ((E, a, U.quant_pitch(b)), (E, U.quant_pitch(a) // 128, U.quant_scale_pitch(b)))]
        U.ultraep_weight_quant(ctx, U.pointer_table(list(src)), E, N, K, *out)
        return [U.pointer_table([t[of[p]] for p in range(ctx.P)]) for t in out], out

    (w1, w1s, w1t, w1ts), keep1 = weights(2 * F, H)
    (w2, w2s, w2t, w2ts), keep2 = weights(H, F)
    xq = Forms(rows, H, blocks)
    U.ultraep_permute_quant(ctx, plan, inv, k, y, 0, ctx.P, *xq.all)
    up, out = empty(rows, 2 * F, dtype=torch.bfloat16), empty(rows, H, dtype=torch.bfloat16)
    U.ultraep_expert_gemm(ctx, plan, xq.q, xq.s, H, w1, w1s, 2 * F, 0, ctx.P, up)
    aq = Forms(rows, F, blocks)
    U.ultraep_glu_quant(ctx, plan, up, 0, ctx.P, *aq.all)
    act = Y.glu(host(up))
    slack = 2.0 ** -14 * np.abs(act)
    check_rows_form(host(aq.q), host(aq.s), act, slack, F)
    check_cols_form(host(aq.qt), host(aq.st), act, slack, off, blocks)
    U.ultraep_expert_gemm(ctx, plan, aq.q, aq.s, F, w2, w2s, H, 0, ctx.P, out)
    back = empty(tokens, H, dtype=torch.bfloat16)
    U.ultraep_combine(ctx, pos, w, k, out, 0, tokens, back)
    assert (back[tokens - padded:] == 0).all() and not back.isnan().any()
    h2, y2, rstd2 = torch.empty_like(h), torch.empty_like(y), torch.empty_like(rstd)
    U.ultraep_residual_norm(ctx, back, norm_w, 1e-6, residual=h, h=h2, y=y2, rstd=rstd2)
    assert torch.equal(h2[tokens - padded:], h[tokens - padded:])
    say("layer: backward")
    d_y2, d_h2, d_back = bf16(tokens, H, std=0.1), torch.empty_like(h), torch.empty_like(back)
    grad_w, ws = empty(H, dtype=torch.float32), empty(U.residual_norm_workspace_bytes(tokens, H))
    U.ultraep_residual_norm_backward(ctx, d_y2, h2, norm_w, rstd2, d_h2, grad_x=d_back, grad_weight=grad_w, workspace=ws)
    d_out, d_w = empty(rows, H, dtype=torch.bfloat16), empty(tokens, k, dtype=torch.float32)
    U.ultraep_combine_backward(ctx, pos, w, k, out, d_back, 0, tokens, d_out, d_w)
    dq = Forms(rows, H, blocks)
    U.ultraep_permute_quant(ctx, plan, None, 1, d_out, 0, ctx.P, *dq.all)
    d_act = empty(rows, F, dtype=torch.bfloat16)
    U.ultraep_expert_gemm(ctx, plan, dq.q, dq.s, H, w2t, w2ts, F, 0, ctx.P, d_act)
    dup = Forms(rows, 2 * F, blocks)
    U.ultraep_glu_quant_backward(ctx, plan, up, d_act, 0, ctx.P, *dup.all)
    want, mag = Y.glu_backward(host(up), host(d_act))
    check_rows_form(host(dup.q), host(dup.s), want, 2.0 ** -14 * mag, 2 * F)
    check_cols_form(host(dup.qt), host(dup.st), want, 2.0 ** -14 * mag, off, blocks)
    grads = empty(ctx.P, 2 * F, H, dtype=torch.float32)
    U.ultraep_expert_wgrad(ctx, plan, dup.qt, dup.st, 2 * F, xq.qt, xq.st, H, 0, ctx.P, rows, U.pointer_table(list(grads)))
    assert not grads.isnan().any() and grads.abs().sum() > 0
    d_rows, d_y = empty(rows, H, dtype=torch.bfloat16), empty(tokens, H, dtype=torch.bfloat16)
    U.ultraep_expert_gemm(ctx, plan, dup.q, dup.s, 2 * F, w1t, w1ts, H, 0, ctx.P, d_rows)
    U.ultraep_combine(ctx, pos, None, k, d_rows, 0, tokens, d_y)
    d_logits = torch.empty_like(logits)
    U.ultraep_route_backward(ctx, logits, k, idx, d_w, d_logits, **how)
    want, mag = Y.route_backward(host(logits), want_i, host(d_w), True, True, 2.5)
    assert (np.abs(host(d_logits) - want) <= 2 * weight_slack(host(logits), want_i, 1, True)[:, None] * mag + F32_STEP * np.abs(want)).all()
    assert (d_logits[tokens - padded:] == 0).all()
    d_y = (d_y.float() + d_logits @ router.float()).bfloat16()
    d_h, d_x = torch.empty_like(h), torch.empty_like(x)
    U.ultraep_residual_norm_backward(ctx, d_y, h, norm_w, rstd, d_h, grad_in=d_h2, grad_x=d_x, grad_weight=grad_w, workspace=ws, accumulate=True)
    want, mag, _, _ = Y.residual_norm_backward(host(d_y), host(h), host(norm_w), host(rstd), host(d_h2))
    assert (np.abs(host(d_h) - want) <= (2 * norm_slack(H) + 6 * F32_STEP) * mag + F32_STEP * np.abs(want)).all()
    assert torch.equal(d_x, d_h.bfloat16())
    del keep1, keep2


@pytest.mark.parametrize("score", [0, 1])
@pytest.mark.parametrize("renorm", [False, True])
def test_routing_gradients_against_differences(score, renorm):
    """Central differences of sum(g * w) at a fixed choice.  Weights are below 1 and off by 2^-20 of that at
    most, which a step of 2^-6 makes 2^-15 a weight; their third derivatives are below 1, the step's square
    over six below 2^-14."""
    rng = np.random.default_rng(12)
    l, v = logits_of(rng.standard_normal((40, 24)), False)
    idx, w = empty(40, 5, dtype=torch.int32), empty(40, 5, dtype=torch.float32)
    ctx = ctx_of(24)
    how = dict(score=score, renormalize=renorm)
    U.ultraep_route(ctx, l, 5, idx, w, **how)
    g = torch.from_numpy(rng.standard_normal((40, 5)).astype(np.float32)).to(DEV)
    grad = torch.empty_like(l)
    U.ultraep_route_backward(ctx, l, 5, idx, g, grad, **how)
    step = 2.0 ** -6
    for e in range(24):
        side = []
        for sign in (1, -1):
            moved = l.clone()
            moved[:, e] += sign * step
            i2, w2 = torch.empty_like(idx), torch.empty_like(w)
            U.ultraep_route(ctx, moved, 5, i2, w2, **how)
            same = (i2.sort(1)[0] == idx.sort(1)[0]).all(1)
            place = torch.argsort(torch.argsort(idx, 1), 1)
            side.append((torch.gather(w2.gather(1, i2.argsort(1)), 1, place).double() * g).sum(1))
            keep = same if sign == 1 else keep & same
        d = (side[0] - side[1]) / (2 * step)
        assert ((d - grad[:, e])[keep].abs() <= 5 * (2.0 ** -14 + 2.0 ** -14) * g.abs().max()).all()
        assert keep.sum() > 20


@pytest.mark.parametrize("E,k,groups,taken", [(128, 8, 1, 1), (256, 8, 8, 4), (160, 6, 8, 3), (512, 10, 16, 5), (60, 4, 4, 2), (250, 8, 5, 2)])
@pytest.mark.parametrize("score", [0, 1])
@pytest.mark.parametrize("bias", [False, True])
def test_choices_of_many_tokens(E, k, groups, taken, score, bias):
    """Ids of 66000 tokens against fp64 elsewhere: among so many some are nearer than fp32 tells apart."""
    gen = torch.Generator(DEV).manual_seed(E + k)
    l = torch.empty(66000, E, device=DEV).normal_(0, 1.3, generator=gen)
    b = torch.empty(E, device=DEV).normal_(0, 0.05, generator=gen) if bias else None
    ctx = ctx_of(E)
    for n in (66000, 9000, 700):
        for top in (1, 2):
            idx, w = empty(n, k, dtype=torch.int32), empty(n, k, dtype=torch.float32)
            U.ultraep_route(ctx, l[:n], k, idx, w, score=score, bias=b, groups=groups, topk_groups=taken, group_top=top)
            x = l[:n].double()
            s = torch.sigmoid(x) if score else torch.softmax(x, 1)
            key = x if b is None else s + b.double()
            if groups > 1:
                part = (s if b is None and top == 2 else key).view(n, groups, -1)
                worth = part.topk(top, dim=2)[0].sum(2)
                stay = torch.zeros(n, groups, dtype=torch.bool, device=DEV).scatter_(1, worth.topk(taken, dim=1)[1], True)
                key = torch.where(stay.repeat_interleave(E // groups, 1), key, -float("inf"))
            want = key.sort(dim=1, descending=True, stable=True)[1][:, :k]
            assert torch.equal(idx.long(), want), (n, top, int((idx.long() != want).any(1).sum()))


@pytest.mark.parametrize("tokens", [24, 6000, 40000])
def test_choices_that_fp32_cannot_tell_apart(tokens):
    """Scores a few 2^-30 apart at every place of the list, at its end, and between groups."""
    rng = np.random.default_rng(3)
    E, groups = 64, 4
    x = rng.standard_normal((24, E)) * 0.3 - 3
    for t in range(20):
        place = t % 10                       # which of the ten best are close
        order = rng.permutation(E)[:11]
        x[t, order] = 2.0 - 0.2 * np.arange(11)
        x[t, order[place + 1]] = x[t, order[place]]
    x[20:24, ::16] = 2.5                     # groups with the same best, and almost the same second
    x[20:24, 1::16] = 2.0 + rng.integers(-2, 3, (4, 4)) * 2.0 ** -22
    x = np.concatenate([x, rng.standard_normal((tokens - 24, E))]) if tokens > 24 else x
    l, v = logits_of(x, False)
    b = rng.integers(-4, 5, E) * 2.0 ** -30
    for kw in (dict(), dict(groups=groups, topk_groups=2, group_top=2), dict(groups=groups, topk_groups=3, group_top=1)):
        for score in (0, 1):
            for bias in (None, b):
                idx, w = empty(tokens, 8, dtype=torch.int32), empty(tokens, 8, dtype=torch.float32)
                U.ultraep_route(ctx_of(E), l, 8, idx, w, score=score, bias=None if bias is None else dev(bias.astype(np.float32)), **kw)
                want = Y.route(v[:24], 8, bool(score), bias, kw.get("groups", 1), kw.get("topk_groups", 1), kw.get("group_top", 1))[0]
                assert np.array_equal(host(idx)[:24], want), (kw, score, bias is None)


def steps(seed_rows=300):
    """Buffers and one pass through all six calls, with two shapes of every kernel choice that small sizes reach."""
    seg = Segment([200, 0, 97, 3])
    E, k, H, F, n = 64, 6, 520, 128, seed_rows
    ctx = ctx_of(E)
    f32 = lambda *s: torch.zeros(s, device=DEV)  # noqa: E731
    b16 = lambda *s: torch.zeros(s, dtype=torch.bfloat16, device=DEV)  # noqa: E731
    u8 = lambda *s: torch.zeros(s, dtype=torch.uint8, device=DEV)  # noqa: E731
    x, res, h, y, rstd, nw = b16(n, H), f32(n, H), f32(n, H), b16(n, H), f32(n), torch.ones(H, device=DEV)
    q, s = u8(n, U.quant_pitch(H)), u8(n, U.quant_scale_pitch(H))
    logits, bias, idx, w = f32(n, E), f32(E), torch.zeros(n, k, dtype=torch.int32, device=DEV), f32(n, k)
    gw, gl = f32(n, k), f32(n, E)
    up, ga = b16(seg.rows, 2 * F), b16(seg.rows, F)
    aq, gq = [u8(seg.rows, U.quant_pitch(W)) for W in (F, 2 * F)], [u8(seg.rows, U.quant_scale_pitch(W)) for W in (F, 2 * F)]
    at, gt = [u8(seg.blocks, W, 128) for W in (F, 2 * F)], [u8(seg.blocks, W) for W in (F, 2 * F)]
    gy, gh, gin, gx, gnw = b16(n, H), f32(n, H), f32(n, H), b16(n, H), f32(H)
    ws = u8(U.residual_norm_workspace_bytes(n, H))

    def step(stream=None):
        U.ultraep_residual_norm(ctx, x, nw, 1e-6, residual=res, h=h, y=y, q=q, q_scale=s, rstd=rstd, stream=stream)
        U.ultraep_route(ctx, logits, k, idx, w, score=1, bias=bias, groups=4, topk_groups=2, group_top=2, stream=stream)
        U.ultraep_glu_quant(seg.ctx, seg.plan, up, 0, seg.ne, aq[0], gq[0], at[0], gt[0], stream=stream)
        U.ultraep_glu_quant_backward(seg.ctx, seg.plan, up, ga, 0, seg.ne, aq[1], gq[1], at[1], gt[1], activation=1, stream=stream)
        U.ultraep_route_backward(ctx, logits, k, idx, gw, gl, score=1, stream=stream)
        U.ultraep_residual_norm_backward(ctx, gy, h, nw, rstd, gh, grad_in=gin, grad_x=gx, grad_weight=gnw, workspace=ws, stream=stream)

    def fill(i):
        gen = torch.Generator(DEV).manual_seed(i)
        for t in (x, res, logits, up, ga, gw, gy, gin):
            t.normal_(generator=gen)
        bias.normal_(0, 0.05, generator=gen)

    return step, fill, (h, y, rstd, q, s, idx, w, gl, *aq, *gq, *at, *gt, gh, gx, gnw)


def bits(t):
    return t.contiguous().view(torch.uint8)


def test_graph_replays_equal_eager():
    step, fill, outs = steps()
    want = []
    for i in range(3):
        fill(i)
        step()
        torch.cuda.synchronize()
        want.append([t.clone() for t in outs])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for rep, i in enumerate((1, 0, 2, 1)):
        fill(7 + rep)
        step()                      # eager work between replays, on other data
        fill(i)
        for t in outs:
            t.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(want[i], outs):
            assert torch.equal(bits(a), bits(b)), f"replay {rep}"


def test_two_streams_at_once():
    """The same calls on two streams, each with its own buffers, and on the current one."""
    first, second = steps(300), steps(211)
    for step, fill, _ in (first, second):
        fill(5)
        step()
    torch.cuda.synchronize()
    want = [[t.clone() for t in outs] for _, _, outs in (first, second)]
    for _, _, outs in (first, second):
        for t in outs:
            t.zero_()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(5):
        for (step, _, _), stream in zip((first, second), streams):
            step(stream)
    torch.cuda.synchronize()
    for saved, (_, _, outs) in zip(want, (first, second)):
        for a, b in zip(saved, outs):
            assert torch.equal(bits(a), bits(b))


def test_beyond_four_gibibytes():
    """The last tokens and rows of buffers whose bytes do not fit 32 bits."""
    say("large offsets: routing")
    n, E, k, tail = 4_300_011, 256, 4, 50
    l = torch.zeros(n, E, device=DEV)
    l[-tail:].normal_(generator=torch.Generator(DEV).manual_seed(1))
    l[:-tail, 7] = 1.0
    idx, w = empty(n, k, dtype=torch.int32), empty(n, k, dtype=torch.float32)
    U.ultraep_route(ctx_of(E), l, k, idx, w, score=1, scale=2.0)
    want = Y.route(host(l[-tail:]), k, True, scale=2.0)[0]
    assert np.array_equal(host(idx[-tail:]), want) and bool((idx[:-tail] == torch.tensor([7, 0, 1, 2], device=DEV)).all())
    grad = torch.empty_like(l)
    U.ultraep_route_backward(ctx_of(E), l, k, idx, w, grad, score=1, scale=2.0)
    want, mag = Y.route_backward(host(l[-tail:]), want, host(w[-tail:]), True, True, 2.0)
    assert (np.abs(host(grad[-tail:]) - want) <= 2.0 ** -18 * mag).all()
    del l, grad, idx, w
    say("large offsets: norm")
    n, H = 300_100, 7168
    x = torch.zeros(n, H, dtype=torch.bfloat16, device=DEV)
    x[-tail:].normal_(generator=torch.Generator(DEV).manual_seed(2))
    nw, y, rstd = torch.ones(H, device=DEV), torch.empty_like(x), empty(n, dtype=torch.float32)
    q, s = empty(n, H), empty(n, U.quant_scale_pitch(H))
    U.ultraep_residual_norm(ctx_of(8), x, nw, 1e-6, y=y, q=q, q_scale=s, rstd=rstd)
    v, want = Y.residual_norm(host(x[-tail:]), 1.0, float(np.float32(1e-6)))
    slack = (norm_slack(H) + 3 * F32_STEP) * np.abs(want)
    assert (np.abs(host(y[-tail:]) - want) <= slack + BF16_STEP * (np.abs(want) + slack)).all() and (y[:-tail] == 0).all()
    check_rows_form(host(q[-tail:]), host(s[-tail:]), want, slack, H)
    g, gw = torch.empty_like(x), empty(H, dtype=torch.float32)
    ws = empty(U.residual_norm_workspace_bytes(n, H))
    U.ultraep_residual_norm_backward(ctx_of(8), y, x, nw, rstd, g, grad_weight=gw, workspace=ws)
    want, mag, want_w, mag_w = Y.residual_norm_backward(host(y[-tail:]), host(x[-tail:]), 1.0, host(rstd[-tail:]))
    slack = (2 * norm_slack(H) + 6 * F32_STEP) * mag
    assert (np.abs(host(g[-tail:]) - want) <= slack + BF16_STEP * (np.abs(want) + slack)).all()
    assert (np.abs(host(gw) - want_w) <= tail * F32_STEP * mag_w + F32_STEP * np.abs(want_w)).all()
    del x, y, q, g
    say("large offsets: activation")
    F, tail = 3584, 300
    n = 300_500
    seg = Segment([n - tail, tail])
    h = torch.zeros(n, 2 * F, dtype=torch.bfloat16, device=DEV)
    h[-tail:].normal_(generator=torch.Generator(DEV).manual_seed(3))
    grad = torch.zeros(n, F, dtype=torch.bfloat16, device=DEV)
    grad[-tail:].normal_(generator=torch.Generator(DEV).manual_seed(4))
    first = X.first_blocks(seg.off)[1]
    for back in (False, True):
        W = 2 * F if back else F
        q, s = empty(n, U.quant_pitch(W)), empty(n, U.quant_scale_pitch(W))
        qt, st = empty(seg.blocks, W, 128), empty(seg.blocks, W)
        if back:
            U.ultraep_glu_quant_backward(seg.ctx, seg.plan, h, grad, 0, 2, q, s, qt, st)
            want, mag = Y.glu_backward(host(h[-tail:]), host(grad[-tail:]))
        else:
            U.ultraep_glu_quant(seg.ctx, seg.plan, h, 0, 2, q, s, qt, st)
            want = Y.glu(host(h[-tail:]))
            mag = np.abs(want)
        check_rows_form(host(q[-tail:]), host(s[-tail:]), want, 2.0 ** -14 * mag, W)
        check_cols_form(host(qt[first:first + 3]), host(st[first:first + 3]), want, 2.0 ** -14 * mag, [0, tail], 3)
        assert bool((q[:-tail] & 0x7F == 0).all())


def test_results_do_not_depend_on_the_others():
    """A token's and a row's results alone equal theirs in a batch, whichever kernel took it."""
    gen = torch.Generator(DEV).manual_seed(8)
    l = torch.empty(20000, 128, device=DEV).normal_(generator=gen)
    ctx = ctx_of(128)
    for score in (0, 1):
        out = []
        for n in (20000, 5000, 3):
            idx, w = empty(n, 8, dtype=torch.int32), empty(n, 8, dtype=torch.float32)
            U.ultraep_route(ctx, l[:n], 8, idx, w, score=score)
            out.append(idx[:3].clone())
        assert torch.equal(out[0], out[1]) and torch.equal(out[0], out[2])
    x = torch.empty(9000, 1024, device=DEV).normal_(generator=gen).bfloat16()
    nw = torch.ones(1024, device=DEV)
    many, one = torch.empty_like(x), torch.empty_like(x[:1])
    U.ultraep_residual_norm(ctx, x, nw, 1e-6, y=many)
    U.ultraep_residual_norm(ctx, x[:1], nw, 1e-6, y=one)
    assert torch.equal(many[:1], one)

"""The experts' steps together, as a program uses them: a training step of a
layer over a balanced plan with replicas, every stage checked on the inputs it
was given; gradients against differences; graphs; offsets beyond 32 bits."""
import numpy as np
import pytest

import moe_expert_load_ultraep_amd as U
import oracle as O
import oracle.experts_oracle as X
import workload as W
from gpu_common import say
from test_gpu_experts import (BF16_STEP, DEV, F32_ADD, F32_STEP, GROUP_CUT, Segment, dev, same_bytes, to_bf16)

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


def host(t):
    """float64 values of a bf16 or fp32 tensor, bytes of the rest."""
    return t.double().cpu().numpy() if t.is_floating_point() else t.cpu().numpy()


class Quantised:
    """Rows form and columns form of a segment's rows, and the checks of both."""

    def __init__(self, layer, x, inv=None, k=1):
        H = x.shape[1]
        self.H, self.layer = H, layer
        self.q = torch.zeros(layer.rows, U.quant_pitch(H), dtype=torch.uint8, device=DEV)
        self.s = torch.zeros(layer.rows, U.quant_scale_pitch(H), dtype=torch.uint8, device=DEV)
        self.qt = torch.zeros(layer.blocks, H, 128, dtype=torch.uint8, device=DEV)
        self.st = torch.zeros(layer.blocks, H, dtype=torch.uint8, device=DEV)
        U.ultraep_permute_quant(layer.ctx, layer.plan, inv, k, x, 0, layer.ctx.P, self.q, self.s, self.qt, self.st)
        v = host(x)
        v = v if inv is None else v[inv.cpu().numpy()[:layer.rows] // k]
        wq, ws = X.quant_rows(v)
        wqt, wst = X.quant_cols(v, layer.off, layer.blocks)
        same_bytes(host(self.q), wq)
        same_bytes(host(self.qt), wqt)
        assert np.array_equal(host(self.s), ws) and np.array_equal(host(self.st), wst)


class Layer:
    """A balanced layer of E experts with replicas: plan, layout and quantised weights."""

    def __init__(self, E=8, R=4, S=1, T=150, k=2, seed=7):
        rng = np.random.default_rng(seed)
        self.k, self.tokens = k, R * T
        pop = np.array([8.0, 1, 1, 3, 1, 1, 0.02, 2])
        idx = np.stack([rng.choice(E, size=k, replace=False, p=pop / pop.sum()) for _ in range(self.tokens)]).astype(np.int32)
        self.w = rng.random((self.tokens, k)).astype(np.float32)
        self.ctx = U.ultraep_create(E, R, S, R)
        self.buf = U.Buffers(self.ctx, 1, T, k, DEV)
        self.d_w = dev(self.w)
        U.ultraep_balance(self.ctx, dev(idx), T, k, self.buf.workspace, self.buf.plans, self.buf.phys_idx, self.buf.pos,
                          topk_w=self.d_w, inv=self.buf.inv, w_perm=self.buf.w_perm, L=1)
        torch.cuda.synchronize()
        self.plan, self.pos, self.inv = self.buf.plans[0], self.buf.pos[0], self.buf.inv[0]
        self.got = self.ctx.decode_plan(self.plan.cpu().numpy())
        self.off = self.got["phys_off"].astype(int).tolist()
        self.rows = self.off[-1]
        self.blocks = U.quant_blocks(self.rows, self.ctx.P)
        assert self.got["replicas"] > 0

    def physical(self, masters, slots):
        """One tensor a physical expert: masters by expert, replicas by slot (None: an empty one)."""
        M, S = self.ctx.M, self.ctx.S
        out = []
        for p in range(self.ctx.P):
            r, j = divmod(p, M + S)
            out.append(masters[r * M + j] if j < M else
                       slots[r * S + j - M] if self.got["slot_expert"][r * S + j - M] >= 0 else None)
        return out

    def weights(self, W, N, K):
        """Quantise the masters, sync bytes and scales to the replicas, build the tables for both orders."""
        E, n = self.ctx.E, self.ctx.R * self.ctx.S
        tables = []
        q, s, qt, st = (torch.empty(shape, dtype=torch.uint8, device=DEV) for a, b in ((N, K), (K, N)) for shape in
                        ((E, a, U.quant_pitch(b)), (E, U.quant_pitch(a) // 128, U.quant_scale_pitch(b))))
        U.ultraep_weight_quant(self.ctx, U.pointer_table(list(W)), E, N, K, q, s, qt, st)
        for i, x in enumerate((q, s, qt, st)):
            rep = torch.full((n, *x.shape[1:]), 0x55, dtype=torch.uint8, device=DEV)
            U.ultraep_weight_sync(self.ctx, self.plan, U.pointer_table(list(x)), rep, x[0].numel() // 2, 0, n)
            tables.append((U.pointer_table(self.physical(list(x), list(rep))), rep))
        torch.cuda.synchronize()
        value = [X.weight_value(host(q[e]), host(s[e])) for e in range(E)]
        value_t = [X.weight_value(host(qt[e]), host(st[e])) for e in range(E)]
        for a, b in zip(value, value_t):
            assert np.array_equal(a[:, :K], b[:, :N].T)
        self.keep = getattr(self, "keep", []) + [q, s, qt, st, tables]
        of = self.expert_of()
        return ((tables[0][0], tables[1][0], [value[e] for e in of]), (tables[2][0], tables[3][0], [value_t[e] for e in of]))

    def expert_of(self):
        out = np.zeros(self.ctx.P, dtype=int)
        for e in range(self.ctx.E):
            a, b = self.got["inst_ptr"][e:e + 2]
            out[self.got["inst_phys"][a:b]] = e
        return out

    def product(self, x: Quantised, weights, N):
        out = torch.empty(self.rows, N, dtype=torch.bfloat16, device=DEV)
        tw, ts, value = weights
        U.ultraep_expert_gemm(self.ctx, self.plan, x.q, x.s, x.H, tw, ts, N, 0, self.ctx.P, out)
        v = X.rows_value(host(x.q), host(x.s))
        want = X.expert_gemm(v, value, self.off)
        mag = X.expert_gemm(np.abs(v), [np.abs(a) for a in value], self.off)
        slack = (GROUP_CUT + x.H * F32_ADD) * mag
        assert (np.abs(host(out) - want) <= slack + BF16_STEP * (np.abs(want) + slack)).all()
        return out

    def gradients(self, dy: Quantised, x: Quantised):
        """Weight gradients of masters and replicas, folded: fp32 [E, N, K], against the oracle's."""
        E, n, N, K = self.ctx.E, self.ctx.R * self.ctx.S, dy.H, x.H
        masters, slots = torch.empty(E, N, K, device=DEV), torch.full((n, N, K), 7.0, device=DEV)
        table = U.pointer_table(self.physical(list(masters), list(slots)))
        U.ultraep_expert_wgrad(self.ctx, self.plan, dy.qt, dy.st, N, x.qt, x.st, K, 0, self.ctx.P, self.rows, table)
        U.ultraep_fold_grads(self.ctx, self.plan, U.pointer_table(list(masters)), slots, N * K, 0, n)
        each = X.expert_wgrad(host(dy.qt), host(dy.st), host(x.qt), host(x.st), self.off)
        mags = X.expert_wgrad(host(dy.qt) & 0x7F, host(dy.st), host(x.qt) & 0x7F, host(x.st), self.off)
        of = self.expert_of()
        for e in range(E):
            ps = [p for p in range(self.ctx.P) if of[p] == e and self.off[p + 1] > self.off[p]]
            want, mag = sum(each[p] for p in ps) + np.zeros((N, K)), sum(mags[p] for p in ps) + np.zeros((N, K))
            count = sum(self.off[p + 1] - self.off[p] for p in ps) + len(ps)
            assert (np.abs(host(masters[e]) - want) <= count * F32_ADD * mag).all(), e
        return masters


def test_training_step_over_a_balanced_plan():
    H, F = 264, 136
    say("chain: balance, weights")
    L = Layer()
    rng = np.random.default_rng(3)
    bf16 = lambda *shape: dev(to_bf16(rng.standard_normal(shape) * 0.2)[0]).view(torch.bfloat16)  # noqa: E731
    hidden, W1, W2 = bf16(L.tokens, H), bf16(L.ctx.E, 2 * F, H), bf16(L.ctx.E, H, F)
    w1, w1t = L.weights(W1, 2 * F, H)
    w2, w2t = L.weights(W2, H, F)
    say("chain: forward")
    x = Quantised(L, hidden, L.inv, L.k)
    h = L.product(x, w1, 2 * F)
    gate, up = h[:, :F].float(), h[:, F:].float()
    act = (torch.nn.functional.silu(gate) * up).bfloat16()
    a = Quantised(L, act)
    y = L.product(a, w2, H)
    out = torch.empty(L.tokens, H, dtype=torch.bfloat16, device=DEV)
    U.ultraep_combine(L.ctx, L.pos, L.d_w, L.k, y, 0, L.tokens, out)
    say("chain: backward")
    d_out = bf16(L.tokens, H)
    dy, dw = torch.empty_like(y), torch.empty(L.tokens, L.k, device=DEV)
    U.ultraep_combine_backward(L.ctx, L.pos, L.d_w, L.k, y, d_out, 0, L.tokens, dy, dw)
    dyq = Quantised(L, dy)
    g2 = L.gradients(dyq, a)
    da = L.product(dyq, w2t, F).float()
    sg = torch.sigmoid(gate)
    dh = torch.cat([da * up * sg * (1 + gate * (1 - sg)), da * gate * sg], 1).bfloat16()
    dhq = Quantised(L, dh)
    g1 = L.gradients(dhq, x)
    dx = L.product(dhq, w1t, H)
    d_hidden = torch.empty_like(hidden)
    U.ultraep_combine(L.ctx, L.pos, None, L.k, dx, 0, L.tokens, d_hidden)
    pos = host(L.pos).reshape(-1)
    want = O.combine(dx.view(torch.int16).cpu().numpy().view(np.uint16), pos, None, L.k, 0, L.tokens)
    assert (np.abs(host(d_hidden) - want) <= (2 * BF16_STEP) * np.abs(want) + L.k * F32_STEP * np.abs(want) + 1e-6).all()
    say("chain: clipping")
    views = [g for t in (g1, g2) for g in t]
    before = [host(v) for v in views]
    tensors, numels = U.pointer_table(views), torch.tensor([v.numel() for v in views]).to(DEV)
    ws = torch.empty(U.GRAD_WORKSPACE_BYTES, dtype=torch.uint8, device=DEV)
    sumsq, norm = torch.empty(1, dtype=torch.float64, device=DEV), torch.empty(1, device=DEV)
    U.ultraep_grad_sumsq(L.ctx, tensors, numels, len(views), torch.float32, sumsq, ws)
    U.ultraep_grad_clip(L.ctx, tensors, numels, len(views), torch.float32, sumsq, 0.5, norm)
    want_norm, want = X.clip(before, 0.5)
    assert want_norm > 0.5 and abs(norm.item() - want_norm) <= 1.01 * F32_STEP * want_norm
    for v, w in zip(views, want):
        assert (np.abs(host(v) - w) <= 1.01 * F32_STEP * np.abs(w) + 1e-45).all()


def test_gradients_against_differences():
    """L = sum(dy * (x W^T)) is linear in x and in W: whole numbers make products,
    gradients and differences exact, so L(x + d) - L(x) = sum(dx * d) to the last bit."""
    rng = np.random.default_rng(17)
    seg = Segment([150, 0, 40], p0=0)
    N, K = 72, 136
    x, d = rng.integers(-1, 2, (seg.rows, K)), rng.integers(-1, 2, (seg.rows, K))
    w, e = rng.integers(-1, 2, (seg.ne, N, K)), rng.integers(-1, 2, (seg.ne, N, K))
    dy = rng.integers(-2, 3, (seg.rows, N))
    bf16 = lambda a: dev(to_bf16(a.astype(np.float64))[0]).view(torch.bfloat16)  # noqa: E731

    def weights(v):
        out = [torch.empty(s, dtype=torch.uint8, device=DEV) for a, b in ((N, K), (K, N)) for s in
               ((seg.ne, a, U.quant_pitch(b)), (seg.ne, U.quant_pitch(a) // 128, U.quant_scale_pitch(b)))]
        src = bf16(v)
        U.ultraep_weight_quant(seg.ctx, U.pointer_table(list(src)), seg.ne, N, K, *out)
        return out

    def rows(v):
        H = v.shape[1]
        out = [torch.zeros(s, dtype=torch.uint8, device=DEV) for s in
               ((seg.rows, U.quant_pitch(H)), (seg.rows, U.quant_scale_pitch(H)), (seg.blocks, H, 128), (seg.blocks, H))]
        U.ultraep_permute_quant(seg.ctx, seg.plan, None, 1, bf16(v), 0, seg.ne, *out)
        return out

    def product(r, q, s, n, kk):
        out = torch.empty(seg.rows, n, dtype=torch.bfloat16, device=DEV)
        U.ultraep_expert_gemm(seg.ctx, seg.plan, r[0], r[1], kk, U.pointer_table(list(q)), U.pointer_table(list(s)), n, 0, seg.ne, out)
        return host(out)

    W = weights(w)
    loss = lambda xv, Wv: float((product(rows(xv), Wv[0], Wv[1], N, K) * dy).sum())  # noqa: E731
    base = loss(x, W)
    dyr, xr = rows(dy), rows(x)
    dx = product(dyr, W[2], W[3], K, N)
    assert loss(x + d, W) - base == float((dx * d).sum())
    grads = torch.empty(seg.ne, N, K, device=DEV)
    U.ultraep_expert_wgrad(seg.ctx, seg.plan, dyr[2], dyr[3], N, xr[2], xr[3], K, 0, seg.ne, seg.rows, U.pointer_table(list(grads)))
    assert loss(x, weights(w + e)) - base == float((host(grads) * e).sum())


def test_graph_replays_equal_eager():
    """All six calls captured once; every replay, between eager calls on other data, equals the eager result."""
    rng = np.random.default_rng(23)
    seg = Segment([300, 0, 129, 60], p0=0)
    small = Segment([2, 0, 1, 3], p0=0)
    N, K = 264, 392
    src = torch.empty(seg.rows, K, dtype=torch.bfloat16, device=DEV)
    wsrc = torch.empty(seg.ne, N, K, dtype=torch.bfloat16, device=DEV)
    u8 = lambda *s: torch.zeros(s, dtype=torch.uint8, device=DEV)  # noqa: E731
    q, s, qt, st = u8(seg.rows, U.quant_pitch(K)), u8(seg.rows, U.quant_scale_pitch(K)), u8(seg.blocks, K, 128), u8(seg.blocks, K)
    w, ws, wt, wst = (u8(*x) for a, b in ((N, K), (K, N)) for x in
                      ((seg.ne, a, U.quant_pitch(b)), (seg.ne, U.quant_pitch(a) // 128, U.quant_scale_pitch(b))))
    yt, yst = u8(seg.blocks, N, 128), u8(seg.blocks, N)
    y, few = (torch.zeros(n, N, dtype=torch.bfloat16, device=DEV) for n in (seg.rows, small.rows))
    g, out = torch.zeros(seg.ne, N, K, device=DEV), torch.zeros(seg.ne, N, K, device=DEV)
    t_src, t_w, t_ws, t_g, t_out = (U.pointer_table(list(t)) for t in (wsrc, w, ws, g, out))
    numels = torch.full((seg.ne,), N * K, dtype=torch.int64, device=DEV)
    sumsq, norm = torch.zeros(1, dtype=torch.float64, device=DEV), torch.zeros(1, device=DEV)
    work = torch.empty(U.GRAD_WORKSPACE_BYTES, dtype=torch.uint8, device=DEV)

    def step():
        U.ultraep_permute_quant(seg.ctx, seg.plan, None, 1, src, 0, seg.ne, q, s, qt, st)
        U.ultraep_weight_quant(seg.ctx, t_src, seg.ne, N, K, w, ws, wt, wst)
        U.ultraep_expert_gemm(seg.ctx, seg.plan, q, s, K, t_w, t_ws, N, 0, seg.ne, y)
        U.ultraep_expert_gemm(small.ctx, small.plan, q, s, K, t_w, t_ws, N, 0, small.ne, few)
        U.ultraep_permute_quant(seg.ctx, seg.plan, None, 1, y, 0, seg.ne, qt=yt, qt_scale=yst, rows=seg.rows)
        U.ultraep_expert_wgrad(seg.ctx, seg.plan, yt, yst, N, qt, st, K, 0, seg.ne, seg.rows, t_g)
        U.ultraep_grad_sumsq(seg.ctx, t_g, numels, seg.ne, torch.float32, sumsq, work)
        U.ultraep_grad_clip(seg.ctx, t_g, numels, seg.ne, torch.float32, sumsq, 1.0, norm, out=t_out)

    def fill(i):
        gen = torch.Generator(DEV).manual_seed(100 + i)
        src.normal_(generator=gen)
        wsrc.normal_(generator=gen)

    outs = (q, s, qt, st, w, ws, wt, wst, y, few, yt, yst, g, out, sumsq, norm)
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
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8)), f"replay {rep}"


def test_rows_beyond_four_gibibytes():
    """The last rows of a segment whose bytes do not fit 32 bits."""
    H, rows, tail = 7168, 600_500, 300
    seg = Segment([rows - tail, tail], p0=0)
    say("large offsets: drawing rows")
    x = torch.zeros(rows, H, dtype=torch.bfloat16, device=DEV)
    x[-tail:].normal_(generator=torch.Generator(DEV).manual_seed(4))
    u8 = lambda *s: torch.empty(s, dtype=torch.uint8, device=DEV)  # noqa: E731
    q, s = u8(rows, H), u8(rows, U.quant_scale_pitch(H))
    qt, st = u8(seg.blocks, H, 128), u8(seg.blocks, H)
    U.ultraep_permute_quant(seg.ctx, seg.plan, None, 1, x, 0, 2, q, s, qt, st)
    v = host(x[-tail:])
    wq, ws = X.quant_rows(v)
    same_bytes(host(q[-tail:]), wq)
    assert np.array_equal(host(s[-tail:]), ws)
    first = X.first_blocks(seg.off)[1]
    wqt, wst = X.quant_cols(v, [0, tail], 3)
    same_bytes(host(qt[first:first + 3]), wqt[:3])
    assert np.array_equal(host(st[first:first + 3]), wst)
    say("large offsets: products")
    N = 72
    rng = np.random.default_rng(5)
    wb = X.to_e4m3(rng.integers(-2, 3, (2, N, H)).astype(np.float64))
    sb = np.full((2, 1, U.quant_scale_pitch(H)), 127, dtype=np.uint8)
    w, sc = dev(wb), dev(sb)
    out = torch.empty(rows, N, dtype=torch.bfloat16, device=DEV)
    U.ultraep_expert_gemm(seg.ctx, seg.plan, q, s, H, U.pointer_table(list(w)), U.pointer_table(list(sc)), N, 0, 2, out)
    xv, wv = X.rows_value(wq, ws), X.weight_value(wb[1], sb[1])
    want, mag = xv @ wv.T, np.abs(xv) @ np.abs(wv).T
    slack = (GROUP_CUT + H * F32_ADD) * mag
    assert (np.abs(host(out[-tail:]) - want) <= slack + BF16_STEP * (np.abs(want) + slack)).all()
    assert (out[:rows - tail] == 0).all()
    g = torch.empty(2, N, H, device=DEV)
    dyt, dys = u8(seg.blocks, N, 128), u8(seg.blocks, N)
    U.ultraep_permute_quant(seg.ctx, seg.plan, None, 1, out, 0, 2, qt=dyt, qt_scale=dys, rows=rows)
    U.ultraep_expert_wgrad(seg.ctx, seg.plan, dyt, dys, N, qt, st, H, 0, 2, rows, U.pointer_table(list(g)))
    last = lambda t: host(t[first:first + 3])  # noqa: E731
    want = X.expert_wgrad(last(dyt), last(dys), last(qt), last(st), [0, tail])[0]
    mag = X.expert_wgrad(last(dyt) & 0x7F, last(dys), last(qt) & 0x7F, last(st), [0, tail])[0]
    assert (g[0] == 0).all()
    assert (np.abs(host(g[1]) - want) <= tail * F32_ADD * mag).all()

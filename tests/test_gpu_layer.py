"""The steps around the experts on the GPU against their 64-bit oracle.

Ids of the routing are compared as they are.  The rest goes by what fp32 can lose:
* Routing weights: an exponential of x - m is off by |x - m| * 2^-24 of itself through
  the difference and two steps through the function, sums of k positive terms by k
  steps, the divisions by two: (k + 8 + |x - m|) * 2^-23 in all, taken at the row's
  spread of chosen logits; with a sum over E experts another E / 64 + 16 (a lane adds
  E / 64 of them, then the lanes are added).  Their gradients the same, of the sum of
  the magnitudes that they are made of, and half a step of their type.
* The norm: a lane adds at most H / 64 squares one after another and then 22 partial
  sums, each addition off by 2^-24: (H / 64 + 32) * 2^-24 with the root and the
  divisions, which goes on into y and the gradients.  A workgroup adds at most
  rows / 256 + 1 rows of grad_weight in fp32 (the rest in fp64).
* The gated activation: z is below 75 where the result is not tiny, its exponential off
  by at most 4 * 75 + 16 steps of 2^-23: less than 2^-14 of the magnitudes.
* Rounding: half a step of the type, 2^-8 for bf16, 2^-4 for e4m3 (2^-10 of the
  scale where e4m3 is subnormal).  A block's scale is the oracle's but where the block's
  largest value is that near to the scale's border.
"""
import numpy as np
import pytest

import moe_expert_load_ultraep_amd as U
import oracle.experts_oracle as X
import oracle.layer_oracle as Y
from test_gpu_experts import LOADS, SENT, Segment, bytes_like, dev, to_bf16

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
DEV = "cuda"
BF16_STEP, F32_STEP, E4M3_STEP = 2.0 ** -8, 2.0 ** -24, 2.0 ** -4
NAN, INF = np.nan, np.inf


def host(t):
    return t.double().cpu().numpy() if t.is_floating_point() else t.cpu().numpy()


def logits_of(x, bf16):
    """(device tensor, its values in 64 bits)."""
    t = torch.from_numpy(np.asarray(x, dtype=np.float32)).to(DEV)
    t = t.bfloat16() if bf16 else t
    return t, host(t)


def ctx_of(E):
    return U.ultraep_create(E, E, 0, 1)


# ---------------------------------------------------------------- routing

def route(l, k, **kw):
    n = l.shape[0]
    idx = torch.full((n + 1, k), -77, dtype=torch.int32, device=DEV)
    w = torch.full((n + 1, k), -7.0, device=DEV)
    U.ultraep_route(ctx_of(l.shape[1]), l, k, idx[:n], w[:n], **kw)
    assert (idx[n] == -77).all() and (w[n] == -7).all(), "rows behind the last token must stay"
    return idx[:n], w[:n]


def weight_slack(v, idx, score, renorm):
    """Relative error of the weights, a row each."""
    masked, l = Y.clean(v)
    some = idx >= 0
    x = np.where(some, np.take_along_axis(l, np.maximum(idx, 0), 1), np.nan)
    spread = np.zeros(len(idx))
    for t in range(len(idx)):
        if some[t].any():
            top = np.nanmax(x[t]) if score or renorm else np.max(np.where(masked[t], -INF, l[t]))
            top = min(top, 0.0) if score else top
            spread[t] = np.nanmax(np.abs(x[t] - top))
    return (idx.shape[1] + 8 + np.minimum(spread, 200.0) + (0 if score or renorm else v.shape[1] / 64 + 16)) * 2.0 ** -23


def check_route(v, l, k, bias=None, **kw):
    idx, w = route(l, k, bias=None if bias is None else dev(np.asarray(bias, dtype=np.float32)), **kw)
    score, renorm = kw.get("score", 0), kw.get("renormalize", True)
    want_i, want_w = Y.route(v, k, bool(score), None if bias is None else np.asarray(bias, dtype=np.float32), kw.get("groups", 1),
                             kw.get("topk_groups", 1), kw.get("group_top", 1), renorm, float(np.float32(kw.get("scale", 1.0))))
    assert np.array_equal(host(idx), want_i)
    got = host(w)
    slack = weight_slack(v, want_i, score, renorm)[:, None]
    assert (np.abs(got - want_w) <= slack * np.abs(want_w) + 2.0 ** -120).all()
    assert (got[want_i < 0] == 0).all()
    return want_i


SHAPES = [(1, 1, 1, 1), (7, 2, 1, 1), (64, 8, 8, 4), (96, 6, 6, 2), (128, 8, 1, 1), (160, 6, 8, 3), (160, 8, 16, 5), (250, 9, 5, 3), (256, 8, 8, 4),
          (256, 12, 4, 4), (320, 8, 4, 2), (512, 10, 64, 7), (513, 3, 27, 4), (1024, 64, 32, 9), (64, 64, 1, 1)]


@pytest.mark.parametrize("E,k,groups,taken", SHAPES)
@pytest.mark.parametrize("score", [0, 1])
@pytest.mark.parametrize("bf16", [False, True])
def test_route(E, k, groups, taken, score, bf16):
    rng = np.random.default_rng(E * 100 + k)
    for tokens in (1, 5, 67):
        l, v = logits_of(rng.standard_normal((tokens, E)) * 1.5, bf16)
        for bias in (None, rng.standard_normal(E) * 0.1):
            for top in (1, 2):
                kw = dict(score=score, groups=groups, topk_groups=taken, group_top=top, scale=2.5, renormalize=(tokens != 5))
                check_route(v, l, min(k, E), bias, **kw)


@pytest.mark.parametrize("score", [0, 1])
@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("E,groups", [(24, 3), (256, 8), (250, 5), (1000, 10)])
def test_route_masks_ties_and_extremes(E, groups, score, bias):
    rng = np.random.default_rng(E)
    x = rng.standard_normal((40, E))
    x[0], x[1], x[2] = -INF, NAN, 0.0                     # nothing left; all the same
    x[3, 1:] = -INF                                       # one left
    x[4, : E - 3], x[5, ::2] = NAN, -INF
    x[6, 5], x[7, [3, 9]], x[8] = INF, INF, INF
    x[9], x[10], x[11] = 1e30, -1e30, np.where(np.arange(E) % 2, -80, 80)
    x[12] = -200 - np.arange(E)
    x[13:20] = np.round(x[13:20])                         # many ties
    x[20:24] = np.round(x[20:24] * 2 ** 10) * 2.0 ** -40  # scores next to each other
    x[24:28] = 1.0 + rng.integers(0, 3, (4, E)) * 2.0 ** -23
    x[28] = 40.0 + np.arange(E) * 0.25                    # sigmoids that round to one
    x[29], x[30] = 5e-324, np.float32(1e-40)
    b = rng.standard_normal(E) * 0.05
    b[::7] = 0.25
    b[1], b[2] = NAN, -INF
    for bf16 in (False, True):
        l, v = logits_of(x, bf16)
        for g, t, top in ((1, 1, 1), (groups, 2, 1), (groups, 2, 2)):
            for renorm in (False, True):
                check_route(v, l, 8, b if bias else None, score=score, groups=g, topk_groups=t, group_top=top, renormalize=renorm)


def test_route_of_an_infinite_bias():
    rng = np.random.default_rng(0)
    l, v = logits_of(rng.standard_normal((9, 32)), False)
    b = np.zeros(32)
    b[[3, 20]] = INF
    assert (check_route(v, l, 4, b, score=1, groups=4, topk_groups=2, group_top=2)[:, :1] == 3).all()
    check_route(v, l, 4, b, score=0)


@pytest.mark.parametrize("E,taken", [(16, 5), (64, 9)])
def test_route_groups_of_one_expert(E, taken):
    rng = np.random.default_rng(E)
    for bf16 in (False, True):
        l, v = logits_of(rng.standard_normal((90, E)), bf16)
        for bias in (None, rng.standard_normal(E) * 0.1):
            for top in (1, 2):
                idx = check_route(v, l, 8, bias, score=1, groups=E, topk_groups=taken, group_top=top)
                assert (idx >= 0).sum() == 90 * min(taken, 8)


@pytest.mark.parametrize("scale", [0.0, -1.5])
def test_route_scales(scale):
    rng = np.random.default_rng(8)
    l, v = logits_of(rng.standard_normal((9, 32)), False)
    check_route(v, l, 4, score=1, scale=scale)


def test_route_many_tokens_and_unaligned_rows():
    """More tokens than waves, from an address that is only the elements' multiple."""
    rng = np.random.default_rng(6)
    for E, bf16 in ((131, False), (131, True), (128, False), (256, True)):
        n = 20011
        flat = rng.standard_normal(n * E + 1).astype(np.float32)
        t = torch.from_numpy(flat).to(DEV)
        t = t.bfloat16() if bf16 else t
        l = t[1:].view(n, E)
        v = host(l)
        idx, w = route(l, 4, score=1)
        pick = rng.integers(0, n, 300)
        want_i, want_w = Y.route(v[pick], 4, True)
        assert np.array_equal(host(idx)[pick], want_i)
        assert (np.abs(host(w)[pick] - want_w) <= weight_slack(v[pick], want_i, 1, True)[:, None] * want_w).all()
        top = torch.topk(l.float(), 4, dim=1)[0]
        assert torch.equal(torch.gather(l.float(), 1, idx.long()), top)


def check_route_backward(v, l, idx, g, score, renorm, scale):
    n, E = v.shape
    out = torch.full((n + 1, E), 9.0, dtype=l.dtype, device=DEV)
    U.ultraep_route_backward(ctx_of(E), l, idx.shape[1], dev(idx), dev(g), out[:n], score=score, renormalize=renorm, scale=scale)
    assert (out[n] == 9).all()
    want, mag = Y.route_backward(v, idx, g.astype(np.float64), bool(score), renorm, float(np.float32(scale)))
    masked, _ = Y.clean(v)
    known = np.where((idx >= 0) & (idx < E) & ~np.take_along_axis(masked, np.clip(idx, 0, E - 1), 1), idx, -1)
    slack = 2 * weight_slack(v, known, score, renorm)[:, None] * mag
    step = BF16_STEP if l.dtype == torch.bfloat16 else F32_STEP
    err = np.abs(host(out[:n]) - want)
    assert (err <= slack + step * (np.abs(want) + slack) + 2.0 ** -120).all(), np.max(err / (mag + 1e-30))
    assert (host(out[:n])[masked] == 0).all()


@pytest.mark.parametrize("E,k", [(1, 1), (7, 2), (64, 8), (131, 5), (160, 6), (256, 8), (513, 12), (1024, 64)])
@pytest.mark.parametrize("score", [0, 1])
@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("bf16", [False, True])
def test_route_backward(E, k, score, renorm, bf16):
    rng = np.random.default_rng(E)
    for tokens in (1, 6, 301):
        x = rng.standard_normal((tokens, E)) * 2
        if tokens > 5 and E > 8:
            x[0], x[1, 3:], x[2, ::3], x[3, 4], x[4] = -INF, NAN, -INF, INF, -30 - np.arange(E) * 0.1
        l, v = logits_of(x, bf16)
        idx = np.stack([rng.permutation(E)[:k] for _ in range(tokens)]).astype(np.int32)
        if tokens > 5:
            idx[:, -1] = idx[:, 0]                     # the same id twice
            idx[5, 0], idx[-1] = E, -1                 # no expert; none at all
        g = rng.standard_normal((tokens, k)).astype(np.float32)
        g[idx < 0] = NAN                               # not looked at
        check_route_backward(v, l, idx, g, score, renorm, 2.5)


# ---------------------------------------------------------------- the 8-bit forms of fp32 values

def check_rows_form(q, scale, want, rel, W):
    """q, scale against `want` [rows, W], each value of which is off by at most rel (an array) before it is rounded."""
    rows, kb = want.shape[0], X.up(W) // 128
    full, slack = np.zeros((rows, kb * 128)), np.zeros((rows, kb * 128))
    full[:, :W], slack[:, :W] = want, rel
    check_blocks(X.VALUES[q].reshape(rows, kb, 128), scale[:, :kb].astype(int) - 127, full.reshape(rows, kb, 128),
                 slack.reshape(rows, kb, 128))
    assert (scale[:, kb:] == 127).all() and (q[:, W:] & 0x7F == 0).all()


def check_blocks(got, e, want, slack):
    """Blocks along the last dimension: the scale, and every value in its steps."""
    bad = ~np.isfinite(want)
    assert np.array_equal(np.isnan(got), bad)
    want, slack, got = np.where(bad, 0, want), np.where(bad, 0, slack), np.where(bad, 0, got)
    low = X.block_exponent(np.maximum(np.abs(want) - slack, 0), want.ndim - 1)
    high = X.block_exponent(np.abs(want) + slack, want.ndim - 1)
    zero = (np.maximum(np.abs(want) - slack, 0) == 0).all(axis=-1)
    assert (((low <= e) & (e <= high)) | (zero & ((e == 0) | (e <= high)))).all()
    value = got * 2.0 ** e[..., None].astype(np.float64)
    step = E4M3_STEP * (np.abs(want) + slack) + 2.0 ** (e[..., None] - 10.0)
    assert (np.abs(value - want) <= slack + step).all()


def check_cols_form(qt, scale, want, rel, off, blocks):
    W = want.shape[1]
    used = np.zeros(blocks, dtype=bool)
    for p, b in enumerate(X.first_blocks(off)[:-1]):
        for i, at in enumerate(range(off[p], off[p + 1], 128)):
            part, slack = np.zeros((128, W)), np.zeros((128, W))
            end = min(at + 128, off[p + 1])
            part[:end - at], slack[:end - at] = want[at:end], rel[at:end]
            check_blocks(X.VALUES[qt[b + i]], scale[b + i].astype(int) - 127, part.T, slack.T)
            assert (qt[b + i][:, end - at:] & 0x7F == 0).all()
            used[b + i] = True
    assert (qt[~used] == SENT).all() and (scale[~used] == SENT).all()


# ---------------------------------------------------------------- norm

WIDTHS = [8, 64, 120, 128, 512, 520, 1000, 1024, 1032, 2048, 2056, 4096, 5120, 7168, 8192, 8200, 16384]


def stream_of(x, dtype):
    return None if dtype is None else torch.from_numpy(x.astype(np.float32)).to(DEV).to(dtype)


def norm_case(rng, rows, H, dtype, w32):
    x = dev(to_bf16(rng.standard_normal((rows, H)))[0]).view(torch.bfloat16)
    r = stream_of(rng.standard_normal((rows, H)) * np.exp(rng.standard_normal(H)), dtype)
    w = torch.from_numpy((1 + 0.2 * rng.standard_normal(H)).astype(np.float32)).to(DEV)
    return x, r, w if w32 else w.bfloat16()


def stored(x, r):
    """The stream's rows as they are stored, in 64 bits."""
    if r is None:
        return host(x)
    return host(torch.from_numpy(host(r) + host(x)).to(r.dtype))


def norm_slack(H):
    return (H / 64 + 32) * F32_STEP


def check_norm(x, r, w, eps, forms="hyqv", in_place=False):
    n, H = x.shape
    want_h = stored(x, r)
    out = {}
    if "h" in forms and r is not None:
        out["h"] = r if in_place else torch.full((n + 1, H), 7.0, dtype=r.dtype, device=DEV)[:n]
    if "y" in forms:
        out["y"] = x if in_place else torch.full((n + 1, H), 7.0, dtype=torch.bfloat16, device=DEV)[:n]
    if "q" in forms:
        out["q"], out["q_scale"] = bytes_like((n + 1, U.quant_pitch(H)))[:n], bytes_like((n + 1, U.quant_scale_pitch(H)))[:n]
    if "v" in forms:
        out["rstd"] = torch.full((n,), 7.0, device=DEV)
    U.ultraep_residual_norm(ctx_of(8), x, w, eps, residual=r, **out)
    torch.cuda.synchronize()
    v, y = Y.residual_norm(want_h, host(w), float(np.float32(eps)))
    slack = norm_slack(H)
    if "h" in out:
        assert np.array_equal(host(out["h"]), want_h)
    if "rstd" in out:
        assert (np.abs(host(out["rstd"]) - v) <= slack * v).all()
    rel = (slack + 3 * F32_STEP) * np.abs(y)
    if "y" in out:
        assert (np.abs(host(out["y"]) - y) <= rel + BF16_STEP * (np.abs(y) + rel)).all()
    if "q" in out:
        check_rows_form(host(out["q"]), host(out["q_scale"]), y, rel, H)
    for name, t in out.items():
        if not in_place and name != "rstd":
            whole = t._base if t._base is not None else t
            assert (whole[n:] == (SENT if t.dtype == torch.uint8 else 7)).all(), name


@pytest.mark.parametrize("H", WIDTHS)
@pytest.mark.parametrize("dtype", [None, torch.bfloat16, torch.float32])
def test_norm(H, dtype):
    rng = np.random.default_rng(H)
    for rows in (1, 5, 131 if H <= 8192 else 19):
        for w32 in (False, True):
            x, r, w = norm_case(rng, rows, H, dtype, w32)
            check_norm(x, r, w, 1e-6)
    for forms in ("h", "y", "q", "v", "hq", "yv") if dtype is not None else ("y", "q", "v"):
        check_norm(*norm_case(rng, 7, H, dtype, True), 1e-5, forms)
    if dtype is not torch.float32:
        check_norm(*norm_case(rng, 7, H, dtype, True), 1e-5, "hy", in_place=True)
    else:
        check_norm(*norm_case(rng, 7, H, dtype, True), 1e-5, "h", in_place=True)


@pytest.mark.parametrize("H", [64, 4096, 7168])
def test_norm_of_unusual_rows(H):
    """Rows of zeros, tiny, large and not finite ones; eps of zero; more rows than workgroups."""
    rng = np.random.default_rng(1)
    x, r, w = norm_case(rng, 12, H, torch.bfloat16, True)
    r[0], x[0] = 0, 0
    r[1], x[1] = 0, x[1] * 2.0 ** -60
    r[2], x[2] = 0, x[2] * 2.0 ** 55
    r[3] = -x[3]
    check_norm(x, r, w, 1e-6)
    w[5] = 0
    x[4:], r[4:] = 1.0, 0
    check_norm(x[4:].clone(), r[4:].clone(), w, 0.0)
    bad = x.clone()
    bad[0, 3], bad[1, 3] = float("nan"), float("inf")
    y = torch.empty_like(x)
    q, s = bytes_like((12, U.quant_pitch(H))), bytes_like((12, U.quant_scale_pitch(H)))
    U.ultraep_residual_norm(ctx_of(8), bad, w, 1e-6, y=y, q=q, q_scale=s)
    good = torch.empty_like(x)
    U.ultraep_residual_norm(ctx_of(8), x, w, 1e-6, y=good)
    assert torch.equal(y[2:], good[2:]) and y[0].isnan().all() and y[1, 3].isnan()
    q = q.view(torch.float8_e4m3fn).float()
    assert q[0, :H].isnan().all() and q[1, 3].isnan() and (q[:, H:] == 0).all() and not q[2:].isnan().any()
    check_norm(*norm_case(rng, 5003, 64, torch.float32, False), 1e-6)


def norm_blocks_slack(rows):
    return (rows / 256 + 8) * F32_STEP


def check_norm_backward(rng, rows, H, dtype, w32, with_in=True, with_x=True, weight="new", in_place=False):
    h = stream_of(rng.standard_normal((rows, H)) * np.exp(rng.standard_normal(H)), dtype)
    g = dev(to_bf16(rng.standard_normal((rows, H)) * 0.1)[0]).view(torch.bfloat16)
    w = torch.from_numpy((1 + 0.2 * rng.standard_normal(H)).astype(np.float32)).to(DEV)
    w = w if w32 else w.bfloat16()
    v = torch.from_numpy((1 / np.sqrt((host(h) ** 2).mean(1) + 1e-6)).astype(np.float32)).to(DEV)
    back = stream_of(rng.standard_normal((rows, H)) * 0.1, dtype) if with_in else None
    want, mag, want_w, mag_w = Y.residual_norm_backward(host(g), host(h), host(w), host(v), None if back is None else host(back))
    to = back if in_place else torch.full((rows + 1, H), 7.0, dtype=dtype, device=DEV)[:rows]
    kw = dict(grad_in=back)
    if dtype == torch.float32 and with_x:
        kw["grad_x"] = torch.full((rows + 1, H), 7.0, dtype=torch.bfloat16, device=DEV)[:rows]
    before = np.zeros(H)
    if weight:
        kw["grad_weight"] = torch.full((H,), 3.0, device=DEV)
        kw["workspace"] = torch.full((U.residual_norm_workspace_bytes(rows, H),), 0xFF, dtype=torch.uint8, device=DEV)
        kw["accumulate"] = weight == "add"
        before += 3.0 if weight == "add" else 0.0
    U.ultraep_residual_norm_backward(ctx_of(8), g, h, w, v, to, **kw)
    torch.cuda.synchronize()
    slack = (2 * norm_slack(H) + 6 * F32_STEP) * mag
    step = BF16_STEP if dtype == torch.bfloat16 else F32_STEP
    assert (np.abs(host(to) - want) <= slack + step * (np.abs(want) + slack)).all()
    if "grad_x" in kw:
        assert torch.equal(kw["grad_x"], to.bfloat16())
        assert (kw["grad_x"]._base[rows:] == 7).all()
    if weight:
        total = want_w + before
        assert (np.abs(host(kw["grad_weight"]) - total) <= norm_blocks_slack(rows) * mag_w + F32_STEP * np.abs(total)).all()
    if not in_place:
        assert (to._base[rows:] == 7).all()


@pytest.mark.parametrize("H", WIDTHS)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_norm_backward(H, dtype):
    rng = np.random.default_rng(H)
    for rows in (1, 5, 131 if H <= 8192 else 19):
        check_norm_backward(rng, rows, H, dtype, True)
    check_norm_backward(rng, 6, H, dtype, False, with_in=False, weight="add")
    check_norm_backward(rng, 6, H, dtype, True, with_x=False, weight=None)
    check_norm_backward(rng, 6, H, dtype, False, in_place=True)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_norm_backward_of_many_rows(dtype):
    check_norm_backward(np.random.default_rng(2), 5003, 64, dtype, True)
    check_norm_backward(np.random.default_rng(2), 3001, 520, dtype, True, weight="add")


def test_norm_without_rows():
    H = 64
    x, w, v = torch.empty(0, H, dtype=torch.bfloat16, device=DEV), torch.ones(H, device=DEV), torch.empty(0, device=DEV)
    U.ultraep_residual_norm(ctx_of(8), x, w, 1e-6, y=x, rstd=v)
    g = torch.full((H,), 5.0, device=DEV)
    U.ultraep_residual_norm_backward(ctx_of(8), x, x, w, v, x, grad_weight=g, workspace=v, accumulate=True)
    assert (g == 5).all()
    U.ultraep_residual_norm_backward(ctx_of(8), x, x, w, v, x, grad_weight=g, workspace=v)
    assert (g == 0).all()


# ---------------------------------------------------------------- gated activation

def glu_case(rng, rows, F):
    return to_bf16(rng.standard_normal((rows, 2 * F)) * np.exp(rng.standard_normal(2 * F)))


def run_glu(seg, h, F, grad, gelu, rows_form, cols_form, capacity):
    W = F if grad is None else 2 * F
    kw = {}
    n, blocks = max(seg.rows, capacity) + 3, U.quant_blocks(capacity, seg.ne) + 1
    if rows_form:
        kw.update(q=bytes_like((n, U.quant_pitch(W))), q_scale=bytes_like((n, U.quant_scale_pitch(W))))
    if cols_form:
        kw.update(qt=bytes_like((blocks, W, 128)), qt_scale=bytes_like((blocks, W)))
    args = (seg.ctx, seg.plan, h) + (() if grad is None else (grad,))
    f = U.ultraep_glu_quant if grad is None else U.ultraep_glu_quant_backward
    f(*args, seg.p0, seg.p1, activation=int(gelu), rows=capacity, **kw)
    torch.cuda.synchronize()
    return {k: host(v) for k, v in kw.items()}


def check_glu(seg, bits, values, F, gelu, grad=None, capacity=None):
    """grad: (bits, values) of the activation's gradients, or None."""
    cap = seg.rows if capacity is None else capacity
    live = min(seg.rows, cap)
    h = dev(bits).view(torch.bfloat16)
    if grad is None:
        want = Y.glu(values, gelu)
        rel = 2.0 ** -14 * np.abs(want) + np.where(np.abs(want) < 2.0 ** -99, 2.0 ** -100, 0)
    else:
        want, mag = Y.glu_backward(values, grad[1], gelu)
        rel = 2.0 ** -14 * mag + np.where(np.abs(want) < 2.0 ** -99, 2.0 ** -100, 0)
    want, rel = want[:live], rel[:live]
    W, off = want.shape[1], np.minimum(seg.off, live).tolist()
    g = None if grad is None else dev(grad[0]).view(torch.bfloat16)
    both = run_glu(seg, h, F, g, gelu, True, True, cap)
    check_rows_form(both["q"][:live], both["q_scale"][:live], want, rel, W)
    assert (both["q"][live:] == SENT).all() and (both["q_scale"][live:] == SENT).all()
    check_cols_form(both["qt"], both["qt_scale"], want, rel, off, U.quant_blocks(cap, seg.ne) + 1)
    rows, cols = run_glu(seg, h, F, g, gelu, True, False, cap), run_glu(seg, h, F, g, gelu, False, True, cap)
    for k in ("q", "q_scale"):
        assert np.array_equal(rows[k], both[k])
    for k in ("qt", "qt_scale"):
        assert np.array_equal(cols[k], both[k])


@pytest.mark.parametrize("loads", LOADS)
@pytest.mark.parametrize("F", [8, 64, 120, 128, 200, 520, 1024])
@pytest.mark.parametrize("back", [False, True])
def test_glu(loads, F, back):
    rng = np.random.default_rng(F)
    seg = Segment(loads, p0=2, before=5)
    bits, values = glu_case(rng, seg.rows, F)
    grad = to_bf16(rng.standard_normal((seg.rows, F)) * 0.01) if back else None
    for gelu in (False, True):
        check_glu(seg, bits, values, F, gelu, grad)
    if seg.rows > 4:
        check_glu(seg, bits, values, F, False, grad, capacity=seg.rows // 2)
        check_glu(seg, np.concatenate([bits, bits]), np.concatenate([values, values]), F, False,
                  None if grad is None else tuple(np.concatenate([x, x]) for x in grad), capacity=2 * seg.rows)


@pytest.mark.parametrize("gelu", [False, True])
@pytest.mark.parametrize("back", [False, True])
def test_glu_of_the_whole_range(gelu, back):
    """Gates from the most negative to the largest: nothing of them is NaN that is finite in fp32."""
    rng = np.random.default_rng(9)
    F, rows = 256, 130
    seg = Segment([rows])
    x = rng.standard_normal((rows, 2 * F))
    x[:, :F] = np.linspace(-130, 130, F) + 0.5 * x[:, :F]
    x[:4, :F] *= 1e3
    x[4, :F], x[5, :F] = np.logspace(-38, 37, F), -np.logspace(-38, 37, F)
    x[6] = 0.0
    x[7, F:] = 0.0
    x[8, :F] = -1.2784645
    bits, values = to_bf16(x)
    grad = to_bf16(rng.standard_normal((rows, F)) * np.exp(3 * rng.standard_normal((rows, 1)))) if back else None
    check_glu(seg, bits, values, F, gelu, grad)


@pytest.mark.parametrize("back", [False, True])
def test_glu_of_what_is_not_finite(back):
    F, rows = 128, 40
    rng = np.random.default_rng(10)
    seg = Segment([rows])
    bits, values = glu_case(rng, rows, F)
    h = dev(bits).view(torch.bfloat16)
    h[3, 5], h[4, F + 6], h[5, F + 7] = float("nan"), float("nan"), float("inf")
    g = None
    if back:
        g = dev(to_bf16(rng.standard_normal((rows, F)))[0]).view(torch.bfloat16)
        g[6, 8] = float("inf")
    got = run_glu(seg, h, F, g, False, True, True, rows)
    good = dev(bits).view(torch.bfloat16)
    v = X.VALUES[got["q"][:rows]]
    bad = np.zeros((rows, F), dtype=bool)
    bad[3, 5] = bad[4, 6] = bad[5, 7] = True
    if back:
        first, second = bad.copy(), bad.copy()
        first[6, 8] = second[6, 8] = True
        second[4, 6] = second[5, 7] = False   # the other half's gradient does not have the factor
        bad = np.concatenate([first, second], axis=1)
    assert np.array_equal(np.isnan(v), bad)
    assert np.array_equal(np.isnan(X.VALUES[got["qt"][0]].T[:rows]), bad)
    g2 = None if g is None else torch.where(g.isfinite(), g, 0)
    other = run_glu(seg, torch.where(h.isfinite(), h, 0), F, g2, False, True, True, rows)
    clean = ~bad.any(axis=1)
    assert np.array_equal(got["q"][:rows][clean], other["q"][:rows][clean])


def test_glu_without_rows_or_experts():
    seg = Segment([0, 0])
    h = torch.zeros(4, 64, dtype=torch.bfloat16, device=DEV)
    q, s = bytes_like((4, 128)), bytes_like((4, 4))
    U.ultraep_glu_quant(seg.ctx, seg.plan, h, 0, 2, q, s)
    U.ultraep_glu_quant(seg.ctx, seg.plan, h, 1, 1, q, s)
    U.ultraep_glu_quant_backward(seg.ctx, seg.plan, h, h[:, :32].contiguous(), 0, 2, q, s, rows=0)
    torch.cuda.synchronize()
    assert (q == SENT).all() and (s == SENT).all()

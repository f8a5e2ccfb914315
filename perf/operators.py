"""The experts' operators, measured: 8-bit quantisers, grouped products, weight gradients, gradient norm and clipping.

Values are e4m3 with one power-of-two scale for each block of 128, held as the byte 127 + exponent.  A rank's segment is
its physical experts' rows, one expert after another (offsets `off`); rows, columns and blocks are laid out as the
framework's entry points document them.  The plain forms compute in 32 bits and round once.
"""
import math

import torch

own = False

DEV = "cuda"
BLOCK = 128


def listed():
    return [
        # one serving step's rows on their way to the experts: latency
        dict(name="quant decode", op="quant", rows=93, experts=6, H=7168, tokens=512, gather=True, cols=False),
        # a training microbatch's rows of one rank, gathered from all ranks' tokens; the forward needs the row form only
        dict(name="quant dispatch", op="quant", rows=32771, experts=6, H=7168, tokens=32768, gather=True, cols=False),
        # gradient rows already in the layout, quantised both ways for the input and the weight gradients
        dict(name="quant gradients", op="quant", rows=16411, experts=4, H=4096, tokens=0, gather=False, cols=True),
        # weights after an optimizer step: small down projections, and a rank's large ones, each with its transpose
        dict(name="weights small", op="weights", experts=2, N=4096, K=1536),
        dict(name="weights large", op="weights", experts=6, N=4096, K=7168),
        # a serving step: few rows an expert, the weights are the traffic
        dict(name="gemm decode", op="gemm", rows=41, experts=6, N=4096, K=7168),
        # many experts with some tens of rows each
        dict(name="gemm ragged", op="gemm", rows=1531, experts=24, N=2048, K=5120),
        # a training microbatch's up projection
        dict(name="gemm training", op="gemm", rows=32768, experts=6, N=4096, K=7168),
        # weight gradients: a short microbatch, a full one
        dict(name="wgrad short", op="wgrad", rows=2999, experts=4, N=1536, K=5120),
        dict(name="wgrad training", op="wgrad", rows=32768, experts=6, N=4096, K=7168),
        # norm and clipping over a layer's small tensors, and over a rank's expert gradients with their small neighbours
        dict(name="clip small", op="clip", tensors=37, elements=600_011, bf16=True),
        dict(name="clip experts", op="clip", tensors=211, elements=400_000_003, bf16=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["quant", "weights", "gemm", "wgrad", "clip"])
    experts = _log(rng, 1, 32)
    if op == "quant":
        gather = rng.random() < 0.5
        return dict(op=op, rows=_log(rng, 1, 20000), experts=experts, H=8 * _log(rng, 8, 896), tokens=_log(rng, 64, 32768) if gather else 0,
                    gather=gather, cols=rng.random() < 0.5)
    if op == "weights":
        return dict(op=op, experts=_log(rng, 1, 6), N=8 * _log(rng, 8, 512), K=8 * _log(rng, 8, 896))
    if op in ("gemm", "wgrad"):
        return dict(op=op, rows=_log(rng, 1, 20000), experts=min(experts, 12) if op == "wgrad" else experts, N=8 * _log(rng, 8, 480), K=8 * _log(rng, 8, 640))
    return dict(op=op, tensors=_log(rng, 1, 400), elements=_log(rng, 1000, 300_000_000), bf16=rng.random() < 0.5)


def work(case):
    op = case["op"]
    if op == "quant":
        n = case["rows"] * case["H"]
        return {"bytes": 2 * min(n, case["tokens"] * case["H"] if case["gather"] else n) + (2 if case["cols"] else 1) * (n + n / BLOCK), "flops": 2 * n}
    if op == "clip":
        size = 2 if case["bf16"] else 4
        return {"bytes": 2 * size * case["elements"], "flops": 3 * case["elements"]}
    full = case["experts"] * case["N"] * case["K"]
    if op == "weights":
        return {"bytes": 4 * full, "flops": 2 * full}
    live = min(case["experts"], case["rows"]) * case["N"] * case["K"]
    flops = 2 * case["rows"] * case["N"] * case["K"]
    if op == "gemm":
        return {"bytes": case["rows"] * (case["K"] + 2 * case["N"]) + live, "flops": flops}
    return {"bytes": case["rows"] * (case["K"] + case["N"]) + 4 * full, "flops": flops}


# ---------------------------------------------------------------- the format, plainly

def _up(n, m=BLOCK):
    return -(-n // m) * m


def _exponent(amax):
    """Smallest e with amax / 2^e <= 448 = 1.75 * 2^8, from the float's own bits; 0 for an empty block."""
    bits = amax.view(torch.int32)
    e = (bits >> 23) - 135 + ((bits & 0x7FFFFF) > 0x600000).int()
    return torch.where(amax == 0, 0, e.clamp(min=-126))


def _pow2(e):
    return ((e + 127) << 23).view(torch.float32)


def _amax(x, dim):
    return torch.where(x.isfinite(), x.abs(), 0).amax(dim)


def _plain_quant(s):
    H, rows = s["H"], s["rows"]
    x = (s["hidden"][s["inv"].long() // s["k"]] if s["inv"] is not None else s["hidden"]).float()
    kb = _up(H) // BLOCK
    g = torch.nn.functional.pad(x, (0, _up(H) - H)).view(rows, kb, BLOCK)
    e = _exponent(_amax(g, 2))
    scale = torch.full((rows, _up(kb, 4)), 127, dtype=torch.uint8, device=DEV)
    scale[:, :kb] = (e + 127).to(torch.uint8)
    out = {"q": (g * _pow2(-e)[:, :, None]).to(torch.float8_e4m3fn).view(rows, kb * BLOCK), "scale": scale}
    if s["cols"]:
        i = torch.arange(rows, device=DEV)
        p = torch.searchsorted(s["off"], i, right=True) - 1
        first = s["off"][p]
        b, r = first // BLOCK + p + (i - first) // BLOCK, (i - first) % BLOCK
        c = torch.zeros(s["blocks"], BLOCK, H, device=DEV)
        c[b, r] = x
        e = _exponent(_amax(c, 1))
        used = torch.zeros(s["blocks"], 1, dtype=torch.bool, device=DEV)
        used[b] = True
        out["qt"] = (c * _pow2(-e)[:, None]).transpose(1, 2).contiguous().to(torch.float8_e4m3fn)
        out["scale_t"] = torch.where(used, e + 127, 0).to(torch.uint8)
    return out


def _quant_blocks(w):
    n, N, K = w.shape
    nb, kb = _up(N) // BLOCK, _up(K) // BLOCK
    g = torch.nn.functional.pad(w, (0, _up(K) - K, 0, _up(N) - N)).view(n, nb, BLOCK, kb, BLOCK)
    e = _exponent(_amax(g, (2, 4)))
    q = (g * _pow2(-e)[:, :, None, :, None]).view(n, nb * BLOCK, kb * BLOCK)[:, :N].to(torch.float8_e4m3fn)
    scale = torch.full((n, nb, _up(kb, 4)), 127, dtype=torch.uint8, device=DEV)
    scale[:, :, :kb] = (e + 127).to(torch.uint8)
    return q, scale


def _plain_weights(s):
    w = s["w"].float()
    q, scale = _quant_blocks(w)
    qt, scale_t = _quant_blocks(w.transpose(1, 2))
    return {"q": q, "scale": scale, "qt": qt, "scale_t": scale_t}


def _value(q, scale, rows_per_scale=1):
    """float32 values of row-form q [..., R, Kp] with scale bytes [..., R / rows_per_scale, >= Kp / 128]."""
    e = scale[..., :q.shape[-1] // BLOCK].int() - 127
    e = e.repeat_interleave(rows_per_scale, -2)[..., :q.shape[-2], :]
    return q.view(torch.float8_e4m3fn).float() * _pow2(e).repeat_interleave(BLOCK, -1)


def _plain_gemm(s):
    x, w = _value(s["q"], s["scale"]), _value(s["w"], s["w_scale"], BLOCK)
    o = s["offsets"]
    return torch.cat([x[o[p]:o[p + 1]] @ w[p].t() for p in range(len(o) - 1)]).bfloat16()


def _plain_wgrad(s):
    dy = s["dyt"].view(torch.float8_e4m3fn).float() * _pow2(s["dyt_scale"].int() - 127)[..., None]
    x = s["xt"].view(torch.float8_e4m3fn).float() * _pow2(s["xt_scale"].int() - 127)[..., None]
    b = s["first_block"]
    flat = lambda t, p: t[b[p]:b[p + 1]].transpose(0, 1).reshape(t.shape[1], -1)  # noqa: E731
    return torch.stack([flat(dy, p) @ flat(x, p).t() for p in range(len(b) - 1)])


def _plain_clip(s):
    g = s["flat"].float()
    sumsq = g.square().sum(dtype=torch.float64)
    coef = (s["max_norm"] / (sumsq.sqrt() + 1e-6)).clamp(max=1.0)
    return {"norm": sumsq.sqrt().float(), "out": (g * coef.float()).to(s["flat"].dtype)}


# ---------------------------------------------------------------- states

def _offsets(case, gen):
    """Row offsets of a segment's experts: popularity is skewed, and with few rows some experts get none."""
    n = case["experts"]
    pop = torch.rand(n, generator=gen).pow(2) + 0.05
    ids = torch.multinomial(pop, case["rows"], replacement=True, generator=gen)
    return [0] + torch.bincount(ids, minlength=n).cumsum(0).tolist()


def _first_blocks(o):
    return [o[p] // BLOCK + p for p in range(len(o))]


def _rows_like(shape, gen):
    """bf16 activations: normal values with a spread of magnitudes over the columns and a few large ones."""
    x = torch.empty(shape, dtype=torch.bfloat16, device=DEV)
    x.normal_(generator=gen)
    return x.mul_(torch.empty(shape[-1], device=DEV).normal_(generator=gen).exp_().bfloat16())


def _e4m3_like(shape, gen):
    """e4m3 bytes as a quantiser leaves them: normal values, the largest of 128 near 448."""
    q = torch.empty(shape, dtype=torch.uint8, device=DEV)
    for part in q.view(-1, BLOCK).split(1 << 18):
        part.copy_(torch.empty(part.shape, device=DEV).normal_(0, 120, generator=gen).clamp_(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8))
    return q


def _exponents_like(shape, gen):
    return torch.randint(112, 122, shape, dtype=torch.uint8, device=DEV, generator=gen)


def _plan(s, case, o):
    """What a user of the entry points holds besides: a context, and the plan record whose segment [0, experts) has the offsets `o`."""
    import moe_expert_load_ultraep_amd as U
    R = -(-case["experts"] // 4)
    ctx = U.ultraep_create(4 * R, R, 0, 1)
    at = ctx.fields["phys_off"][0]
    words = torch.zeros(ctx.plan_words, dtype=torch.int32)
    words[at:at + 4 * R + 1] = o[-1]
    words[at:at + len(o)] = torch.tensor(o, dtype=torch.int32)
    s.update(U=U, ctx=ctx, plan=words.to(DEV))


def _table(tensors):
    return torch.tensor([t.data_ptr() for t in tensors], dtype=torch.int64).to(DEV)


def prepare(case, seed):
    cpu, gen = torch.Generator().manual_seed(seed), torch.Generator(DEV).manual_seed(seed)
    op = case["op"]
    s = {"op": op}
    if op == "clip":
        sizes = torch.rand(case["tensors"], generator=cpu, dtype=torch.float64).pow(4) + 1e-4
        ends = (sizes.cumsum(0) / sizes.sum() * case["elements"]).long()
        ends[-1] = case["elements"]
        dtype = torch.bfloat16 if case["bf16"] else torch.float32
        s["flat"] = torch.empty(case["elements"], dtype=dtype, device=DEV).normal_(0, 0.01, generator=gen)
        s["out"] = torch.empty_like(s["flat"])
        s["max_norm"] = 1.0 if case["elements"] > 100_000 else 0.1
        ends = [0] + ends.tolist()
        s["tensors"] = _table([s["flat"][a:b] for a, b in zip(ends, ends[1:])])
        s["outs"] = _table([s["out"][a:b] for a, b in zip(ends, ends[1:])])
        s["numels"] = torch.tensor([b - a for a, b in zip(ends, ends[1:])], dtype=torch.int64).to(DEV)
        s["sumsq"], s["norm"] = torch.empty(1, dtype=torch.float64, device=DEV), torch.empty(1, dtype=torch.float32, device=DEV)
        if own:
            import moe_expert_load_ultraep_amd as U
            s.update(U=U, ctx=U.ultraep_create(8, 4, 0, 1), workspace=torch.empty(U.GRAD_WORKSPACE_BYTES, dtype=torch.uint8, device=DEV))
        return s
    n = s["experts"] = case["experts"]
    if op == "weights":
        N, K = s["N"], s["K"] = case["N"], case["K"]
        s["w"] = torch.empty(n, N, K, dtype=torch.bfloat16, device=DEV).normal_(0, 0.02, generator=gen)
        s["table"] = _table(s["w"])
        for name, a, b in (("", N, K), ("t", K, N)):
            s["q" + name] = torch.empty(n, a, _up(b), dtype=torch.uint8, device=DEV)
            s["scale" + name] = torch.empty(n, _up(a) // BLOCK, _up(_up(b) // BLOCK, 4), dtype=torch.uint8, device=DEV)
        if own:
            _plan(s, case, [0] * (n + 1))
        return s
    o = s["offsets"] = _offsets(case, cpu)
    rows = s["rows"] = case["rows"]
    s["off"] = torch.tensor(o, dtype=torch.int64).to(DEV)
    s["blocks"] = rows // BLOCK + n
    if own:
        _plan(s, case, o)
    if op == "quant":
        H, k = s["H"], s["k"] = case["H"], 8
        s["cols"] = case["cols"]
        s["hidden"] = _rows_like((case["tokens"] or rows, H), gen)
        s["inv"] = None
        if case["gather"]:  # each expert's pairs in ascending order, as the layout lists them
            pair = torch.randint(0, case["tokens"] * k, (rows,), generator=cpu)
            expert = torch.bucketize(torch.arange(rows), torch.tensor(o[1:]), right=True)
            s["inv"] = (pair + expert * (case["tokens"] * k)).sort()[0].remainder(case["tokens"] * k).int().to(DEV)
        s["q"] = torch.zeros(rows, _up(H), dtype=torch.uint8, device=DEV)
        s["scale"] = torch.zeros(rows, _up(_up(H) // BLOCK, 4), dtype=torch.uint8, device=DEV)
        if case["cols"]:
            s["qt"] = torch.zeros(s["blocks"], H, BLOCK, dtype=torch.uint8, device=DEV)
            s["scale_t"] = torch.zeros(s["blocks"], H, dtype=torch.uint8, device=DEV)
        return s
    N, K = s["N"], s["K"] = case["N"], case["K"]
    if op == "gemm":
        kb = _up(K) // BLOCK
        s["q"], s["w"] = _e4m3_like((rows, _up(K)), gen), _e4m3_like((n, N, _up(K)), gen)
        s["q"][:, K:], s["w"][:, :, K:] = 0, 0
        s["scale"] = _exponents_like((rows, _up(kb, 4)), gen)
        s["w_scale"] = _exponents_like((n, _up(N) // BLOCK, _up(kb, 4)), gen)
        s["w_table"], s["w_scale_table"] = _table(s["w"]), _table(s["w_scale"])
        s["out"] = torch.empty(rows, N, dtype=torch.bfloat16, device=DEV)
        return s
    b = s["first_block"] = _first_blocks(o)
    row = torch.arange(b[-1] * BLOCK).view(-1, BLOCK)  # the slots behind an expert's last row hold zeros
    block = torch.bucketize(row[:, 0] // BLOCK, torch.tensor(b[1:]), right=True).clamp(max=n - 1)
    live = (row - torch.tensor(b)[block][:, None] * BLOCK) < (torch.tensor(o)[block + 1] - torch.tensor(o)[block])[:, None]
    live = torch.nn.functional.pad(live, (0, 0, 0, s["blocks"] - live.shape[0])).to(DEV)
    for name, width in (("dyt", N), ("xt", K)):
        s[name] = _e4m3_like((s["blocks"], width, BLOCK), gen)
        s[name].mul_(live[:, None].to(torch.uint8))
        s[name + "_scale"] = _exponents_like((s["blocks"], width), gen)
    s["grads"] = torch.empty(n, N, K, dtype=torch.float32, device=DEV)
    s["grad_table"] = _table(s["grads"])
    return s


# ---------------------------------------------------------------- one pass

def run(s):
    if not own:
        return {"quant": _plain_quant, "weights": _plain_weights, "gemm": _plain_gemm, "wgrad": _plain_wgrad, "clip": _plain_clip}[s["op"]](s)
    U, ctx, op = s["U"], s["ctx"], s["op"]
    f8 = torch.float8_e4m3fn
    if op == "quant":
        cols = {"qt": s["qt"], "qt_scale": s["scale_t"]} if s["cols"] else {}
        U.ultraep_permute_quant(ctx, s["plan"], s["inv"], s["k"], s["hidden"], 0, s["experts"], s["q"], s["scale"], **cols)
        return {"q": s["q"].view(f8), "scale": s["scale"], **({"qt": s["qt"].view(f8), "scale_t": s["scale_t"]} if s["cols"] else {})}
    if op == "weights":
        U.ultraep_weight_quant(ctx, s["table"], s["experts"], s["N"], s["K"], s["q"], s["scale"], s["qt"], s["scalet"])
        return {"q": s["q"].view(f8), "scale": s["scale"], "qt": s["qt"].view(f8), "scale_t": s["scalet"]}
    if op == "gemm":
        U.ultraep_expert_gemm(ctx, s["plan"], s["q"], s["scale"], s["K"], s["w_table"], s["w_scale_table"], s["N"], 0, s["experts"], s["out"])
        return s["out"]
    if op == "wgrad":
        U.ultraep_expert_wgrad(ctx, s["plan"], s["dyt"], s["dyt_scale"], s["N"], s["xt"], s["xt_scale"], s["K"], 0, s["experts"], s["rows"], s["grad_table"])
        return s["grads"]
    n = s["numels"].numel()
    U.ultraep_grad_sumsq(ctx, s["tensors"], s["numels"], n, s["flat"].dtype, s["sumsq"], s["workspace"])
    U.ultraep_grad_clip(ctx, s["tensors"], s["numels"], n, s["flat"].dtype, s["sumsq"], s["max_norm"], s["norm"], out=s["outs"])
    return {"norm": s["norm"][0], "out": s["out"]}


# ---------------------------------------------------------------- the definitions in 64 bits

def _exact_blocks(g):
    """Quantised values of blocks that lie along the last dimension, and the exponents."""
    amax = torch.where(g.isfinite(), g.abs(), 0).amax(-1, keepdim=True)
    e = torch.ceil(torch.log2(torch.where(amax == 0, 448.0, amax) / 448.0)).clamp(min=-126)
    v = g / torch.exp2(e)
    step = torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6))) - 3)
    return torch.round(v / step) * step, (e[..., 0] + 127).to(torch.uint8)


def _exact_rows(x):
    rows, H = x.shape
    padded = x.new_zeros(rows, _up(H))
    padded[:, :H] = x
    v, byte = _exact_blocks(padded.view(rows, -1, BLOCK))
    scale = byte.new_full((rows, _up(byte.shape[1], 4)), 127)
    scale[:, :byte.shape[1]] = byte
    return v.view(rows, -1), scale


def _exact_weight(w):
    N, K = w.shape
    nb, kb = _up(N) // BLOCK, _up(K) // BLOCK
    padded = w.new_zeros(_up(N), _up(K))
    padded[:N, :K] = w
    v, byte = _exact_blocks(padded.view(nb, BLOCK, kb, BLOCK).permute(0, 2, 1, 3).reshape(nb, kb, -1))
    scale = byte.new_full((nb, _up(kb, 4)), 127)
    scale[:, :kb] = byte
    return v.view(nb, kb, BLOCK, BLOCK).permute(0, 2, 1, 3).reshape(_up(N), _up(K))[:N], scale


def exact(case, seed):
    s = prepare(case, seed)
    op = s["op"]
    f8 = torch.float8_e4m3fn
    if op == "clip":
        g = s["flat"].double()
        norm = torch.linalg.vector_norm(g)
        return {"norm": norm, "out": g.mul_(min(1.0, s["max_norm"] / (norm.item() + 1e-6)))}
    if op == "weights":
        got = [[f(s["w"][p].double()) for p in range(s["experts"])] for f in (_exact_weight, lambda w: _exact_weight(w.t()))]
        (q, scale), (qt, scale_t) = [[torch.stack(list(t)) for t in zip(*side)] for side in got]
        return {"q": q, "scale": scale, "qt": qt, "scale_t": scale_t}
    o = s["offsets"]
    if op == "quant":
        pick = torch.arange(s["rows"], device=DEV) if s["inv"] is None else torch.div(s["inv"], s["k"], rounding_mode="floor").long()
        x = s["hidden"].double()[pick]
        q, scale = _exact_rows(x)
        out = {"q": q.float(), "scale": scale}
        if s["cols"]:
            out["qt"] = torch.zeros(s["blocks"], s["H"], BLOCK, device=DEV)
            out["scale_t"] = torch.zeros(s["blocks"], s["H"], dtype=torch.uint8, device=DEV)
            for p in range(s["experts"]):
                for i, at in enumerate(range(o[p], o[p + 1], BLOCK)):
                    part = x[at:min(at + BLOCK, o[p + 1])]
                    block = part.new_zeros(BLOCK, s["H"])
                    block[:part.shape[0]] = part
                    v, byte = _exact_blocks(block.t())
                    out["qt"][o[p] // BLOCK + p + i], out["scale_t"][o[p] // BLOCK + p + i] = v.float(), byte
        return out
    if op == "gemm":
        out = torch.empty(s["rows"], s["N"], dtype=torch.float64, device=DEV)
        kb = _up(s["K"]) // BLOCK
        x = s["q"].view(f8).double().view(s["rows"], kb, BLOCK) * torch.exp2(s["scale"][:, :kb].double() - 127)[..., None]
        for p in range(s["experts"]):
            e = torch.exp2(s["w_scale"][p, :, :kb].double() - 127)
            w = s["w"][p].view(f8).double().view(s["N"], kb, BLOCK) * e[torch.arange(s["N"], device=DEV) // BLOCK][..., None]
            out[o[p]:o[p + 1]] = torch.mm(x[o[p]:o[p + 1]].reshape(-1, kb * BLOCK), w.view(s["N"], -1).t())
        return out
    out = torch.empty(s["experts"], s["N"], s["K"], dtype=torch.float64, device=DEV)
    for p in range(s["experts"]):
        part = slice(o[p] // BLOCK + p, o[p] // BLOCK + p + -(-(o[p + 1] - o[p]) // BLOCK))
        dy, x = ((s[t][part].view(f8).double() * torch.exp2(s[t + "_scale"][part].double() - 127)[..., None]).permute(0, 2, 1) for t in ("dyt", "xt"))
        out[p] = torch.mm(dy.reshape(-1, s["N"]).t(), x.reshape(-1, s["K"]))
    return out

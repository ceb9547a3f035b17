"""The operators around the attention, as they are measured: the block norms with gate and
residual scale, the per-head norm and grid rotation of Q and K, and the expert sort.

Formulas (rows r, channels c, g = r // rows_per_group the row of scale, shift and gate):

  norm      z = res_scale x + gate_g ∘ [N_post(h) ∘ w_post], or z = x where there is no branch h
            y = N(z) ∘ w ∘ (1 + scale_g) + b ∘ (1 + scale_g) + shift_g
            N: layer (v - mean) / sqrt(var + eps), or rms v / sqrt(mean v² + eps)
  rotate    n = N_rms(x) ∘ w over a head's channels, then each pair (n_a, n_b) of it is turned
            by its angle: (n_a cos - n_b sin, n_a sin + n_b cos)
  experts   the slots (token, choice) sorted by expert, stably, each expert's rows from a
            multiple of `align` on; the tokens' rows copied there; the experts' outputs summed
            back with the router's weights; and the gradients of both

``run`` computes them with elementary torch operations in 32 bits, or, where ``own`` is
true, through the framework.
"""
import math

import torch

own = False

_DT = {"f32": torch.float32, "bf16": torch.bfloat16}


# ------------------------------------------------------------------ cases
def _norm_case(rows, channels, rpg, way, stream="bf16", branch="bf16", norm="layer", post="none", mod=True,
               affine=False, gated=True, res_scale=1.0):
    return {"op": "norm", "way": way, "rows": rows, "channels": channels, "rpg": rpg, "stream": stream,
            "branch": branch, "norm": norm, "post": post, "mod": mod, "affine": affine, "gated": gated,
            "res_scale": res_scale}


def _rotate_case(T, H, W, heads, d, way, dtype="bf16", pairs="interleaved", norm=True):
    return {"op": "rotate", "way": way, "T": T, "H": H, "W": W, "heads": heads, "d": d, "dtype": dtype,
            "pairs": pairs, "norm": norm}


def _expert_case(rows, k, experts, channels, way, dtype="bf16", align=1, dropped=0.0):
    return {"op": "experts", "way": way, "rows": rows, "k": k, "experts": experts, "channels": channels,
            "dtype": dtype, "align": align, "dropped": dropped}


def listed():
    named = lambda name, c: dict(c, name=name)
    return [
        # a conditional and an unconditional token (a class or register token): the call's latency
        named("norm 2 rows", _norm_case(2, 1536, 1, "fwd", gated=False)),
        # inference at 131,072 tokens, two samples: attention out, gate and next norm in one pass,
        # the residual stream kept in 32 bits
        named("gate+norm 131072x2048", _norm_case(131072, 2048, 65536, "fwd", stream="f32")),
        # the training backward of a modulated block on the 720p grid
        named("gate+norm 61440x2048 bwd", _norm_case(61440, 2048, 30720, "bwd")),
        # norms before and after a wide block, learned weights, odd number of tokens
        named("sandwich 8191x5120 bwd", _norm_case(8191, 5120, 8191, "bwd", norm="rms", post="rms", mod=False,
                                                   affine=True, res_scale=0.5)),
        # ragged everything: odd width, groups that do not divide the rows
        named("sandwich 1371x1001 f32", _norm_case(1371, 1001, 97, "bwd", stream="f32", branch="f32", norm="layer",
                                                   post="layer", affine=True)),
        # the 2K layer's Q and K before its attention
        named("rotate 2K", _rotate_case(32, 72, 128, 24, 128, "fwd")),
        # the training backward on the 720p grid
        named("rotate 720p bwd", _rotate_case(16, 48, 80, 24, 128, "bwd")),
        # one small frame, odd grid, the other pairing
        named("rotate 1x9x13 f32", _rotate_case(1, 9, 13, 5, 64, "fwd", dtype="f32", pairs="half")),
        # a handful of tokens over many experts: latency
        named("experts 8 tokens", _expert_case(8, 4, 64, 2048, "fwd")),
        # training on the 720p grid, two experts a token
        named("experts 61440x2048 train", _expert_case(61440, 2, 16, 2048, "train")),
        # many small experts, rows padded to the tiles of a grouped product
        named("experts 32768x1024 top8", _expert_case(32768, 8, 128, 1024, "fwd", align=128)),
        # odd sizes, some slots dropped (padding tokens, capacity)
        named("experts 2049x333 f32", _expert_case(2049, 3, 7, 333, "train", dtype="f32", align=4, dropped=0.2)),
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng, lo, hi):
    c = _spread(rng, lo, hi)
    step = rng.choice((1, 2, 8, 64, 128))
    return max(lo, c // step * step)


def draw(rng):
    op = rng.choice(("norm", "norm", "rotate", "experts", "experts"))
    if op == "norm":
        channels = _width(rng, 64, 8192)
        rows = _spread(rng, 1, min(131072, 200_000_000 // channels))
        rpg = rng.choice((1, rows, max(1, rows // 2), max(1, rows // 7), _spread(rng, 1, max(2, rows))))
        stream, branch = rng.choice((("bf16", "bf16"), ("f32", "bf16"), ("f32", "f32")))
        return _norm_case(rows, channels, rpg, rng.choice(("fwd", "bwd")), stream, branch,
                          rng.choice(("layer", "rms")), rng.choice(("none", "layer", "rms")),
                          rng.random() < 0.6, rng.random() < 0.5, rng.random() < 0.7, rng.choice((1.0, 0.5)))
    if op == "rotate":
        d, heads = rng.choice((64, 128)), rng.randint(1, 40)
        T, H, W = _spread(rng, 1, 32), _spread(rng, 1, 72), _spread(rng, 1, 128)
        while T * H * W * heads * d > 400_000_000:
            T = (T + 1) // 2
            heads = (heads + 1) // 2
        return _rotate_case(T, H, W, heads, d, rng.choice(("fwd", "bwd")), rng.choice(("f32", "bf16", "bf16")),
                            rng.choice(("interleaved", "half")), rng.random() < 0.7)
    channels, k = _width(rng, 64, 5120), rng.randint(1, 8)
    experts = max(k, _spread(rng, 2, 256))
    rows = _spread(rng, 1, min(65536, 200_000_000 // (channels * k)))
    return _expert_case(rows, k, experts, channels, rng.choice(("fwd", "train")), rng.choice(("f32", "bf16", "bf16")),
                        rng.choice((1, 8, 128)), rng.choice((0.0, 0.0, 0.3)))


# ------------------------------------------------------------------ inputs
def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed * 3 + 1)

    def normal(*shape, std=1.0, dt=torch.float32):
        return (torch.randn(*shape, generator=gen, device="cuda", dtype=torch.float32) * std).to(dt)

    s = {"case": dict(case)}
    if case["op"] == "norm":
        R, C = case["rows"], case["channels"]
        G = -(-R // case["rpg"])
        sdt, bdt = _DT[case["stream"]], _DT[case["branch"]]
        # a residual stream: some channels much larger than the rest, a common offset
        spread = torch.exp(normal(C, std=0.7))
        s["x"] = (normal(R, C) * spread + 0.3).to(sdt)
        s["h"] = normal(R, C, dt=bdt) if case["gated"] or case["post"] != "none" else None
        s["gate"] = normal(G, C, std=0.5) if case["gated"] else None
        s["scale"], s["shift"] = (normal(G, C, std=0.3), normal(G, C, std=0.3)) if case["mod"] else (None, None)
        s["weight"] = 1 + normal(C, std=0.2) if case["affine"] else None
        s["bias"] = normal(C, std=0.2) if case["affine"] and case["norm"] == "layer" else None
        s["post_weight"] = 1 + normal(C, std=0.2) if case["affine"] and case["post"] != "none" else None
        if case["way"] == "bwd":
            s["dz"], s["dy"] = normal(R, C, dt=sdt), normal(R, C, dt=bdt)
    elif case["op"] == "rotate":
        T, H, W, h, d = (case[k] for k in ("T", "H", "W", "heads", "d"))
        dt = _DT[case["dtype"]]
        n = d // 6
        s["axes"] = (d // 2 - 2 * n, n, n)
        parts = []
        for length, pairs in zip((T, H, W), s["axes"]):
            freq = 10000.0 ** (-torch.arange(pairs, device="cuda", dtype=torch.float64) / pairs)
            angle = torch.arange(length, device="cuda", dtype=torch.float64)[:, None] * freq
            parts.append(torch.stack((angle.cos(), angle.sin()), -1).reshape(-1, 2))
        s["table"] = torch.cat(parts).float()
        s["Q"], s["K"] = normal(T * H * W, h, d, dt=dt), normal(T * H * W, h, d, dt=dt)
        s["wq"], s["wk"] = (1 + normal(d, std=0.2), 1 + normal(d, std=0.2)) if case["norm"] else (None, None)
        if case["way"] == "bwd":
            s["dQr"], s["dKr"] = normal(T * H * W, h, d, dt=dt), normal(T * H * W, h, d, dt=dt)
    else:
        R, k, E, C = (case[n] for n in ("rows", "k", "experts", "channels"))
        dt = _DT[case["dtype"]]
        # a router whose experts are not equally liked
        logits = normal(R, E) + normal(E, std=0.7)
        top, ids = torch.topk(logits, k, dim=1)
        if case["dropped"]:
            out = torch.rand(R, k, generator=gen, device="cuda") < case["dropped"]
            ids = torch.where(out, torch.full_like(ids, -1), ids)
        s["ids"], s["weights"] = ids, torch.softmax(top, 1)
        cap = _capacity(R, k, E, case["align"])
        s["x"], s["ys"] = normal(R, C, dt=dt), normal(cap, C, dt=dt)
        s["xs"] = torch.zeros(cap, C, device="cuda", dtype=dt)
        if case["way"] == "train":
            s["dout"], s["dxs"] = normal(R, C, dt=dt), normal(cap, C, dt=dt)
            s["dys"] = torch.zeros(cap, C, device="cuda", dtype=dt)
    return s


def _capacity(rows, k, experts, align):
    """Rows that the sorted layout can take at most: each expert with rows may end in a part of a unit."""
    return rows * k + min(experts, rows * k) * (align - 1)


# ------------------------------------------------------------------ the framework's calls
def _run_own(s):
    from dynamic_block_sparse_macro_b200 import block
    c = s["case"]
    if c["op"] == "norm":
        kw = dict(gate=s["gate"], post_weight=s["post_weight"], weight=s["weight"], bias=s["bias"], scale=s["scale"],
                  norm=c["norm"], post_norm=None if c["post"] == "none" else c["post"], eps=1e-6,
                  res_scale=c["res_scale"], rows_per_group=c["rpg"])
        if c["way"] == "fwd":
            z, y = block.norm_forward(s["x"], s["h"], shift=s["shift"], out_dtype=_DT[c["branch"]], **kw)
            return {"y": y} if s["h"] is None else {"z": z, "y": y}
        g = block.norm_backward(s["x"], s["h"], s["dz"], s["dy"], **kw)
        return {n: t for n, t in g.items() if t is not None}
    if c["op"] == "rotate":
        kw = dict(grid=(c["T"], c["H"], c["W"]), axes=s["axes"], q_weight=s["wq"], k_weight=s["wk"], norm=c["norm"],
                  eps=1e-6, pairs=c["pairs"])
        if c["way"] == "fwd":
            Q, K = block.rotate_forward(s["Q"], s["K"], s["table"], **kw)
            return {"Q": Q, "K": K}
        g = block.rotate_backward(s["Q"], s["K"], s["dQr"], s["dKr"], s["table"], **kw)
        return {n: t for n, t in g.items() if t is not None}
    plan = block.expert_plan(s["ids"], c["experts"], align=c["align"])
    r = {"counts": plan.counts, "offsets": plan.offsets, "pos": plan.pos, "src": plan.src,
         "xs": block.expert_dispatch(s["x"], plan, out=s["xs"]),
         "out": block.expert_combine(s["ys"], plan, s["weights"])}
    if c["way"] == "train":
        r["dys"], r["dweights"] = block.expert_combine_backward(s["dout"], s["ys"], plan, s["weights"], out=s["dys"])
        r["dx"] = block.expert_combine(s["dxs"], plan)
    return r


# ------------------------------------------------------------------ plain forms
def _plain_stats(v, kind, eps):
    if kind == "layer":
        v = v - v.mean(-1, keepdim=True)
    r = torch.rsqrt((v * v).mean(-1, keepdim=True) + eps)
    return v * r, r


def _plain_unnorm(dn, n, r, kind):
    d = dn - n * (dn * n).mean(-1, keepdim=True)
    if kind == "layer":
        d = d - dn.mean(-1, keepdim=True)
    return d * r


def _of_rows(v, rows, rpg):
    return v[torch.arange(rows, device=v.device) // rpg]


def _group_sums(v, rpg):
    R, C = v.shape
    G = -(-R // rpg)
    if G * rpg > R:
        v = torch.cat((v, v.new_zeros(G * rpg - R, C)))
    return v.view(G, rpg, C).sum(1)


def _plain_norm(s):
    c = s["case"]
    R, rpg, eps = c["rows"], c["rpg"], 1e-6
    sdt, bdt = _DT[c["stream"]], _DT[c["branch"]]
    w = 1.0 if s["weight"] is None else s["weight"]
    b = 0.0 if s["bias"] is None else s["bias"]
    wp = 1.0 if s["post_weight"] is None else s["post_weight"]
    gate = 1.0 if s["gate"] is None else _of_rows(s["gate"], R, rpg)
    one = 1.0 if s["scale"] is None else 1 + _of_rows(s["scale"], R, rpg)
    x = s["x"].float()
    nh = rh = None
    if s["h"] is not None:
        nh = s["h"].float()
        if c["post"] != "none":
            nh, rh = _plain_stats(nh, c["post"], eps)
    if c["way"] == "fwd":
        z = x if nh is None else c["res_scale"] * x + gate * (nh * wp)
        n, _ = _plain_stats(z, c["norm"], eps)
        y = (n * w + b) * one
        if s["shift"] is not None:
            y = y + _of_rows(s["shift"], R, rpg)
        return {"y": y.to(bdt)} if nh is None else {"z": z.to(sdt), "y": y.to(bdt)}
    dy = s["dy"].float()
    n, r = _plain_stats(x, c["norm"], eps)
    dzt = s["dz"].float() + _plain_unnorm(dy * (one * w), n, r, c["norm"])
    A, D = _group_sums(dy * n, rpg), _group_sums(dy, rpg)
    scale1 = 1.0 if s["scale"] is None else 1 + s["scale"]
    g = {"dx": (dzt if nh is None else c["res_scale"] * dzt).to(sdt)}
    if nh is not None:
        t = dzt * gate
        dnh = t * wp
        g["dh"] = (dnh if rh is None else _plain_unnorm(dnh, nh, rh, c["post"])).to(bdt)
        if s["gate"] is not None:
            g["dgate"] = _group_sums(dzt * (nh * wp), rpg)
        if s["post_weight"] is not None:
            g["dpost_weight"] = (t * nh).sum(0)
    if s["weight"] is not None:
        g["dweight"] = (A * scale1).sum(0)
    if s["bias"] is not None:
        g["dbias"] = (D * scale1).sum(0)
    if s["scale"] is not None:
        g["dscale"], g["dshift"] = A * w + D * b, D
    return g


def _plain_angles(s):
    c = s["case"]
    T, H, W = c["T"], c["H"], c["W"]
    nT, nH, nW = s["axes"]
    r = torch.arange(T * H * W, device="cuda")
    tT, tH, tW = s["table"].split((T * nT, H * nH, W * nW))
    cs = torch.cat((tT.view(T, nT, 2)[r // (H * W)], tH.view(H, nH, 2)[r // W % H], tW.view(W, nW, 2)[r % W]), 1)
    return cs[:, None, :, 0], cs[:, None, :, 1]


def _split(v, pairs):
    h = v.shape[-1] // 2
    return (v[..., 0::2], v[..., 1::2]) if pairs == "interleaved" else (v[..., :h], v[..., h:])


def _join(a, b, pairs):
    return torch.stack((a, b), -1).flatten(-2) if pairs == "interleaved" else torch.cat((a, b), -1)


def _plain_rotate_one(s, x, w, cos, sin):
    v = x.float()
    if s["case"]["norm"]:
        v = _plain_stats(v, "rms", 1e-6)[0] * w
    a, b = _split(v, s["case"]["pairs"])
    return _join(a * cos - b * sin, a * sin + b * cos, s["case"]["pairs"]).to(x.dtype)


def _plain_rotate_one_bwd(s, x, w, dr, cos, sin):
    a, b = _split(dr.float(), s["case"]["pairs"])
    dn = _join(a * cos + b * sin, b * cos - a * sin, s["case"]["pairs"])
    if not s["case"]["norm"]:
        return dn.to(x.dtype), None
    n, r = _plain_stats(x.float(), "rms", 1e-6)
    return _plain_unnorm(dn * w, n, r, "rms").to(x.dtype), (dn * n).sum((0, 1))


def _plain_rotate(s):
    cos, sin = _plain_angles(s)
    if s["case"]["way"] == "fwd":
        return {"Q": _plain_rotate_one(s, s["Q"], s["wq"], cos, sin),
                "K": _plain_rotate_one(s, s["K"], s["wk"], cos, sin)}
    g = {}
    g["dQ"], g["dq_weight"] = _plain_rotate_one_bwd(s, s["Q"], s["wq"], s["dQr"], cos, sin)
    g["dK"], g["dk_weight"] = _plain_rotate_one_bwd(s, s["K"], s["wk"], s["dKr"], cos, sin)
    return {n: t for n, t in g.items() if t is not None}


def _plain_plan(ids, E, align, cap):
    R, k = ids.shape
    flat = ids.reshape(-1)
    n = flat.numel()
    valid = (flat >= 0) & (flat < E)
    key = torch.where(valid, flat, torch.full_like(flat, E))
    order = torch.sort(key, stable=True).indices
    counts = (key[:, None] == torch.arange(E, device=key.device)).sum(0)
    first = torch.cumsum(counts, 0) - counts
    units = (counts + align - 1) // align * align
    offsets = torch.cat((units.new_zeros(1), torch.cumsum(units, 0)))
    place = torch.cat((offsets[:E] - first, offsets.new_zeros(1)))[key[order]] + torch.arange(n, device=key.device)
    pos = torch.empty_like(flat)
    pos[order] = place
    pos = torch.where(valid, pos, torch.full_like(pos, -1))
    src = torch.full((cap + 1,), -1, device=key.device, dtype=torch.int64)
    src[torch.where(valid, pos, torch.full_like(pos, cap))] = torch.arange(n, device=key.device)
    return counts, offsets, pos.view(R, k), src[:cap]


def _plain_experts(s):
    c = s["case"]
    R, k = s["ids"].shape
    cap = s["xs"].shape[0]
    dt = s["x"].dtype
    counts, offsets, pos, src = _plain_plan(s["ids"], c["experts"], c["align"], cap)
    r = {n: t.to(torch.int32) for n, t in (("counts", counts), ("offsets", offsets), ("pos", pos), ("src", src))}
    there, has = (pos >= 0)[..., None], (src >= 0)[:, None]
    at, token = pos.clamp(min=0), src.clamp(min=0) // k
    zero = torch.zeros((), device="cuda")
    r["xs"] = torch.where(has, s["x"][token], zero.to(dt))
    y = torch.where(there, s["ys"][at].float(), zero)
    r["out"] = (y * s["weights"][..., None]).sum(1).to(dt)
    if c["way"] == "train":
        dout = s["dout"].float()
        dys = dout[token] * s["weights"].reshape(-1)[src.clamp(min=0)][:, None]
        r["dys"] = torch.where(has, dys, zero).to(dt)
        r["dweights"] = (y * dout[:, None]).sum(-1)
        r["dx"] = torch.where(there, s["dxs"][at].float(), zero).sum(1).to(dt)
    return r


def run(state):
    if own:
        return _run_own(state)
    return {"norm": _plain_norm, "rotate": _plain_rotate, "experts": _plain_experts}[state["case"]["op"]](state)


# ------------------------------------------------------------------ work
def work(case):
    size = {"f32": 4, "bf16": 2}
    if case["op"] == "norm":
        R, C = case["rows"], case["channels"]
        G = -(-R // case["rpg"])
        sb, bb = size[case["stream"]], size[case["branch"]]
        h = case["gated"] or case["post"] != "none"
        vectors = 4 * C * (G * (2 * case["mod"] + case["gated"]) + case["affine"] *
                           (1 + (case["norm"] == "layer") + (case["post"] != "none")))
        if case["way"] == "fwd":
            return {"bytes": R * C * (sb + bb + h * (sb + bb)) + vectors, "flops": R * C * (10 + 8 * h)}
        # z, dz, dx of the stream's type, dy and h, dh of the branch's; the vectors and their gradients
        return {"bytes": R * C * (3 * sb + bb + h * 2 * bb) + 2 * vectors, "flops": R * C * (20 + 15 * h)}
    if case["op"] == "rotate":
        n = 2 * case["T"] * case["H"] * case["W"] * case["heads"] * case["d"]
        table = 8 * (case["T"] + case["H"] + case["W"]) * case["d"] // 6
        return {"bytes": n * size[case["dtype"]] * (2 if case["way"] == "fwd" else 2 + case["norm"]) + table,
                "flops": n * (8 if case["way"] == "fwd" else 16)}
    R, k, E, C = (case[n] for n in ("rows", "k", "experts", "channels"))
    slots = R * k * (1 - case["dropped"])
    row = C * size[case["dtype"]]
    total = R * k * (8 + 4 + 4 + 4) + 8 * E + 2 * (R * row + slots * row)
    flops = 2 * slots * C
    if case["way"] == "train":
        total += R * row + 2 * slots * row + R * k * 4 + slots * row + R * row
        flops += 4 * slots * C
    return {"bytes": int(total), "flops": int(flops)}


# ------------------------------------------------------------------ 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    return {"norm": _exact_norm, "rotate": _exact_rotate, "experts": _exact_experts}[case["op"]](case, s)


def _exact_norm(case, s):
    """Group by group, from the definitions; the gradients through torch's own differentiation of them."""
    R, C, rpg = case["rows"], case["channels"], case["rpg"]
    d64 = lambda t: None if t is None else t.to(torch.float64)

    def normed(v, kind):
        mu = v.sum(1, keepdim=True) / C if kind == "layer" else 0.0
        return (v - mu) / torch.sqrt(((v - mu) ** 2).sum(1, keepdim=True) / C + 1e-6)

    bwd = case["way"] == "bwd"
    blocks = [(g, r0, min(R, r0 + rpg), None) for g, r0 in enumerate(range(0, R, rpg))]
    if len(blocks) > 64:
        # many groups: all rows at once, each with its group's vectors picked out
        blocks = [(slice(None), 0, R, torch.arange(R, device="cuda").div(rpg, rounding_mode="floor"))]
    shared = {n: d64(s[n]) for n in ("weight", "bias", "post_weight")}
    if bwd:
        shared = {n: t if t is None else t.requires_grad_() for n, t in shared.items()}
    out = {}
    for g, r0, r1, at in blocks:
        one = lambda t: None if t is None else d64(t[g]) if at is not None else d64(t[g:g + 1])
        rows = lambda t: t if at is None else t[at]
        gate, scale, shift = one(s["gate"]), one(s["scale"]), one(s["shift"])
        x = d64(s["x"][r0:r1])
        h = None if s["h"] is None else d64(s["h"][r0:r1])

        def branch(h, gate):
            v = h if case["post"] == "none" else normed(h, case["post"])
            if shared["post_weight"] is not None:
                v = v * shared["post_weight"]
            return v if gate is None else v * rows(gate)

        def head(z, scale, shift):
            y = normed(z, case["norm"])
            if shared["weight"] is not None:
                y = y * shared["weight"]
            if shared["bias"] is not None:
                y = y + shared["bias"]
            return y if scale is None else y * (1 + rows(scale)) + rows(shift)

        if not bwd:
            z = x if h is None else x * case["res_scale"] + branch(h, gate)
            part = {"y": head(z, scale, shift)}
            if h is not None:
                part["z"] = z
            for n, t in part.items():
                out.setdefault(n, []).append(t)
            continue
        # two steps: through the norm to the stream's whole gradient, then through the branch to it
        leaf = {"z": x, "scale": scale, "shift": shift}
        leaf = {n: t.requires_grad_() for n, t in leaf.items() if t is not None}
        want = dict(leaf, **{n: shared[n] for n in ("weight", "bias") if shared[n] is not None})
        got = torch.autograd.grad((head(x, scale, shift) * d64(s["dy"][r0:r1])).sum(), list(want.values()))
        got = dict(zip(want, got))
        dz = d64(s["dz"][r0:r1]) + got["z"]
        part = {"dx": dz if h is None else dz * case["res_scale"]}
        for n in ("scale", "shift"):
            if n in got:
                part["d" + n] = got[n]
        sums = {"d" + n: got[n] for n in ("weight", "bias") if n in got}
        if h is not None:
            want = {"h": h.requires_grad_()}
            if gate is not None:
                want["gate"] = gate.requires_grad_()
            if shared["post_weight"] is not None:
                want["post_weight"] = shared["post_weight"]
            got = dict(zip(want, torch.autograd.grad((branch(h, gate) * dz.detach()).sum(), list(want.values()))))
            part["dh"] = got["h"]
            if gate is not None:
                part["dgate"] = got["gate"]
            if "post_weight" in got:
                sums["dpost_weight"] = got["post_weight"]
        for n, t in part.items():
            out.setdefault(n, []).append(t.detach())
        for n, t in sums.items():
            out[n] = [out[n][0] + t.detach()] if n in out else [t.detach()]
    return {n: torch.cat(t) if len(t) > 1 else t[0] for n, t in out.items()}


def _exact_rotate(case, s):
    """As complex numbers: a pair is a + ib, and the rotation a product with cos + i sin."""
    T, H, W, d = (case[n] for n in ("T", "H", "W", "d"))
    nT, nH, nW = s["axes"]
    t64 = torch.view_as_complex(s["table"].to(torch.float64))
    turn = torch.empty(T, H, W, nT + nH + nW, dtype=torch.complex128, device="cuda")
    turn[..., :nT] = t64[:T * nT].view(T, 1, 1, nT)
    turn[..., nT:nT + nH] = t64[T * nT:T * nT + H * nH].view(1, H, 1, nH)
    turn[..., nT + nH:] = t64[T * nT + H * nH:].view(1, 1, W, nW)
    turn = turn.view(T * H * W, 1, -1)

    def to_complex(v):
        v = v.unflatten(-1, (d // 2, 2)) if case["pairs"] == "interleaved" else v.unflatten(-1, (2, d // 2)).transpose(-1, -2)
        return torch.view_as_complex(v.contiguous())

    def to_real(v):
        v = torch.view_as_real(v)
        return (v if case["pairs"] == "interleaved" else v.transpose(-1, -2)).flatten(-2)

    out = {}
    for name, w in (("Q", s["wq"]), ("K", s["wk"])):
        parts, dw = [], 0.0
        for r0 in range(0, T * H * W, 65536):
            rows = slice(r0, r0 + 65536)
            x = s[name][rows].to(torch.float64)
            size = torch.sqrt((x * x).sum(-1, keepdim=True) / d + 1e-6)
            if case["way"] == "fwd":
                n = x / size * w.to(torch.float64) if case["norm"] else x
                parts.append(to_real(to_complex(n) * turn[rows]))
                continue
            dn = to_real(to_complex(s["d" + name + "r"][rows].to(torch.float64)) * turn[rows].conj())
            if case["norm"]:
                dw = dw + (dn * x / size).sum((0, 1))
                dn = dn * w.to(torch.float64)
                dn = dn / size - x * (dn * x).sum(-1, keepdim=True) / (d * size ** 3)
            parts.append(dn)
        out[name if case["way"] == "fwd" else "d" + name] = torch.cat(parts)
        if case["way"] == "bwd" and case["norm"]:
            out["d%s_weight" % name.lower()] = dw
    return out


def _exact_experts(case, s):
    """Expert by expert and choice by choice."""
    R, k = s["ids"].shape
    E, align, cap = case["experts"], case["align"], s["xs"].shape[0]
    flat = s["ids"].reshape(-1)
    counts, offsets, at = [], [0], 0
    pos = torch.full((R * k,), -1, dtype=torch.int64, device="cuda")
    src = torch.full((cap,), -1, dtype=torch.int64, device="cuda")
    for e in range(E):
        slots = torch.nonzero(flat == e).reshape(-1)
        m = slots.numel()
        pos[slots] = at + torch.arange(m, device="cuda")
        src[at:at + m] = slots
        counts.append(m)
        at += -(-m // align) * align
        offsets.append(at)
    C = case["channels"]
    train = case["way"] == "train"
    xs = torch.zeros(cap, C, dtype=torch.float64, device="cuda")
    dys = torch.zeros_like(xs) if train else None
    out = torch.zeros(R, C, dtype=torch.float64, device="cuda")
    dx, dw = torch.zeros_like(out), torch.zeros(R, k, dtype=torch.float64, device="cuda")
    for j in range(k):
        p = pos.view(R, k)[:, j]
        t = torch.nonzero(p >= 0).reshape(-1)
        p, w = p[t], s["weights"][t, j].to(torch.float64)[:, None]
        y = s["ys"][p].to(torch.float64)
        xs[p] = s["x"][t].to(torch.float64)
        out[t] += w * y
        if train:
            do = s["dout"][t].to(torch.float64)
            dys[p] = w * do
            dw[t, j] = (y * do).sum(1)
            dx[t] += s["dxs"][p].to(torch.float64)
    i32 = lambda v: torch.as_tensor(v, device="cuda").to(torch.int32)
    r = {"counts": i32(counts), "offsets": i32(offsets), "pos": i32(pos.view(R, k)), "src": i32(src), "xs": xs,
         "out": out}
    if train:
        r.update(dys=dys, dweights=dw, dx=dx)
    return r

"""The operators around the attention in a transformer block, on torch tensors.

  norm          the norm before a block, and after it the gated, scaled residual sum with the
                norms on either side of it, in one pass
  rotate        the norm of each head's channels and the rotation by the token's place in the
                grid, for raster Q and K (``layer.prism_attention`` calls it with ``rotation=``)
  expert_plan, dispatch, combine
                tokens sorted by expert and back, beside the permutation by block

Each has a differentiable form (``norm``, ``rotate``, ``dispatch``, ``combine``) and the explicit
calls it is made of (``*_forward``, ``*_backward``, ``expert_*``), which allocate their outputs and
workspaces on the current stream, synchronise nothing and may be captured into a CUDA graph.  The
differentiable forms refuse to run under capture: autograd would tie the captured backward to
gradient accumulators that may belong to another stream.  Capture the explicit calls instead.

Every step runs in ``libprism.so`` (contracts in ``include/prism.h``), on the current stream of the
tensors' device.  Checks of shapes, types and devices raise ``ValueError``; what the library refuses
raises ``PrismError``.
"""
from __future__ import annotations

import contextlib
import functools

import torch
from torch.autograd.function import once_differentiable

from . import _abi

_DT = {torch.float32: _abi.PRISM_F32, torch.bfloat16: _abi.PRISM_BF16}
_NORMS = {None: 0, "none": 0, "rms": 1, "layer": 2}
_PAIRS = {"interleaved": 0, "half": 1}


# ------------------------------------------------------------------ shared checks
def _need(ok, what):
    if not ok:
        raise ValueError(what)


def _same_device(dev, *tensors):
    _need(dev.type == "cuda", f"the tensors must be on a CUDA device, not {dev}")
    for t in tensors:
        if t is not None and t.device != dev:
            raise ValueError(f"tensors on {dev} and {t.device}")


def _on(dev):
    """The device as the current one, where it is another."""
    return contextlib.nullcontext() if dev.index == torch.cuda.current_device() else torch.cuda.device(dev)


def _rows(t, C, what):
    """t as rows of C contiguous channels, copied only where it cannot be viewed so."""
    if t.dim() == 0 or t.shape[-1] != C:
        raise ValueError(f"{what} must be [..., {C}], not {tuple(t.shape)}")
    if t.dim() != 2:
        t = t.reshape(-1, C) if t.numel() or C == 0 else t.new_empty(_count(t), C)
    if (C > 1 and t.stride(1) != 1) or (t.shape[0] > 1 and t.stride(0) < C):
        t = t.contiguous()
    return t


def _count(t):
    n = 1
    for s in t.shape[:-1]:
        n *= s
    return n


def _ld(t):
    """Row stride for the library (0: dense rows)."""
    return t.stride(0) if t is not None and t.shape[0] > 1 else 0


def _bytes(t):
    """First and last address of a tensor's elements."""
    a = t.data_ptr()
    return a, a + (sum((n - 1) * s for n, s in zip(t.shape, t.stride())) + 1) * t.element_size()


def _apart(a, b):
    """Whether two tensors of rows share no element: other memory, or other columns of the same rows."""
    if a is None or b is None or not a.numel() or not b.numel():
        return True
    (a0, a1), (b0, b1) = _bytes(a), _bytes(b)
    if a1 <= b0 or b1 <= a0:
        return True
    step = a.stride(0) * a.element_size()
    if a.dim() < 2 or step != b.stride(0) * b.element_size() or step <= 0:
        return False
    (_, ae), (_, be) = _bytes(a[0]), _bytes(b[0])
    off = (b0 - a0) % step
    return ae - a0 <= off and off + be - b0 <= step


def _itself(a, b):
    return a.data_ptr() == b.data_ptr() and a.shape == b.shape and a.stride() == b.stride() and a.dtype == b.dtype


def _check_out(out, what, allowed, *others):
    """An output may be the tensor ``allowed`` itself, and has to be apart from all others."""
    for t in others:
        if t is not None and not _apart(out, t) and not (t is allowed or (allowed is not None and _itself(t, allowed))
                                                         and _itself(out, t)):
            raise ValueError(f"{what} overlaps another argument")
    if allowed is not None and not _apart(out, allowed) and not _itself(out, allowed):
        raise ValueError(f"{what} overlaps an input without being it")


def _refuse_capture(name, instead):
    if torch.cuda.is_current_stream_capturing():
        raise RuntimeError(f"{name} records an autograd graph and cannot be captured; capture {instead}")


def _wants_graph(*tensors):
    return torch.is_grad_enabled() and any(t is not None and t.requires_grad for t in tensors)


# ------------------------------------------------------------------ block norms
@functools.lru_cache(maxsize=256)
def _norm_desc(*fields):
    d = _abi.BlockNormT(*fields)
    return d, _abi.block_norm_ws_bytes(d)


def _vector(v, shape, what):
    if v is None:
        return None
    if v.dtype != torch.float32:
        raise ValueError(f"{what} must be float32, not {v.dtype}")
    if tuple(v.shape) != shape:
        raise ValueError(f"{what} must be {shape}, not {tuple(v.shape)}")
    if len(shape) == 1:
        return v.contiguous()
    return v if (shape[1] == 1 or v.stride(1) == 1) and (shape[0] < 2 or v.stride(0) >= shape[1]) else v.contiguous()


def _norm_setup(x, h, gate, post_weight, weight, bias, scale, shift, norm, post_norm, rows_per_group, branch):
    _need(norm in _NORMS, f"norm is 'layer', 'rms' or None, not {norm!r}")
    _need(post_norm in _NORMS, f"post_norm is 'layer', 'rms' or None, not {post_norm!r}")
    _need(x.dim() >= 1 and x.shape[-1] >= 1, f"x must be [..., C], not {tuple(x.shape)}")
    _need(x.dtype in _DT and branch in _DT, f"float32 or bfloat16, not {x.dtype} and {branch}")
    C = x.shape[-1]
    _same_device(x.device, h, gate, post_weight, weight, bias, scale, shift)
    if h is not None:
        _need(h.shape == x.shape, f"h must have x's shape {tuple(x.shape)}, not {tuple(h.shape)}")
        _need(h.dtype == branch, f"h is {h.dtype} and the next branch {branch}")
    R = _count(x)
    rpg = rows_per_group
    if rpg is None:
        rpg = x.shape[-2] if x.dim() > 2 else R
    _need(rpg >= 1 or R == 0, "rows_per_group must be at least 1")
    rpg = max(1, int(rpg))
    G = -(-R // rpg)
    return (C, R, rpg, _vector(gate, (G, C), "gate"), _vector(post_weight, (C,), "post_weight"),
            _vector(weight, (C,), "weight"), _vector(bias, (C,), "bias"), _vector(scale, (G, C), "scale"),
            _vector(shift, (G, C), "shift"))


def norm_forward(x, h=None, *, gate=None, post_weight=None, weight=None, bias=None, scale=None, shift=None,
                 norm="layer", post_norm=None, eps=1e-6, res_scale=1.0, rows_per_group=None, out_dtype=None, z=None,
                 y=None):
    """(z, y) with z = res_scale x + gate ∘ N_post(h) ∘ post_weight and
    y = N(z) ∘ weight ∘ (1 + scale) + bias ∘ (1 + scale) + shift.

    x [..., C] is the residual stream, h [..., C] the block's output (None: z is x); gate, scale and shift are
    float32 [groups, C], one row for each ``rows_per_group`` rows (default: x's last-but-one dimension where it has
    three or more, else all rows); weight, bias and post_weight float32 [C].  ``norm=None`` gives no y.  y has
    ``out_dtype`` (default: h's type, else x's).  ``z`` and ``y`` may be given as outputs; z may be x itself.
    """
    branch = out_dtype or (h if h is not None else x).dtype
    C, R, rpg, gate, post_weight, weight, bias, scale, shift = _norm_setup(
        x, h, gate, post_weight, weight, bias, scale, shift, norm, post_norm, rows_per_group, branch)
    dev = x.device
    given = []
    for t, dt, what in ((z, x.dtype, "z"), (y, branch, "y")):
        if t is not None:
            _need(t.shape == x.shape and t.dtype == dt and t.device == dev,
                  f"{what} must be {dt} of shape {tuple(x.shape)} on {dev}")
            v = t.flatten(0, -2) if t.dim() > 1 else t.view(1, C)
            _need(not t.numel() or (v.data_ptr() == t.data_ptr() and (C == 1 or v.stride(1) == 1)
                                    and (v.shape[0] < 2 or v.stride(0) >= C)), f"{what}'s rows must lie evenly")
            given.append((v, what))
    _need(z is None or h is not None, "without h there is no z to write")
    _need(y is None or norm not in (None, "none"), "without a norm there is no y to write")
    xr, hr = _rows(x, C, "x"), None if h is None else _rows(h, C, "h")
    for i, (v, what) in enumerate(given):
        _check_out(v, what, xr if what == "z" else None, xr, hr, gate, post_weight, weight, bias, scale, shift,
                   *(o for o, _ in given[:i]))
    with _on(dev):
        has_y = norm not in (None, "none")
        if z is None and h is not None:
            z = torch.empty(x.shape, dtype=x.dtype, device=dev)
        if y is None and has_y:
            y = torch.empty(x.shape, dtype=branch, device=dev)
        zr, yr = (None if t is None else t.view(-1, C) if t.is_contiguous() and t.numel() else t.flatten(0, -2)
                  if t.dim() > 1 else t.view(1, C) for t in (z, y))
        d, _ = _norm_desc(R, rpg, C, _DT[x.dtype], _DT[branch], _NORMS[norm], _NORMS[post_norm], eps, res_scale,
                          _ld(xr), _ld(hr), _ld(zr), _ld(yr), 0, 0, 0, 0, _ld(gate), _ld(scale), _ld(shift))
        _abi.prism_block_norm_fwd(d, xr, hr, gate, post_weight, weight, bias, scale, shift, zr, yr)
    return (x if h is None else z), y


def norm_backward(z, h, dz, dy, *, gate=None, post_weight=None, weight=None, bias=None, scale=None, norm="layer",
                  post_norm=None, eps=1e-6, res_scale=1.0, rows_per_group=None, wants=None):
    """Gradients of ``norm_forward``, from the stored stream z (x where there was no h) and the branch h.

    dz (None: zero) is the gradient that reaches z past this norm, dy that of y.  Returns a dict of ``dx``, ``dh``
    and, for the vectors that are given, ``dgate``, ``dpost_weight``, ``dweight``, ``dbias``, ``dscale`` and, with
    scale, ``dshift``; the others are None.  ``wants``: names of the vectors' gradients to take instead
    (``dshift`` needs no vector).
    """
    branch = (dy if dy is not None else h if h is not None else z).dtype
    C, R, rpg, gate, post_weight, weight, bias, scale, _ = _norm_setup(
        z, h, gate, post_weight, weight, bias, scale, None, norm, post_norm, rows_per_group, branch)
    dev, G = z.device, -(-R // rpg)
    _same_device(dev, dz, dy)
    has_y = norm not in (None, "none")
    _need(not has_y or dy is not None, "a norm's backward needs dy")
    _need(has_y or dz is not None, "without a norm the backward needs dz")
    for t, dt, what in ((dz, z.dtype, "dz"), (dy, branch, "dy")):
        _need(t is None or (t.shape == z.shape and t.dtype == dt), f"{what} must be {dt} of shape {tuple(z.shape)}")
    if wants is None:
        wants = [n for n, v in (("dgate", gate), ("dpost_weight", post_weight), ("dweight", weight), ("dbias", bias),
                                ("dscale", scale), ("dshift", scale)) if v is not None]
    else:
        for n in wants:
            _need(n in ("dgate", "dpost_weight", "dweight", "dbias", "dscale", "dshift"), f"no gradient {n!r}")
    zr, hr, dzr, dyr = (None if t is None else _rows(t, C, n) for t, n in ((z, "z"), (h, "h"), (dz, "dz"), (dy, "dy")))
    with _on(dev):
        g = dict.fromkeys(("dx", "dh", "dgate", "dpost_weight", "dweight", "dbias", "dscale", "dshift"))
        g["dx"] = torch.empty(z.shape, dtype=z.dtype, device=dev)
        if h is not None:
            g["dh"] = torch.empty(z.shape, dtype=branch, device=dev)
        for n in wants:
            g[n] = torch.empty((G, C) if n in ("dgate", "dscale", "dshift") else (C,), dtype=torch.float32, device=dev)
        d, ws_bytes = _norm_desc(R, rpg, C, _DT[z.dtype], _DT[branch], _NORMS[norm], _NORMS[post_norm], eps,
                                 res_scale, 0, _ld(hr), _ld(zr), 0, 0, 0, _ld(dzr), _ld(dyr), _ld(gate), _ld(scale), 0)
        ws = torch.empty(ws_bytes, dtype=torch.uint8, device=dev) if wants else None
        _abi.prism_block_norm_bwd(d, zr, hr, gate, post_weight, weight, bias, scale, dzr, dyr, g["dx"], g["dh"],
                                  g["dgate"], g["dpost_weight"], g["dweight"], g["dbias"], g["dscale"], g["dshift"],
                                  ws, ws_bytes if wants else 0)
    return g


class _NormFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, h, gate, post_weight, weight, bias, scale, shift, kw, out_dtype):
        ctx.set_materialize_grads(False)
        z, y = norm_forward(x, h, gate=gate, post_weight=post_weight, weight=weight, bias=bias, scale=scale,
                            shift=shift, out_dtype=out_dtype, **kw)
        ctx.save_for_backward(z, h, gate, post_weight, weight, bias, scale)
        ctx.kw, ctx.y_dtype = kw, None if y is None else y.dtype
        return (z, y) if h is not None else y

    @staticmethod
    @once_differentiable
    def backward(ctx, *grads):
        z, h, gate, post_weight, weight, bias, scale = ctx.saved_tensors
        dz, dy = grads if h is not None else (None, grads[0])
        if dz is None and dy is None:
            return (None,) * 10
        need = ctx.needs_input_grad
        if dy is None and ctx.y_dtype is not None:
            dy = torch.zeros(z.shape, dtype=ctx.y_dtype, device=z.device)
        if dz is None and ctx.y_dtype is None:
            dz = torch.zeros_like(z)
        wants = [n for n, k in (("dgate", 2), ("dpost_weight", 3), ("dweight", 4), ("dbias", 5), ("dscale", 6),
                                ("dshift", 7)) if need[k]]
        g = norm_backward(z, h, dz, dy, gate=gate, post_weight=post_weight, weight=weight, bias=bias, scale=scale,
                          wants=wants, **ctx.kw)
        return (g["dx"] if need[0] else None, g["dh"] if need[1] else None, g["dgate"], g["dpost_weight"], g["dweight"],
                g["dbias"], g["dscale"], g["dshift"], None, None)


def norm(x, h=None, *, gate=None, post_weight=None, weight=None, bias=None, scale=None, shift=None, norm="layer",
         post_norm=None, eps=1e-6, res_scale=1.0, rows_per_group=None, out_dtype=None):
    """Differentiable ``norm_forward``: returns (z, y); z is x itself where there is no h."""
    tensors = (x, h, gate, post_weight, weight, bias, scale, shift)
    kw = dict(norm=norm, post_norm=post_norm, eps=eps, res_scale=res_scale, rows_per_group=rows_per_group)
    if not _wants_graph(*tensors):
        return norm_forward(x, h, gate=gate, post_weight=post_weight, weight=weight, bias=bias, scale=scale,
                            shift=shift, out_dtype=out_dtype, **kw)
    _refuse_capture("block.norm", "norm_forward and norm_backward")
    if h is None:
        return x, _NormFn.apply(*tensors, kw, out_dtype)
    return _NormFn.apply(*tensors, kw, out_dtype)


# ------------------------------------------------------------------ head norm and rotation
@functools.lru_cache(maxsize=256)
def _rotate_desc(*fields):
    d = _abi.RotateT(*fields)
    return d, _abi.head_rotate_ws_bytes(d)


def rotation_table(grid, axes, base=10000.0, device="cuda", positions=None):
    """The (cos, sin) rows that ``rotate`` reads: for each axis of ``grid`` = (T, H, W) a row for each place with
    ``axes`` = (pairs_t, pairs_h, pairs_w) pairs, pair i of n at place p turned by p base^(-i/n).  ``positions``:
    three sequences of places instead of 0, 1, 2, ...  Angles in 64 bits, rounded once to float32."""
    parts = []
    for a, (length, pairs) in enumerate(zip(grid, axes)):
        p = torch.arange(length, dtype=torch.float64) if positions is None else torch.as_tensor(
            positions[a], dtype=torch.float64)
        _need(p.shape == (length,), f"axis {a} has {length} places, not {tuple(p.shape)}")
        angle = p[:, None] * base ** (-torch.arange(pairs, dtype=torch.float64) / max(1, pairs))
        parts.append(torch.stack((angle.cos(), angle.sin()), -1).reshape(-1, 2))
    return torch.cat(parts).float().to(device)


def _heads(t, what):
    """t as [tokens, heads, d] rows that the library can walk, copied where it cannot be viewed so."""
    _need(t.dim() == 3, f"{what} must be [tokens, heads, head_dim], not {tuple(t.shape)}")
    n, h, d = t.shape
    step = 16 // t.element_size()
    if ((d > 1 and t.stride(2) != 1) or (h > 1 and t.stride(1) != d)
            or (n > 1 and (t.stride(0) < h * d or t.stride(0) % step)) or t.data_ptr() % 16):
        t = t.contiguous()
        if t.data_ptr() % 16:
            t = t.clone()
    return t


def _rotate_setup(sides, table, grid, axes, weights, norm, pairs):
    _need(pairs in _PAIRS, f"pairs is 'interleaved' or 'half', not {pairs!r}")
    _need(len(grid) == 3 and len(axes) == 3, "grid and axes have three entries: (T, H, W)")
    first = next((t for t in sides if t is not None), None)
    _need(first is not None, "neither Q nor K")
    _same_device(first.device, table, *sides, *weights)
    for t in sides:
        _need(t is None or t.dim() == 3, "Q and K must be [tokens, heads, head_dim]")
        _need(t is None or (t.shape[0] == first.shape[0] and t.shape[2] == first.shape[2] and t.dtype == first.dtype),
              "Q and K must agree in tokens, head_dim and type")
    _need(first.dtype in _DT, f"float32 or bfloat16, not {first.dtype}")
    rows = sum(n * p for n, p in zip(grid, axes))
    _need(table.dtype == torch.float32 and tuple(table.shape) == (rows, 2),
          f"table must be float32 [{rows}, 2], not {table.dtype} {tuple(table.shape)}")
    ws = [_vector(w, (first.shape[2],), "a head's weight") for w in weights]
    _need(norm or (ws[0] is None and ws[1] is None), "weights without a norm")
    ws = [w if w is None or w.data_ptr() % 16 == 0 else w.clone() for w in ws]
    table = table.contiguous()
    return first, table if table.data_ptr() % 16 == 0 else table.clone(), ws


def _rotate_fields(first, sides, grid, axes, norm, eps, pairs, lds):
    hq, hk = (0 if t is None else t.shape[1] for t in sides)
    return (first.shape[0], *grid, hq, hk, first.shape[2], *axes, _PAIRS[pairs], _DT[first.dtype], int(bool(norm)), eps,
            *lds)


def rotate_forward(Q, K, table, *, grid, axes, q_weight=None, k_weight=None, norm=True, eps=1e-6, pairs="interleaved",
                   out=None):
    """(Q, K) with each head's channels RMS-normed (``norm``), weighted (q_weight, k_weight float32 [d]) and its
    channel pairs turned by the token's place: token i lies at place i mod T H W of ``grid`` = (T, H, W) in raster
    order, the first axes[0] pairs turn with its t, the next axes[1] with h, the next axes[2] with w, the rest not
    at all.  ``table`` float32 [T axes[0] + H axes[1] + W axes[2], 2] as ``rotation_table`` makes it; ``pairs``
    'interleaved' (channels 2i, 2i + 1) or 'half' (i, i + d/2).  Q or K may be None, and have different numbers of
    heads.  ``out`` = (Qr, Kr) takes the results, and may be (Q, K) themselves.
    """
    first, table, ws = _rotate_setup((Q, K), table, grid, axes, (q_weight, k_weight), norm, pairs)
    dev = first.device
    src = [None if t is None else _heads(t, "Q or K") for t in (Q, K)]
    if out is not None:
        _need(len(out) == 2, "out is (Qr, Kr)")
        for i, (o, t, s) in enumerate(zip(out, (Q, K), src)):
            _need((o is None) == (t is None), "out must have a tensor for each of Q and K")
            if o is None:
                continue
            _need(o.shape == t.shape and o.dtype == t.dtype and o.device == dev, "out must be like Q and K")
            _need(not o.numel() or _heads(o, "out") is o, "out's heads must lie densely on 16-byte boundaries")
            _check_out(o, "out", s, table, *ws, *(out[:i]))
            # one tensor as Q and K would be read by one side while the other writes it
            _need(_apart(o, src[1 - i]), "out overlaps the other of Q and K")
    with _on(dev):
        if out is None:
            out = [None if t is None else torch.empty(t.shape, dtype=t.dtype, device=dev) for t in (Q, K)]
        d, _ = _rotate_desc(*_rotate_fields(first, (Q, K), grid, axes, norm, eps, pairs,
                                            (_ld(src[0]), _ld(src[1]), _ld(out[0]), _ld(out[1]), 0, 0)))
        _abi.prism_head_rotate_fwd(d, src[0], src[1], ws[0], ws[1], table, out[0], out[1])
    return tuple(out)


def rotate_backward(Q, K, dQr, dKr, table, *, grid, axes, q_weight=None, k_weight=None, norm=True, eps=1e-6,
                    pairs="interleaved", wants=None):
    """Gradients of ``rotate_forward`` from its inputs Q, K and its outputs' gradients: a dict of ``dQ``, ``dK`` and,
    for the weights that are given, ``dq_weight``, ``dk_weight`` (``wants``: names of these to take instead); the
    others are None.  Without a norm Q and K are not read and may be None."""
    first, table, ws = _rotate_setup((dQr, dKr), table, grid, axes, (q_weight, k_weight), norm, pairs)
    dev = first.device
    _same_device(dev, Q, K)
    xs, drs = [], []
    for x, dr in ((Q, dQr), (K, dKr)):
        _need(x is None or (dr is not None and x.shape == dr.shape and x.dtype == dr.dtype),
              "Q and K must be like their gradients")
        _need(dr is None or x is not None or not norm, "the norm's backward needs Q and K")
        xs.append(None if x is None or not norm else _heads(x, "Q or K"))
        drs.append(None if dr is None else _heads(dr, "dQr or dKr"))
    if wants is None:
        wants = [n for n, w in (("dq_weight", ws[0]), ("dk_weight", ws[1])) if w is not None]
    for n in wants:
        _need(n in ("dq_weight", "dk_weight") and norm, f"no gradient {n!r} here")
        _need((dQr if n == "dq_weight" else dKr) is not None, f"no gradient {n!r} here")
    g = dict.fromkeys(("dQ", "dK", "dq_weight", "dk_weight"))
    with _on(dev):
        for n, dr in (("dQ", dQr), ("dK", dKr)):
            if dr is not None:
                g[n] = torch.empty(dr.shape, dtype=dr.dtype, device=dev)
        for n in wants:
            g[n] = torch.empty(first.shape[2], dtype=torch.float32, device=dev)
        d, ws_bytes = _rotate_desc(*_rotate_fields(first, (dQr, dKr), grid, axes, norm, eps, pairs,
                                                   (_ld(xs[0]), _ld(xs[1]), 0, 0, _ld(drs[0]), _ld(drs[1]))))
        buf = torch.empty(ws_bytes, dtype=torch.uint8, device=dev) if wants else None
        _abi.prism_head_rotate_bwd(d, xs[0], xs[1], ws[0], ws[1], table, drs[0], drs[1], g["dQ"], g["dK"],
                                   g["dq_weight"], g["dk_weight"], buf, ws_bytes if wants else 0)
    return g


class _RotateFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, Q, K, q_weight, k_weight, table, kw):
        ctx.set_materialize_grads(False)
        ctx.kw = kw
        keep = kw["norm"]
        ctx.save_for_backward(Q if keep else None, K if keep else None, q_weight, k_weight, table)
        return rotate_forward(Q, K, table, q_weight=q_weight, k_weight=k_weight, **kw)

    @staticmethod
    @once_differentiable
    def backward(ctx, dQr, dKr):
        Q, K, wq, wk, table = ctx.saved_tensors
        if dQr is None and dKr is None:
            return (None,) * 6
        need = ctx.needs_input_grad
        wants = [n for n, k, d in (("dq_weight", 2, dQr), ("dk_weight", 3, dKr)) if need[k] and d is not None]
        g = rotate_backward(None if dQr is None else Q, None if dKr is None else K, dQr, dKr, table,
                            q_weight=None if dQr is None else wq, k_weight=None if dKr is None else wk, wants=wants,
                            **ctx.kw)
        return (g["dQ"] if need[0] else None, g["dK"] if need[1] else None, g["dq_weight"], g["dk_weight"], None, None)


def rotate(Q, K, table, *, grid, axes, q_weight=None, k_weight=None, norm=True, eps=1e-6, pairs="interleaved"):
    """Differentiable ``rotate_forward`` (the table gets no gradient)."""
    kw = dict(grid=tuple(grid), axes=tuple(axes), norm=norm, eps=eps, pairs=pairs)
    if not _wants_graph(Q, K, q_weight, k_weight):
        return rotate_forward(Q, K, table, q_weight=q_weight, k_weight=k_weight, **kw)
    _refuse_capture("block.rotate", "rotate_forward and rotate_backward")
    return _RotateFn.apply(Q, K, q_weight, k_weight, table, kw)


# ------------------------------------------------------------------ experts
class ExpertPlan:
    """Where each slot (token, choice) lies in the layout sorted by expert.

    counts [experts] and offsets [experts + 1]: each expert's slots and first row (a multiple of ``align``);
    pos [rows, top_k]: the slot's row, -1 where it is dropped; src [rows_sorted]: the row's slot t top_k + j, -1
    where there is none.  All int32 on the device; ``rows_sorted`` is the host's bound on the sorted rows, of which
    offsets[experts] are in use.
    """

    def __init__(self, rows, top_k, experts, align, id_bytes, device):
        self.desc, self.rows_sorted, self.ws_bytes = _expert_desc(rows, top_k, experts, align, id_bytes)
        self.rows, self.top_k, self.experts, self.align, self.device = rows, top_k, experts, align, device
        # one allocation, its parts on 16-byte boundaries
        sizes = (experts, experts + 1, rows * top_k, self.rows_sorted, self.ws_bytes // 4)
        starts = [0]
        for n in sizes:
            starts.append(starts[-1] + (n + 3) // 4 * 4)
        buf = torch.empty(starts[-1], dtype=torch.int32, device=device)
        part = [buf[a:a + n] for a, n in zip(starts, sizes)]
        self.counts, self.offsets, pos, self.src, self._ws = part
        self.pos = pos.view(rows, top_k)


@functools.lru_cache(maxsize=256)
def _expert_desc(*fields):
    d = _abi.ExpertsT(*fields)
    return (d, *_abi.expert_sizes(d))


def expert_plan(ids, experts, align=1) -> ExpertPlan:
    """Sort the slots of ids [rows, top_k] (int32 or int64) by expert, stably; an id outside [0, experts) drops its
    slot.  Each expert's rows start at a multiple of ``align``."""
    _need(ids.dim() == 2, f"ids must be [rows, top_k], not {tuple(ids.shape)}")
    _need(ids.dtype in (torch.int32, torch.int64), f"ids must be int32 or int64, not {ids.dtype}")
    _same_device(ids.device)
    ids = ids.contiguous()
    with _on(ids.device):
        p = ExpertPlan(ids.shape[0], ids.shape[1], int(experts), int(align), ids.element_size(), ids.device)
        _abi.prism_expert_plan(p.desc, ids, p.counts, p.offsets, p.pos, p.src, p._ws if p.ws_bytes else None,
                               p.ws_bytes)
    return p


def _by_token(t, plan, C, what):
    _need(t.dim() == 2 and t.shape[0] == plan.rows and (C is None or t.shape[1] == C),
          f"{what} must be [{plan.rows}, channels], not {tuple(t.shape)}")
    _need(t.dtype in _DT, f"float32 or bfloat16, not {t.dtype}")
    _same_device(plan.device, t)
    return _rows(t, t.shape[1], what)


def _sorted(t, plan, C, dtype, what):
    _need(t.dim() == 2 and tuple(t.shape) == (plan.rows_sorted, C if C is not None else t.shape[1]),
          f"{what} must be [{plan.rows_sorted}, channels], not {tuple(t.shape)}")
    _need(t.dtype in _DT and (dtype is None or t.dtype == dtype), f"{what} has type {t.dtype}")
    _same_device(plan.device, t)
    return t


def _weights(w, plan):
    if w is None:
        return None
    _need(w.dtype == torch.float32 and tuple(w.shape) == (plan.rows, plan.top_k),
          f"weights must be float32 [{plan.rows}, {plan.top_k}]")
    _same_device(plan.device, w)
    return w.contiguous()


def expert_dispatch(x, plan, *, out=None):
    """xs [rows_sorted, C]: x's rows [rows, C] copied to their slots' rows; the rows between an expert's last slot
    and the next multiple of ``align`` are 0, as are those behind the last expert.  A given ``out`` (dense, not
    overlapping x) keeps the rows behind the last expert as they are."""
    xr = _by_token(x, plan, None, "x")
    C = xr.shape[1]
    with _on(plan.device):
        clear = out is None
        if clear:
            out = torch.empty((plan.rows_sorted, C), dtype=x.dtype, device=plan.device)
        else:
            _need(_sorted(out, plan, C, x.dtype, "out").is_contiguous(), "out must be dense")
            _check_out(out, "out", None, xr, plan.pos, plan.counts, plan.offsets)
        _abi.prism_expert_dispatch(plan.desc, _DT[x.dtype], C, xr, _ld(xr), plan.pos, plan.counts, plan.offsets,
                                   int(clear), out)
    return out


def expert_combine(ys, plan, weights=None, *, add=None, out=None):
    """out [rows, C]: add[t] + sum over t's choices j of weights[t, j] ys[pos[t, j]], without the dropped ones
    (weights float32 [rows, top_k], None: 1; add None: 0).  Summed in float32 in j's order, rounded once.  Without
    weights it is the gradient of ``expert_dispatch``.  ``out`` may be ``add`` itself."""
    y = _sorted(ys, plan, None, None, "ys").contiguous()
    C = y.shape[1]
    w = _weights(weights, plan)
    addr = None if add is None else _by_token(add, plan, C, "add")
    _need(add is None or add.dtype == y.dtype, "add must have ys' type")
    with _on(plan.device):
        if out is None:
            out = torch.empty((plan.rows, C), dtype=y.dtype, device=plan.device)
        else:
            _need(_by_token(out, plan, C, "out") is out and out.dtype == y.dtype, "out must be rows of ys' type")
            _check_out(out, "out", addr, y, w, addr, plan.pos)
        _abi.prism_expert_combine(plan.desc, _DT[y.dtype], C, y, plan.pos, w, addr, _ld(addr), out, _ld(out))
    return out


def expert_combine_backward(dout, ys, plan, weights=None, *, out=None, want_weights=True):
    """(dys, dweights) of ``expert_combine``: dys[pos[t, j]] = weights[t, j] dout[t] and dweights[t, j] =
    ys[pos[t, j]] . dout[t] (0 where dropped; None with ``want_weights=False``, where ys may be None).  Rows of dys
    without a slot as in ``expert_dispatch``; ``out`` may be ys itself."""
    d = _by_token(dout, plan, None, "dout")
    C = d.shape[1]
    w = _weights(weights, plan)
    _need(ys is not None or not want_weights, "the weights' gradient needs ys")
    y = None if ys is None or not want_weights else _sorted(ys, plan, C, dout.dtype, "ys").contiguous()
    with _on(plan.device):
        clear = out is None
        if clear:
            out = torch.empty((plan.rows_sorted, C), dtype=dout.dtype, device=plan.device)
        else:
            _need(_sorted(out, plan, C, dout.dtype, "out").is_contiguous(), "out must be dense")
            _check_out(out, "out", y, d, y, w, plan.pos, plan.counts, plan.offsets)
        dw = torch.empty((plan.rows, plan.top_k), dtype=torch.float32, device=plan.device) if want_weights else None
        _abi.prism_expert_combine_bwd(plan.desc, _DT[dout.dtype], C, d, _ld(d), y, plan.pos, w, plan.counts,
                                      plan.offsets, int(clear), out, dw)
    return out, dw


class _DispatchFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, plan):
        ctx.plan = plan
        return expert_dispatch(x, plan)

    @staticmethod
    @once_differentiable
    def backward(ctx, dxs):
        return expert_combine(dxs, ctx.plan), None


class _CombineFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, ys, weights, add, plan):
        ctx.plan = plan
        need_w = weights is not None and ctx.needs_input_grad[1]
        ctx.save_for_backward(ys if need_w else None, weights)
        return expert_combine(ys, plan, weights, add=add)

    @staticmethod
    @once_differentiable
    def backward(ctx, dout):
        ys, weights = ctx.saved_tensors
        need = ctx.needs_input_grad
        dys = dw = None
        if need[0] or need[1]:
            dys, dw = expert_combine_backward(dout, ys, ctx.plan, weights, want_weights=need[1])
        return dys if need[0] else None, dw, dout if need[2] else None, None


def dispatch(x, plan):
    """Differentiable ``expert_dispatch``."""
    if not _wants_graph(x):
        return expert_dispatch(x, plan)
    _refuse_capture("block.dispatch", "expert_dispatch and expert_combine")
    return _DispatchFn.apply(x, plan)


def combine(ys, plan, weights=None, *, add=None):
    """Differentiable ``expert_combine`` (gradients of ys, weights and add)."""
    if not _wants_graph(ys, weights, add):
        return expert_combine(ys, plan, weights, add=add)
    _refuse_capture("block.combine", "expert_combine and expert_combine_backward")
    return _CombineFn.apply(ys, weights, add, plan)

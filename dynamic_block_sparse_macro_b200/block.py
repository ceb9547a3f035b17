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
gradient accumulators that may belong to another stream.  Capture the explicit calls instead.  They have no
forward-mode derivatives, and refuse inputs with tangents.

Outputs given to the explicit calls are written in place: tensors that autograd has saved for a backward are known to
have changed, and one that requires grad is refused outside of ``torch.no_grad()``.

Every step runs in ``libprism.so`` (contracts in ``include/prism.h``), on the current stream of the
tensors' device.  Checks of shapes, types and devices raise ``ValueError``; what the library refuses
raises ``PrismError``.

A call's checks and its descriptor depend on its arguments' shapes, strides, types and devices alone; they are
made once a signature and kept (``_plans``), so that a repeated call costs little more than its launch.
"""
from __future__ import annotations

import ctypes
from operator import index

import torch
from torch.autograd import forward_ad
from torch.autograd.graph import increment_version
from torch.autograd.function import once_differentiable

from . import _abi

_DT = {torch.float32: _abi.PRISM_F32, torch.bfloat16: _abi.PRISM_BF16}
_NORMS = {None: 0, "none": 0, "rms": 1, "layer": 2}
_PAIRS = {"interleaved": 0, "half": 1}


# ------------------------------------------------------------------ shared checks
_plans = {}             # signature -> the checked call: descriptor, output shapes
_MAX_PLANS = 2048


def _need(ok, what):
    if not ok:
        raise ValueError(what)


def _real(v, what):
    """A number that a kept call holds: its value now, where it is a tensor of one element."""
    if type(v) is float:
        return v
    if isinstance(v, torch.Tensor) and v.requires_grad:
        raise ValueError(f"{what} is a number and gets no gradient")
    return float(v)


def _fits(**fields):
    """A descriptor's 32-bit fields, which would take the low half of a larger number."""
    for name, v in fields.items():
        _need(abs(v) < 1 << 31, f"{name} = {v} is out of range")


def _group_rows(v):
    return None if v is None else int(v)


def _whole(values):
    if len(values) != 3:
        raise ValueError("grid and axes have three entries: (T, H, W)")
    a, b, c = values
    return (a, b, c) if type(a) is type(b) is type(c) is int else (index(a), index(b), index(c))


def _sig(t):
    return None if t is None else (t.shape, t.stride(), t.dtype, t.device)


def _ptr(t):
    return None if t is None else t.data_ptr()


def _there(t):
    """As ``_ptr``, where the library is to see that a tensor is given: one without elements has no address of its own."""
    return None if t is None else t.data_ptr() or 256


def _keep(key, plan):
    """Keeps a finished plan: another thread may take it at once."""
    if len(_plans) >= _MAX_PLANS:
        _plans.clear()
    _plans[key] = plan
    return plan


class _Plan:
    """A checked call.  ``copy``: an argument's layout is not one that the library walks, so the arguments are laid
    out anew and the call is made with those."""
    __slots__ = ("desc", "addr", "index", "copy", "ws_bytes", "a", "b", "c")

    def __init__(self, desc, dev, copy=False):
        self.desc, self.addr, self.index, self.copy = desc, ctypes.addressof(desc), dev.index, copy
        self.ws_bytes = 0
        self.a = self.b = self.c = None


def _current(index):
    return torch._C._cuda_getDevice() == index


def _stream(index):
    return torch._C._cuda_getCurrentRawStream(index)


def _check(name, code):
    if code:
        raise _abi.PrismError(name, code)


def _same_device(dev, *tensors):
    _need(dev.type == "cuda", f"the tensors must be on a CUDA device, not {dev}")
    for t in tensors:
        if t is not None and t.device != dev:
            raise ValueError(f"tensors on {dev} and {t.device}")


def _count(shape):
    n = 1
    for s in shape[:-1]:
        n *= s
    return n


def _row_stride(t):
    """Elements between rows of C contiguous channels, 0 for dense ones or one row; None where t is not laid out so."""
    shape, stride = t.shape, t.stride()
    C = shape[-1]
    dims = [(n, s) for n, s in zip(shape[:-1], stride[:-1]) if n != 1]
    if any(n == 0 for n, _ in dims):
        return 0
    if C > 1 and stride[-1] != 1:
        return None
    for (_, s), (n, inner) in zip(dims, dims[1:]):
        if s != n * inner:
            return None
    if not dims:
        return 0
    return dims[-1][1] if dims[-1][1] >= C else None


def _like(t, dtype):
    """A dense tensor of t's shape."""
    if t.dtype == dtype and t.is_contiguous():
        return torch.empty_like(t)
    return torch.empty(*t.shape, dtype=dtype, device=t.device)


def _dense(t):
    """t where its rows lie evenly, else a copy."""
    return t if t is None or _row_stride(t) is not None else t.contiguous()


def _bytes(t):
    """First and last address of a tensor's elements."""
    a = t.data_ptr()
    if t.is_contiguous():
        return a, a + t.numel() * t.element_size()
    return a, a + (sum((n - 1) * s for n, s in zip(t.shape, t.stride())) + 1) * t.element_size()


def _apart(a, b):
    """Whether two tensors share no element: other memory, or other columns of the same rows."""
    if a is None or b is None or not a.numel() or not b.numel():
        return True
    (a0, a1), (b0, b1) = _bytes(a), _bytes(b)
    if a1 <= b0 or b1 <= a0:
        return True
    if a.dim() < 2 or a.dim() != b.dim():
        return False
    # the dimensions that hold more than a row, from the outermost on, have to run alike
    while a.dim() > 1 and (a.dim() > 2 and a.stride(0) == a.shape[1] * a.stride(1)
                           and b.stride(0) == b.shape[1] * b.stride(1)):
        a, b = a.flatten(0, 1), b.flatten(0, 1)
    step = a.stride(0) * a.element_size()
    if step != b.stride(0) * b.element_size() or step <= 0:
        return False
    (a0, ae), (b0, be) = _bytes(a[0]), _bytes(b[0])
    off = (b0 - a0) % step
    return ae - a0 <= off and off + be - b0 <= step


def _itself(a, b):
    return a.data_ptr() == b.data_ptr() and a.shape == b.shape and a.stride() == b.stride() and a.dtype == b.dtype


def _writable(out, what):
    if out.requires_grad and torch.is_grad_enabled():
        raise ValueError(f"{what} requires grad and is written without autograd's knowledge: use torch.no_grad()")


def _written(t):
    """Tells autograd that a given output has new values: a backward that needs the old ones then raises."""
    if t is not None and not t.is_inference():               # inference tensors have no version
        increment_version(t)


def _check_out(out, what, allowed, *others):
    """An output may be the tensor ``allowed`` itself, and has to be apart from all others."""
    _writable(out, what)
    o0, o1 = _bytes(out)
    near = False
    for t in (allowed, *others):
        if t is not None:
            t0, t1 = _bytes(t)
            near = near or (t0 < o1 and o0 < t1)
    if not near:
        return
    if allowed is not None and not _apart(out, allowed):
        _need(_itself(out, allowed), f"{what} overlaps an input without being it")
    for t in others:
        _need(_apart(out, t), f"{what} overlaps another argument")


def _refuse_capture(name, instead):
    if torch.cuda.is_initialized() and torch.cuda.is_current_stream_capturing():
        raise RuntimeError(f"{name} works on an autograd graph and cannot be captured; capture {instead}")


def _wants_graph(*tensors):
    """Whether a gradient may be asked for.  Tangents of forward mode are refused: a result without them would be taken
    for a constant."""
    if forward_ad._current_level >= 0 and any(t is not None and forward_ad.unpack_dual(t).tangent is not None
                                              for t in tensors):
        raise NotImplementedError("no forward-mode derivatives")
    return torch.is_grad_enabled() and any(t is not None and t.requires_grad for t in tensors)


# ------------------------------------------------------------------ block norms
def _vector(v, shape, what):
    if v is None:
        return
    _need(v.dtype == torch.float32, f"{what} must be float32, not {v.dtype}")
    _need(tuple(v.shape) == shape, f"{what} must be {shape}, not {tuple(v.shape)}")


def _norm_plan(x, h, gate, post_weight, weight, bias, scale, shift, norm, post_norm, eps, res_scale, rows_per_group,
               branch, rows):
    """The call's plan; ``rows``: its other tensors like x, as (field of the descriptor, name, tensor, type)."""
    _need(norm in _NORMS, f"norm is 'layer', 'rms' or None, not {norm!r}")
    _need(post_norm in _NORMS, f"post_norm is 'layer', 'rms' or None, not {post_norm!r}")
    _need(x.dim() >= 1 and x.shape[-1] >= 1, f"x must be [..., C], not {tuple(x.shape)}")
    _need(x.dtype in _DT and branch in _DT, f"float32 or bfloat16, not {x.dtype} and {branch}")
    C, R, dev = x.shape[-1], _count(x.shape), x.device
    _fits(channels=C)
    _same_device(dev, h, gate, post_weight, weight, bias, scale, shift, *(t for _, _, t, _ in rows))
    if h is not None:
        _need(h.shape == x.shape, f"h must have x's shape {tuple(x.shape)}, not {tuple(h.shape)}")
        _need(h.dtype == branch, f"h is {h.dtype} and the next branch {branch}")
    for _, what, t, dt in rows:
        _need(t is None or (t.shape == x.shape and t.dtype == dt),
              f"{what} must be {dt} of shape {tuple(x.shape)}")
    rpg = rows_per_group
    if rpg is None:
        rpg = x.shape[-2] if x.dim() > 2 else R
    _need(rpg >= 1 or R == 0, "rows_per_group must be at least 1")
    rpg = min(max(1, rpg), max(1, R))
    G = -(-R // rpg)
    if R == 0:
        # groups without rows: as many as the vectors have, or as x's leading dimensions make
        G = next((v.shape[0] for v in (gate, scale, shift) if v is not None and v.dim() == 2),
                 _count(x.shape[:-1]) if x.dim() > 2 and rows_per_group is None else 0)
    for v, shape, what in ((gate, (G, C), "gate"), (scale, (G, C), "scale"), (shift, (G, C), "shift"),
                           (post_weight, (C,), "post_weight"), (weight, (C,), "weight"), (bias, (C,), "bias")):
        _vector(v, shape, what)
    lds = dict.fromkeys(("x", "h", "z", "y", "dx", "dh", "dz", "dy", "gate", "scale", "shift"), 0)
    copy = any(v is not None and v.stride(0) != 1 and C > 1 for v in (post_weight, weight, bias))
    for field, t in ([("x", x), ("h", h), ("gate", gate), ("scale", scale), ("shift", shift)]
                     + [(f, t) for f, _, t, _ in rows]):
        if t is not None:
            ld = _row_stride(t)
            copy = copy or ld is None
            lds[field] = ld or 0
    if rows and rows[0][0] == "dz":                # the backward reads the stream as z
        lds["z"], lds["x"] = lds["x"], 0
    desc = _abi.BlockNormT(R, rpg, C, _DT[x.dtype], _DT[branch], _NORMS[norm], _NORMS[post_norm], eps, res_scale,
                           *lds.values())
    p = _Plan(desc, dev, copy)
    p.ws_bytes = _abi.block_norm_ws_bytes(desc)
    p.a, p.b = _NORMS[norm] != 0, (G, C)
    return p


def norm_forward(x, h=None, *, gate=None, post_weight=None, weight=None, bias=None, scale=None, shift=None,
                 norm="layer", post_norm=None, eps=1e-6, res_scale=1.0, rows_per_group=None, out_dtype=None, z=None,
                 y=None):
    """(z, y) with z = res_scale x + gate ∘ N_post(h) ∘ post_weight and
    y = N(z) ∘ weight ∘ (1 + scale) + bias ∘ (1 + scale) + shift.

    x [..., C] is the residual stream, h [..., C] the block's output (None: z is x); gate, scale and shift are
    float32 [groups, C], one row for each ``rows_per_group`` rows (default: x's last-but-one dimension where it has
    three or more, else all rows; without rows any number of groups); weight, bias and post_weight float32 [C].
    ``norm=None`` gives no y.  y has ``out_dtype`` (default: h's type, else x's).  ``z`` and ``y`` may be given as
    outputs; z may be x itself.
    """
    eps, res_scale, rows_per_group = _real(eps, "eps"), _real(res_scale, "res_scale"), _group_rows(rows_per_group)
    key = ("norm", x.shape, x.stride(), x.dtype, x.device, _sig(h), _sig(gate), _sig(post_weight), _sig(weight), _sig(bias),
           _sig(scale), _sig(shift), norm, post_norm, eps, res_scale, rows_per_group, out_dtype, _sig(z), _sig(y))
    p = _plans.get(key)
    if p is None:
        branch = out_dtype or (h if h is not None else x).dtype
        _need(z is None or h is not None, "without h there is no z to write")
        _need(y is None or norm not in (None, "none"), "without a norm there is no y to write")
        for t, what in ((z, "z"), (y, "y")):
            _need(t is None or t.dim() < 1 or _row_stride(t) is not None, f"{what}'s rows must lie evenly")
        p = _norm_plan(x, h, gate, post_weight, weight, bias, scale, shift, norm, post_norm, eps, res_scale,
                       rows_per_group, branch, (("z", "z", z, x.dtype), ("y", "y", y, branch)))
        p.c = branch
        _keep(key, p)
    if p.copy:
        x0 = x
        vecs = [None if v is None else v.contiguous() for v in (post_weight, weight, bias)]
        x, h, gate, scale, shift = (_dense(t) for t in (x, h, gate, scale, shift))
        zo, yo = norm_forward(x, h, gate=gate, post_weight=vecs[0], weight=vecs[1], bias=vecs[2], scale=scale,
                              shift=shift, norm=norm, post_norm=post_norm, eps=eps, res_scale=res_scale,
                              rows_per_group=rows_per_group, out_dtype=out_dtype, z=z, y=y)
        return (x0 if h is None else zo), yo
    if not _current(p.index):
        with torch.cuda.device(p.index):
            return norm_forward(x, h, gate=gate, post_weight=post_weight, weight=weight, bias=bias, scale=scale,
                                shift=shift, norm=norm, post_norm=post_norm, eps=eps, res_scale=res_scale,
                                rows_per_group=rows_per_group, out_dtype=out_dtype, z=z, y=y)
    given = () if z is None and y is None else (z, y)
    if z is not None:
        # h may be x, in place too: a row's h is read before its z is written
        _check_out(z, "z", x, None if _itself(h, x) else h, gate, post_weight, weight, bias, scale, shift)
    elif h is not None:
        z = _like(x, x.dtype)
    if y is not None:
        _check_out(y, "y", None, x, h, gate, post_weight, weight, bias, scale, shift, z)
    elif p.a:
        y = _like(x, p.c)
    _check("prism_block_norm_fwd", _abi.lib().prism_block_norm_fwd(
        p.addr, x.data_ptr(), _there(h), _ptr(gate), _ptr(post_weight), _ptr(weight), _ptr(bias), _ptr(scale),
        _ptr(shift), _ptr(z), _ptr(y), _stream(p.index)))
    for t in given:
        _written(t)
    return (x if h is None else z), y


_NORM_GRADS = ("dgate", "dscale", "dshift", "dpost_weight", "dweight", "dbias")      # [groups, C], then [C]


def norm_backward(z, h, dz, dy, *, gate=None, post_weight=None, weight=None, bias=None, scale=None, norm="layer",
                  post_norm=None, eps=1e-6, res_scale=1.0, rows_per_group=None, wants=None):
    """Gradients of ``norm_forward``, from the stored stream z (x where there was no h) and the branch h.

    dz (None: zero) is the gradient that reaches z past this norm, dy that of y.  Returns a dict of ``dx``, ``dh``
    and, for the vectors that are given, ``dgate``, ``dpost_weight``, ``dweight``, ``dbias``, ``dscale`` and, with
    scale, ``dshift``; the others are None.  ``wants``: names of the vectors' gradients to take instead
    (``dshift`` needs no vector).
    """
    if wants is not None:
        wants = tuple(wants)
    eps, res_scale, rows_per_group = _real(eps, "eps"), _real(res_scale, "res_scale"), _group_rows(rows_per_group)
    key = ("dnorm", z.shape, z.stride(), z.dtype, z.device, _sig(h), _sig(dz), _sig(dy), _sig(gate), _sig(post_weight),
           _sig(weight), _sig(bias), _sig(scale), norm, post_norm, eps, res_scale, rows_per_group, wants)
    p = _plans.get(key)
    if p is None:
        branch = (dy if dy is not None else h if h is not None else z).dtype
        has_y = norm not in (None, "none")
        _need(not has_y or dy is not None, "a norm's backward needs dy")
        _need(has_y or dz is not None, "without a norm the backward needs dz")
        have = dict(dgate=gate, dscale=scale, dshift=scale, dpost_weight=post_weight, dweight=weight, dbias=bias)
        names = [n for n in _NORM_GRADS if have[n] is not None] if wants is None else wants
        for n in names:
            _need(n in _NORM_GRADS, f"no gradient {n!r}")
        p = _norm_plan(z, h, gate, post_weight, weight, bias, scale, None, norm, post_norm, eps, res_scale,
                       rows_per_group, branch, (("dz", "dz", dz, z.dtype), ("dy", "dy", dy, branch)))
        p.a, p.c = branch, ([n for n in _NORM_GRADS[:3] if n in names], [n for n in _NORM_GRADS[3:] if n in names])
        _keep(key, p)
    if p.copy:
        vecs = [None if v is None else v.contiguous() for v in (post_weight, weight, bias)]
        z, h, dz, dy, gate, scale = (_dense(t) for t in (z, h, dz, dy, gate, scale))
        return norm_backward(z, h, dz, dy, gate=gate, post_weight=vecs[0], weight=vecs[1], bias=vecs[2], scale=scale,
                             norm=norm, post_norm=post_norm, eps=eps, res_scale=res_scale,
                             rows_per_group=rows_per_group, wants=wants)
    if not _current(p.index):
        with torch.cuda.device(p.index):
            return norm_backward(z, h, dz, dy, gate=gate, post_weight=post_weight, weight=weight, bias=bias, scale=scale,
                                 norm=norm, post_norm=post_norm, eps=eps, res_scale=res_scale,
                                 rows_per_group=rows_per_group, wants=wants)
    dev = z.device
    g = dict.fromkeys(("dx", "dh", "dgate", "dpost_weight", "dweight", "dbias", "dscale", "dshift"))
    g["dx"] = _like(z, z.dtype)
    if h is not None:
        g["dh"] = _like(z, p.a)
    groups, vectors = p.c
    G, C = p.b
    make = torch.empty if p.desc.rows else torch.zeros           # the library has no groups where it has no rows
    for n in groups:
        g[n] = make(G, C, dtype=torch.float32, device=dev)
    for n in vectors:
        g[n] = torch.empty(C, dtype=torch.float32, device=dev)
    ws = torch.empty(p.ws_bytes, dtype=torch.uint8, device=dev) if groups or vectors else None
    _check("prism_block_norm_bwd", _abi.lib().prism_block_norm_bwd(
        p.addr, z.data_ptr(), _there(h), _ptr(gate), _ptr(post_weight), _ptr(weight), _ptr(bias), _ptr(scale), _there(dz),
        _ptr(dy), _ptr(g["dx"]), _ptr(g["dh"]), _ptr(g["dgate"]), _ptr(g["dpost_weight"]), _ptr(g["dweight"]),
        _ptr(g["dbias"]), _ptr(g["dscale"]), _ptr(g["dshift"]), _ptr(ws), p.ws_bytes, _stream(p.index)))
    return g


class _NormFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, h, gate, post_weight, weight, bias, scale, shift, kw, out_dtype):
        ctx.set_materialize_grads(False)
        z, y = norm_forward(x, h, gate=gate, post_weight=post_weight, weight=weight, bias=bias, scale=scale,
                            shift=shift, out_dtype=out_dtype, **kw)
        ctx.save_for_backward(z, h, gate, post_weight, weight, bias, scale)
        ctx.kw, ctx.y_dtype, ctx.shift = kw, None if y is None else y.dtype, None if shift is None else shift.shape
        return (z, y) if h is not None else y

    @staticmethod
    @once_differentiable
    def backward(ctx, *grads):
        _refuse_capture("block.norm's backward", "norm_backward")
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
        if g["dshift"] is not None and g["dshift"].shape != ctx.shift:       # without rows its groups are not known
            g["dshift"] = g["dshift"].new_zeros(ctx.shift)
        return (g["dx"] if need[0] else None, g["dh"] if need[1] else None, g["dgate"], g["dpost_weight"], g["dweight"],
                g["dbias"], g["dscale"], g["dshift"], None, None)


def norm(x, h=None, *, gate=None, post_weight=None, weight=None, bias=None, scale=None, shift=None, norm="layer",
         post_norm=None, eps=1e-6, res_scale=1.0, rows_per_group=None, out_dtype=None):
    """Differentiable ``norm_forward``: returns (z, y); z is x itself where there is no h."""
    tensors = (x, h, gate, post_weight, weight, bias, scale, shift)
    kw = dict(norm=norm, post_norm=post_norm, eps=_real(eps, "eps"), res_scale=_real(res_scale, "res_scale"),
              rows_per_group=_group_rows(rows_per_group))
    if not _wants_graph(*tensors):
        return norm_forward(x, h, gate=gate, post_weight=post_weight, weight=weight, bias=bias, scale=scale,
                            shift=shift, out_dtype=out_dtype, **kw)
    _refuse_capture("block.norm", "norm_forward and norm_backward")
    if h is None:
        return x, _NormFn.apply(*tensors, kw, out_dtype)
    return _NormFn.apply(*tensors, kw, out_dtype)


# ------------------------------------------------------------------ head norm and rotation
def rotation_table(grid, axes, base=10000.0, device="cuda", positions=None):
    """The (cos, sin) rows that ``rotate`` reads: for each axis of ``grid`` = (T, H, W) a row for each place with
    ``axes`` = (pairs_t, pairs_h, pairs_w) pairs, pair i of n at place p turned by p base^(-i/n).  ``positions``:
    three sequences of places instead of 0, 1, 2, ...  Angles in 64 bits, rounded once to float32."""
    parts = []
    for a, (length, pairs) in enumerate(zip(grid, axes)):
        p = torch.arange(length, dtype=torch.float64) if positions is None else torch.as_tensor(
            positions[a], dtype=torch.float64, device="cpu")
        _need(p.shape == (length,), f"axis {a} has {length} places, not {tuple(p.shape)}")
        angle = p[:, None] * base ** (-torch.arange(pairs, dtype=torch.float64) / max(1, pairs))
        parts.append(torch.stack((angle.cos(), angle.sin()), -1).reshape(-1, 2))
    return torch.cat(parts).float().to(device)


def _head_stride(t):
    """Elements between tokens of t [tokens, heads, d], 0 for dense ones; None where the library cannot walk it."""
    n, h, d = t.shape
    s = t.stride()
    if t.numel() == 0:
        return 0
    if (d > 1 and s[2] != 1) or (h > 1 and s[1] != d):
        return None
    if n == 1:
        return 0
    return s[0] if s[0] >= h * d and s[0] * t.element_size() % 16 == 0 else None


def _aligned(t):
    """A dense copy of t, on 16 bytes (heads laid out otherwise, or starting elsewhere)."""
    if t is None or (_head_stride(t) is not None and t.data_ptr() % 16 == 0):
        return t
    return t.clone(memory_format=torch.contiguous_format)


def _on16(*tensors):
    m = 0
    for t in tensors:
        if t is not None:
            m |= t.data_ptr()
    return m % 16 == 0


def _rotate_plan(ins, outs, table, grid, axes, weights, norm, eps, pairs):
    """ins, outs: pairs of tensors (Q's, K's) by descriptor fields, the first of ins deciding the shapes."""
    _need(pairs in _PAIRS, f"pairs is 'interleaved' or 'half', not {pairs!r}")
    tensors = [t for f, pair in (*ins, *outs) for t in pair if t is not None]
    _need(tensors, "neither Q nor K")
    first = tensors[0]
    _same_device(first.device, table, *tensors, *weights)
    for t in tensors:
        _need(t.dim() == 3, "Q and K must be [tokens, heads, head_dim]")
        _need(t.shape[0] == first.shape[0] and t.shape[2] == first.shape[2] and t.dtype == first.dtype,
              "Q and K must agree in tokens, head_dim and type")
    _need(first.dtype in _DT, f"float32 or bfloat16, not {first.dtype}")
    rows = sum(n * p for n, p in zip(grid, axes))
    _need(table.dtype == torch.float32 and tuple(table.shape) == (rows, 2),
          f"table must be float32 [{rows}, 2], not {table.dtype} {tuple(table.shape)}")
    for w in weights:
        _vector(w, (first.shape[2],), "a head's weight")
        _need(norm or w is None, "weights without a norm")
    copy = not table.is_contiguous() or any(w is not None and w.stride(0) != 1 for w in weights)
    lds = {}
    for fields, pair in (*ins, *outs):
        for f, t in zip(fields, pair):
            ld = 0 if t is None else _head_stride(t)
            copy = copy or ld is None
            lds[f] = ld or 0
    heads = [0 if t is None else t.shape[1] for t in ins[0][1]]
    for _, pair in (*ins[1:], *outs):
        for t, n in zip(pair, heads):
            _need(t is None or t.shape[1] == n, "Q and K must be like their gradients and results")
    T, H, W = grid
    _fits(T=T, H=H, W=W, pairs_t=axes[0], pairs_h=axes[1], pairs_w=axes[2], head_dim=first.shape[2], heads=max(heads))
    desc = _abi.RotateT(first.shape[0], *grid, *heads, first.shape[2], *axes, _PAIRS[pairs], _DT[first.dtype],
                        int(norm), eps, *(lds.get(f, 0) for f in ("q", "k", "qo", "ko", "dq", "dk")))
    p = _Plan(desc, first.device, copy)
    p.ws_bytes = _abi.head_rotate_ws_bytes(desc)
    return p


def rotate_forward(Q, K, table, *, grid, axes, q_weight=None, k_weight=None, norm=True, eps=1e-6, pairs="interleaved",
                   out=None):
    """(Q, K) with each head's channels RMS-normed (``norm``), weighted (q_weight, k_weight float32 [d]) and its
    channel pairs turned by the token's place: token i lies at place i mod T H W of ``grid`` = (T, H, W) in raster
    order, the first axes[0] pairs turn with its t, the next axes[1] with h, the next axes[2] with w, the rest not
    at all.  ``table`` float32 [T axes[0] + H axes[1] + W axes[2], 2] as ``rotation_table`` makes it; ``pairs``
    'interleaved' (channels 2i, 2i + 1) or 'half' (i, i + d/2).  Q or K may be None, and have different numbers of
    heads.  ``out`` = (Qr, Kr) takes the results, and may be (Q, K) themselves.
    """
    oq, ok = (None, None) if out is None else out
    grid, axes, norm, eps = _whole(grid), _whole(axes), bool(norm), _real(eps, "eps")
    key = ("rotate", _sig(Q), _sig(K), _sig(table), grid, axes, _sig(q_weight), _sig(k_weight), norm, eps,
           pairs, _sig(oq), _sig(ok))
    p = _plans.get(key)
    if p is None:
        _need(out is None or ((oq is None) == (Q is None) and (ok is None) == (K is None)),
              "out must have a tensor for each of Q and K")
        for o in (oq, ok):
            _need(o is None or (o.dim() == 3 and _head_stride(o) is not None),
                  "out's heads must lie densely on 16-byte boundaries")
        p = _rotate_plan(((("q", "k"), (Q, K)),), ((("qo", "ko"), (oq, ok)),), table, grid, axes,
                         (q_weight, k_weight), norm, eps, pairs)
        _keep(key, p)
    if p.copy or not _on16(Q, K, table, q_weight, k_weight):
        vecs = [None if v is None else v.clone(memory_format=torch.contiguous_format) for v in (q_weight, k_weight)]
        _need(_on16(oq, ok), "out must lie on 16-byte boundaries")
        return rotate_forward(_aligned(Q), _aligned(K), table.clone(memory_format=torch.contiguous_format), grid=grid,
                              axes=axes, q_weight=vecs[0], k_weight=vecs[1], norm=norm, eps=eps, pairs=pairs, out=out)
    if not _current(p.index):
        with torch.cuda.device(p.index):
            return rotate_forward(Q, K, table, grid=grid, axes=axes, q_weight=q_weight, k_weight=k_weight, norm=norm,
                                  eps=eps, pairs=pairs, out=out)
    if out is None:
        oq = None if Q is None else _like(Q, Q.dtype)
        ok = None if K is None else _like(K, K.dtype)
    else:
        # one tensor as Q and K would be read by one side while the other writes it
        for o, own, other in ((oq, Q, K), (ok, K, Q)):
            if o is not None:
                _check_out(o, "out", own, table, q_weight, k_weight)
                _need(_apart(o, other), "out overlaps the other of Q and K")
        _need(_apart(oq, ok), "the outputs overlap")
    _check("prism_head_rotate_fwd", _abi.lib().prism_head_rotate_fwd(
        p.addr, _ptr(Q), _ptr(K), _ptr(q_weight), _ptr(k_weight), table.data_ptr(), _ptr(oq), _ptr(ok),
        _stream(p.index)))
    if out is not None:
        _written(oq)
        _written(ok)
    return oq, ok


def rotate_backward(Q, K, dQr, dKr, table, *, grid, axes, q_weight=None, k_weight=None, norm=True, eps=1e-6,
                    pairs="interleaved", wants=None):
    """Gradients of ``rotate_forward`` from its inputs Q, K and its outputs' gradients: a dict of ``dQ``, ``dK`` and,
    for the weights that are given, ``dq_weight``, ``dk_weight`` (``wants``: names of these to take instead); the
    others are None.  Without a norm Q and K are not read and may be None."""
    if wants is not None:
        wants = tuple(wants)
    grid, axes, norm, eps = _whole(grid), _whole(axes), bool(norm), _real(eps, "eps")
    if not norm:
        Q = K = None
    key = ("drotate", _sig(Q), _sig(K), _sig(dQr), _sig(dKr), _sig(table), grid, axes, _sig(q_weight), _sig(k_weight),
           norm, eps, pairs, wants)
    p = _plans.get(key)
    if p is None:
        for x, dr in ((Q, dQr), (K, dKr)):
            _need(x is None or dr is not None, "Q and K must be like their gradients")
            _need(dr is None or x is not None or not norm, "the norm's backward needs Q and K")
        names = wants if wants is not None else [n for n, w in (("dq_weight", q_weight), ("dk_weight", k_weight))
                                                 if w is not None]
        for n in names:
            _need(n in ("dq_weight", "dk_weight") and norm and (dQr if n == "dq_weight" else dKr) is not None,
                  f"no gradient {n!r} here")
        p = _rotate_plan(((("dq", "dk"), (dQr, dKr)), (("q", "k"), (Q, K))), (), table, grid, axes,
                         (q_weight, k_weight), norm, eps, pairs)
        p.a = names
        _keep(key, p)
    if p.copy or not _on16(Q, K, dQr, dKr, table, q_weight, k_weight):
        vecs = [None if v is None else v.clone(memory_format=torch.contiguous_format) for v in (q_weight, k_weight)]
        return rotate_backward(_aligned(Q), _aligned(K), _aligned(dQr), _aligned(dKr),
                               table.clone(memory_format=torch.contiguous_format), grid=grid, axes=axes,
                               q_weight=vecs[0], k_weight=vecs[1], norm=norm, eps=eps, pairs=pairs, wants=wants)
    if not _current(p.index):
        with torch.cuda.device(p.index):
            return rotate_backward(Q, K, dQr, dKr, table, grid=grid, axes=axes, q_weight=q_weight, k_weight=k_weight,
                                   norm=norm, eps=eps, pairs=pairs, wants=wants)
    dev = table.device
    g = dict.fromkeys(("dQ", "dK", "dq_weight", "dk_weight"))
    if dQr is not None:
        g["dQ"] = _like(dQr, dQr.dtype)
    if dKr is not None:
        g["dK"] = _like(dKr, dKr.dtype)
    ws = None
    if p.a:
        d = p.desc.head_dim
        for n in p.a:
            g[n] = torch.empty(d, dtype=torch.float32, device=dev)
        ws = torch.empty(p.ws_bytes, dtype=torch.uint8, device=dev)
    _check("prism_head_rotate_bwd", _abi.lib().prism_head_rotate_bwd(
        p.addr, _ptr(Q), _ptr(K), _ptr(q_weight), _ptr(k_weight), table.data_ptr(), _ptr(dQr), _ptr(dKr), _ptr(g["dQ"]),
        _ptr(g["dK"]), _ptr(g["dq_weight"]), _ptr(g["dk_weight"]), _ptr(ws), p.ws_bytes, _stream(p.index)))
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
        _refuse_capture("block.rotate's backward", "rotate_backward")
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
    kw = dict(grid=_whole(grid), axes=_whole(axes), norm=bool(norm), eps=_real(eps, "eps"), pairs=pairs)
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
    __slots__ = ("rows", "top_k", "experts", "align", "device", "rows_sorted", "counts", "offsets", "pos", "src",
                 "_call")

    def __init__(self, rows, top_k, experts, align, id_bytes, device):
        key = ("experts", rows, top_k, experts, align, id_bytes, device)
        p = _plans.get(key)
        if p is None:
            _fits(top_k=top_k, experts=experts, align=align)
            p = _Plan(_abi.ExpertsT(rows, top_k, experts, align, id_bytes), device)
            p.a, p.ws_bytes = _abi.expert_sizes(p.desc)
            _keep(key, p)
        self._call, self.rows_sorted = p, p.a
        self.rows, self.top_k, self.experts, self.align, self.device = rows, top_k, experts, align, device
        e = torch.empty
        self.counts = e(experts, dtype=torch.int32, device=device)
        self.offsets = e(experts + 1, dtype=torch.int32, device=device)
        self.pos = e(rows, top_k, dtype=torch.int32, device=device)
        self.src = e(p.a, dtype=torch.int32, device=device)


def expert_plan(ids, experts, align=1) -> ExpertPlan:
    """Sort the slots of ids [rows, top_k] (int32 or int64) by expert, stably; an id outside [0, experts) drops its
    slot.  Each expert's rows start at a multiple of ``align``."""
    _need(ids.dim() == 2, f"ids must be [rows, top_k], not {tuple(ids.shape)}")
    _need(ids.dtype in (torch.int32, torch.int64), f"ids must be int32 or int64, not {ids.dtype}")
    dev = ids.device
    _same_device(dev)
    if not ids.is_contiguous():
        ids = ids.contiguous()
    if not _current(dev.index):
        with torch.cuda.device(dev.index):
            return expert_plan(ids, experts, align)
    rows, top_k = ids.shape
    p = ExpertPlan(rows, top_k, int(experts), int(align), ids.element_size(), dev)
    c = p._call
    ws = torch.empty(c.ws_bytes, dtype=torch.uint8, device=dev) if c.ws_bytes else None
    code = _abi.lib().prism_expert_plan(c.addr, ids.data_ptr(), p.counts.data_ptr(), p.offsets.data_ptr(),
                                        p.pos.data_ptr(), p.src.data_ptr(), _ptr(ws),
                                        c.ws_bytes, _stream(dev.index))
    if code:
        raise _abi.PrismError("prism_expert_plan", code)
    return p


def _extent(t):
    """Bytes from a tensor's first element to its last one's end."""
    if t is None or not t.numel():
        return 0
    a, b = _bytes(t)
    return b - a


def _by_token(t, plan, C, dtype, what):
    """Row stride of t [rows, C] (None: to be copied)."""
    if t is None:
        return 0
    _need(t.dim() == 2 and t.shape[0] == plan.rows and t.shape[1] >= 1 and (C is None or t.shape[1] == C),
          f"{what} must be [{plan.rows}, channels], not {tuple(t.shape)}")
    _need(t.dtype in _DT and (dtype is None or t.dtype == dtype), f"{what} has type {t.dtype}")
    _same_device(plan.device, t)
    return _row_stride(t)


def _sorted(t, plan, C, dtype, what):
    if t is not None:
        _need(t.dim() == 2 and t.shape[0] == plan.rows_sorted and t.shape[1] >= 1 and (C is None or t.shape[1] == C),
              f"{what} must be [{plan.rows_sorted}, channels], not {tuple(t.shape)}")
        _need(t.dtype in _DT and (dtype is None or t.dtype == dtype), f"{what} has type {t.dtype}")
        _same_device(plan.device, t)


def _weights(w, plan):
    if w is not None:
        _need(w.dtype == torch.float32 and tuple(w.shape) == (plan.rows, plan.top_k),
              f"weights must be float32 [{plan.rows}, {plan.top_k}]")
        _same_device(plan.device, w)


def expert_dispatch(x, plan, *, out=None):
    """xs [rows_sorted, C]: x's rows [rows, C] copied to their slots' rows; the rows between an expert's last slot
    and the next multiple of ``align`` are 0, as are those behind the last expert.  A given ``out`` (dense, not
    overlapping x) keeps the rows behind the last expert as they are."""
    call = plan._call
    key = ("dispatch", call, _sig(x), _sig(out))
    p = _plans.get(key)
    if p is None:
        ld = _by_token(x, plan, None, None, "x")
        _sorted(out, plan, x.shape[1], x.dtype, "out")
        _need(out is None or out.is_contiguous(), "out must be dense")
        p = _Plan(call.desc, plan.device, ld is None)
        p.a = (_DT[x.dtype], x.shape[1], ld, _extent(x), _extent(out))
        _keep(key, p)
    if p.copy:
        return expert_dispatch(x.contiguous(), plan, out=out)
    if not _current(p.index):
        with torch.cuda.device(p.index):
            return expert_dispatch(x, plan, out=out)
    dt, C, ld, n_x, n_out = p.a
    clear = out is None
    if clear:
        out = torch.empty(plan.rows_sorted, C, dtype=x.dtype, device=x.device)
    else:
        _writable(out, "out")
    p_x, p_out = x.data_ptr(), out.data_ptr()
    if p_x < p_out + n_out and p_out < p_x + n_x:
        _check_out(out, "out", None, x)
    code = _abi.lib().prism_expert_dispatch(p.addr, dt, C, p_x, ld, plan.pos.data_ptr(), plan.counts.data_ptr(),
                                            plan.offsets.data_ptr(), clear, p_out, _stream(p.index))
    if code:
        raise _abi.PrismError("prism_expert_dispatch", code)
    if not clear:
        _written(out)
    return out


def expert_combine(ys, plan, weights=None, *, add=None, out=None):
    """out [rows, C]: add[t] + sum over t's choices j of weights[t, j] ys[pos[t, j]], without the dropped ones
    (weights float32 [rows, top_k], None: 1; add None: 0).  Summed in float32 in j's order, rounded once.  Without
    weights it is the gradient of ``expert_dispatch``.  ``out`` may be ``add`` itself."""
    call = plan._call
    key = ("combine", call, _sig(ys), _sig(weights), _sig(add), _sig(out))
    p = _plans.get(key)
    if p is None:
        _sorted(ys, plan, None, None, "ys")
        _weights(weights, plan)
        C = ys.shape[1]
        ld_add, ld_out = _by_token(add, plan, C, ys.dtype, "add"), _by_token(out, plan, C, ys.dtype, "out")
        _need(ld_out is not None, "out's rows must lie evenly")
        p = _Plan(call.desc, plan.device, ld_add is None or not ys.is_contiguous()
                  or (weights is not None and not weights.is_contiguous()))
        p.a = (_DT[ys.dtype], C, ld_add, ld_out)
        _keep(key, p)
    if p.copy:
        return expert_combine(ys.contiguous(), plan, None if weights is None else weights.contiguous(),
                              add=_dense(add), out=out)
    if not _current(p.index):
        with torch.cuda.device(p.index):
            return expert_combine(ys, plan, weights, add=add, out=out)
    dt, C, ld_add, ld_out = p.a
    given = out
    if out is None:
        out = torch.empty(plan.rows, C, dtype=ys.dtype, device=ys.device)
    else:
        _check_out(out, "out", add, ys, weights)
    code = _abi.lib().prism_expert_combine(p.addr, dt, C, ys.data_ptr(), plan.pos.data_ptr(),
                                           _ptr(weights),
                                           _ptr(add), ld_add, out.data_ptr(), ld_out,
                                           _stream(p.index))
    if code:
        raise _abi.PrismError("prism_expert_combine", code)
    if given is not None:
        _written(given)
    return out


def expert_combine_backward(dout, ys, plan, weights=None, *, out=None, want_weights=True):
    """(dys, dweights) of ``expert_combine``: dys[pos[t, j]] = weights[t, j] dout[t] and dweights[t, j] =
    ys[pos[t, j]] . dout[t] (0 where dropped; None with ``want_weights=False``, where ys may be None).  Rows of dys
    without a slot as in ``expert_dispatch``; ``out`` may be ys itself."""
    if not want_weights:
        ys = None
    call = plan._call
    key = ("dcombine", call, _sig(dout), _sig(ys), _sig(weights), _sig(out), want_weights)
    p = _plans.get(key)
    if p is None:
        ld = _by_token(dout, plan, None, None, "dout")
        C = dout.shape[1]
        _weights(weights, plan)
        _need(ys is not None or not want_weights, "the weights' gradient needs ys")
        _sorted(ys, plan, C, dout.dtype, "ys")
        _sorted(out, plan, C, dout.dtype, "out")
        _need(out is None or out.is_contiguous(), "out must be dense")
        p = _Plan(call.desc, plan.device, ld is None or (ys is not None and not ys.is_contiguous())
                  or (weights is not None and not weights.is_contiguous()))
        p.a = (_DT[dout.dtype], C, ld, _extent(out), _extent(ys), _extent(dout), _extent(weights))
        _keep(key, p)
    if p.copy:
        return expert_combine_backward(_dense(dout), None if ys is None else ys.contiguous(), plan,
                                       None if weights is None else weights.contiguous(), out=out,
                                       want_weights=want_weights)
    if not _current(p.index):
        with torch.cuda.device(p.index):
            return expert_combine_backward(dout, ys, plan, weights, out=out, want_weights=want_weights)
    dt, C, ld, n_out, n_y, n_d, n_w = p.a
    p_d = dout.data_ptr()
    p_y = _ptr(ys)
    p_w = _ptr(weights)
    clear = out is None
    if clear:
        out = torch.empty(plan.rows_sorted, C, dtype=dout.dtype, device=dout.device)
        p_out = out.data_ptr()
    else:
        _writable(out, "out")
        p_out = out.data_ptr()
        end = p_out + n_out
        if (p_d < end and p_out < p_d + n_d or p_y is not None and p_y < end and p_out < p_y + n_y
                or p_w is not None and p_w < end and p_out < p_w + n_w):
            _check_out(out, "out", ys, dout, weights)
    dw = p_dw = None
    if want_weights:
        dw = torch.empty(plan.rows, plan.top_k, dtype=torch.float32, device=dout.device)
        p_dw = dw.data_ptr()
    code = _abi.lib().prism_expert_combine_bwd(p.addr, dt, C, p_d, ld, p_y, plan.pos.data_ptr(), p_w,
                                               plan.counts.data_ptr(), plan.offsets.data_ptr(), clear, p_out, p_dw,
                                               _stream(p.index))
    if code:
        raise _abi.PrismError("prism_expert_combine_bwd", code)
    if not clear:
        _written(out)
    return out, dw


class _DispatchFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, plan):
        ctx.plan = plan
        return expert_dispatch(x, plan)

    @staticmethod
    @once_differentiable
    def backward(ctx, dxs):
        _refuse_capture("block.dispatch's backward", "expert_combine")
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
        _refuse_capture("block.combine's backward", "expert_combine_backward")
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

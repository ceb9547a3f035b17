"""Plain forms of the operators around the attention, in 64 bits, for the tests.

Gradients come from torch's differentiation of the definitions.  Beside each value the norms' and the
rotation's forms give the sum of the absolute values of the terms it is made of (``*_terms``), from which
the tests' error bounds follow.
"""
import torch

U = 2.0 ** -24                                     # half a step of float32


def half_step(dt):
    return torch.finfo(dt).eps / 2


def d64(t):
    return None if t is None else t.detach().double()


def normed(v, kind, eps):
    if kind is None:
        return v
    if kind == "layer":
        v = v - v.mean(-1, keepdim=True)
    return v / torch.sqrt((v * v).mean(-1, keepdim=True) + eps)


def of_rows(v, R, rpg):
    return v[torch.arange(R, device=v.device) // rpg]


def block_norm(x, h, a, norm, post, eps, res, rpg):
    """(z, y) of 64-bit tensors; a: dict of gate, post_weight, weight, bias, scale, shift or None."""
    R = x.shape[0]
    z = x
    if h is not None:
        t = normed(h, post, eps)
        if a["post_weight"] is not None:
            t = t * a["post_weight"]
        if a["gate"] is not None:
            t = t * of_rows(a["gate"], R, rpg)
        z = res * x + t
    if norm is None:
        return z, None
    y = normed(z, norm, eps)
    if a["weight"] is not None:
        y = y * a["weight"]
    if a["bias"] is not None:
        y = y + a["bias"]
    if a["scale"] is not None:
        y = y * (1 + of_rows(a["scale"], R, rpg))
    if a["shift"] is not None:
        y = y + of_rows(a["shift"], R, rpg)
    return z, y


def _mean(v):
    return v.mean(-1, keepdim=True)


def _norm_terms(v, kind, eps):
    """For n = N(v): r, the size A of the terms n is made of (v and its mean), and the row's S >= 1, by which an
    error of v relative to its terms can grow in r: the mean square of A."""
    if kind is None:
        return 1.0, v.abs(), 1.0
    c = v - _mean(v) if kind == "layer" else v
    r = 1 / torch.sqrt(_mean(c * c) + eps)
    A = r * (v.abs() + (_mean(v.abs()) if kind == "layer" else 0))
    return r, A, 1 + _mean(A * A)


def norm_forward_terms(x, h, a, norm, post, eps, res, rpg):
    """Sizes of the terms of z and of y.  An error of z relative to its own terms passes to y through r."""
    R = x.shape[0]
    one = lambda n: 1.0 if a[n] is None else a[n].abs()
    rows = lambda n: 0.0 if a[n] is None else of_rows(a[n], R, rpg)
    z, _ = block_norm(x, h, a, None, post, eps, res, rpg)
    mz = x.abs()
    if h is not None:
        _, A, S = _norm_terms(h, post, eps)
        g = 1.0 if a["gate"] is None else rows("gate").abs()
        mz = abs(res) * x.abs() + g * one("post_weight") * A * S
    if norm is None:
        return mz, None
    r, A, _ = _norm_terms(z, norm, eps)
    B = r * (mz + (_mean(mz) if norm == "layer" else 0))      # n's terms, and those of z behind them
    my = B * (1 + _mean(B * B)) * one("weight") * (1 + abs(rows("scale")))
    if a["bias"] is not None:
        my = my + a["bias"].abs() * (1 + abs(rows("scale")))
    return mz, my + abs(rows("shift"))


def norm_backward_terms(z, h, dz, dy, a, norm, post, eps, res, rpg):
    """Sizes of the terms of every gradient."""
    R, C = z.shape
    G = -(-R // rpg)
    one = lambda n: 1.0 if a[n] is None else a[n].abs()
    rows = lambda n: 0.0 if a[n] is None else of_rows(a[n], R, rpg).abs()
    gate = 1.0 if a["gate"] is None else rows("gate")

    def groups(v):
        out = v.new_zeros(G, C)
        return out.index_add_(0, torch.arange(R, device=v.device) // rpg, v)

    m = {}
    d = torch.zeros_like(z) if dz is None else dz.abs()
    if norm is not None:
        r, A, S = _norm_terms(z, norm, eps)
        c = dy.abs() * one("weight") * (1 + rows("scale"))
        d = d + r * S * (c + _mean(c) + A * _mean(c * A))
        nA, nD = groups(dy.abs() * A * S), groups(dy.abs())
        s1 = 1.0 if a["scale"] is None else 1 + a["scale"].abs()
        m["dscale"] = nA * one("weight") + (0 if a["bias"] is None else nD * a["bias"].abs())
        m["dshift"] = nD
        m["dweight"], m["dbias"] = (nA * s1).sum(0), (nD * s1).sum(0)
    m["dx"] = d if h is None else abs(res) * d
    if h is not None:
        rh, Ah, Sh = _norm_terms(h, post, eps)
        t = d * gate * one("post_weight")
        m["dh"] = t if post is None else rh * Sh * (t + _mean(t) + Ah * _mean(t * Ah))
        m["dgate"] = groups(d * Ah * Sh) * one("post_weight")
        m["dpost_weight"] = (d * gate * Ah * Sh).sum(0)
    return m


def rotate(x, w, cos, sin, pairs, eps):
    """Head norm (where w is not None) and rotation of 64-bit x [tokens, heads, d]; cos, sin [tokens, 1, d/2]."""
    if w is not None:
        x = normed(x, "rms", eps) * w
    h = x.shape[-1] // 2
    a, b = (x[..., 0::2], x[..., 1::2]) if pairs == "interleaved" else (x[..., :h], x[..., h:])
    p, q = a * cos - b * sin, a * sin + b * cos
    return torch.stack((p, q), -1).flatten(-2) if pairs == "interleaved" else torch.cat((p, q), -1)


def angles(table, grid, axes, tokens, d):
    """cos, sin [tokens, 1, d/2] of the table that the framework reads, in 64 bits."""
    (T, H, W), (nT, nH, nW) = grid, axes
    i = torch.arange(tokens, device=table.device) % (T * H * W)
    t, h, w = i // (H * W), i // W % H, i % W
    a, b, c = table.double().split((T * nT, H * nH, W * nW))
    cs = torch.cat((a.view(T, nT, 2)[t], b.view(H, nH, 2)[h], c.view(W, nW, 2)[w]), 1)
    rest = d // 2 - cs.shape[1]
    still = torch.tensor([1.0, 0.0], dtype=torch.float64, device=table.device).expand(tokens, rest, 2)
    cs = torch.cat((cs, still), 1)
    return cs[:, None, :, 0], cs[:, None, :, 1]


def experts(ids, E, align, cap):
    """counts, offsets, pos, src of the sort, slot by slot on the host."""
    flat = ids.reshape(-1).tolist()
    lists = [[] for _ in range(E)]
    for i, e in enumerate(flat):
        if 0 <= e < E:
            lists[e].append(i)
    pos, src, offsets = [-1] * len(flat), [-1] * cap, [0]
    for slots in lists:
        for j, i in enumerate(slots):
            pos[i] = offsets[-1] + j
            src[offsets[-1] + j] = i
        offsets.append(offsets[-1] + -(-len(slots) // align) * align)
    t = lambda v: torch.tensor(v, dtype=torch.int32)
    return t([len(s) for s in lists]), t(offsets), t(pos).view(ids.shape), t(src)

"""The operators around the attention on the GPU against plain forms in 64 bits (block_forms).

Bounds.  Every result is held in float32 until its one rounding, so it is off by at most half a step of its
type, relative to it, and K half steps of float32 relative to the sum of its terms' sizes: a term passes at
most 8 sums in a thread, 5 in a warp and 5 over the warps of each of up to four reductions (mean, second
moment, both again of the branch) and about twenty products, so K = 128 covers them; a sum over n rows adds
at most n.  All but a few terms stay far below that.
"""
import ctypes

import pytest
import torch

import block_forms as bf
from dynamic_block_sparse_macro_b200 import _abi, block, inputs
from dynamic_block_sparse_macro_b200.configs import get_config
from dynamic_block_sparse_macro_b200.layer import PrismSparseAttention, prism_attention

pytestmark = pytest.mark.gpu

K = 128
F32, BF16 = torch.float32, torch.bfloat16


def close(got, want, terms, extra=0, what=""):
    bound = bf.half_step(got.dtype) * want.abs() * 1.01 + (K + extra) * bf.U * terms + 1e-37
    err = (got.double() - want).abs()
    bad = ~(err <= bound)                                  # NaN is bad
    if bool(bad.any()):
        pytest.fail(f"{what}: {int(bad.sum())} of {bad.numel()} off, up to {float((err / bound).max())} of the bound, "
                    f"first at {bad.nonzero()[0].tolist()}: {float(got[bad][0])} for {float(want[bad][0])}")


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return lambda *s, std=1.0, dt=F32: (torch.randn(*s, generator=g, device="cuda") * std).to(dt)


# ------------------------------------------------------------------ block norms
def vectors(n, R, C, rpg, have):
    G = -(-R // rpg)
    a = dict.fromkeys(("gate", "post_weight", "weight", "bias", "scale", "shift"))
    for k in have.split():
        a[k] = n(G, C, std=0.5) if k in ("gate", "scale", "shift") else 1 + n(C, std=0.3)
    return a


ALL = "gate post_weight weight bias scale shift"
NORM_CASES = [
    # rows, channels, rows a group, stream, branch, norm, post, vectors, res_scale
    (1, 1, 1, F32, F32, "rms", "rms", ALL, 1.0),
    (2, 7, 1, BF16, BF16, "layer", "layer", ALL, 0.5),
    (5, 64, 2, F32, BF16, "rms", None, "gate scale shift", 1.0),
    (3, 100, 5, BF16, BF16, "layer", "rms", "gate weight bias", 1.0),
    (33, 256, 33, F32, F32, "layer", None, "gate scale shift", 1.0),
    (700, 333, 97, F32, BF16, "layer", "layer", ALL, -0.7),
    (257, 1001, 64, BF16, BF16, "rms", "layer", ALL, 0.5),
    (301, 2048, 100, BF16, BF16, "layer", None, "gate scale shift", 1.0),
    (130, 2050, 130, F32, F32, "rms", "rms", "post_weight weight", 1.0),
    (64, 5120, 64, BF16, BF16, "rms", "rms", "post_weight weight", 0.5),
    (19, 4104, 7, F32, BF16, "layer", "layer", ALL, 1.0),
    (11, 8192, 3, F32, F32, "layer", "rms", ALL, 1.0),
    (9, 8191, 9, BF16, BF16, "rms", "layer", ALL, 1.0),
    (4099, 64, 1, BF16, BF16, "layer", None, "gate scale shift", 1.0),
    (3001, 72, 1500, BF16, BF16, None, "rms", "gate post_weight", 1.0),
    (2500, 128, 2500, F32, F32, "rms", None, "weight", 1.0),
    # teams of several warps whose rows share barriers: one norm behind a plain branch, two rms norms; many rows a team
    (997, 4096, 997, BF16, BF16, "layer", None, "gate scale shift", 1.0),
    (1500, 3000, 499, F32, BF16, "rms", "rms", "gate post_weight weight", 0.5),
    (611, 6000, 611, F32, F32, "layer", None, "gate weight bias scale shift", -1.0),
    (2111, 264, 700, BF16, BF16, "rms", "rms", ALL, 1.0),
    (4999, 1100, 4999, F32, F32, "layer", None, "scale shift", 1.0),
    # groups that are not cut, more of them than teams: runs of groups with all gradients
    (10007, 64, 1, F32, F32, "layer", "rms", ALL, 1.0),
    (1203, 2048, 2, BF16, BF16, "layer", "layer", ALL, 0.5),
    (900, 1001, 1, BF16, BF16, "rms", "rms", ALL, 1.0),
    # few groups, cut, on both sides of what one cluster's first CTA adds up, and many cut ones
    (4000, 64, 1000, F32, BF16, "layer", None, ALL.replace("post_weight ", ""), 1.0),
    (5000, 520, 1000, BF16, BF16, "layer", "rms", ALL, 1.0),
    (20000, 40, 700, F32, F32, "rms", "layer", ALL, 1.0),
    (40000, 96, 40000, BF16, BF16, "layer", "rms", ALL, 1.0),
    (6001, 320, 6001, BF16, BF16, "layer", "rms", ALL, 1.0),
]


@pytest.mark.parametrize("R,C,rpg,sdt,bdt,norm,post,have,res", NORM_CASES)
@pytest.mark.parametrize("branch", [True, False])
def test_norm_forward_and_backward(R, C, rpg, sdt, bdt, norm, post, have, res, branch):
    if not branch and norm is None:
        pytest.skip("neither a branch nor a norm: nothing to do")
    n = gen(R * 10007 + C)
    a = vectors(n, R, C, rpg, have)
    x = n(R, C, std=2.0, dt=sdt) + 0.5
    h = n(R, C, dt=bdt)
    if not branch:
        h, post = None, None
        a["gate"] = a["post_weight"] = None
    kw = dict(norm=norm, post_norm=post, eps=1e-5, res_scale=res, rows_per_group=rpg)
    z, y = block.norm_forward(x, h, out_dtype=bdt, **a, **kw)
    a64 = {k: bf.d64(v) for k, v in a.items()}
    fa = (norm, post, 1e-5, res, rpg)
    zw, yw = bf.block_norm(bf.d64(x), bf.d64(h), a64, *fa)
    mz, my = bf.norm_forward_terms(bf.d64(x), bf.d64(h), a64, *fa)
    if branch:
        close(z, zw, mz, what="z")
    else:
        assert z is x
    if norm is not None:
        close(y, yw, my, what="y")

    # the backward from the stored stream, which bf16 has rounded: two leaves, z and h
    dz, dy = n(R, C, dt=sdt), None if norm is None else n(R, C, dt=bdt)
    av = {k: a[k] for k in a if k != "shift"}
    g = block.norm_backward(z, h, dz, dy, **av, **kw)
    la = {k: None if v is None else v.clone().requires_grad_() for k, v in a64.items()}
    z64 = bf.d64(z).requires_grad_()
    tot = bf.d64(dz)
    want = {}
    if norm is not None:
        _, yv = bf.block_norm(z64, None, dict(la, gate=None, post_weight=None), norm, None, 1e-5, 1.0, rpg)
        ks = [k for k in ("weight", "bias", "scale", "shift") if la[k] is not None]
        gs = torch.autograd.grad((yv * bf.d64(dy)).sum(), [z64] + [la[k] for k in ks])
        tot = tot + gs[0]
        want.update({"d" + k: v for k, v in zip(ks, gs[1:])})
    want["dx"] = tot * res if branch else tot
    if branch:
        h64 = bf.d64(h).requires_grad_()
        zb, _ = bf.block_norm(torch.zeros_like(h64), h64, la, None, post, 1e-5, res, rpg)
        ks = [k for k in ("gate", "post_weight") if la[k] is not None]
        gs = torch.autograd.grad((zb * tot.detach()).sum(), [h64] + [la[k] for k in ks])
        want["dh"] = gs[0]
        want.update({"d" + k: v for k, v in zip(ks, gs[1:])})
    m = bf.norm_backward_terms(bf.d64(z), bf.d64(h), bf.d64(dz), bf.d64(dy), a64, *fa)
    for k, v in g.items():
        assert (v is not None) == (k in want) or (k == "dshift" and a["scale"] is None), k
        if v is not None and k in want:
            close(v, want[k].detach(), m[k], 0 if k in ("dx", "dh") else R, what=k)


def test_norm_without_dz_takes_zero_and_gives_only_what_is_wanted():
    n = gen(3)
    x, dy = n(50, 96), n(50, 96)
    w, s = 1 + n(96, std=0.1), n(5, 96)
    kw = dict(weight=w, scale=s, rows_per_group=10)
    a = block.norm_backward(x, None, torch.zeros_like(x), dy, **kw)
    b = block.norm_backward(x, None, None, dy, wants=("dshift",), **kw)
    assert torch.equal(a["dx"], b["dx"]) and torch.equal(a["dshift"], b["dshift"])
    assert b["dweight"] is None and b["dscale"] is None


@pytest.mark.parametrize("C,off", [(256, 0), (256, 1), (256, 4), (100, 2), (333, 3)])
def test_norm_of_strided_and_unaligned_rows(C, off):
    """Rows cut out of wider ones, starting anywhere, give the bits of dense ones."""
    n = gen(C + off)
    wide = n(40, 2 * C + 16, dt=BF16)
    x, h = wide[:, off:off + C], wide[:, C + 8 + off:2 * C + 8 + off]
    vec = n(4, 3 * C + 1)
    gate, scale, shift = (vec[:, i * C + 1:(i + 1) * C + 1] for i in range(3))
    kw = dict(rows_per_group=10, norm="layer", post_norm="rms")
    # the width of an access, and with it the order of a row's sums, follows the alignment: the bound, not the bits
    z, y = block.norm_forward(x, h, gate=gate, scale=scale, shift=shift, **kw)
    a = dict.fromkeys(("post_weight", "weight", "bias"))
    a.update(gate=bf.d64(gate), scale=bf.d64(scale), shift=bf.d64(shift))
    f = ("layer", "rms", 1e-6, 1.0, 10)
    zw, yw = bf.block_norm(bf.d64(x), bf.d64(h), a, *f)
    mz, my = bf.norm_forward_terms(bf.d64(x), bf.d64(h), a, *f)
    close(z, zw, mz)
    close(y, yw, my)
    dz, dy = n(40, C, dt=BF16), n(40, C, dt=BF16)
    g1 = block.norm_backward(z, h, dz, dy, gate=gate, scale=scale, **kw)
    zs = torch.empty(40, C + 24, dtype=BF16, device="cuda")[:, 1:C + 1].copy_(z)
    g2 = block.norm_backward(zs, h, dz, dy, gate=gate, scale=scale, **kw)
    m = bf.norm_backward_terms(bf.d64(z), bf.d64(h), bf.d64(dz), bf.d64(dy), a, *f)
    for k in ("dx", "dh", "dgate", "dscale", "dshift"):
        close(g2[k], g1[k].double(), 2 * m[k] + (bf.half_step(BF16) / bf.U / K if k in ("dx", "dh") else 0)
              * g1[k].double().abs(), 40, what=k)


def test_norm_leaves_what_lies_behind_strided_outputs():
    n = gen(8)
    x, h = n(6, 64), n(6, 64)
    big = torch.full((8, 80), 7.0, device="cuda")
    z, y = block.norm_forward(x, h, z=big[1:7, 8:72])
    z0, y0 = block.norm_forward(x, h)
    assert torch.equal(z, z0) and torch.equal(y, y0)
    big[1:7, 8:72] = 7.0
    assert bool((big == 7.0).all())


def test_norm_in_place_and_empty_and_constant_rows():
    n = gen(9)
    x, h = n(40, 512, dt=BF16), n(40, 512, dt=BF16)
    z, y = block.norm_forward(x, h)
    x2 = x.clone()
    z2, y2 = block.norm_forward(x2, h, z=x2)
    assert z2 is x2 and torch.equal(x2, z) and torch.equal(y, y2)
    # no rows
    e = torch.empty(0, 64, device="cuda")
    w = torch.ones(64, device="cuda")
    z, y = block.norm_forward(e, e, weight=w)
    assert z.shape == (0, 64) and y.shape == (0, 64)
    g = block.norm_backward(e, e, e, e, weight=w, gate=torch.empty(0, 64, device="cuda"))
    assert g["dx"].shape == (0, 64) and bool((g["dweight"] == 0).all()) and g["dgate"].shape == (0, 64)
    # rows without variance: finite, and 0 after a layer norm
    c = torch.full((3, 1000), 4.0, device="cuda")
    assert bool((block.norm_forward(c)[1] == 0).all())
    g = block.norm_backward(c, None, None, torch.ones_like(c))
    assert bool(torch.isfinite(g["dx"]).all())
    assert bool((block.norm_forward(torch.zeros_like(c), norm="rms")[1] == 0).all())


def test_norm_of_one_channel_one_row_and_other_shapes():
    n = gen(13)
    # one channel: nothing is left of it after a layer norm but the shift
    x, b = n(5, 1), n(1)
    assert torch.equal(block.norm_forward(x, bias=b)[1], b.expand(5, 1))
    g = block.norm_backward(x, None, None, n(5, 1), bias=b)
    assert bool((g["dx"] == 0).all())
    # a vector alone, and rows of a view with leading dimensions that cannot be walked
    v = n(64)
    want = block.norm_forward(v.view(1, 64), norm="rms")[1]
    assert torch.equal(block.norm_forward(v, norm="rms")[1], want.view(64))
    w = n(4, 3, 5, 64, dt=BF16)
    for t in (w, w.transpose(0, 2), w[:, :, ::2], w.transpose(2, 3).contiguous().transpose(2, 3)):
        z, y = block.norm_forward(t, t, norm="rms")
        z0, y0 = block.norm_forward(t.contiguous().view(-1, 64), t.contiguous().view(-1, 64), norm="rms")
        assert z.shape == t.shape and torch.equal(z.reshape(-1, 64), z0) and torch.equal(y.reshape(-1, 64), y0)
        g = block.norm_backward(t, t, t, t, norm="rms")
        g0 = block.norm_backward(*(t.contiguous().view(-1, 64),) * 4, norm="rms")
        assert torch.equal(g["dx"].reshape(-1, 64), g0["dx"])


def test_offsets_past_32_bits():
    """More than 2^31 elements: the last rows' bits are those of a call on them alone."""
    R, C = 524289 + 37, 4096
    x = torch.empty(R, C, dtype=BF16, device="cuda")
    x.view(-1)[: 1 << 20].normal_()
    x[-100:].normal_()
    x[-200:-100].fill_(0)
    w = 1 + gen(14)(C, std=0.2)
    y = block.norm_forward(x, weight=w)[1]
    assert torch.equal(y[-50:], block.norm_forward(x[-50:].contiguous(), weight=w)[1])
    g = block.norm_backward(x, None, None, y, wants=(), weight=w)["dx"]
    assert torch.equal(g[-50:], block.norm_backward(x[-50:].contiguous(), None, None, y[-50:].contiguous(), wants=(),
                                                    weight=w)["dx"])
    del g
    ids = torch.arange(R, device="cuda").view(R, 1) % 3
    plan = block.expert_plan(ids, 3)
    xs = block.expert_dispatch(x, plan, out=y)                    # every row of it has a slot
    assert torch.equal(xs[plan.pos[-50:, 0].long()], x[-50:])
    out = block.expert_combine(xs, plan)
    assert torch.equal(out[-50:], x[-50:]) and torch.equal(out[:50], x[:50])
    del out, xs, y
    q = x[:262144 + 9].view(-1, 32, 128)[:524288 + 16]            # 2^31 + 2^16 elements
    grid, axes = (8, 32, 32), (22, 21, 21)
    table = block.rotation_table(grid, axes)
    qr = block.rotate_forward(q, None, table, grid=grid, axes=axes)[0]
    tail = q[-16:].contiguous()
    at = (torch.arange(q.shape[0] - 16, q.shape[0]) % 8192)
    full = torch.zeros(8192, 32, 128, dtype=BF16, device="cuda")
    full[at] = tail
    assert torch.equal(qr[-16:], block.rotate_forward(full, None, table, grid=grid, axes=axes)[0][at])


def test_norm_row_with_nan_stays_alone():
    n = gen(10)
    x = n(64, 256)
    y0 = block.norm_forward(x, norm="rms")[1]
    x[17, 3], x[40, 9] = float("nan"), float("inf")
    y1 = block.norm_forward(x, norm="rms")[1]
    ok = torch.ones(64, dtype=torch.bool, device="cuda")
    ok[17] = ok[40] = False
    assert torch.equal(y0[ok], y1[ok]) and bool(torch.isnan(y1[17]).all())


def test_norm_autograd_against_the_formula_and_differences():
    n = gen(11)
    B, N, C = 2, 6, 40
    x, h = n(B, N, C).requires_grad_(), n(B, N, C).requires_grad_()
    v = {k: n(B, C, std=0.5).requires_grad_() for k in ("gate", "scale", "shift")}
    v.update({k: (1 + n(C, std=0.2)).requires_grad_() for k in ("weight", "bias", "post_weight")})
    a, b = n(B, N, C), n(B, N, C)

    def loss():
        z, y = block.norm(x, h, norm="layer", post_norm="rms", eps=1e-4, **v)
        return (z * a).sum() + (y * b).sum()

    loss().backward()
    leaves = dict(v, x=x, h=h)
    l64 = {k: t.detach().double().requires_grad_() for k, t in leaves.items()}

    def loss64(l):
        z, y = bf.block_norm(l["x"].reshape(-1, C), l["h"].reshape(-1, C),
                             {k: l[k] for k in v}, "layer", "rms", 1e-4, 1.0, N)
        return (z * a.double().view(-1, C)).sum() + (y * b.double().view(-1, C)).sum()

    loss64(l64).backward()
    for k, t in leaves.items():
        # gradients of order one, of at most 12 x 40 terms: 1e-5 is 168 half steps
        assert torch.allclose(t.grad.double(), l64[k].grad, rtol=1e-5, atol=1e-4), k
        # a central difference in 64 bits along one direction: its error is of order step^2
        d = torch.randn_like(l64[k])
        up, dn = ({**l64, k: l64[k] + s * d} for s in (1e-4, -1e-4))
        diff = (loss64(up) - loss64(dn)).detach() / 2e-4
        assert abs(float(diff - (t.grad.double() * d).sum())) <= 1e-3 * (1 + float((t.grad.double() * d).abs().sum()))


def test_norm_autograd_parts():
    """Only y used, only z used, only some inputs with gradients; shared leaves add up."""
    n = gen(12)
    x, h, g = n(9, 32).requires_grad_(), n(9, 32), n(1, 32).requires_grad_()
    z, y = block.norm(x, h, gate=g, norm="rms")
    y.sum().backward()
    gx, gg = x.grad.clone(), g.grad.clone()
    x.grad = g.grad = None
    z, y = block.norm(x, h, gate=g, norm="rms")
    (2 * z.sum()).backward()
    assert torch.equal(x.grad, torch.full_like(x, 2.0))
    assert torch.allclose(g.grad, 2 * h.sum(0, keepdim=True), rtol=1e-5, atol=1e-5)
    assert gx.abs().sum() > 0 and gg.abs().sum() > 0
    # no branch: z is x, and y's gradient joins x's others
    x.grad = None
    z, y = block.norm(x, norm="rms")
    assert z is x
    (z.sum() + 0 * y.sum()).backward()
    assert torch.allclose(x.grad, torch.ones_like(x))
    # x and h one tensor
    x.grad = None
    z, _ = block.norm(x, x, norm="rms")
    z.sum().backward()
    assert torch.equal(x.grad, torch.full_like(x, 2.0))


# ------------------------------------------------------------------ rotation
ROT_CASES = [
    # tokens, grid, axes, heads q, heads k, d, type, pairs, norm
    (1, (1, 1, 1), (12, 10, 10), 1, 1, 64, F32, "interleaved", True),
    (117, (1, 9, 13), (12, 10, 10), 5, 5, 64, F32, "half", True),
    (117, (1, 9, 13), (22, 21, 21), 3, 1, 128, BF16, "interleaved", True),
    (200, (4, 5, 10), (22, 21, 21), 24, 24, 128, BF16, "half", True),
    (400, (4, 5, 10), (8, 8, 8), 7, 2, 64, BF16, "interleaved", True),     # two samples, pairs that do not turn
    (90, (2, 5, 9), (0, 32, 0), 33, 0, 64, BF16, "half", False),
    (90, (2, 5, 9), (0, 0, 0), 0, 4, 128, F32, "interleaved", False),
    (5000, (8, 25, 25), (22, 21, 21), 2, 3, 128, F32, "half", True),
    (333, (1, 9, 37), (10, 30, 20), 0, 3, 128, BF16, "interleaved", True),
    (3000, (2, 30, 50), (10, 11, 11), 0, 5, 64, F32, "half", True),
]


@pytest.mark.parametrize("N,grid,axes,hq,hk,d,dt,pairs,norm", ROT_CASES)
def test_rotate_forward_and_backward(N, grid, axes, hq, hk, d, dt, pairs, norm):
    n = gen(N + d)
    table = block.rotation_table(grid, axes)
    Q, Kt = (n(N, h, d, std=3.0, dt=dt) if h else None for h in (hq, hk))
    wq, wk = (1 + n(d, std=0.3) if norm and h else None for h in (hq, hk))
    kw = dict(grid=grid, axes=axes, norm=norm, eps=1e-6, pairs=pairs)
    got = block.rotate_forward(Q, Kt, table, q_weight=wq, k_weight=wk, **kw)
    dr = [None if t is None else n(*t.shape, dt=dt) for t in (Q, Kt)]
    g = block.rotate_backward(Q, Kt, *dr, table, q_weight=wq, k_weight=wk, **kw)
    cos, sin = bf.angles(table, grid, axes, N, d)
    for x, w, o, dro, dx, dw in ((Q, wq, got[0], dr[0], g["dQ"], g["dq_weight"]),
                                 (Kt, wk, got[1], dr[1], g["dK"], g["dk_weight"])):
        if x is None:
            assert o is None and dx is None
            continue
        x64 = bf.d64(x).requires_grad_()
        w64 = None if not norm else bf.d64(w).requires_grad_()
        want = bf.rotate(x64, w64, cos, sin, pairs, 1e-6)
        # a pair's terms: |n_a cos| + |n_b sin|
        nx = x64 if not norm else bf.normed(x64, "rms", 1e-6) * w64
        close(o, want.detach(), bf.rotate(nx.detach().abs(), None, cos.abs(), -sin.abs(), pairs, 0).abs()
              + bf.rotate(nx.detach().abs(), None, cos.abs(), sin.abs(), pairs, 0).abs())
        gs = torch.autograd.grad((want * bf.d64(dro)).sum(), [x64] + ([w64] if norm else []))
        a = bf.d64(dro).abs()
        t = (bf.rotate(a, None, cos.abs(), -sin.abs(), pairs, 0).abs()
             + bf.rotate(a, None, cos.abs(), sin.abs(), pairs, 0).abs())
        if not norm:
            close(dx, gs[0], t)
            continue
        r = 1 / torch.sqrt((x64 * x64).mean(-1, keepdim=True) + 1e-6).detach()
        nn = (x64.detach() * r).abs()
        tw = t * w64.detach().abs()
        close(dx, gs[0], r * (tw + nn * (tw * nn).mean(-1, keepdim=True)))
        close(dw, gs[1], (t * nn).sum((0, 1)), N * x.shape[1], what="dw")


def test_rotation_table_places():
    t = block.rotation_table((2, 3, 4), (1, 2, 1), base=100.0, positions=([0, 5], [1, 2, 3], [0, 0.5, 1, 1.5]))
    assert t.shape == (2 + 6 + 4, 2)
    want = torch.tensor([0, 5, 1, 0.1, 2, 0.2, 3, 0.3, 0, 0.5, 1, 1.5], dtype=torch.float64)
    assert torch.equal(t.cpu(), torch.stack((want.cos(), want.sin()), 1).float())


def test_rotate_of_a_fused_projection_in_place():
    """Q and K cut out of one [N, 3, heads, d] tensor, dense results and in place."""
    n = gen(21)
    grid, axes = (2, 4, 8), (22, 21, 21)
    qkv = n(64, 3, 4, 128, dt=BF16)
    table = block.rotation_table(grid, axes)
    w = 1 + n(128, std=0.2)
    kw = dict(grid=grid, axes=axes, q_weight=w, k_weight=w)
    a = block.rotate_forward(qkv[:, 0].contiguous(), qkv[:, 1].contiguous(), table, **kw)
    b = block.rotate_forward(qkv[:, 0], qkv[:, 1], table, **kw)
    v = qkv[:, 2].clone()
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    block.rotate_forward(qkv[:, 0], qkv[:, 1], table, out=(qkv[:, 0], qkv[:, 1]), **kw)
    assert torch.equal(qkv[:, 0], a[0]) and torch.equal(qkv[:, 1], a[1]) and torch.equal(qkv[:, 2], v)


def test_rotate_keeps_inner_products_of_places():
    """Turned by the angles' differences only: q(p) . k(p + s) is the same at every p along an axis."""
    grid, axes, d = (1, 1, 24), (0, 0, 32), 64
    n = gen(22)
    q, k = n(1, 1, d).expand(24, 1, d).contiguous(), n(1, 1, d).expand(24, 1, d).contiguous()
    table = block.rotation_table(grid, axes)
    qr, kr = block.rotate_forward(q, k, table, grid=grid, axes=axes, norm=False)
    s = (qr[:-5, 0] * kr[5:, 0]).sum(-1)
    # 64 products of sizes whose sum is about |q||k| ~ 64, each off by a few half steps
    assert float((s - s[0]).abs().max()) <= 64 * 64 * 4 * bf.U


def test_rotate_autograd_through_the_layer():
    """prism_attention(rotation=): bits of the calls it is made of, and their gradients."""
    cfg = get_config("720p", T=8, H=16, W=16, heads=2)
    x = inputs.make_inputs(cfg, "cuda")
    mod = PrismSparseAttention(cfg.T, cfg.H, cfg.W, cfg.heads, cfg.head_dim, cfg.audio_dim, cfg.dtype, cfg.top_k,
                               cfg.top_p)
    grid, axes = (cfg.T, cfg.H, cfg.W), (22, 21, 21)
    table = block.rotation_table(grid, axes)
    n = gen(23)
    w = (1 + n(128, std=0.2)).requires_grad_()          # one weight for Q and K: its gradients add up
    Q, Kt, V = (x[k].clone().requires_grad_() for k in ("Q", "K", "V"))
    O = prism_attention(Q, Kt, V, x["hhat"], mod, rotation=dict(table=table, axes=axes, q_weight=w, k_weight=w))
    O.backward(x["dO"])
    kw = dict(grid=grid, axes=axes, q_weight=w.detach(), k_weight=w.detach())
    Qr, Kr = block.rotate_forward(x["Q"], x["K"], table, **kw)
    O2 = mod.forward(Qr, Kr, x["V"], x["hhat"])
    assert torch.equal(O, O2)
    dQr, dKr, dV = mod.backward(x["dO"])
    g = block.rotate_backward(x["Q"], x["K"], dQr, dKr, table, **kw)
    assert torch.equal(Q.grad, g["dQ"]) and torch.equal(Kt.grad, g["dK"]) and torch.equal(V.grad, dV)
    assert torch.allclose(w.grad, g["dq_weight"] + g["dk_weight"], rtol=1e-6, atol=0)


# ------------------------------------------------------------------ experts
def routed(n, R, k, E, dropped, id_dt=torch.int64, even=False):
    if even:
        ids = (torch.arange(R * k, device="cuda") % E).view(R, k)
    else:
        ids = torch.topk(n(R, E) + n(E, std=1.0), k, 1).indices if k <= E else torch.randint(
            0, E, (R, k), device="cuda")
    if dropped:
        ids = torch.where(torch.rand(R, k, device="cuda") < dropped, torch.full_like(ids, -1), ids)
    return ids.to(id_dt)


EXPERT_CASES = [
    # rows, k, experts, channels, type, align, dropped, id type
    (1, 1, 1, 1, F32, 1, 0.0, torch.int64),
    (8, 4, 64, 256, BF16, 1, 0.0, torch.int64),
    (8, 4, 64, 257, BF16, 128, 0.5, torch.int32),
    (33, 16, 16, 100, F32, 3, 0.2, torch.int64),
    (700, 2, 1024, 64, BF16, 8, 0.0, torch.int32),
    (2049, 3, 7, 333, F32, 4, 0.2, torch.int64),
    (2731, 3, 5, 72, BF16, 16, 0.0, torch.int64),       # 8193 slots
    (8192, 1, 9, 40, BF16, 1, 0.0, torch.int64),
    (4096, 1, 300, 24, F32, 2, 0.0, torch.int32),       # as many slots as one CTA sorts
    (4097, 1, 300, 24, F32, 2, 0.1, torch.int32),
    (20000, 8, 128, 48, BF16, 128, 0.1, torch.int64),
    (31, 9, 12, 2048, F32, 1, 0.0, torch.int64),
    (77777, 2, 1000, 8, F32, 1, 0.0, torch.int32),
]


@pytest.mark.parametrize("R,k,E,C,dt,align,dropped,idt", EXPERT_CASES)
def test_experts_there_and_back(R, k, E, C, dt, align, dropped, idt):
    n = gen(R + C)
    ids = routed(n, R, k, E, dropped, idt)
    plan = block.expert_plan(ids, E, align=align)
    want = bf.experts(ids.cpu(), E, align, plan.rows_sorted)
    for got, w in zip((plan.counts, plan.offsets, plan.pos, plan.src), want):
        assert torch.equal(got.cpu(), w)
    pos, used = plan.pos.long(), int(want[1][-1])
    there = pos >= 0
    x, w = n(R, C, dt=dt), torch.rand(R, k, device="cuda")
    w = torch.where(there, w, torch.full_like(w, float("nan")))       # a dropped slot's weight is not read
    xs = block.expert_dispatch(x, plan)
    src = plan.src.long()
    assert torch.equal(xs, torch.where((src >= 0)[:, None], x[src.clamp(min=0) // k], torch.zeros((), dtype=dt,
                                                                                                  device="cuda")))
    # what no slot reads may hold anything
    ys = n(plan.rows_sorted, C, dt=dt)
    ys[src < 0] = float("nan")
    add = n(R, C, dt=dt)
    y64 = torch.where(there[..., None], bf.d64(ys)[pos.clamp(min=0)], 0.0)
    w64 = torch.where(there, bf.d64(w), 0.0)
    t = (y64 * w64[..., None])
    close(block.expert_combine(ys, plan, w), t.sum(1), t.abs().sum(1))
    close(block.expert_combine(ys, plan, w, add=add), t.sum(1) + bf.d64(add), t.abs().sum(1) + bf.d64(add).abs())
    close(block.expert_combine(ys, plan), y64.sum(1), y64.abs().sum(1))
    # gradients: a given output keeps the rows behind the last expert
    dout = n(R, C, dt=dt)
    out = torch.full((plan.rows_sorted, C), 5.0, dtype=dt, device="cuda")
    dys, dw = block.expert_combine_backward(dout, ys, plan, w, out=out)
    row_w = torch.where(src >= 0, bf.d64(w).reshape(-1)[src.clamp(min=0)], 0.0)
    dwant = bf.d64(dout)[src.clamp(min=0) // k] * row_w[:, None]
    close(dys[:used], dwant[:used], dwant[:used].abs())
    assert bool((dys[used:] == 5.0).all())
    p = y64 * bf.d64(dout)[:, None]
    close(dw, p.sum(-1), p.abs().sum(-1), C)
    d2, none = block.expert_combine_backward(dout, None, plan, w, want_weights=False)
    assert none is None and torch.equal(d2[:used], dys[:used]) and bool((d2[used:] == 0).all())
    # in place of ys
    dys3, _ = block.expert_combine_backward(dout, ys, plan, w, out=ys)
    assert torch.equal(dys3[:used], dys[:used])


def test_expert_plan_of_runs_longer_than_a_batch():
    """More slots than 148 CTAs take at eight a thread: 1.3 million and odd."""
    R, k, E = 650011, 2, 40
    ids = torch.randint(-1, E, (R, k), device="cuda", generator=torch.Generator("cuda").manual_seed(5))
    plan = block.expert_plan(ids, E, align=8)
    flat = ids.view(-1)
    key = torch.where(flat < 0, torch.full_like(flat, E), flat)
    order = torch.sort(key, stable=True).indices
    counts = torch.bincount(key, minlength=E + 1)[:E]
    assert torch.equal(plan.counts.long(), counts)
    offsets = torch.cumsum((counts + 7) // 8 * 8, 0)
    assert torch.equal(plan.offsets[1:].long(), offsets) and int(plan.offsets[0]) == 0
    used = plan.src[plan.src >= 0].long()
    assert torch.equal(used, order[:int(counts.sum())])           # stable, expert by expert
    there = plan.pos.view(-1) >= 0
    assert torch.equal(there, flat >= 0)
    slots = torch.nonzero(there).view(-1)
    assert torch.equal(plan.src[plan.pos.view(-1)[slots].long()].long(), slots)
    assert int((plan.src >= 0).sum()) == int(counts.sum())


@pytest.mark.parametrize("align", [1, 16])
def test_experts_empty_and_one_sided(align):
    # no rows
    plan = block.expert_plan(torch.empty(0, 2, dtype=torch.int64, device="cuda"), 5, align=align)
    assert plan.counts.tolist() == [0] * 5 and plan.offsets.tolist() == [0] * 6
    x = torch.empty(0, 8, device="cuda")
    assert block.expert_dispatch(x, plan).shape == (0, 8) and block.expert_combine(x, plan).shape == (0, 8)
    # every slot dropped, by ids on either side of the range and past 32 bits
    ids = torch.tensor([[-1, 5], [1 << 40, -(1 << 40)]], device="cuda")
    plan = block.expert_plan(ids, 5, align=align)
    assert plan.offsets.tolist() == [0] * 6 and plan.pos.tolist() == [[-1, -1]] * 2
    x = torch.ones(2, 8, device="cuda")
    assert bool((block.expert_dispatch(x, plan) == 0).all())
    assert bool((block.expert_combine(torch.full((plan.rows_sorted, 8), float("nan"), device="cuda"), plan) == 0).all())
    # all to one expert, one token twice to it
    ids = torch.full((300, 2), 3, device="cuda")
    plan = block.expert_plan(ids, 5, align=align)
    assert plan.counts.tolist() == [0, 0, 0, 600, 0]
    assert torch.equal(plan.pos.cpu().view(-1), torch.arange(600, dtype=torch.int32))
    x = gen(1)(300, 24)
    assert torch.equal(block.expert_combine(block.expert_dispatch(x, plan), plan), 2 * x)


def test_experts_strided_and_unaligned_rows():
    n = gen(31)
    ids = routed(n, 50, 2, 6, 0.1)
    plan = block.expert_plan(ids, 6, align=8)
    wide = n(50, 75, dt=BF16)
    for x in (wide[:, :64], wide[:, 1:65], wide[:, 3:36], wide[::2, 8:72].repeat_interleave(2, 0)):
        assert torch.equal(block.expert_dispatch(x, plan), block.expert_dispatch(x.contiguous(), plan))
    ys, add = n(plan.rows_sorted, 64, dt=BF16), wide[:, 5:69]
    assert torch.equal(block.expert_combine(ys, plan, add=add), block.expert_combine(ys, plan, add=add.contiguous()))
    out = torch.full((50, 66), 9.0, dtype=BF16, device="cuda")
    o = block.expert_combine(ys, plan, out=out[:, 1:65])
    assert torch.equal(o, block.expert_combine(ys, plan)) and bool((out[:, 0] == 9).all() and (out[:, 65] == 9).all())


def test_experts_autograd():
    n = gen(32)
    R, k, E, C = 60, 3, 4, 20
    ids = routed(n, R, k, E, 0.2)
    plan = block.expert_plan(ids, E, align=4)
    x, w, add = (t.requires_grad_() for t in (n(R, C), torch.rand(R, k, device="cuda"), n(R, C)))
    wE = n(E, C, C).requires_grad_()
    a = n(R, C)

    def experts(xs, wE):
        off = plan.offsets.tolist()
        return torch.cat([xs[off[e]:off[e + 1]] @ wE[e] for e in range(E)] + [xs[off[E]:]])

    out = block.combine(experts(block.dispatch(x, plan), wE), plan, w, add=add)
    (out * a).sum().backward()
    l = [t.detach().double().requires_grad_() for t in (x, w, add, wE)]
    t = torch.einsum("rc,rkcd->rkd", l[0], l[3][ids.clamp(min=0)]) * l[1][..., None]
    o64 = torch.where((ids >= 0)[..., None], t, 0.0).sum(1) + l[2]
    (o64 * a.double()).sum().backward()
    for got, want in zip((x, w, add, wE), l):
        # sums of up to 60 products of order one beside the library's float32 products
        assert torch.allclose(got.grad.double(), want.grad, rtol=1e-4, atol=1e-4)


# ------------------------------------------------------------------ together
def test_block_run_forward_and_backward():
    """Norm, projections, rotation, attention, gate and next norm, experts and the last gate, as a block runs them,
    with all gradients, against 64 bits (every block selected, so that the attention is the dense one)."""
    T, H, W, heads, d = 8, 8, 8, 2, 64
    N, C, E, k = T * H * W, 96, 4, 2
    n = gen(41)
    mod = PrismSparseAttention(T, H, W, heads, d, 16, "f32", top_k=8, top_p=1.0)
    grid, axes = (T, H, W), (12, 10, 10)
    table = block.rotation_table(grid, axes)
    hhat = n(N, 16)
    P = {"x": n(N, C), "mod": n(1, 6 * C, std=0.2), "qkv": n(C, 3 * heads * d, std=C ** -0.5), "wq": 1 + n(d, std=0.1),
         "wk": 1 + n(d, std=0.1), "o": n(heads * d, C, std=(heads * d) ** -0.5), "router": n(C, E, std=0.2),
         "w1": n(E, C, C, std=C ** -0.5)}
    a = n(N, C)
    ids = []

    def run(p, own):
        m = [p["mod"][:, i * C:(i + 1) * C] for i in range(6)]
        if own:
            z, y = block.norm(p["x"], scale=m[0], shift=m[1])
        else:
            z, y = bf.block_norm(p["x"], None, dict(none, scale=m[0], shift=m[1]), "layer", None, 1e-6, 1.0, N)
        Q, Kt, V = (y @ p["qkv"]).view(N, 3, heads, d).unbind(1)
        if own:
            O = prism_attention(Q, Kt, V, hhat, mod, rotation=dict(table=table, axes=axes, q_weight=p["wq"],
                                                                   k_weight=p["wk"]))
        else:
            cos, sin = bf.angles(table, grid, axes, N, d)
            q, kk = (bf.rotate(t, w, cos, sin, "interleaved", 1e-6) for t, w in ((Q, p["wq"]), (Kt, p["wk"])))
            O = torch.einsum("hqk,khd->qhd", torch.softmax(torch.einsum("qhd,khd->hqk", q, kk) / d ** 0.5, -1), V)
        o = O.reshape(N, heads * d) @ p["o"]
        if own:
            z, y = block.norm(z, o, gate=m[2], scale=m[3], shift=m[4], post_norm="rms")
        else:
            z, y = bf.block_norm(z, o, dict(none, gate=m[2], scale=m[3], shift=m[4]), "layer", "rms", 1e-6, 1.0, N)
        logits = y @ p["router"]
        if own:
            ids.append(torch.topk(logits, k, 1).indices)
        w = torch.softmax(logits.gather(1, ids[0]), 1)
        if own:
            plan = block.expert_plan(ids[0], E, align=8)
            xs, off = block.dispatch(y, plan), plan.offsets.tolist()
            ys = torch.cat([torch.tanh(xs[off[e]:off[e + 1]] @ p["w1"][e]) for e in range(E)] + [xs[off[E]:]])
            f = block.combine(ys, plan, w)
            return block.norm(z, f, gate=m[5], norm=None)[0]
        f = (torch.tanh(torch.einsum("rc,rkcd->rkd", y, p["w1"][ids[0]])) * w[..., None]).sum(1)
        return bf.block_norm(z, f, dict(none, gate=m[5]), None, None, 1e-6, 1.0, N)[0]

    none = dict.fromkeys(("gate", "post_weight", "weight", "bias", "scale", "shift"))
    torch.backends.cuda.matmul.allow_tf32 = False
    p32 = {k_: v.clone().requires_grad_() for k_, v in P.items()}
    p64 = {k_: v.double().requires_grad_() for k_, v in P.items()}
    o32 = run(p32, True)
    o64 = run(p64, False)
    o32.backward(a)
    o64.backward(a.double())
    # a chain of about ten float32 steps, each within some hundred half steps relative to its norm: 10 x 100 x 2^-24
    tol = 6e-5
    rel = lambda g, r: float((g.double() - r).norm() / r.norm())
    assert rel(o32.detach(), o64.detach()) <= tol
    for k_ in P:
        assert rel(p32[k_].grad, p64[k_].grad) <= tol, (k_, rel(p32[k_].grad, p64[k_].grad))


def _everything(n):
    """Explicit calls of every operator on fixed inputs; returns a function that runs them all."""
    x, h, dz, dy = (n(300, 192, dt=BF16) for _ in range(4))
    gate, w = n(3, 192), 1 + n(192, std=0.1)
    Q, Kt, dQ, dK = (n(64, 3, 64, dt=BF16) for _ in range(4))
    grid, axes = (2, 4, 8), (12, 10, 10)
    table = block.rotation_table(grid, axes)
    wq = 1 + n(64, std=0.1)
    ids = routed(n, 3000, 4, 8, 0.1)
    t, wt = n(3000, 64), torch.rand(3000, 4, device="cuda")

    def run():
        kw = dict(gate=gate, weight=w, rows_per_group=100, norm="rms")
        z, y = block.norm_forward(x, h, **kw)
        g = block.norm_backward(z, h, dz, dy, **kw)
        r = block.rotate_forward(Q, Kt, table, grid=grid, axes=axes, q_weight=wq, k_weight=wq)
        rg = block.rotate_backward(Q, Kt, dQ, dK, table, grid=grid, axes=axes, q_weight=wq, k_weight=wq)
        plan = block.expert_plan(ids, 8, align=16)
        xs = block.expert_dispatch(t, plan)
        o = block.expert_combine(xs, plan, wt)
        dys, dw = block.expert_combine_backward(t, xs, plan, wt)
        return [z, y, *r, plan.counts, plan.offsets, plan.pos, plan.src, xs, o, dys, dw,
                *(v for d_ in (g, rg) for v in d_.values() if v is not None)]

    return run, (x, t, Q)


def test_same_bits_again_on_another_stream_and_in_two_graphs():
    run, ins = _everything(gen(51))
    want = run()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        got = run()
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = run()
        graphs.append((g, out))
    s2 = torch.cuda.Stream()
    for _ in range(3):
        for t in graphs[0][1] + graphs[1][1]:
            t.zero_()
        torch.cuda.synchronize()
        with torch.cuda.stream(s):
            graphs[0][0].replay()
        with torch.cuda.stream(s2):
            graphs[1][0].replay()
        torch.cuda.synchronize()
        for _, out in graphs:
            assert all(torch.equal(a, b) for a, b in zip(want, out))
    # new values in the same inputs are seen by a replay
    for t in ins:
        t.mul_(1.5)
    want = run()
    graphs[0][0].replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, graphs[0][1]))


def test_differentiable_forms_refuse_capture():
    n = gen(52)
    x = n(16, 64).requires_grad_()
    ids = routed(n, 16, 2, 4, 0.0)
    plan = block.expert_plan(ids, 4)
    table = block.rotation_table((1, 4, 4), (12, 10, 10))
    q = n(16, 2, 64).requires_grad_()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        g = torch.cuda.CUDAGraph()
        g.capture_begin()
        try:
            for f in (lambda: block.norm(x), lambda: block.dispatch(x, plan),
                      lambda: block.rotate(q, q.detach(), table, grid=(1, 4, 4), axes=(12, 10, 10))):
                with pytest.raises(RuntimeError, match="captured"):
                    f()
            with torch.no_grad():
                y = block.norm(x)[1]
        finally:
            g.capture_end()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, block.norm_forward(x.detach())[1])


def test_a_captured_backward_of_an_eager_graph_is_refused():
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        x = gen(54)(16, 64).requires_grad_()
        y = block.norm(x, norm="rms")[1]
        one = torch.ones_like(y)
        s.synchronize()
        g = torch.cuda.CUDAGraph()
        g.capture_begin()
        try:
            with pytest.raises(RuntimeError, match="captured"):
                y.backward(one)
        finally:
            g.capture_end()
    torch.cuda.synchronize()
    assert x.grad is None


def test_calls_from_two_threads():
    """Two threads, a stream each, calls of many signatures for the first time."""
    import threading
    n = gen(55)
    cases = [(n(r, c), n(r, c), n(r, c)) for r in (3, 17, 64) for c in (32, 100, 513, 2048)]
    want = [(block.norm_forward(x, h, norm="rms", eps=2e-6), block.norm_backward(x, h, x, dy, norm="rms", eps=2e-6))
            for x, h, dy in cases]
    torch.cuda.synchronize()
    block._plans.clear()
    bad, streams = [], [torch.cuda.Stream() for _ in range(2)]

    def work(i):
        try:
            with torch.cuda.stream(streams[i]):
                for _ in range(20):
                    for (x, h, dy), (f, g) in zip(cases, want):
                        z, y = block.norm_forward(x, h, norm="rms", eps=2e-6)
                        b = block.norm_backward(x, h, x, dy, norm="rms", eps=2e-6)
                        if not (torch.equal(z, f[0]) and torch.equal(y, f[1]) and torch.equal(b["dh"], g["dh"])):
                            bad.append(tuple(x.shape))
        except Exception as e:                  # to be seen by the test, not lost with the thread
            bad.append(e)
    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad


def test_results_in_place_of_inputs_through_the_library():
    """The overlaps that include/prism.h allows give the bits of separate outputs."""
    n = gen(56)
    L = _abi.lib()
    st = torch.cuda.current_stream().cuda_stream
    for R, C in ((70, 2048), (70, 96), (40, 5120)):
        for norm in ("layer", "rms"):
            z, h, dz, dy = (n(R, C, dt=BF16) for _ in range(4))
            g = block.norm_backward(z, h, dz, dy, norm=norm, post_norm="rms")
            d = _abi.BlockNormT(R, R, C, 1, 1, {"rms": 1, "layer": 2}[norm], 1, 1e-6, 1.0)
            assert L.prism_block_norm_bwd(ctypes.addressof(d), z.data_ptr(), h.data_ptr(), None, None, None, None, None,
                                          dz.data_ptr(), dy.data_ptr(), dz.data_ptr(), h.data_ptr(), None, None, None,
                                          None, None, None, None, 0, st) == 0
            assert torch.equal(dz, g["dx"]) and torch.equal(h, g["dh"])
    grid, axes = (1, 8, 8), (10, 11, 11)
    table = block.rotation_table(grid, axes)
    for dt, pairs in ((BF16, 0), (BF16, 1), (F32, 0)):
        Q, dr, w = n(64, 3, 64, dt=dt), n(64, 3, 64, dt=dt), 1 + n(64, std=0.2)
        g = block.rotate_backward(Q, None, dr, None, table, grid=grid, axes=axes, q_weight=w,
                                  pairs=("interleaved", "half")[pairs])
        d = _abi.RotateT(64, *grid, 3, 0, 64, *axes, pairs, int(dt == BF16), 1, 1e-6)
        ws = torch.empty(_abi.head_rotate_ws_bytes(d), dtype=torch.uint8, device="cuda")
        dw = torch.empty(64, device="cuda")
        assert L.prism_head_rotate_bwd(ctypes.addressof(d), Q.data_ptr(), None, w.data_ptr(), None, table.data_ptr(),
                                       dr.data_ptr(), None, dr.data_ptr(), None, dw.data_ptr(), None, ws.data_ptr(),
                                       ws.numel(), st) == 0
        assert torch.equal(dr, g["dQ"]) and torch.equal(dw, g["dq_weight"])
    ids = routed(n, 50, 2, 6, 0.1)
    plan = block.expert_plan(ids, 6)
    ys, add = n(plan.rows_sorted, 40), n(50, 40)
    want = block.expert_combine(ys, plan, add=add)
    assert block.expert_combine(ys, plan, add=add, out=add) is add and torch.equal(add, want)


def test_launches_are_counted():
    n = gen(53)
    x = n(4, 64)
    n0 = _abi.launch_count()
    block.norm_forward(x)
    assert _abi.launch_count() == n0 + 1

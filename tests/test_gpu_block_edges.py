"""The operators around the attention on the GPU, where a fault would be lost among roundings or needs two callers:
column sums of whole numbers, which show a single lost or doubled row; both sides of the plan's switch between one CTA
and several; threads in one kernel with rows of different widths; infinities beside pairs that do not turn."""
import ctypes
import threading

import pytest
import torch

import block_forms as bf
from dynamic_block_sparse_macro_b200 import _abi, block

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def signs(g, *shape, balanced=False):
    """-1 and 1 at random; `balanced`: as many of either in a row."""
    if balanced:
        return (torch.rand(*shape, generator=g, device="cuda").argsort(-1) % 2).float() * 2 - 1
    return torch.randint(0, 2, shape, generator=g, device="cuda").float() * 2 - 1


# ------------------------------------------------------------------ sums of whole numbers
# Rows of -1 and 1 have the mean square 1, and the norm leaves them as they are but for the roundings of the mean square
# (two half steps), of its reciprocal root (CUDA's bound: two units, four half steps) and of the product: seven half
# steps.  With gradients of -1 and 1 the column sums of dy and of dz ∘ h are whole numbers below 2^24, exact in any
# order, and those of dy ∘ N(z) and dz ∘ N(h) are off whole ones by at most R (7 + n) 2^-24, n the additions that a value
# passes: rows a team, teams a CTA, segments and groups over 16 warps, these, and up to 8 CTAs.  n is at most 60 where
# R is 40000, 64 at 20000 and 110 at 10007 and below: 0.16.  A lost or doubled row moves a sum by 1.
SUM_CASES = [
    # rows, channels, rows a group, stream, branch: the lengths at which groups are cut, run together and joined
    (1, 64, 1, F32, F32),
    (4999, 1100, 4999, F32, F32),
    (6001, 320, 6001, BF16, BF16),
    (6000, 320, 2999, F32, BF16),
    (10007, 64, 1, F32, F32),
    (20000, 40, 700, F32, F32),
    (19999, 40, 700, BF16, BF16),
    (40000, 96, 40000, BF16, BF16),
    (39999, 96, 13333, BF16, BF16),
    (5000, 520, 1000, BF16, BF16),
    (2111, 264, 700, BF16, BF16),
    (1203, 2048, 2, BF16, BF16),
    (4097, 2048, 4097, F32, BF16),
    (997, 4096, 997, BF16, BF16),
    (1500, 3000, 499, F32, BF16),
    (901, 1001, 1, BF16, BF16),
    (1371, 1001, 97, F32, F32),
    (611, 6000, 611, F32, F32),
    (333, 8192, 100, BF16, BF16),
]


def group_sums(v, rpg):
    R, C = v.shape
    G = -(-R // rpg)
    return v.new_zeros(G, C).index_add_(0, torch.arange(R, device="cuda") // rpg, v)


@pytest.mark.parametrize("R,C,rpg,sdt,bdt", SUM_CASES)
@pytest.mark.parametrize("norm", ["layer", "rms"])
@pytest.mark.parametrize("form", ["none", "plain", "normed"])
def test_column_sums_hold_every_row_once(R, C, rpg, sdt, bdt, norm, form):
    g = gen(R + C)
    if norm == "layer" and C % 2:
        pytest.skip("a row of odd width has no mean of 0")
    z, dy, dz, h = (signs(g, R, C, balanced=i == 0) for i in range(4))
    G = -(-R // rpg)
    near = lambda got, want: bool(((got.double() - want).abs() <= 0.25).all())
    kw = dict(norm=norm, eps=1e-9, rows_per_group=rpg)
    D, A = group_sums(dy.double(), rpg), group_sums((dy * z).double(), rpg)
    if form == "none":
        # weight 1: dscale is A; all the vectors' gradients of the groups, then only those of all rows
        one, zero = torch.ones(C, device="cuda"), torch.zeros(G, C, device="cuda")
        b = block.norm_backward(z.to(sdt), None, dz.to(sdt), dy.to(bdt), weight=one, bias=one, scale=zero, **kw)
        assert torch.equal(b["dshift"].double(), D) and near(b["dscale"], A + D)
        assert torch.equal(b["dbias"].double(), D.sum(0)) and near(b["dweight"], A.sum(0))
        b = block.norm_backward(z.to(sdt), None, None, dy.to(bdt), weight=one, bias=one, **kw)
        assert torch.equal(b["dbias"].double(), D.sum(0)) and near(b["dweight"], A.sum(0))
        return
    # weight 0: nothing of y reaches dz', which stays dz; gates of 1 and 2
    w = torch.zeros(C, device="cuda")
    gate = 1.0 + torch.randint(0, 2, (G, C), generator=g, device="cuda")
    B = group_sums((dz * h).double(), rpg)
    post = dict(post_norm="rms", post_weight=torch.ones(C, device="cuda")) if form == "normed" else {}
    b = block.norm_backward(z.to(sdt), h.to(bdt), dz.to(sdt), dy.to(bdt), weight=w, bias=w, gate=gate,
                            scale=torch.zeros(G, C, device="cuda"), **kw, **post)
    assert torch.equal(b["dshift"].double(), D) and torch.equal(b["dbias"].double(), D.sum(0))
    assert near(b["dweight"], A.sum(0)) and near(b["dgate"], B)
    if form == "normed":
        # a row counts once or twice by its gate, and so does the bound
        assert bool(((b["dpost_weight"].double() - (gate.double() * B).sum(0)).abs() <= 0.5).all())
    else:
        assert torch.equal(b["dgate"].double(), B)


# Quarter turns: cosines and sines of 0, 1 and -1, whole numbers again.  The bound is as above with R = tokens x heads; n
# counts a group of lanes' heads, the 16 or 32 groups of a CTA, the CTAs over 16 warps and these.  It is largest for
# 12345 x 3 heads: 4 + 32 + 28 + 16 = 80, 0.19.
@pytest.mark.parametrize("N,grid,hq,hk,d,dt,pairs", [
    (5000, (8, 25, 25), 2, 3, 128, F32, "half"), (5001, (8, 25, 25), 3, 2, 128, BF16, "interleaved"),
    (2999, (2, 30, 50), 0, 5, 64, F32, "half"), (117, (1, 9, 13), 5, 1, 64, BF16, "half"),
    (12345, (5, 47, 53), 3, 0, 64, BF16, "interleaved"), (1, (1, 1, 1), 1, 1, 64, F32, "interleaved")])
def test_rotation_weight_sums_hold_every_head_once(N, grid, hq, hk, d, dt, pairs):
    g = gen(N)
    axes = (d // 8, d // 8, d // 8)                 # a quarter of the pairs does not turn
    rows = sum(n * p for n, p in zip(grid, axes))
    turn = torch.randint(0, 4, (rows,), generator=g, device="cuda")
    table = torch.tensor([[1, 0], [0, 1], [-1, 0], [0, -1]], dtype=F32, device="cuda")[turn]
    x = [signs(g, N, h, d) if h else None for h in (hq, hk)]
    dr = [signs(g, N, h, d) if h else None for h in (hq, hk)]
    w = [torch.ones(d, device="cuda") if h else None for h in (hq, hk)]
    to = lambda t: None if t is None else t.to(dt)
    got = block.rotate_backward(*map(to, x), *map(to, dr), table, grid=grid, axes=axes, q_weight=w[0], k_weight=w[1],
                                eps=1e-9, pairs=pairs)
    cos, sin = bf.angles(table, grid, axes, N, d)
    for a, b, name in ((x[0], dr[0], "dq_weight"), (x[1], dr[1], "dk_weight")):
        if a is not None:
            want = (bf.rotate(b.double(), None, cos, -sin, pairs, 0) * a.double()).sum((0, 1))
            assert bool(((got[name].double() - want).abs() <= 0.25).all()), name


def test_groups_without_rows():
    """Samples of no tokens on the GPU: gradients of the vectors are 0, those of all rows' vectors too."""
    x = torch.empty(3, 0, 64, device="cuda", requires_grad=True)
    v = {k: torch.ones(3, 64, device="cuda", requires_grad=True) for k in ("gate", "scale", "shift")}
    w = torch.ones(64, device="cuda", requires_grad=True)
    z, y = block.norm(x, torch.empty(3, 0, 64, device="cuda"), weight=w, **v)
    (z.sum() + y.sum()).backward()
    assert x.grad.shape == x.shape and all(torch.equal(t.grad, torch.zeros_like(t)) for t in (w, *v.values()))


# ------------------------------------------------------------------ expert plan
@pytest.mark.parametrize("R,k", [(2047, 1), (2048, 1), (2049, 1), (1024, 2), (683, 3), (128, 16), (129, 16), (1025, 2)])
@pytest.mark.parametrize("E,align,dropped", [(7, 1, 0.0), (300, 8, 0.1), (1024, 3, 0.0)])
def test_expert_plan_where_one_cta_ends(R, k, E, align, dropped):
    """2048 slots are sorted by one CTA, 2049 by two launches, whose third CTA has a single slot."""
    g = gen(R * k + E)
    ids = torch.randint(0, E, (R, k), generator=g, device="cuda")
    ids[torch.rand(R, k, generator=g, device="cuda") < dropped] = -1
    plan = block.expert_plan(ids, E, align=align)
    want = bf.experts(ids.cpu(), E, align, plan.rows_sorted)
    for got, w in zip((plan.counts, plan.offsets, plan.pos, plan.src), want):
        assert torch.equal(got.cpu(), w)
    x = torch.randn(R, 24, generator=g, device="cuda")
    src = plan.src.long()
    xs = block.expert_dispatch(x, plan)
    assert torch.equal(xs, torch.where((src >= 0)[:, None], x[src.clamp(min=0) // k], torch.zeros((), device="cuda")))


# ------------------------------------------------------------------ two callers
@pytest.mark.parametrize("widths", [(2048, 1024, 1536), (4096, 3200, 4096)])
def test_threads_in_one_kernel_with_rows_of_other_widths(widths):
    """Widths that share a kernel but not the size of its shared memory, straight into the library, so that the threads
    are in it together: every call is accepted, and gives the bits that it gives alone."""
    g = gen(7)
    L = _abi.lib()
    calls = []
    for C in widths:
        z, h, dz, dy = (torch.randn(2, C, generator=g, device="cuda") for _ in range(4))
        d = _abi.BlockNormT(2, 2, C, 0, 0, 2, 0, 1e-6, 1.0)
        outs = [torch.empty_like(z) for _ in range(4)]
        want = [*block.norm_forward(z, h), *(block.norm_backward(z, h, dz, dy)[k] for k in ("dx", "dh"))]
        calls.append((d, z, h, dz, dy, outs, want))
    torch.cuda.synchronize()
    codes, go = [set() for _ in widths], threading.Barrier(len(widths))
    streams = [torch.cuda.Stream() for _ in widths]

    def work(i):
        d, z, h, dz, dy, outs, _ = calls[i]
        a, st, p = ctypes.addressof(d), streams[i].cuda_stream, [t.data_ptr() for t in (z, h, dz, dy, *outs)]
        fwd = (a, p[0], p[1], None, None, None, None, None, None, p[4], p[5], st)
        bwd = (a, p[0], p[1], None, None, None, None, None, p[2], p[3], p[6], p[7], None, None, None, None, None, None,
               None, 0, st)
        go.wait(60)
        for _ in range(20000):
            codes[i].add(L.prism_block_norm_fwd(*fwd))
            codes[i].add(L.prism_block_norm_bwd(*bwd))
    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(widths))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert codes == [{0}] * len(widths)
    for _, _, _, _, _, outs, want in calls:
        assert all(torch.equal(a, b) for a, b in zip(outs, want))


# ------------------------------------------------------------------ rotation
@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("pairs", ["interleaved", "half"])
@pytest.mark.parametrize("d,axes", [(64, (8, 8, 7)), (64, (0, 0, 0)), (128, (20, 20, 20)), (128, (0, 5, 0))])
def test_a_pair_that_does_not_turn_is_left_alone(d, axes, pairs, dt):
    """An infinity or NaN in one member of such a pair does not reach the other: without a norm the channels of these
    pairs are copied, forwards and backwards."""
    g = gen(d)
    N, grid, n = 24, (2, 3, 4), sum(axes)
    table = block.rotation_table(grid, axes)
    x = torch.randn(N, 5, d, generator=g, device="cuda").to(dt)
    ch = torch.arange(d, device="cuda")
    pair = ch // 2 if pairs == "interleaved" else ch % (d // 2)
    second = ch % 2 == 1 if pairs == "interleaved" else ch >= d // 2
    still = pair >= n
    y = x.clone()
    y[0:8, :, still & second] = float("inf")
    y[8:16, :, still & ~second] = float("-inf")
    y[16:24, :, still & second] = float("nan")
    kw = dict(grid=grid, axes=axes, norm=False, pairs=pairs)
    same = lambda a, b: torch.equal(a.nan_to_num(7.0, 8.0, 9.0), b.nan_to_num(7.0, 8.0, 9.0))
    for call in (lambda t: block.rotate_forward(t, None, table, **kw)[0],
                 lambda t: block.rotate_backward(None, None, t, None, table, **kw)["dQ"]):
        a, b = call(x), call(y)
        assert torch.equal(a[..., still], x[..., still])
        assert same(b[..., still], y[..., still]) and torch.equal(b[..., ~still], a[..., ~still])
    # with the norm an infinity makes the row's root mean square infinite: it becomes NaN and all else 0
    y = x.clone()
    y[:, :, still & second] = float("inf")
    out = block.rotate_forward(y, None, table, grid=grid, axes=axes, pairs=pairs)[0]
    assert bool((out[..., still & ~second] == 0).all()) and bool(out[..., still & second].isnan().all())
    assert bool((out[..., ~still] == 0).all())
    # nor does an infinite weight
    w = torch.ones(d, device="cuda")
    w[still & second] = float("inf")
    out = block.rotate_forward(x, None, table, grid=grid, axes=axes, pairs=pairs, q_weight=w)[0]
    assert torch.equal(out[..., still & ~second], block.rotate_forward(x, None, table, grid=grid, axes=axes,
                                                                       pairs=pairs)[0][..., still & ~second])


@pytest.mark.parametrize("pairs", ["interleaved", "half"])
def test_rotation_backward_of_rows_of_zeros_with_the_smallest_eps(pairs):
    """dx = r c for rows of zeros, r = eps^-1/2 up to 10^21: r is squared only with what makes it small again."""
    g = gen(77)
    grid, axes, eps = (1, 4, 4), (10, 11, 11), 1e-42
    table = block.rotation_table(grid, axes)
    x, dr = torch.zeros(16, 2, 64, device="cuda"), torch.randn(16, 2, 64, generator=g, device="cuda") * 1e-10
    got = block.rotate_backward(x, None, dr, None, table, grid=grid, axes=axes, eps=eps, pairs=pairs)["dQ"]
    cos, sin = bf.angles(table, grid, axes, 16, 64)
    r = torch.tensor(eps, dtype=F32).double().item() ** -0.5
    want = bf.rotate(dr.double(), None, cos, -sin, pairs, 0) * r
    terms = dr.double().abs().amax() * 2 * r
    # two products and a sum, the reciprocal root (four half steps), a product with it and one with the weight: 9
    assert bool(((got.double() - want).abs() <= 9 * bf.U * terms).all())


def test_rotation_table_of_places_on_the_gpu():
    places = [torch.tensor(p) for p in ([0.0, 5.0], [1.0, 2.0, 3.0], [0.0, 0.5])]
    kw = dict(grid=(2, 3, 2), axes=(2, 1, 3))
    assert torch.equal(block.rotation_table(positions=[p.cuda() for p in places], **kw),
                       block.rotation_table(positions=places, **kw))

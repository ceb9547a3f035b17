"""The operators around the attention on the GPU, where a fault would be lost among roundings or needs two callers."""
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


def test_groups_without_rows():
    """Samples of no tokens on the GPU: gradients of the vectors are 0, those of all rows' vectors too."""
    x = torch.empty(3, 0, 64, device="cuda", requires_grad=True)
    v = {k: torch.ones(3, 64, device="cuda", requires_grad=True) for k in ("gate", "scale", "shift")}
    w = torch.ones(64, device="cuda", requires_grad=True)
    z, y = block.norm(x, torch.empty(3, 0, 64, device="cuda"), weight=w, **v)
    (z.sum() + y.sum()).backward()
    assert x.grad.shape == x.shape and all(torch.equal(t.grad, torch.zeros_like(t)) for t in (w, *v.values()))


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

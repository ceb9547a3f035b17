"""Calls of the operators around the attention that have to be refused or prepared alike whatever came before them,
in the library and in the tensor calls: nothing here launches."""
import ctypes

import pytest
import torch
from torch.autograd import forward_ad

from dynamic_block_sparse_macro_b200 import _abi, block

OK, ARG, SHAPE, UNSUP = 0, 1, 2, 3
P = 1 << 40                                   # aligned, never dereferenced on the host


@pytest.fixture(scope="module")
def L():
    from dynamic_block_sparse_macro_b200 import build
    build.build()
    return _abi.lib()


def test_leaves_off_the_gpu_are_refused_as_other_tensors_are():
    x, q = torch.zeros(4, 8, requires_grad=True), torch.zeros(4, 2, 64, requires_grad=True)
    for f in (lambda: block.norm(x), lambda: block.norm(x.detach(), x),
              lambda: block.rotate(q, None, torch.zeros(1, 2), grid=(1, 1, 1), axes=(1, 0, 0))):
        with pytest.raises(ValueError, match="CUDA"):
            f()


@pytest.fixture
def host(monkeypatch):
    """The tensor calls on CPU tensors, up to the library: the device check is passed over, and a call that gets
    through every check raises ``Through``."""
    class Through(Exception):
        pass

    def through(index):
        raise Through
    monkeypatch.setattr(block, "_same_device", lambda dev, *t: None)
    monkeypatch.setattr(block, "_stream", through)
    monkeypatch.setattr(block, "_current", lambda index: True)
    monkeypatch.setattr(block, "_plans", {})
    return Through


@pytest.fixture
def unlaunched(L, host, monkeypatch):
    """As ``host``, and every call of the library that would launch answers that it has."""
    class Library:
        def __getattr__(self, name):
            return getattr(L, name) if name.endswith(("_bytes", "_sizes")) else lambda *a: OK
    library = Library()
    monkeypatch.setattr(_abi, "lib", lambda: library)
    monkeypatch.setattr(block, "_stream", lambda index: 0)


def test_tangents_of_forward_mode_are_refused(unlaunched):
    """No result without its tangent, whichever input carries one, with or without gradients beside it."""
    x, h, v, q, t = torch.zeros(6, 8), torch.zeros(6, 8), torch.zeros(1, 8), torch.zeros(6, 2, 64), torch.zeros(62, 2)
    p = block.ExpertPlan(6, 2, 3, 1, 8, torch.device("cpu"))
    ys, w, qw = torch.zeros(p.rows_sorted, 8), torch.zeros(6, 2), torch.ones(64)
    kw = dict(grid=(1, 2, 3), axes=(12, 10, 10))
    with forward_ad.dual_level():
        dual = lambda a: forward_ad.make_dual(a, torch.ones_like(a))
        for f in (lambda: block.norm(dual(x)), lambda: block.norm(x, dual(h)), lambda: block.norm(x, gate=None, scale=dual(v)),
                  lambda: block.norm(x.clone().requires_grad_(), dual(h)),
                  lambda: block.rotate(dual(q), None, t, **kw), lambda: block.rotate(q, dual(q), t, **kw),
                  lambda: block.rotate(q, None, t, q_weight=dual(qw), **kw), lambda: block.dispatch(dual(x), p),
                  lambda: block.combine(dual(ys), p), lambda: block.combine(ys, p, dual(w)),
                  lambda: block.combine(ys, p, add=dual(x))):
            with pytest.raises(NotImplementedError):
                f()
            with pytest.raises(NotImplementedError), torch.no_grad():
                f()
        # none of the inputs carries one
        assert block.norm(x, h)[0].shape == x.shape and block.combine(ys, p, w).shape == x.shape
    assert block.norm(x.clone().requires_grad_(), h)[0].requires_grad


def test_numbers_held_in_tensors_are_read_at_each_call(unlaunched, monkeypatch):
    """A number may come in a tensor of one element, whose value may change between two calls of one signature."""
    seen = []

    class Library:
        def __getattr__(self, name):
            of = {"prism_block_norm_fwd": _abi.BlockNormT, "prism_block_norm_bwd": _abi.BlockNormT,
                  "prism_head_rotate_fwd": _abi.RotateT, "prism_head_rotate_bwd": _abi.RotateT}.get(name)
            if of is None:
                return getattr(answering, name)
            return lambda addr, *a: seen.append(of.from_buffer_copy(ctypes.string_at(addr, ctypes.sizeof(of)))) or OK
    answering, library = _abi.lib(), Library()
    monkeypatch.setattr(_abi, "lib", lambda: library)
    x, h, q, t = torch.zeros(6, 8), torch.zeros(6, 8), torch.zeros(6, 2, 64), torch.zeros(62, 2)
    n = {k: torch.tensor(v) for k, v in dict(eps=0.25, res_scale=0.5, rows_per_group=2).items()}
    grid, norm = [torch.tensor(v) for v in (1, 2, 3)], torch.tensor(True)
    for f in (lambda: block.norm_forward(x, h, **n), lambda: block.norm_backward(x, h, x, x, **n),
              lambda: block.norm(x, h, **n)):
        for scale in (0.5, 2.0):
            n["res_scale"].fill_(scale)
            n["eps"].fill_(scale / 8)
            n["rows_per_group"].fill_(int(2 * scale))
            f()
            assert (seen[-1].res_scale, seen[-1].eps, seen[-1].rows_per_group) == (scale, scale / 8, int(2 * scale))
    for f in (lambda: block.rotate_forward(q, None, t, grid=grid, axes=(12, 10, 10), norm=norm),
              lambda: block.rotate_backward(q, None, q, None, t, grid=grid, axes=(12, 10, 10), norm=norm)):
        for T, H, flag in ((1, 2, True), (1, 2, False), (1, 2, True)):
            norm.fill_(flag)
            f()
            assert (seen[-1].T, seen[-1].H, seen[-1].norm) == (T, H, flag)
    t2 = torch.zeros(6, 2)
    for T, H in ((2, 3), (6, 1)):
        grid[0].fill_(T), grid[1].fill_(H)
        block.rotate_forward(q, None, t2[:T], grid=grid, axes=(1, 0, 0))
        assert (seen[-1].T, seen[-1].H) == (T, H)
        block.rotate_forward(q, None, t2, grid=[T, 6, 1], axes=(0, 1, 0))
        assert seen[-1].T == T
    grid = [torch.tensor(v) for v in (2, 1, 1)]
    for T in (2, 5):
        grid[0].fill_(T)
        block.rotate_forward(q, None, t2[:1], grid=grid, axes=(0, 0, 1))
        assert seen[-1].T == T
    # the differentiable form's backward has the forward's numbers
    n = {k: torch.tensor(v) for k, v in dict(eps=0.25, res_scale=0.5, rows_per_group=6).items()}
    z, _ = block.norm(x.clone().requires_grad_(), h, **n)
    n["res_scale"].fill_(3.0)
    z.sum().backward()
    assert seen[-1].res_scale == 0.5
    with pytest.raises(ValueError, match="three"):
        block.rotate(q, None, t, grid=(1, 2, 3, 1), axes=(12, 10, 10))
    # a number that is to be learned would get no gradient
    for k in ("eps", "res_scale"):
        with pytest.raises(ValueError, match="gradient"):
            block.norm(x, h, **{k: torch.tensor(0.5, requires_grad=True)})


def test_numbers_past_the_descriptors_32_bits_are_refused(unlaunched):
    """2^32 and a small number, which would be taken for the small one: sizes of expanded tensors, of which nothing but
    the shape is looked at."""
    big = (1 << 32) + 8
    x, h = torch.zeros(6, 8), torch.zeros(6, 8)
    q, t = torch.zeros(6, 2, 64), torch.zeros(62, 2)
    wide = torch.zeros(1, 1).expand(1, big)
    for f in (lambda: block.norm_forward(wide), lambda: block.norm_backward(wide, None, None, wide),
              lambda: block.rotate_forward(torch.zeros(1, 1, 1).expand(1, 1, (1 << 32) + 64), None, t[:0],
                                           grid=(1, 1, 1), axes=(0, 0, 0)),
              lambda: block.rotate_forward(torch.zeros(1, 1, 1).expand(1, (1 << 32) + 1, 64), None, t[:0],
                                           grid=(1, 1, 1), axes=(0, 0, 0)),
              lambda: block.rotate_forward(q, None, t[:12], grid=(1, (1 << 32) + 2, 3), axes=(12, 0, 0)),
              lambda: block.expert_plan(torch.zeros(6, 2, dtype=torch.int64), big),
              lambda: block.expert_plan(torch.zeros(6, 2, dtype=torch.int64), 8, align=(1 << 32) + 1),
              lambda: block.ExpertPlan(6, (1 << 32) + 2, 8, 1, 8, torch.device("cpu"))):
        with pytest.raises(ValueError, match="out of range"):
            f()
    # more rows a group than there are rows, however many, are all of them
    z, y = block.norm_forward(x, h, gate=torch.zeros(1, 8), rows_per_group=(1 << 64) + 2)
    assert z.shape == x.shape


@pytest.mark.parametrize("shape,rpg,G", [((2, 0, 8), None, 2), ((2, 0, 8), 5, 3), ((0, 4, 8), None, 0), ((0, 8), None, 1),
                                         ((0, 8), 7, 2), ((0, 8), None, 0), ((3, 2, 0, 8), None, 6)])
def test_groups_without_rows_have_their_vectors_and_gradients(unlaunched, shape, rpg, G):
    """Samples of no tokens: a row of gate, scale and shift each, whose gradients are 0."""
    x, h = torch.zeros(shape, requires_grad=True), torch.zeros(shape)
    for names in (("gate", "scale", "shift"), ("shift",), ("scale",)):
        v = {k: torch.ones(G, 8, requires_grad=True) for k in names}
        z, y = block.norm(x, h, rows_per_group=rpg, **v)
        assert z.shape == y.shape == shape
        (z.sum() + y.sum()).backward()
        for k in names:
            assert torch.equal(v[k].grad, torch.zeros(G, 8)), k
    g = block.norm_backward(x.detach(), h, h, h, gate=torch.ones(G, 8), scale=torch.ones(G, 8), rows_per_group=rpg)
    assert all(torch.equal(g[k], torch.zeros(G, 8)) for k in ("dgate", "dscale", "dshift"))
    if shape == (3, 2, 0, 8):
        assert block.norm_backward(x.detach(), None, None, h, wants=("dshift",))["dshift"].shape == (6, 8)
    with pytest.raises(ValueError):
        block.norm_forward(x.detach(), h, gate=torch.ones(G, 8), scale=torch.ones(G + 1, 8), rows_per_group=rpg)


def test_calls_without_rows_reach_the_library_as_given(L, host, monkeypatch):
    """A tensor without elements has no address; the library, which launches nothing for it, still sees it as given."""
    monkeypatch.setattr(block, "_stream", lambda index: 0)
    e, v, c = torch.empty(2, 0, 8), torch.ones(2, 8), torch.ones(8)
    z, y = block.norm_forward(e, e, gate=v, scale=v, shift=v, post_weight=c, post_norm="rms")
    assert z.shape == y.shape == e.shape
    assert block.norm_forward(e, e, gate=v, norm=None)[0].shape == e.shape
    g = block.norm_backward(e, e, None, e, gate=v, scale=v)
    assert all(torch.equal(g[k], torch.zeros(2, 8)) for k in ("dgate", "dscale", "dshift"))
    g = block.norm_backward(e, e, e, None, gate=v, norm=None)
    assert torch.equal(g["dgate"], torch.zeros(2, 8)) and g["dh"].shape == e.shape
    # what is refused with rows is refused without them
    with pytest.raises(_abi.PrismError):
        block.norm_forward(e, gate=v)
    with pytest.raises(_abi.PrismError):
        block.norm_forward(e, e, post_weight=c)


def given_outputs():
    """(name, output, call that writes it) of every output that a caller may give, in place or apart."""
    z = lambda *s: torch.zeros(*s)
    t = torch.zeros(62, 2)
    p, kw = block.ExpertPlan(6, 2, 3, 1, 8, torch.device("cpu")), dict(grid=(1, 2, 3), axes=(12, 10, 10))
    n = p.rows_sorted
    return [
        ("z", z(6, 8), lambda o: block.norm_forward(z(6, 8), z(6, 8), z=o)),
        ("z is x", z(6, 8), lambda o: block.norm_forward(o, z(6, 8), z=o)),
        ("y", z(6, 8), lambda o: block.norm_forward(z(6, 8), y=o)),
        ("a part of y's buffer", z(6, 24)[:, 8:16], lambda o: block.norm_forward(z(6, 8), y=o)),
        ("y, of a copied input", z(6, 8), lambda o: block.norm_forward(z(8, 6).t(), y=o)),
        ("Qr", z(6, 2, 64), lambda o: block.rotate_forward(z(6, 2, 64), None, t, out=(o, None), **kw)),
        ("Kr is K", z(6, 2, 64), lambda o: block.rotate_forward(z(6, 2, 64), o, t, out=(z(6, 2, 64), o), **kw)),
        ("xs", z(n, 8), lambda o: block.expert_dispatch(z(6, 8), p, out=o)),
        ("combined", z(6, 8), lambda o: block.expert_combine(z(n, 8), p, out=o)),
        ("combined is add", z(6, 8), lambda o: block.expert_combine(z(n, 8), p, add=o, out=o)),
        ("dys", z(n, 8), lambda o: block.expert_combine_backward(z(6, 8), z(n, 8), p, out=o)),
        ("dys is ys", z(n, 8), lambda o: block.expert_combine_backward(z(6, 8), o, p, out=o)),
    ]


@pytest.mark.parametrize("i", range(12))
def test_autograd_knows_of_given_outputs(unlaunched, i):
    name, o, call = given_outputs()[i]
    # a tensor that autograd has saved: the call goes through, the backward that needs its old values does not
    a = torch.ones_like(o).requires_grad_()
    prod = (a * o).sum()
    before = o._version
    call(o)
    assert o._version > before, name
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        prod.backward()
    call(o)                                                # kept signatures behave alike
    assert o._version > before + 1, name
    # a leaf, and a tensor with a history
    for g in (given_outputs()[i][1].requires_grad_(), given_outputs()[i][1].requires_grad_() * 1):
        with pytest.raises(ValueError, match="requires grad"):
            call(g)
        with torch.no_grad():
            call(g)
    with torch.inference_mode():
        call(given_outputs()[i][1])


def test_results_that_are_not_given_keep_their_version(unlaunched):
    x, h = torch.zeros(6, 8), torch.zeros(6, 8)
    z, y = block.norm_forward(x, h)
    assert x._version == h._version == 0
    x = x.clone().requires_grad_()
    z, y = block.norm(x, h)
    block.norm_forward(x, h)
    (z.sum() + y.sum()).backward()
    assert x.grad is not None


def test_an_output_that_is_also_a_second_input_is_refused(L, host):
    """With one choice a token and no padding, sorted and token buffers have one shape, and the tensor that an output
    may take the place of can be another argument too, which other tokens still read."""
    p = block.ExpertPlan(6, 1, 3, 1, 8, torch.device("cpu"))
    t, o = torch.zeros(6, 8), torch.zeros(6, 8)
    assert p.rows_sorted == 6
    for f in (lambda: block.expert_combine(t, p, add=t, out=t),
              lambda: block.expert_combine(t, p, torch.zeros(6, 1), add=t, out=t),
              lambda: block.expert_combine_backward(t, t, p, out=t),
              lambda: block.expert_dispatch(t, p, out=t)):
        with pytest.raises(ValueError, match="overlaps"):
            f()
    # each alone is allowed, and so is one tensor as both inputs
    for f in (lambda: block.expert_combine(o, p, add=t, out=t), lambda: block.expert_combine(t, p, add=t, out=o),
              lambda: block.expert_combine_backward(o, t, p, out=t), lambda: block.expert_combine(t, p, add=t)):
        with pytest.raises(host):
            f()
    # the norms' vectors of a row each: read after the row of z is written
    x, h = torch.zeros(6, 8), torch.zeros(6, 8)
    for k in ("scale", "shift", "gate"):
        with pytest.raises(ValueError, match="overlaps"):
            block.norm_forward(x, h, z=x, rows_per_group=1, **{k: x})
    with pytest.raises(ValueError, match="overlaps"):
        block.norm_forward(x, h, z=h)
    # the stream itself as the branch, in place or not
    for z in (None, x, torch.zeros(6, 8)):
        with pytest.raises(host):
            block.norm_forward(x, x, z=z)


# grids whose number of places passes 64 bits: cut to 64 bits, the products are 0 or below it but for the last
@pytest.mark.parametrize("grid", [(1 << 16, 1 << 24, 1 << 24), (1 << 24, 1 << 24, 1 << 16), (1 << 21, 1 << 21, 1 << 21),
                                  (1 << 30, 1 << 30, 1 << 4), (2 ** 31 - 1, 2 ** 31 - 1, 2 ** 31 - 1)])
def test_rotation_grids_past_64_bits_refused(L, grid):
    # no tokens: not even an accepted grid launches anything
    d = _abi.RotateT(0, *grid, 1, 0, 64, 0, 0, 0, 0, _abi.PRISM_BF16, 1, 1e-6)
    assert L.prism_head_rotate_fwd(ctypes.addressof(d), P, None, None, None, P, P, None, None) == UNSUP
    out = ctypes.c_size_t(0)
    assert L.prism_head_rotate_ws_bytes(ctypes.addressof(d), ctypes.addressof(out)) == UNSUP

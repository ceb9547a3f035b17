"""What the operators around the attention refuse, in the library and in the tensor calls, and the host-side
sizes: nothing here launches."""
import ctypes

import pytest
import torch

from dynamic_block_sparse_macro_b200 import _abi, block

OK, ARG, SHAPE, UNSUP, WS = 0, 1, 2, 3, 4
P = 1 << 40                                   # aligned, never dereferenced on the host
F, B = _abi.PRISM_F32, _abi.PRISM_BF16
INT_MAX = 2 ** 31 - 1


@pytest.fixture(scope="module")
def L():
    from dynamic_block_sparse_macro_b200 import build
    build.build()
    return _abi.lib()


def norm_desc(**kw):
    d = dict(rows=10, rows_per_group=5, channels=64, stream_dtype=B, branch_dtype=B, norm=2, post_norm=0, eps=1e-6,
             res_scale=1.0)
    d.update(kw)
    return _abi.BlockNormT(**d)


def fwd(L, n, x=P, h=P, gate=None, w_post=None, w=None, b=None, scale=None, shift=None, z=P, y=P):
    return L.prism_block_norm_fwd(ctypes.addressof(n) if n is not None else None, x, h, gate, w_post, w, b, scale, shift,
                                  z, y, None)


def bwd(L, n, z=P, h=P, gate=None, w_post=None, w=None, b=None, scale=None, dz=P, dy=P, dx=P, dh=P, dgate=None,
        dw_post=None, dw=None, db=None, dscale=None, dshift=None, ws=None, ws_bytes=0):
    return L.prism_block_norm_bwd(ctypes.addressof(n), z, h, gate, w_post, w, b, scale, dz, dy, dx, dh, dgate, dw_post,
                                  dw, db, dscale, dshift, ws, ws_bytes, None)


@pytest.mark.parametrize("kw,code", [
    (dict(rows=-1), SHAPE), (dict(rows_per_group=0), SHAPE), (dict(channels=0), SHAPE), (dict(channels=8193), UNSUP),
    (dict(rows=1 << 41), UNSUP), (dict(stream_dtype=B, branch_dtype=F), UNSUP), (dict(stream_dtype=2), UNSUP),
    (dict(norm=3), ARG), (dict(post_norm=-1), ARG), (dict(eps=0.0), ARG), (dict(eps=float("nan")), ARG),
    (dict(eps=float("inf")), ARG), (dict(res_scale=float("nan")), ARG), (dict(ld_x=63), SHAPE), (dict(ld_gate=1), SHAPE),
    (dict(ld_z=-64), SHAPE),
])
def test_norm_descriptors_refused(L, kw, code):
    assert fwd(L, norm_desc(**kw)) == code
    if not {"ld_x", "ld_gate", "ld_z"} & set(kw):
        assert bwd(L, norm_desc(**kw)) == code
        out = ctypes.c_size_t(0)
        n = norm_desc(**kw)
        assert L.prism_block_norm_ws_bytes(ctypes.addressof(n), ctypes.addressof(out)) == code


def test_norm_arguments_refused(L):
    n = norm_desc()
    assert fwd(L, None) == ARG
    assert fwd(L, n, x=None) == fwd(L, n, z=None) == fwd(L, n, y=None) == ARG
    assert fwd(L, n, x=P + 1) == fwd(L, n, y=P + 1) == fwd(L, n, gate=P + 2) == ARG      # not on an element
    assert fwd(L, n, h=None) == ARG                                  # z without a branch
    assert fwd(L, n, h=None, z=None, gate=P) == ARG
    assert fwd(L, n, w_post=P) == ARG                                # without its norm
    assert fwd(L, norm_desc(norm=0), y=None, h=None, z=None) == ARG  # nothing to do
    assert fwd(L, norm_desc(norm=0)) == ARG                          # y without a norm
    assert fwd(L, norm_desc(norm=0), y=None, shift=P) == ARG
    assert bwd(L, n, dy=None) == bwd(L, n, dx=None) == bwd(L, n, dh=None) == bwd(L, n, h=None) == ARG
    assert bwd(L, n, dgate=P) == bwd(L, n, dw=P) == bwd(L, n, db=P) == bwd(L, n, dscale=P) == ARG   # without the vector
    assert bwd(L, n, w_post=P) == ARG
    assert bwd(L, norm_desc(norm=0), dz=None, dy=None) == ARG
    n = norm_desc(rows=100, rows_per_group=50)                       # cut groups: their sums meet in the workspace
    assert bwd(L, n, dshift=P) == WS and bwd(L, n, dshift=P, ws=P, ws_bytes=64) == WS
    assert bwd(L, n, dshift=P, ws=P + 4, ws_bytes=1 << 30) == ARG
    assert fwd(L, norm_desc(rows=0), x=None, h=P, z=None, y=None) == OK     # no rows: nothing launched


def test_norm_workspace_grows_with_the_split_only(L):
    def size(**kw):
        return _abi.block_norm_ws_bytes(norm_desc(**kw))
    # [segments][3][C] floats.  64 channels: CTAs of 32 teams of 8 threads, two an SM; segments of two rows a team at least
    assert size(rows=1) == 1 * 3 * 64 * 4
    assert size(rows=128, rows_per_group=128) == 2 * 3 * 64 * 4
    assert size(rows=10 ** 6, rows_per_group=10 ** 6) == 296 * 3 * 64 * 4
    # groups of one row are not cut, and shared out among the teams
    assert size(rows=1000, rows_per_group=1) == 1000 * 3 * 64 * 4
    assert size(rows=10 ** 5, rows_per_group=1) == 148 * 64 * 3 * 64 * 4
    # 2048 channels: a team a CTA
    assert size(rows=1, channels=2048) == 1 * 3 * 2048 * 4
    assert size(rows=8, rows_per_group=8, channels=2048) == 4 * 3 * 2048 * 4
    assert size(rows=61440, rows_per_group=30720, channels=2048) == 296 * 3 * 2048 * 4


def rot_desc(**kw):
    d = dict(tokens=10, T=1, H=2, W=5, heads_q=2, heads_k=2, head_dim=64, pairs_t=12, pairs_h=10, pairs_w=10, pairing=0,
             dtype=B, norm=1, eps=1e-6)
    d.update(kw)
    return _abi.RotateT(**d)


def rot(L, p, Q=P, K=P, wq=None, wk=None, table=P, Qr=P, Kr=P):
    return L.prism_head_rotate_fwd(ctypes.addressof(p), Q, K, wq, wk, table, Qr, Kr, None)


@pytest.mark.parametrize("kw,code", [
    (dict(tokens=-1), SHAPE), (dict(T=0), SHAPE), (dict(head_dim=96), UNSUP), (dict(heads_q=1025), UNSUP),
    (dict(heads_q=0, heads_k=0), SHAPE), (dict(pairs_t=13), SHAPE), (dict(pairs_h=-1), SHAPE), (dict(pairing=2), ARG),
    (dict(dtype=7), UNSUP), (dict(norm=2), ARG), (dict(eps=-1.0), ARG), (dict(ld_q=64), SHAPE), (dict(ld_q=132), SHAPE),
    (dict(T=INT_MAX, H=2), UNSUP), (dict(T=1 << 28), UNSUP),
])
def test_rotation_descriptors_refused(L, kw, code):
    assert rot(L, rot_desc(**kw)) == code


def test_rotation_arguments_refused(L):
    p = rot_desc()
    assert L.prism_head_rotate_fwd(None, P, P, None, None, P, P, P, None) == ARG
    for k in ("Q", "K", "Qr", "Kr", "table"):
        assert rot(L, p, **{k: None}) == ARG and rot(L, p, **{k: P + 8}) == ARG
    assert rot(L, rot_desc(norm=0), wq=P) == ARG
    assert rot(L, rot_desc(heads_k=0)) == ARG                        # K without heads
    assert rot(L, rot_desc(tokens=0), Q=None, K=None, Qr=None, Kr=None) == OK
    b = lambda p, dwq, ws, n: L.prism_head_rotate_bwd(ctypes.addressof(p), P, P, None, None, P, P, P, P, P, dwq, None,
                                                      ws, n, None)
    assert b(p, P, None, 0) == WS and b(p, P, P, 1024) == WS
    assert b(rot_desc(norm=0), P, P, 1 << 30) == ARG


def ex(**kw):
    d = dict(rows=10, top_k=2, experts=4, align=1, id_bytes=8)
    d.update(kw)
    return _abi.ExpertsT(**d)


def plan(L, e, ids=P, counts=P, offsets=P, pos=P, src=P, ws=P, n=1 << 30):
    return L.prism_expert_plan(ctypes.addressof(e), ids, counts, offsets, pos, src, ws, n, None)


@pytest.mark.parametrize("kw,code", [
    (dict(rows=-1), SHAPE), (dict(top_k=0), SHAPE), (dict(top_k=17), UNSUP), (dict(experts=0), SHAPE),
    (dict(experts=1025), UNSUP), (dict(align=0), SHAPE), (dict(align=4097), UNSUP), (dict(rows=(1 << 29) + 1), UNSUP),
    (dict(id_bytes=2), ARG),
])
def test_expert_descriptors_refused(L, kw, code):
    e = ex(**kw)
    assert plan(L, e) == code
    assert L.prism_expert_dispatch(ctypes.addressof(e), B, 64, P, 0, P, P, P, 0, P, None) == code
    assert L.prism_expert_combine(ctypes.addressof(e), B, 64, P, P, None, None, 0, P, 0, None) == code
    r, w = ctypes.c_int64(0), ctypes.c_size_t(0)
    assert L.prism_expert_sizes(ctypes.addressof(e), ctypes.addressof(r), ctypes.addressof(w)) == code


def test_expert_arguments_refused(L):
    e = ex()
    assert plan(L, e, ids=None) == plan(L, e, ids=P + 4) == plan(L, e, counts=None) == plan(L, e, src=P + 2) == ARG
    assert plan(L, ex(rows=100000), ws=None, n=0) == WS and plan(L, ex(rows=100000), n=8) == WS
    a = ctypes.addressof(e)
    d = lambda dt=B, C=64, x=P, ld=0, pos=P, tail=0, xs=P: L.prism_expert_dispatch(a, dt, C, x, ld, pos, P, P, tail, xs,
                                                                                   None)
    assert d(dt=5) == UNSUP and d(C=0) == SHAPE and d(C=(1 << 20) + 1) == UNSUP and d(ld=63) == SHAPE
    assert d(x=None) == d(x=P + 1) == d(pos=None) == d(tail=2) == d(xs=None) == ARG
    c = lambda y=P, out=P, add=None, ld=0: L.prism_expert_combine(a, F, 64, y, P, None, add, 0, out, ld, None)
    assert c(y=None) == c(out=None) == c(add=P + 2) == ARG and c(ld=10) == SHAPE
    b = lambda dout=P, y=P, dy=P, dw=P: L.prism_expert_combine_bwd(a, F, 64, dout, 0, y, P, None, P, P, 0, dy, dw, None)
    assert b(dout=None) == b(y=None) == b(dy=None) == b(dw=P + 1) == ARG


def test_expert_sizes():
    # each expert with slots may end in a part of a unit
    assert _abi.expert_sizes(ex(rows=10, top_k=2, experts=4, align=1)) == (20, 0)
    assert _abi.expert_sizes(ex(rows=10, top_k=2, experts=4, align=8)) == (20 + 4 * 7, 0)
    assert _abi.expert_sizes(ex(rows=1, top_k=2, experts=64, align=128)) == (2 + 2 * 127, 0)
    assert _abi.expert_sizes(ex(rows=0)) == (0, 0)
    rows, ws = _abi.expert_sizes(ex(rows=61440, top_k=2, experts=16))
    assert rows == 122880 and ws == -(-122880 // 1024) * 16 * 4


def test_tensors_off_the_gpu_are_refused():
    x = torch.zeros(4, 8)
    for f in (lambda: block.norm_forward(x), lambda: block.norm(x),
              lambda: block.rotate_forward(x[:, None], None, torch.zeros(1, 2), grid=(1, 1, 1), axes=(1, 0, 0)),
              lambda: block.expert_plan(torch.zeros(4, 2, dtype=torch.int64), 4)):
        with pytest.raises(ValueError, match="CUDA"):
            f()


@pytest.fixture
def host(monkeypatch):
    """The tensor calls' checks on CPU tensors: the device check is passed over, and no call gets through."""
    monkeypatch.setattr(block, "_same_device", lambda dev, *t: None)

    def refuse(*a):
        raise AssertionError("the call was not refused")
    monkeypatch.setattr(block, "_stream", refuse)
    monkeypatch.setattr(block, "_current", lambda index: True)
    monkeypatch.setattr(block, "_plans", {})


def test_norm_tensor_checks(L, host):
    x, h, v = torch.zeros(6, 8), torch.zeros(6, 8), torch.zeros(8)
    bad = [
        lambda: block.norm_forward(x, norm="group"),
        lambda: block.norm_forward(x, h, post_norm="l2"),
        lambda: block.norm_forward(x.half()),
        lambda: block.norm_forward(x, h[:, :4]),
        lambda: block.norm_forward(x, h.bfloat16(), out_dtype=torch.float32),
        lambda: block.norm_forward(x, weight=v.bfloat16()),
        lambda: block.norm_forward(x, weight=v[:4]),
        lambda: block.norm_forward(x, h, gate=torch.zeros(2, 8)),                      # one group by default
        lambda: block.norm_forward(x, h, gate=torch.zeros(2, 8), rows_per_group=2),    # three groups
        lambda: block.norm_forward(x, rows_per_group=0),
        lambda: block.norm_forward(x, z=x),                                            # no branch
        lambda: block.norm_forward(x, h, y=torch.zeros(6, 4)),
        lambda: block.norm_forward(x, h, y=x),                                         # only z may be x
        lambda: block.norm_forward(x, h, z=h),
        lambda: block.norm_forward(x, h, norm=None, y=torch.zeros(6, 8)),
        lambda: block.norm_forward(x[:5], h[:5], z=x[1:]),                             # shifted by a row
        lambda: block.norm_forward(x, h, z=torch.zeros(1, 8).expand(6, 8)),
        lambda: block.norm_backward(x, h, x, None),
        lambda: block.norm_backward(x, h, None, None, norm=None),
        lambda: block.norm_backward(x, h, x[:, :4], x),
        lambda: block.norm_backward(x, h, x, x, wants=("dz",)),
    ]
    for f in bad:
        with pytest.raises(ValueError):
            f()


def test_rotation_tensor_checks(L, host):
    q, t = torch.zeros(6, 2, 64), torch.zeros(12 + 20 + 30, 2)
    kw = dict(grid=(1, 2, 3), axes=(12, 10, 10))
    bad = [
        lambda: block.rotate_forward(None, None, t, **kw),
        lambda: block.rotate_forward(q, q[:3], t, **kw),
        lambda: block.rotate_forward(q, torch.zeros(6, 2, 128), t, **kw),
        lambda: block.rotate_forward(q, q.bfloat16(), t, **kw),
        lambda: block.rotate_forward(q.half(), None, t, **kw),
        lambda: block.rotate_forward(q[0], None, t, **kw),
        lambda: block.rotate_forward(q, None, t[:-1], **kw),
        lambda: block.rotate_forward(q, None, t.double(), **kw),
        lambda: block.rotate_forward(q, None, t, pairs="split", **kw),
        lambda: block.rotate_forward(q, None, t, q_weight=torch.ones(64), norm=False, **kw),
        lambda: block.rotate_forward(q, None, t, q_weight=torch.ones(32), **kw),
        lambda: block.rotate_forward(q, q, t, out=(q, torch.zeros_like(q)), **kw),     # K is read while Q is written
        lambda: block.rotate_forward(q, None, t, out=(q, q), **kw),
        lambda: block.rotate_forward(q[:5], None, t, out=(q[1:], None), **kw),
        lambda: block.rotate_backward(None, None, q, None, t, **kw),                   # the norm needs Q
        lambda: block.rotate_backward(q, q, q, None, t, **kw),
        lambda: block.rotate_backward(q, None, q, None, t, wants=("dk_weight",), **kw),
    ]
    for f in bad:
        with pytest.raises(ValueError):
            f()
    with pytest.raises(ValueError):
        block.rotation_table((2, 1, 1), (1, 1, 1), device="cpu", positions=([0], [0], [0]))


def test_expert_tensor_checks(L, host):
    p = block.ExpertPlan(6, 2, 3, 4, 8, torch.device("cpu"))
    x, ys, w = torch.zeros(6, 8), torch.zeros(p.rows_sorted, 8), torch.zeros(6, 2)
    assert p.rows_sorted == 12 + 3 * 3 and p.pos.shape == (6, 2) and p.counts.data_ptr() % 16 == 0
    bad = [
        lambda: block.expert_plan(torch.zeros(6, dtype=torch.int64), 3),
        lambda: block.expert_plan(torch.zeros(6, 2), 3),
        lambda: block.expert_dispatch(x[:5], p),
        lambda: block.expert_dispatch(x.half(), p),
        lambda: block.expert_dispatch(x, p, out=torch.zeros(p.rows_sorted, 9)),
        lambda: block.expert_dispatch(x, p, out=torch.zeros(p.rows_sorted, 16)[:, :8]),
        lambda: block.expert_dispatch(ys[:6], p, out=ys),
        lambda: block.expert_combine(ys[:-1], p),
        lambda: block.expert_combine(ys, p, w[:, :1]),
        lambda: block.expert_combine(ys, p, w.double()),
        lambda: block.expert_combine(ys, p, add=x.bfloat16()),
        lambda: block.expert_combine(ys, p, add=x, out=torch.zeros(6, 9)[:, :8].t().contiguous().t()),
        lambda: block.expert_combine(ys, p, out=ys[:6]),
        lambda: block.expert_combine_backward(x, None, p, w),
        lambda: block.expert_combine_backward(x, ys.bfloat16(), p, w),
        lambda: block.expert_combine_backward(x, ys, p, w, out=torch.zeros(p.rows_sorted, 9)),
    ]
    for i, f in enumerate(bad):
        with pytest.raises(ValueError):
            f()
    with pytest.raises(_abi.PrismError):
        block.ExpertPlan(6, 17, 3, 4, 8, torch.device("cpu"))


def test_columns_of_one_buffer_are_apart():
    b = torch.zeros(6, 24)
    assert block._apart(b[:, :8], b[:, 8:16]) and block._apart(b[:, 16:], b[:, :16])
    assert not block._apart(b[:, :9], b[:, 8:16]) and not block._apart(b[:4], b[3:])
    assert block._apart(b[:3], b[3:]) and not block._apart(b[1:, :8], b.view(-1, 12)[:, :8])
    assert not block._apart(b[:3, 20:], b.view(-1)[20:20 + 72].view(3, 24)[:, :8])     # runs over the row's end


def test_calls_move_to_the_tensors_device(L, host, monkeypatch):
    """A call on tensors of another device than the current one is made with theirs as the current one."""
    current = [0]

    class Device:
        def __init__(self, index):
            self.index = index

        def __enter__(self):
            current[0] = "theirs"

        def __exit__(self, *a):
            current[0] = 0

    class Reached(Exception):
        pass

    def stream(index):
        assert current[0] == "theirs"
        raise Reached
    monkeypatch.setattr(block, "_current", lambda index: current[0] == "theirs")
    monkeypatch.setattr(block, "_stream", stream)
    monkeypatch.setattr(torch.cuda, "device", Device)
    x, t = torch.zeros(6, 8), torch.zeros(62, 2)
    q = torch.zeros(6, 2, 64)
    kw = dict(grid=(1, 2, 3), axes=(12, 10, 10))
    p = block.ExpertPlan(6, 2, 3, 1, 8, torch.device("cpu"))
    ys = torch.zeros(p.rows_sorted, 8)
    for f in (lambda: block.norm_forward(x, x), lambda: block.norm_backward(x, x, x, x),
              lambda: block.rotate_forward(q, None, t, **kw), lambda: block.rotate_backward(q, None, q, None, t, **kw),
              lambda: block.expert_plan(torch.zeros(6, 2, dtype=torch.int64), 3), lambda: block.expert_dispatch(x, p),
              lambda: block.expert_combine(ys, p), lambda: block.expert_combine_backward(x, ys, p)):
        with pytest.raises(Reached):
            f()
        assert current[0] == 0


def test_kept_signatures_are_bounded(monkeypatch):
    monkeypatch.setattr(block, "_plans", {})
    monkeypatch.setattr(block, "_MAX_PLANS", 3)
    for i in range(10):
        block._keep(i, i)
        assert len(block._plans) <= 3 and block._plans[i] == i

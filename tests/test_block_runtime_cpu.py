"""What the row operators' host code asks of the CUDA runtime, seen through a stand-in for it (fake_runtime.cpp):
launches, limits of shared memory, and what happens when one of these calls fails.  Nothing runs on a GPU."""
import ctypes
import os
import subprocess

import pytest

from dynamic_block_sparse_macro_b200 import _abi, build

HERE = os.path.dirname(os.path.abspath(__file__))
OBJS = ("block_norm", "block_norm_bb", "block_norm_fb", "block_norm_ff", "head_rotate", "experts")
P = 1 << 40
OK, CUDA = 0, 5
F, B = _abi.PRISM_F32, _abi.PRISM_BF16


@pytest.fixture(scope="module")
def L(tmp_path_factory):
    build.build()
    out = str(tmp_path_factory.mktemp("fake") / "librows_fake.so")
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(build.nvcc()))), "include")
    subprocess.run(["g++", "-O1", "-std=c++17", "-fPIC", "-shared", "-Wl,-z,defs,-Bsymbolic", "-I", cuda, "-o", out,
                    os.path.join(HERE, "fake_runtime.cpp"), *(os.path.join(build.OBJ, o + ".o") for o in OBJS)], check=True)
    lib = ctypes.CDLL(out)
    for name, sig in _abi._SIGS.items():
        if name.startswith(("prism_block_norm", "prism_head_rotate", "prism_expert")):
            getattr(lib, name).argtypes = sig
    return lib


def events(L):
    """(kind, kernel, bytes, grid, block) of the calls since the last reset."""
    out = []
    for i in range(L.fake_count()):
        name, n, dims = ctypes.c_char_p(), ctypes.c_ulonglong(), (ctypes.c_uint * 6)()
        kind = L.fake_event(i, ctypes.byref(name), ctypes.byref(n), dims)
        out.append((("launch", "limit", "memset")[kind], name.value.decode(), n.value, tuple(dims[:3]), tuple(dims[3:])))
    return out


def norm_calls(L, C, sdt, bdt, branch, post, rows=5):
    n = _abi.BlockNormT(rows, rows, C, sdt, bdt, 2, post if branch else 0, 1e-6, 1.0)
    a, h = ctypes.addressof(n), P if branch else None
    yield L.prism_block_norm_fwd(a, P, h, None, None, None, None, None, None, h, P, None)
    yield L.prism_block_norm_bwd(a, P, h, None, None, P, None, None, P, P, P, h, None, None, P, None, None, None, P,
                                 1 << 40, None)


def test_a_kernels_shared_memory_limit_is_the_same_for_all_its_rows(L):
    """The limit belongs to the kernel and to all host threads: whatever the width, a call sets the same one, which
    holds its own launch and every other of the kernel's."""
    limits, used = {}, {}
    for sdt, bdt in ((F, F), (F, B), (B, B)):
        for branch, post in ((False, 0), (True, 0), (True, 1)):
            for C in (1, 8, 64, 100, 256, 264, 333, 512, 1000, 1001, 1024, 1536, 2048, 2056, 2304, 2500, 2560, 2568, 3000,
                      3001, 3080, 3200, 4096, 4104, 5000, 5120, 5121, 6000, 6144, 6152, 7000, 8184, 8191, 8192):
                L.fake_reset(-1)
                assert list(norm_calls(L, C, sdt, bdt, branch, post)) == [OK, OK]
                for kind, kernel, n, _, _ in events(L):
                    if kind == "limit":
                        limits.setdefault(kernel, set()).add(n)
                    elif kind == "launch":
                        used[kernel] = max(used.get(kernel, 0), n)
    assert len(limits) > 20
    for kernel, n in limits.items():
        assert len(n) == 1, (kernel, sorted(n))
        assert used[kernel] <= max(n) <= 227 << 10
    for kernel, n in used.items():
        assert n <= 40 << 10 or kernel in limits


def calls(L):
    """One call of each entry point, in the forms that differ in what they launch."""
    out = {}
    for C in (64, 2048, 8192):
        for rows in (0, 1, 5000):
            n = _abi.BlockNormT(rows, max(1, rows), C, B, B, 2, 0, 1e-6, 1.0)
            a = ctypes.addressof(n)
            out["norm", C, rows] = n, lambda a=a: L.prism_block_norm_fwd(a, P, P, None, None, None, None, None, None, P, P,
                                                                        None)
            for want in (None, P):
                out["norm backward", C, rows, want] = n, lambda a=a, want=want: L.prism_block_norm_bwd(
                    a, P, P, None, None, P, P, None, P, P, P, P, None, None, want, want, None, None, P, 1 << 40, None)
    for rows in (0, 117):
        p = _abi.RotateT(rows, 1, 9, 13, 3, 2, 64, 10, 10, 10, 0, B, 1, 1e-6)
        a = ctypes.addressof(p)
        out["rotate", rows] = p, lambda a=a: L.prism_head_rotate_fwd(a, P, P, None, None, P, P, P, None)
        for want in (None, P):
            out["rotate backward", rows, want] = p, lambda a=a, want=want: L.prism_head_rotate_bwd(
                a, P, P, None, None, P, P, P, P, P, want, want, P, 1 << 40, None)
    for rows in (0, 2048, 2049):
        e = _abi.ExpertsT(rows, 1, 8, 4, 8)
        a = ctypes.addressof(e)
        out["plan", rows] = e, lambda a=a: L.prism_expert_plan(a, P, P, P, P, P, P, 1 << 40, None)
        out["dispatch", rows] = e, lambda a=a: L.prism_expert_dispatch(a, B, 64, P, 0, P, P, P, 1, P, None)
        out["combine", rows] = e, lambda a=a: L.prism_expert_combine(a, B, 64, P, P, None, None, 0, P, 0, None)
        out["combine backward", rows] = e, lambda a=a: L.prism_expert_combine_bwd(a, B, 64, P, 0, P, P, None, P, P, 1, P, P,
                                                                                None)
    return out


def test_a_refused_launch_ends_its_call_and_leaves_no_error(L):
    """Whichever of a call's steps the runtime refuses, the call reports it, launches nothing more (a sum over what was
    never written), and the next call's check does not find the error."""
    seen = set()
    for name, (_, f) in calls(L).items():
        L.fake_reset(-1)
        assert f() == OK, name
        n = L.fake_count()
        seen.add((name[0], n))
        for i in range(n):
            L.fake_reset(i)
            assert f() == CUDA, (name, i)
            assert L.fake_count() == i + 1, (name, i)
            assert L.fake_last_error() == 0, (name, i)
    # the forms of more than one step are among them: a limit, a kernel and its join; two memsets; count and placement
    assert {("norm backward", 3), ("norm backward", 2), ("rotate backward", 2), ("plan", 1), ("plan", 2)} <= seen

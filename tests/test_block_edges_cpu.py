"""Calls of the operators around the attention that have to be refused or prepared alike whatever came before them,
in the library and in the tensor calls: nothing here launches."""
import ctypes

import pytest
import torch

from dynamic_block_sparse_macro_b200 import _abi, block

OK, ARG, SHAPE, UNSUP = 0, 1, 2, 3
P = 1 << 40                                   # aligned, never dereferenced on the host


@pytest.fixture(scope="module")
def L():
    from dynamic_block_sparse_macro_b200 import build
    build.build()
    return _abi.lib()


# grids whose number of places passes 64 bits: cut to 64 bits, the products are 0 or below it but for the last
@pytest.mark.parametrize("grid", [(1 << 16, 1 << 24, 1 << 24), (1 << 24, 1 << 24, 1 << 16), (1 << 21, 1 << 21, 1 << 21),
                                  (1 << 30, 1 << 30, 1 << 4), (2 ** 31 - 1, 2 ** 31 - 1, 2 ** 31 - 1)])
def test_rotation_grids_past_64_bits_refused(L, grid):
    # no tokens: not even an accepted grid launches anything
    d = _abi.RotateT(0, *grid, 1, 0, 64, 0, 0, 0, 0, _abi.PRISM_BF16, 1, 1e-6)
    assert L.prism_head_rotate_fwd(ctypes.addressof(d), P, None, None, None, P, P, None, None) == UNSUP
    out = ctypes.c_size_t(0)
    assert L.prism_head_rotate_ws_bytes(ctypes.addressof(d), ctypes.addressof(out)) == UNSUP

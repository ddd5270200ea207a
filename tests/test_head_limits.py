"""The largest vocabulary of the cross entropy calls, without a GPU: entries are
numbered in 32 bits, padded to whole tiles of 256."""
from __future__ import annotations

import ctypes

import sparse_linear_layers_02_amd as sbn

OK, SHAPE = 0, 2


def test_tiles_of_the_largest_vocabulary_stay_in_32_bits():
    L, b = sbn.lib(), ctypes.c_size_t()
    most = 2 ** 31 - 256                                # its last tile ends at 2^31 - 256
    P, big = ctypes.c_void_p(0x100000), 1 << 50
    for f in (L.sbn_cross_entropy_workspace_bytes, L.sbn_cross_entropy_backward_workspace_bytes):
        assert f(1, most, 64, ctypes.byref(b)) == OK
        for V in (most + 1, 2 ** 31 - 200, 2 ** 31 - 128, 2 ** 31 - 1):
            assert f(1, V, 64, ctypes.byref(b)) == SHAPE, V
    for V in (most + 1, 2 ** 31 - 128):
        assert L.sbn_cross_entropy(P, 64, P, 64, P, 8, 1, V, 64, P, P, P, big, None) == SHAPE
        assert L.sbn_cross_entropy_backward(P, 64, P, 64, P, 8, P, P, 1, V, 64, P, 0, 64, P, 0, 64, P, big, None) == SHAPE

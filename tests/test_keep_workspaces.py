"""Workspaces of include/sbn_keep.h, without a GPU: a row of partial sums for each block that is on the
machine at once."""
from __future__ import annotations

import ctypes

import pytest

import sparse_linear_layers_02_amd as sbn


@pytest.mark.parametrize("fn", ["sbn_rmsnorm_backward_kept_workspace_bytes", "sbn_activation_backward_workspace_bytes"])
def test_partial_sums(fn):
    def blocks(T, K):
        b = ctypes.c_size_t()
        assert getattr(sbn.lib(), fn)(T, K, ctypes.byref(b)) == 0
        return -(-b.value // (4 * K)) if b.value % (4 * K) else b.value // (4 * K)

    assert blocks(0, 4096) == 0 and blocks(17, 4096) == 17
    for K in (12288, 12296, 14344, 16384, 16392, 32768):            # one block a unit
        assert 256 <= blocks(8192, K) <= 257
    assert 512 <= blocks(8192, 4096) <= 513                          # two

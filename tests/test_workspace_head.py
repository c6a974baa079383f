"""The head of a workspace: what calls keep between them lies at the same place for every shape (CPU)."""

import ctypes
import os
import re

import pytest

from mixture_experts_layer_counts_amd import _lib, shape_for


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(_lib.LIB_PATH):
        from mixture_experts_layer_counts_amd import build
        build.build()
    return _lib.load()


SHAPES = [
    dict(T=0, D=64, I=64, E=1, k=1), dict(T=1, D=64, I=64, E=1, k=1), dict(T=4, D=2048, I=768, E=128, k=8),
    dict(T=5, D=2048, I=768, E=128, k=8), dict(T=64, D=512, I=128, E=1024, k=16), dict(T=65, D=64, I=64, E=1, k=1),
    dict(T=16, D=65536, I=64, E=4, k=2), dict(T=3, D=128, I=128, E=8, k=2, precision="mxfp8"),
    dict(T=3, D=128, I=128, E=8, k=2, precision="int8", shared_precision="int8"), dict(T=8, D=64, I=64, E=8, k=2, R=4),
    dict(T=256, D=128, I=64, E=8, k=2, minibatch_rows=64, ring_rows=128, pipeline=True, mem_workgroups=8),
]


@pytest.mark.parametrize("kw", SHAPES)
def test_data_lies_behind_the_head(lib, kw):
    head = int(re.search(r"#define MOE_WORKSPACE_HEAD_BYTES (\d+)", open(_lib.HEADER).read()).group(1))
    s, n = shape_for(**kw), ctypes.c_size_t()
    assert lib.moe_workspace_bytes(ctypes.byref(s), ctypes.byref(n)) == 0
    assert n.value >= head
    rows, count = ctypes.c_void_p(), ctypes.c_int64()
    ws = 1 << 32
    assert lib.moe_routed_rows(ctypes.byref(s), ctypes.c_void_p(ws), n.value, ctypes.byref(rows),
                               ctypes.byref(count)) == 0
    assert head <= rows.value - ws <= n.value

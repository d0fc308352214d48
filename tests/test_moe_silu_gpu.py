"""SiLU as the tile kernel evaluates it has tq_silu's bits for every fp32 gate."""
import ctypes

import pytest

from _native import compile_library

pytestmark = pytest.mark.gpu


def test_every_gate(tmp_path):
    import torch
    lib = compile_library("silu_compare", tmp_path)
    lib.silu_compare.argtypes = [ctypes.c_void_p, ctypes.c_void_p]
    differ = torch.zeros(1, dtype=torch.int64, device="cuda")
    example = torch.zeros(1, dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    assert lib.silu_compare(differ.data_ptr(), example.data_ptr()) == 0
    torch.cuda.synchronize()
    assert int(differ) == 0, hex(int(example) & 0xffffffff)

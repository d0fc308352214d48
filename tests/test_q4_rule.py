"""Which form of the tile kernel a call of 4-bit products takes, and that its workspace holds either.  No GPU needed."""
import ctypes

import pytest

from _native import compile_library
from ternary_weight_dp4a_gb300 import build as tqbuild
from ternary_weight_dp4a_gb300 import tq

SMS = 152


@pytest.fixture(scope="module")
def rule(tmp_path_factory):
    lib = compile_library("q4_rule", tmp_path_factory.mktemp("native"))
    lib.scaled.argtypes = [ctypes.c_int, ctypes.c_int, ctypes.c_int, ctypes.c_longlong, ctypes.c_int]
    return lib


def test_the_rule_looks_at_the_tiles_that_would_run(rule):
    """With minima a scaled tile has 176 rows and a folded one 192: 177 to 192 rows are two tiles against one, and groups of
    64 are folded there, unless the two of every tile of the weights run at once."""
    assert rule.scaled_cols() == 176 and rule.tile_cols() == 192
    for m in range(17, 600):
        two = rule.row_tiles(m, 176) == 2 and rule.row_tiles(m, 192) == 1
        assert two == (177 <= m <= 192)
        for tiles in (1, SMS // 2, SMS // 2 + 1, 1024, 1 << 15):
            want = m > 64 and not (two and 2 * tiles > SMS)
            assert rule.scaled(m, 64, 1, tiles, SMS) == want, (m, tiles)
            assert rule.scaled(m, 32, 1, tiles, SMS) == (m > 32), m
            assert rule.scaled(m, 32, 0, tiles, SMS) == (m > 64) and rule.scaled(m, 64, 0, tiles, SMS) == (m > 96)
            assert not rule.scaled(m, 128, 0, tiles, SMS) and not rule.scaled(m, 128, 1, tiles, SMS)


def test_a_workspace_holds_what_either_form_writes(rule):
    tqbuild.build()
    lib, k = tq.load(), 1024
    for group in (32, 64, 128):
        for m in range(17, 600):
            have = lib.tq_q4_workspace_bytes(m, k, group)
            for tiles in (1, 1024):
                need = m * (k // 128) * 64 if rule.scaled(m, group, 1, tiles, SMS) else -(-m // 16) * 16 * (k // group) * 4
                assert have >= need, (group, m)

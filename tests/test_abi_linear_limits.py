"""Sizes at the ends of their types: refused before anything is launched, and never wrapped round."""
import ctypes

import pytest

import gated_delta_rule_31_gb300 as gdr
from gated_delta_rule_31_gb300 import LinearProblem, NormProblem

OK, INVALID, UNSUPPORTED, WORKSPACE = range(4)
FAKE = ctypes.c_void_p(0x100000)
BIG = ctypes.c_size_t((1 << 64) - 1)
LIMIT = 2 ** 31 - 2 ** 20  # of tokens


@pytest.fixture(scope="module")
def L():
    gdr.build()
    return gdr.lib()


@pytest.mark.parametrize("dtype", [0, 1])
@pytest.mark.parametrize("T", [LIMIT + 1, 2 ** 31 - 128, 2 ** 31 - 1])
def test_too_many_tokens(L, T, dtype):
    p = ctypes.byref(LinearProblem(1, T, 1, 1, 32, 32, dtype, 0.1))
    for f in (L.gdr_linear_fwd_workspace, L.gdr_linear_bwd_workspace, L.gdr_linear_states_bytes, L.gdr_linear_bwd_states_workspace):
        assert f(p) == 0
    assert L.gdr_linear_fwd(p, *[FAKE] * 8, FAKE, BIG, None) == UNSUPPORTED
    assert L.gdr_linear_bwd(p, *[FAKE] * 12, FAKE, BIG, None) == UNSUPPORTED


@pytest.mark.parametrize("heads", [1, 3, 40])
@pytest.mark.parametrize("T", [LIMIT, LIMIT - 1, LIMIT - 127, LIMIT - 128, 10 ** 9 + 7])
def test_as_many_tokens_as_there_can_be(L, T, heads):
    p = ctypes.byref(LinearProblem(1, T, 1, heads, 128, 128, 1, 0.1))
    chunks = (T + 127) // 128
    assert L.gdr_linear_states_bytes(p) == chunks * heads * 32768
    kept, both = L.gdr_linear_bwd_states_workspace(p), L.gdr_linear_bwd_workspace(p)
    segments = L.gdr_linear_fwd_workspace(p) - 256
    assert segments % (heads * 65536) == 0 and 1 <= segments // (heads * 65536) <= 1216
    assert kept == 256 + segments + chunks * heads * 32768
    assert both == kept + chunks * heads * 32768 + T * heads * 256


@pytest.mark.parametrize("rows,groups,D", [(2 ** 63 - 1, 1, 1), (2 ** 63 - 1, 2, 64), (2 ** 60 + 1, 1, 1), (2 ** 53 + 1, 2, 64)])
def test_too_many_rows(L, rows, groups, D):
    p = ctypes.byref(NormProblem(rows, groups, D, 1, 1, 1, 1e-5))
    assert L.gdr_group_norm_bwd_workspace(p) == 0
    assert L.gdr_group_norm_fwd(p, *[FAKE] * 5, None) == UNSUPPORTED
    assert L.gdr_group_norm_bwd(p, *[FAKE] * 9, FAKE, BIG, None) == UNSUPPORTED


def test_many_rows(L):
    assert 256 < L.gdr_group_norm_bwd_workspace(ctypes.byref(NormProblem(2 ** 40, 2, 64, 1, 1, 1, 1e-5))) < 2 ** 24

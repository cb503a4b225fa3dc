"""CPU checks of the hybrid step's entry points, of calls that they once refused or let pass."""
import ctypes

import pytest
import torch

from linear_attention_rule_b200 import kda
from tests.test_hybrid_refusals_cpu import INVALID, Rope, _append, _cache, _decode, _lib, _pool  # noqa: F401 (_lib: a fixture)

OK = kda.KDA_OK


@pytest.mark.parametrize("empty", [dict(T=0), dict(N=0), dict(N=0, T=0)])
def test_empty_steps_may_have_no_addresses(empty):
    """A tensor without elements has a null pointer: a step without tokens or sequences is nothing to do."""
    none = dict(q=None, k=None, v=None, out=None)
    assert _append(_cache(), **none, **empty) == OK
    assert _append(_cache(block_table=None, seq_lens=None), **none, **empty) == OK
    assert _append(_cache(), q=None, **{**empty, "Hq": 0}) == OK
    for axes, pairs in ((1, (16, 0, 0, 0)), (3, (8, 4, 4, 0))):
        rope = Rope(None, None, 32, axes, (ctypes.c_int32 * 4)(*pairs), 0)
        assert _append(_cache(), rope, **none, **empty) == OK
    assert _pool(**none, g=None, beta=None, sout=None, **empty) == OK
    assert _decode(_cache(), q=None, out=None, ws=None, ws_bytes=0, **empty) == OK


@pytest.mark.parametrize("empty", [dict(T=0), dict(N=0)])
def test_empty_steps_still_name_bad_sizes(empty):
    assert _append(_cache(), **{"Hq": -1, **empty}) == INVALID
    rope = Rope(None, None, 32, 5, (ctypes.c_int32 * 4)(16, 0, 0, 0), 0)
    assert _append(_cache(), rope, **empty) == INVALID
    rope = Rope(None, None, 32, 2, (ctypes.c_int32 * 4)(8, 4, 0, 0), 0)
    assert _append(_cache(), rope, **empty) == INVALID


def test_steps_with_tokens_want_their_addresses():
    rope = Rope(1 << 20, None, 32, 2, (ctypes.c_int32 * 4)(8, 8, 0, 0), 0)
    assert _append(_cache(), rope) == INVALID
    for bad in (dict(q=None), dict(out=None), dict(Hq=0), dict(k=None), dict(v=None)):
        assert _append(_cache(), **bad) == INVALID


@pytest.mark.parametrize("cap", [2.0 ** -149, 2.0 ** -127, 2.0 ** -101, 2.0 ** 101, 2.0 ** 126, 3.4e38])
def test_decode_refuses_caps_that_it_cannot_divide_by(cap):
    """Far out the quotient of scale and cap loses its bits or overflows (0 times infinity for a score of 0)."""
    assert _decode(_cache(), cap=cap) == kda.KDA_ERR_UNSUPPORTED


@pytest.mark.parametrize("cap", [2.0 ** -100, 2.0 ** 100])
def test_decode_takes_caps_up_to_there(cap):
    assert _decode(_cache(), cap=cap, N=0) == OK

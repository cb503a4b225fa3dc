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


def test_strides_of_axes_of_one_do_not_matter():
    """One kv head, one page or pages of one row: the stride of such an axis is used by nothing, and torch
    gives it different values by how a tensor came about.  On the CPU the call ends at the device check."""
    D = 64
    k = torch.zeros(6, 16, D)
    for pages, a, b in ((6, k.unsqueeze(1), k.as_strided((6, 1, 16, D), (16 * D, 7 * D, D, 1))),
                        (1, k[:1].unsqueeze(1), k.as_strided((1, 1, 16, D), (3, 5, D, 1))),
                        (1, torch.zeros(1, 1, 1, D), k.as_strided((1, 1, 1, D), (9 * D, 9 * D, 9 * D, 1)))):
        ps = a.shape[2]
        for kc, vc in ((a, b), (b, a)):
            assert kc.stride() != vc.stride()
            with pytest.raises(ValueError, match="must be on"):
                kda.kda_kv_append(k=torch.zeros(4, 1, D), v=torch.zeros(4, 1, D), k_cache=kc, v_cache=vc, block_table=torch.zeros(4, 3, dtype=torch.int32),
                                  seq_lens=torch.zeros(4, dtype=torch.int32))
    with pytest.raises(ValueError, match="strides"):   # those of longer axes do
        kda.kda_kv_append(k=torch.zeros(4, 1, D), v=torch.zeros(4, 1, D), k_cache=k.unsqueeze(1), v_cache=torch.zeros(6, 32, D)[:, ::2].unsqueeze(1),
                          block_table=torch.zeros(4, 3, dtype=torch.int32), seq_lens=torch.zeros(4, dtype=torch.int32))

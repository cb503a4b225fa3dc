"""CPU checks of the hybrid step's entry points: the C calls reject bad arguments with a status before
anything is launched, and the Python ones raise before any pointer reaches the library."""
import ctypes

import pytest
import torch

from linear_attention_rule_b200 import kda

P = ctypes.c_void_p
A = 1 << 20   # an aligned address that is never looked at
INVALID, UNSUPPORTED = kda.KDA_ERR_INVALID_ARG, kda.KDA_ERR_UNSUPPORTED


class Cache(ctypes.Structure):   # kda_kv_cache
    _fields_ = [("k", P), ("v", P), ("k_scale", P), ("v_scale", P), ("block_table", P), ("seq_lens", P),
                ("page_stride", ctypes.c_int64), ("head_stride", ctypes.c_int64), ("row_stride", ctypes.c_int64),
                ("table_stride", ctypes.c_int64), ("num_pages", ctypes.c_int32), ("page_size", ctypes.c_int32),
                ("max_pages", ctypes.c_int32), ("Hkv", ctypes.c_int32), ("D", ctypes.c_int32), ("dt", ctypes.c_int)]


class Rope(ctypes.Structure):   # kda_rope
    _fields_ = [("inv_freq", P), ("positions", P), ("rot_dim", ctypes.c_int32), ("num_axes", ctypes.c_int32),
                ("axis_pairs", ctypes.c_int32 * 4), ("adjacent", ctypes.c_int32)]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from linear_attention_rule_b200 import build
    build.build()
    kda.load()


def _pool(**kw):
    a = dict(q=A, k=A, v=A, g=A, beta=A, qs=128, ks=128, vs=256, pool=A, slots=4, sin=A, sout=A, cu=A, N=2, T=3, Hk=2, Hv=4,
             dk=64, dv=64, dt=kda.KDA_F32, out=A, flags=0, stream=None)
    a.update(kw)
    return kda.load().kda_decode_pool(*a.values())


@pytest.mark.parametrize("bad,status", [
    (dict(N=-1), INVALID), (dict(T=-1), INVALID), (dict(slots=-1), INVALID), (dict(Hk=0), INVALID), (dict(Hv=3), INVALID),
    (dict(Hv=0), INVALID), (dict(flags=64), INVALID), (dict(dt=kda.KDA_E4M3), INVALID), (dict(cu=None), INVALID),
    (dict(cu=A + 2), INVALID), (dict(dk=96, dv=96), UNSUPPORTED), (dict(dv=128), UNSUPPORTED), (dict(T=1 << 31), UNSUPPORTED),
    (dict(N=1 << 30), UNSUPPORTED), (dict(q=None), INVALID), (dict(k=A + 8), INVALID), (dict(pool=A + 4), INVALID),
    (dict(pool=None), INVALID), (dict(sin=None), INVALID), (dict(sout=A + 1), INVALID), (dict(g=A + 2), INVALID),
    (dict(out=A + 8), INVALID), (dict(qs=124), INVALID), (dict(ks=130), INVALID), (dict(vs=255), INVALID),
])
def test_pool_refuses(bad, status):
    assert _pool(**bad) == status


def _cache(**kw):
    a = dict(k=A, v=A, k_scale=None, v_scale=None, block_table=A, seq_lens=A, page_stride=2 * 16 * 64, head_stride=16 * 64,
             row_stride=64, table_stride=8, num_pages=9, page_size=16, max_pages=8, Hkv=2, D=64, dt=kda.KDA_BF16)
    a.update(kw)
    return Cache(*a.values())


CACHE_REFUSALS = [
    (dict(num_pages=-1), INVALID), (dict(max_pages=-1), INVALID), (dict(Hkv=0), INVALID), (dict(page_size=0), INVALID),
    (dict(page_size=24), UNSUPPORTED), (dict(page_size=8192), UNSUPPORTED), (dict(D=96, row_stride=96), UNSUPPORTED),
    (dict(dt=kda.KDA_F32), UNSUPPORTED), (dict(dt=5), INVALID), (dict(seq_lens=None), INVALID), (dict(block_table=None), INVALID),
    (dict(k=None), INVALID), (dict(v=A + 8), INVALID), (dict(block_table=A + 2), INVALID), (dict(k_scale=A), INVALID),
    (dict(row_stride=32), INVALID), (dict(head_stride=1025), INVALID), (dict(page_stride=1), INVALID), (dict(table_stride=7), INVALID),
    (dict(dt=kda.KDA_E4M3, k_scale=A + 1), INVALID), (dict(dt=kda.KDA_E4M3, row_stride=72), INVALID),
]


def _append(c, rope=None, **kw):
    a = dict(k=A, v=A, q=A, ks=128, vs=128, qs=256, dt=kda.KDA_BF16, cache=ctypes.byref(c), cu=A, N=2, T=3, Hq=4,
             rope=None if rope is None else ctypes.byref(rope), out=A + 4096, stream=None)
    a.update(kw)
    return kda.load().kda_kv_append(*a.values())


@pytest.mark.parametrize("bad,status", CACHE_REFUSALS)
def test_append_refuses_caches(bad, status):
    assert _append(_cache(**bad)) == status


@pytest.mark.parametrize("bad,status", [
    (dict(N=-1), INVALID), (dict(T=-1), INVALID), (dict(dt=kda.KDA_E4M3), INVALID), (dict(Hq=-1), INVALID), (dict(Hq=0), INVALID),
    (dict(q=None), INVALID), (dict(out=None), INVALID), (dict(cu=None), INVALID), (dict(T=1 << 31), UNSUPPORTED),
    (dict(k=None), INVALID), (dict(v=A + 2), INVALID), (dict(qs=192), INVALID), (dict(ks=120), INVALID), (dict(vs=132), INVALID),
    (dict(out=A, qs=512), INVALID),   # in place only when dense
    (dict(cache=None), INVALID),
])
def test_append_refuses(bad, status):
    assert _append(_cache(), **bad) == status


@pytest.mark.parametrize("bad", [dict(rot_dim=0), dict(rot_dim=24), dict(rot_dim=80), dict(num_axes=0), dict(num_axes=5),
                                 dict(axis_pairs=(8, 0, 0, 0)), dict(axis_pairs=(-8, 24, 0, 0), num_axes=2),
                                 dict(axis_pairs=(8, 8, 0, 0), num_axes=2, positions=None), dict(axis_pairs=(2 ** 31 - 1, 0, 0, 0)),
                                 dict(inv_freq=None), dict(inv_freq=A + 2), dict(positions=A + 1)])
def test_append_refuses_rotations(bad):
    a = dict(inv_freq=A, positions=A, rot_dim=32, num_axes=1, axis_pairs=(16, 0, 0, 0), adjacent=0)
    a.update(bad)
    a["axis_pairs"] = (ctypes.c_int32 * 4)(*a["axis_pairs"])
    assert _append(_cache(), Rope(*a.values())) == INVALID


def _decode(c, **kw):
    a = dict(q=A, qs=256, dt=kda.KDA_BF16, cache=ctypes.byref(c), cu=A, N=2, T=3, max_q=2, Hq=4, scale=0.1, cap=0.0, window=0,
             slopes=None, start=None, out=A, lse=None, ws=A, ws_bytes=1 << 30, stream=None)
    a.update(kw)
    return kda.load().kda_kv_decode(*a.values())


@pytest.mark.parametrize("bad,status", CACHE_REFUSALS + [(dict(dt=kda.KDA_E4M3, page_size=1), UNSUPPORTED)])
def test_decode_refuses_caches(bad, status):
    assert _decode(_cache(**bad)) == status


@pytest.mark.parametrize("bad,status", [
    (dict(N=-1), INVALID), (dict(Hq=0), INVALID), (dict(Hq=3), INVALID), (dict(max_q=0), INVALID), (dict(max_q=17), UNSUPPORTED),
    (dict(Hq=1 << 17, qs=1 << 23), UNSUPPORTED), (dict(window=-1), INVALID), (dict(cap=-1.0), INVALID), (dict(cap=float("nan")), INVALID),
    (dict(cap=float("inf")), INVALID), (dict(scale=float("nan")), INVALID), (dict(scale=float("inf")), INVALID),
    (dict(q=None), INVALID), (dict(q=A + 8), INVALID), (dict(out=A + 2), INVALID), (dict(qs=252), INVALID), (dict(slopes=A + 1), INVALID),
    (dict(start=A + 2), INVALID), (dict(lse=A + 2), INVALID), (dict(ws=None), INVALID), (dict(ws=A + 128), INVALID),
    (dict(ws_bytes=1000), INVALID), (dict(cu=None), INVALID), (dict(cache=None), INVALID),
])
def test_decode_refuses(bad, status):
    assert _decode(_cache(), **bad) == status


def test_empty_calls_are_fine():
    assert _pool(N=0) == kda.KDA_OK and _pool(T=0) == kda.KDA_OK
    assert _append(_cache(), T=0) == kda.KDA_OK and _decode(_cache(), N=0) == kda.KDA_OK


def test_decode_workspace_size():
    size = kda.kda_kv_decode_workspace_size
    assert size(4, 8, 2, 128, 1) > 0
    assert size(4, 8, 2, 128, 16) >= size(4, 8, 2, 128, 4) >= size(4, 8, 2, 128, 1)
    for bad in ((-1, 8, 2, 128, 1), (4, 0, 2, 128, 1), (4, 8, 0, 128, 1), (4, 8, 3, 128, 1), (4, 8, 2, 96, 1), (4, 8, 2, 128, 0),
                (4, 8, 2, 128, 17)):
        assert size(*bad) == 0


# ------------------------------------------------------------------------------- the Python calls

def _ints(*shape):
    return torch.zeros(shape, dtype=torch.int32)


def _pool_args(**kw):
    T, Hk, Hv, D = 4, 1, 2, 64
    a = dict(q=torch.zeros(T, Hk, D), k=torch.zeros(T, Hk, D), v=torch.zeros(T, Hv, D), g=torch.zeros(T, Hv, D),
             beta=torch.zeros(T, Hv), state_pool=torch.zeros(5, Hv, D, D), slots_in=_ints(2), slots_out=_ints(T),
             out=torch.zeros(T, Hv, D), cu_seqlens=_ints(3))
    a.update(kw)
    return a


@pytest.mark.parametrize("bad,exc,match", [
    ({}, ValueError, "must be on"), (dict(k=torch.zeros(3, 1, 64)), ValueError, "shape"), (dict(q=None), TypeError, "Tensor"),
    (dict(q=torch.zeros(4, 1, 64, dtype=torch.float16)), TypeError, "float32 or bfloat16"), (dict(v=torch.zeros(4, 2, 64).double()), TypeError, "v must"),
    (dict(g=torch.zeros(4, 2)), ValueError, "shape"), (dict(in_flags=kda.KDA_IN_G_SCALAR), ValueError, "shape"),
    (dict(slots_in=_ints(3)), ValueError, "shape"), (dict(slots_out=_ints(4).long()), TypeError, "slots_out"), (dict(slots_out=None), TypeError, "slots_out"),
    (dict(state_pool=torch.zeros(5, 2, 64, 128)), ValueError, "shape"), (dict(state_pool=torch.zeros(5, 2, 64, 64).transpose(2, 3)), ValueError, "contiguous"),
    (dict(out=torch.zeros(4, 2, 64, dtype=torch.bfloat16)), TypeError, "out must"), (dict(cu_seqlens=_ints(3, 1)), ValueError, "cu_seqlens"),
    (dict(q=torch.zeros(4, 64, 1).transpose(1, 2)[:, :, ::2]), ValueError, "dense"), (dict(in_flags=-1), ValueError, "in_flags"),
    (dict(beta=torch.zeros(4, 2)[:, :1]), ValueError, "shape"),
])
def test_pool_binding_checks(bad, exc, match):
    with pytest.raises(exc, match=match):
        kda.kda_decode_pool(**_pool_args(**bad))


def _append_args(**kw):
    T, H, D = 4, 2, 64
    a = dict(k=torch.zeros(T, H, D), v=torch.zeros(T, H, D), k_cache=torch.zeros(6, H, 16, D), v_cache=torch.zeros(6, H, 16, D),
             block_table=_ints(4, 3), seq_lens=_ints(4))
    a.update(kw)
    return a


F = torch.zeros(16)


@pytest.mark.parametrize("bad,exc,match", [
    ({}, ValueError, "must be on"), (dict(v=torch.zeros(4, 1, 64)), ValueError, "shape"), (dict(k_cache=torch.zeros(6, 2, 16)), ValueError, "k_cache"),
    (dict(k_cache=torch.zeros(6, 2, 16, 64).double()), ValueError, "k_cache"), (dict(v_cache=torch.zeros(6, 16, 2, 64).transpose(1, 2)), ValueError, "strides"),
    (dict(k_cache=torch.zeros(6, 1, 16, 64), v_cache=torch.zeros(6, 1, 16, 64)), ValueError, "heads"),
    (dict(block_table=_ints(4, 3).long()), ValueError, "block_table"), (dict(block_table=_ints(3, 3)), ValueError, "block_table"),
    (dict(block_table=_ints(3, 4).t()), ValueError, "block_table"), (dict(seq_lens=None), TypeError, "seq_lens"), (dict(seq_lens=_ints(3)), ValueError, "shape"),
    (dict(positions=_ints(4)), ValueError, "inv_freq"), (dict(axis_pairs=(4,)), ValueError, "inv_freq"),
    (dict(inv_freq=F, positions=_ints(3, 4)), ValueError, "axis_pairs"), (dict(inv_freq=F, positions=_ints(3, 4), axis_pairs=(8, 8)), ValueError, "axis_pairs"),
    (dict(inv_freq=F, positions=_ints(5, 4), axis_pairs=(4, 4, 4, 2, 2)), ValueError, "axis_pairs"), (dict(inv_freq=F, positions=_ints(5)), ValueError, "shape"),
    (dict(inv_freq=F.double()), TypeError, "inv_freq"), (dict(inv_freq=F, positions=_ints(1, 1, 4)), ValueError, "positions"),
    (dict(q_out=torch.zeros(4, 2, 64)), ValueError, "q_out"), (dict(k_scale=torch.zeros(3)), ValueError, "shape"),
    (dict(inv_freq=F, axis_pairs=("a",)), TypeError, "."),
])
def test_append_binding_checks(bad, exc, match):
    with pytest.raises(exc, match=match):
        kda.kda_kv_append(**_append_args(**bad))


@pytest.mark.parametrize("bad,exc,match", [
    ({}, ValueError, "must be on"), (dict(q=torch.zeros(4, 3, 64)), ValueError, "divide"), (dict(q=torch.zeros(4, 64)), ValueError, "q must be"),
    (dict(q=torch.zeros(4, 4, 128)), ValueError, "channels"), (dict(out=torch.zeros(4, 2, 64)), ValueError, "shape"),
    (dict(lse=torch.zeros(4, 3)), ValueError, "shape"), (dict(alibi_slopes=torch.zeros(2)), ValueError, "shape"), (dict(kv_start=_ints(3)), ValueError, "shape"),
    (dict(workspace=torch.zeros(9)), TypeError, "workspace"), (dict(max_q=1 << 40), ValueError, "max_q"), (dict(scale="x"), TypeError, "."),
])
def test_decode_binding_checks(bad, exc, match):
    a = dict(q=torch.zeros(4, 4, 64), k_cache=torch.zeros(6, 2, 16, 64), v_cache=torch.zeros(6, 2, 16, 64), block_table=_ints(4, 3),
             seq_lens=_ints(4), out=torch.zeros(4, 4, 64), workspace=torch.zeros(1 << 10, dtype=torch.uint8))
    a.update(bad)
    with pytest.raises(exc, match=match):
        kda.kda_kv_decode(**a)


@pytest.mark.parametrize("cu", [[0, 1, 2, 3, 4], 4])
def test_decode_without_a_workspace_names_a_bad_argument(cu):
    with pytest.raises(ValueError, match="cu_seqlens"):
        kda.kda_kv_decode(q=torch.zeros(4, 4, 64), k_cache=torch.zeros(6, 2, 16, 64), v_cache=torch.zeros(6, 2, 16, 64),
                          block_table=_ints(4, 3), seq_lens=_ints(4), out=torch.zeros(4, 4, 64), cu_seqlens=cu)

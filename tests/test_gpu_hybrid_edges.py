"""The hybrid step's operators where they can go wrong: pages smaller than a tile's parts, row blocks and
stretches of every kind, many short sequences, extreme scores and queries, bad values in the cache."""
import math

import pytest
import torch

from linear_attention_rule_b200 import kda
from tests import hybrid_reference as ref
from tests.test_gpu_hybrid_step import BF16, E4M3, F32, _attend_inputs, _cu, _ints, _new_cache, _ok, _pool_inputs, _within

pytestmark = pytest.mark.gpu


def _attend(q, kc, vc, table, sl, lens, ks, vs, max_q=None, **opt):
    T, Hq, D = sum(lens), q.shape[1], q.shape[2]
    out = torch.full((T, Hq, D), 7.0, dtype=q.dtype, device="cuda")
    lse = torch.full((T, Hq), 7.0, device="cuda")
    kda.kda_kv_decode(q[:T], kc, vc, table, sl, out, cu_seqlens=_cu(lens), max_q=max_q or max(lens + [1]), lse=lse, k_scale=ks, v_scale=vs, **opt)
    _ok()
    return out, lse


def _matches(q, kc, vc, table, sl, lens, ks, vs, scale=None, cap=0.0, window=0, slopes=None, start=None):
    D = q.shape[2]
    out, lse = _attend(q, kc, vc, table, sl, lens, ks, vs, scale=scale, softcap=cap, window=window, alibi_slopes=slopes,
                       kv_start=None if start is None else _ints(start))
    T = sum(lens)
    o, l, ob, lb = ref.attend(q[:T], kc, vc, table, sl, lens, D ** -0.5 if scale is None else scale, cap, window, slopes, start, ks, vs)
    seen = torch.isfinite(l)
    _within(out, o, ob)
    _within(lse.cpu()[seen], l[seen], lb[seen])
    assert (lse.cpu()[~seen] == -math.inf).all() and (out.cpu()[~seen] == 0).all()
    return out, lse


@pytest.mark.parametrize("dtype,cdt,D,ps", [(BF16, BF16, 128, 1), (BF16, BF16, 64, 2), (BF16, BF16, 128, 4), (BF16, E4M3, 128, 1),
                                            (BF16, E4M3, 64, 2), (BF16, E4M3, 64, 4), (BF16, E4M3, 128, 256), (F32, F32, 128, 1),
                                            (F32, F32, 64, 2), (F32, F32, 128, 4), (F32, F32, 64, 512), (BF16, BF16, 128, 4096)])
@pytest.mark.parametrize("order", ["heads", "rows"])
def test_pages_of_any_size(dtype, cdt, D, ps, order):
    seq, lens = [1, 130, 37], [1, 2, 1]
    q, kc, vc, table, sl, (ks, vs) = _attend_inputs(dtype, cdt, D, 4, 2, ps, order, seq, lens)
    _matches(q, kc, vc, table, sl, lens, ks, vs)
    _matches(q, kc, vc, table, sl, lens, ks, vs, window=20)


def test_a_page_of_one_64_byte_row_is_refused():
    q, kc, vc, table, sl, (ks, vs) = _attend_inputs(BF16, E4M3, 64, 2, 1, 1, "heads", [3], [1])
    with pytest.raises(kda.KdaError) as e:
        _attend(q, kc, vc, table, sl, [1], ks, vs)
    assert e.value.status == kda.KDA_ERR_UNSUPPORTED


@pytest.mark.parametrize("dtype,cdt", [(BF16, BF16), (BF16, E4M3), (F32, F32)])
@pytest.mark.parametrize("D,Hq,Hkv,new", [(64, 2, 1, 5), (128, 16, 1, 2), (64, 20, 1, 2), (128, 12, 2, 5), (64, 16, 1, 4), (128, 16, 1, 5),
                                          (64, 48, 2, 6), (128, 3, 3, 1)])
def test_row_blocks_split_over_stretches(dtype, cdt, D, Hq, Hkv, new):
    """10 to 144 query rows a kv head in blocks of every size, sequences split at every kind of place;
    the same bits each time."""
    seq = [3000, new, 640, 127 + new, 1025, 32]
    lens = [new, new, 1, new, max(1, new - 1), new]
    q, kc, vc, table, sl, (ks, vs) = _attend_inputs(dtype, cdt, D, Hq, Hkv, 64, "heads", seq, lens)
    out, lse = _matches(q, kc, vc, table, sl, lens, ks, vs)
    for _ in range(12):
        o2, l2 = _attend(q, kc, vc, table, sl, lens, ks, vs)
        assert torch.equal(out, o2) and torch.equal(lse, l2)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Hq,new", [(2, 1), (2, 2), (6, 1), (8, 1), (10, 1), (8, 2), (6, 3)])
def test_fp32_rows_in_groups(D, Hq, new):
    """1 to 9 rows a kv head: one row, two, groups of four that are full or not; sequences without a visible
    key, split ones, and bad values where a row does not see."""
    seq, lens = [2500, 3 + new, 190, 64], [new, new, 1, new]
    q, kc, vc, table, sl, _ = _attend_inputs(F32, F32, D, Hq, 2, 16, "heads", seq, lens)
    slopes = 0.5 ** torch.arange(1, Hq + 1, device="cuda", dtype=torch.float32)
    _matches(q, kc, vc, table, sl, lens, None, None, slopes=slopes, start=[0, 2, 190, 63])
    _matches(q, kc, vc, table, sl, lens, None, None, cap=4.0, window=70, slopes=slopes, start=[2400, 0, 7, 64])
    clean, _ = _attend(q, kc, vc, table, sl, lens, None, None, kv_start=_ints([2450, 0, 0, 60]))
    for c in (kc, vc):   # before the first visible keys, in their pages
        c[table[0, 2449 // 16].long(), :, : 2450 % 16] = math.nan
        c[table[3, 59 // 16].long(), :, : 60 % 16] = -math.inf
    out, _ = _attend(q, kc, vc, table, sl, lens, None, None, kv_start=_ints([2450, 0, 0, 60]))
    assert torch.equal(out, clean)


@pytest.mark.parametrize("dtype,cdt", [(BF16, BF16), (BF16, E4M3), (F32, F32)])
def test_many_short_sequences(dtype, cdt):
    """More sequences than the table of work has entries, a third of them without new tokens."""
    gen = torch.Generator().manual_seed(8)
    N = 2500
    seq = torch.randint(1, 40, (N,), generator=gen).tolist()
    lens = [min(int(x), s) for x, s in zip(torch.randint(0, 3, (N,), generator=gen), seq)]
    q, kc, vc, table, sl, (ks, vs) = _attend_inputs(dtype, cdt, 64, 2, 1, 16, "heads", seq, lens)
    _matches(q, kc, vc, table, sl, lens, ks, vs)


def test_no_sequence_has_new_tokens():
    q, kc, vc, table, sl, _ = _attend_inputs(BF16, BF16, 64, 2, 1, 16, "heads", [40, 3], [1, 1])
    out = torch.full((2, 2, 64), 7.0, dtype=BF16, device="cuda")
    kda.kda_kv_decode(q, kc, vc, table, sl, out, cu_seqlens=_ints([0, 0, 0]))
    _ok()
    assert (out == 7).all()


@pytest.mark.parametrize("dtype,cdt", [(BF16, BF16), (BF16, E4M3), (F32, F32)])
@pytest.mark.parametrize("scale,cap", [(3.0, 2.0), (0.5, 50.0), (0.0, 0.0), (-0.3, 5.0), (8.0, 0.0)])
def test_scores_far_from_one(dtype, cdt, scale, cap):
    """Scores into and far below the cap, all equal, of the other sign, hundreds apart."""
    seq, lens = [300, 65], [2, 1]
    q, kc, vc, table, sl, (ks, vs) = _attend_inputs(dtype, cdt, 128, 4, 2, 32, "heads", seq, lens)
    _matches(q, kc, vc, table, sl, lens, ks, vs, scale=scale, cap=cap)


@pytest.mark.parametrize("dtype,cdt", [(BF16, BF16), (BF16, E4M3), (F32, F32)])
def test_queries_of_all_sizes(dtype, cdt):
    """Rows of zeros, tiny and huge ones, and one large channel beside small ones."""
    seq, lens = [200] * 4, [1] * 4
    q, kc, vc, table, sl, (ks, vs) = _attend_inputs(dtype, cdt, 64, 4, 2, 16, "heads", seq, lens)
    q = q.clone()
    q[0] = 0
    q[1] *= 2.0 ** -100
    q[2] *= 2.0 ** 8
    q[3, :, 5] = 3.0
    q[3, :, 6:] *= 2.0 ** -7
    _matches(q, kc, vc, table, sl, lens, ks, vs)
    q[1] *= 2.0 ** 100
    _matches(q, kc, vc, table, sl, lens, ks, vs)


@pytest.mark.parametrize("dtype,cdt", [(BF16, BF16), (BF16, E4M3), (F32, F32)])
def test_a_sink_and_a_long_tail(dtype, cdt):
    """One key with half of the weight, the rest shared by thousands: each of those counts."""
    seq, lens, D = [6000], [1], 64
    q, kc, vc, table, sl, (ks, vs) = _attend_inputs(dtype, cdt, D, 2, 1, 64, "heads", seq, lens)
    page, row = table[0].long()[torch.arange(6000, device="cuda") // 64], torch.arange(6000, device="cuda") % 64
    kc[page, :, row] = (0.05 * torch.randn(6000, 1, D, device="cuda") / (ks.max() if ks is not None else 1)).to(cdt)
    # a key along the query with a score of 9
    one = q[0, 0].float() / q[0, 0].float().square().sum() * 9.0 * D ** 0.5
    kc[page[1234], :, row[1234]] = (one / (ks[:, None] if ks is not None else 1)).to(cdt)
    q[0, 1] = q[0, 0]
    _matches(q, kc, vc, table, sl, lens, ks, vs)


def test_rising_maxima():
    """Scores that grow along the keys, so that every tile raises the maximum; and that fall."""
    seq, lens, D = [900, 900], [3, 3], 64
    for cdt in (BF16, E4M3):
        q, kc, vc, table, sl, (ks, vs) = _attend_inputs(BF16, cdt, D, 4, 1, 64, "heads", seq, lens)
        slopes = torch.tensor([0.1, 0.02, -0.1, -0.02], device="cuda")
        _matches(q, kc, vc, table, sl, lens, ks, vs, slopes=slopes)


@pytest.mark.parametrize("cdt", [BF16, F32])
def test_infinite_values_keep_to_their_channel_and_rows(cdt):
    """Infinities among the values of the newest keys, seen by some of the tokens: their channel is
    infinite (or NaN, where both signs meet) for those tokens, all else is as the formula has it."""
    seq, lens, D, Hq = [300], [6], 128, 4
    q, kc, vc, table, sl, _ = _attend_inputs(cdt, cdt, D, Hq, 2, 16, "heads", seq, lens)
    at = lambda j: (int(table[0, j // 16]), j % 16)
    p, r = at(296)   # seen by tokens 2 .. 5
    vc[p, 0, r, 7] = math.inf
    vc[p, 1, r, 100] = -math.inf
    p, r = at(298)   # seen by tokens 4 and 5
    vc[p, 0, r, 7] = -math.inf
    vc[p, 1, r, 9] = math.nan
    out, _ = _attend(q, kc, vc, table, sl, lens, None, None)
    clean = vc.clone()
    clean[~torch.isfinite(clean)] = 0
    o, _, ob, _ = ref.attend(q, kc, clean, table, sl, lens, D ** -0.5)
    want = o.clone()
    want[2:4, :2, 7] = math.inf
    want[4:6, :2, 7] = math.nan
    want[2:6, 2:, 100] = -math.inf
    want[4:6, 2:, 9] = math.nan
    got = out.double().cpu()
    fin = torch.isfinite(want)
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    assert torch.equal(got[torch.isinf(want)], want[torch.isinf(want)])
    assert ((got - o).abs()[fin] <= ob[fin]).all()


@pytest.mark.parametrize("dtype,cdt", [(BF16, BF16), (BF16, E4M3), (F32, F32)])
def test_nan_at_the_windows_rear_and_in_bad_pages(dtype, cdt):
    """Keys that only the oldest of the new tokens still sees; a page that is missing in the middle."""
    seq, lens, D, Hq = [400, 333], [5, 2], 64, 6
    q, kc, vc, table, sl, (ks, vs) = _attend_inputs(dtype, cdt, D, Hq, 2, 16, "heads", seq, lens)
    clean, _ = _attend(q, kc, vc, table, sl, lens, ks, vs, window=150)
    j = 395 - 149   # the first key of token 0 (position 395), of no other
    for c in (kc, vc):
        c[int(table[0, j // 16]), :, j % 16] = float("nan")
    out, _ = _attend(q, kc, vc, table, sl, lens, ks, vs, window=150)
    assert torch.equal(out[1:], clean[1:]) and not torch.isfinite(out[0].float()).all(-1).any()
    t2 = table.clone()
    t2[0, j // 16] = -1
    t2[1, 12] = kc.shape[0] + 3
    out = torch.zeros_like(clean)
    kda.kda_kv_decode(q, kc, vc, t2, sl, out, cu_seqlens=_cu(lens), max_q=5, window=150, k_scale=ks, v_scale=vs)
    assert kda.kda_get_device_status() == kda.KDA_ERR_BAD_PAGE
    o, _, ob, _ = ref.attend(q, kc, vc, t2, sl, lens, D ** -0.5, 0.0, 150, None, None, ks, vs)
    _within(out, o, ob)
    _ok()


def test_workspaces_hold_what_earlier_calls_left():
    """One workspace for calls of other shapes in turn, filled with NaN in between."""
    ws = torch.full((64 << 18,), float("nan"), device="cuda").view(torch.uint8)
    for dtype, cdt, D, Hq, Hkv, new in ((BF16, BF16, 128, 16, 1, 5), (F32, F32, 64, 2, 2, 1), (BF16, E4M3, 64, 8, 2, 3), (BF16, BF16, 64, 4, 2, 1)):
        seq, lens = [2000, 500, new], [new] * 3
        q, kc, vc, table, sl, (ks, vs) = _attend_inputs(dtype, cdt, D, Hq, Hkv, 16, "heads", seq, lens)
        a, la = _attend(q, kc, vc, table, sl, lens, ks, vs)
        b, lb = _attend(q, kc, vc, table, sl, lens, ks, vs, workspace=ws)
        ws.view(torch.float32).fill_(float("nan"))
        c, lc = _attend(q, kc, vc, table, sl, lens, ks, vs, workspace=ws)
        assert torch.equal(a, b) and torch.equal(a, c) and torch.equal(la, lb) and torch.equal(la, lc)


# ------------------------------------------------------------------------------- appending

@pytest.mark.parametrize("dtype,cdt", [(BF16, BF16), (BF16, E4M3), (F32, F32)])
def test_append_of_many_tokens_has_the_bits_of_few(dtype, cdt):
    """A call for 2,500 tokens (a warp each), in three (two warps a token) and in tens (four)."""
    gen = torch.Generator().manual_seed(4)
    T, Hq, Hkv, D, ps = 2500, 5, 3, 128, 16
    q, k, v = (torch.randn(T, h, D, generator=gen).to(dtype).cuda() for h in (Hq, Hkv, Hkv))
    inv = (10000.0 ** (-torch.arange(32, dtype=torch.float64) / 32)).float().cuda()
    table = torch.randperm(160, generator=gen).to(torch.int32).view(1, -1).cuda()
    sc = [torch.full((Hkv,), 0.013, device="cuda")] * 2 if cdt == E4M3 else [None, None]
    results = []
    for step in (2500, 1300, 37):
        kc, vc = _new_cache(160, Hkv, ps, D, cdt, fill=0.0)
        outs = []
        for i in range(0, T, step):
            n = min(step, T - i)
            outs.append(kda.kda_kv_append(k[i:i + n], v[i:i + n], kc, vc, table, _ints([i + n]), cu_seqlens=_ints([0, n]), q=q[i:i + n],
                                          inv_freq=inv, k_scale=sc[0], v_scale=sc[1]))
        results.append((torch.cat(outs), kc.float(), vc.float()))
    _ok()
    for r in results[1:]:
        assert all(torch.equal(x, y) for x, y in zip(r, results[0]))


def test_append_of_extreme_values_in_8_bits():
    """Infinities and large values are held at 448 scales, NaN stays NaN, quotients are rounded once."""
    gen = torch.Generator().manual_seed(6)
    H, D = 2, 64
    x = torch.randn(300, H, D, generator=gen).mul(torch.logspace(-6, 6, 300)[:, None, None]).to(BF16).cuda()
    x[0, 0, 0], x[0, 0, 1], x[0, 1, 2], x[1, 0, 5] = math.inf, -math.inf, math.nan, 3e38
    kc, vc = _new_cache(20, H, 16, D, E4M3, fill=0.0)
    sc = torch.tensor([0.0123, 1.0 / 3], device="cuda")
    kda.kda_kv_append(x, x, kc, vc, _ints([list(range(20))]), _ints([300]), cu_seqlens=_ints([0, 300]), k_scale=sc, v_scale=sc)
    _ok()
    want = (x.float() / sc[:, None]).clamp(-448, 448).to(E4M3).float()
    j = torch.arange(300, device="cuda")
    for c in (kc, vc):
        got = c[j // 16, :, j % 16].float()
        assert torch.equal(torch.isnan(got), torch.isnan(x.float()))
        ok = ~torch.isnan(got)
        assert torch.equal(got[ok], want[ok])


# ------------------------------------------------------------------------------- the state pool

@pytest.mark.parametrize("dtype,D", [(BF16, 128), (F32, 64)])
def test_pool_many_tokens_have_the_bits_of_one_by_one(dtype, D):
    """13 tokens in a call (groups of four, the last partial) and in 13 calls."""
    lens, Hv = [13, 5], 2
    q, k, v, g, b, pool, order = _pool_inputs(lens, 1, Hv, D, dtype, 3, raw=True)
    flags = kda.KDA_IN_NORMALIZE_QK | kda.KDA_IN_G_LOGITS | kda.KDA_IN_BETA_LOGITS
    T = 18
    keep = order[2:2 + T].cuda()
    one, out = pool.clone(), torch.empty(T, Hv, D, dtype=dtype, device="cuda")
    kda.kda_decode_pool(q, k, v, g, b, one, order[:2].cuda(), keep, out, cu_seqlens=_cu(lens), in_flags=flags)
    two = pool.clone()
    for n, (t0, length) in enumerate(((0, 13), (13, 5))):
        for i in range(length):
            t = t0 + i
            o = torch.empty(1, Hv, D, dtype=dtype, device="cuda")
            src = order[n:n + 1].cuda() if i == 0 else keep[t - 1:t]
            kda.kda_decode_pool(q[t:t + 1], k[t:t + 1], v[t:t + 1], g[t:t + 1], b[t:t + 1], two, src, keep[t:t + 1], o, in_flags=flags)
            assert torch.equal(o[0], out[t])
    _ok()
    assert torch.equal(one, two)

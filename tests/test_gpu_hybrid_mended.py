"""The hybrid step's operators in calls that they once answered wrongly, or that nothing had tested."""
import math

import pytest
import torch

from linear_attention_rule_b200 import kda
from tests import hybrid_reference as ref
from tests.test_gpu_hybrid_step import BF16, E4M3, F32, _attend_inputs, _cu, _ints, _new_cache, _ok, _table, _within

pytestmark = pytest.mark.gpu


def _attend(q, kc, vc, table, sl, ks=None, vs=None, **opt):
    out = torch.full_like(q, 7.0, memory_format=torch.contiguous_format)
    lse = torch.full(q.shape[:2], 7.0, device="cuda")
    kda.kda_kv_decode(q, kc, vc, table, sl, out, lse=lse, k_scale=ks, v_scale=vs, **opt)
    _ok()
    return out, lse


@pytest.mark.parametrize("dtype,cdt", [(BF16, BF16), (BF16, E4M3), (F32, F32)])
def test_first_tile_lands_where_the_table_of_work_lay(dtype, cdt):
    """With more than 32 sequences a table lies where the first tile comes next.  A CTA's first tile
    decides here (stretches of one to three tiles): right, and the same bits each time, with a table of
    few entries, a full one, and one whose entries stand for several sequences."""
    for N, length in ((33, 300), (1024, 40), (1500, 20)):
        seq = [1 + (length * (n + 1)) // N for n in range(N)]
        q, kc, vc, table, sl, (ks, vs) = _attend_inputs(dtype, cdt, 128, 4, 2, 16, "heads", seq, [1] * N)
        out, lse = _attend(q, kc, vc, table, sl, ks, vs)
        o, l, ob, lb = ref.attend(q, kc, vc, table, sl, [1] * N, 128 ** -0.5, k_scale=ks, v_scale=vs)
        _within(out, o, ob)
        _within(lse, l, lb)
        for _ in range(30):
            again, l2 = _attend(q, kc, vc, table, sl, ks, vs)
            assert torch.equal(out, again) and torch.equal(lse, l2)


@pytest.mark.parametrize("cdt", [BF16, E4M3])
@pytest.mark.parametrize("Hq,new", [(8, 1), (8, 4), (16, 4)])
def test_items_of_one_tile_follow_one_another(cdt, Hq, new):
    """Each warp sets an item's maxima and scales for itself.  Here each tile begins an item, and
    queries alternate between large and small, so that a maximum or scale of the item before would show."""
    N = 300
    seq, lens = [new + n % 100 for n in range(N)], [new] * N
    q, kc, vc, table, sl, (ks, vs) = _attend_inputs(BF16, cdt, 64, Hq, 1, 16, "heads", seq, lens)
    q = (q.contiguous().unflatten(0, (N, new)) * torch.tensor([4.0, 2.0 ** -6], device="cuda").repeat(N // 2)[:, None, None, None]).flatten(0, 1).to(BF16)
    cu = _cu(lens)
    out, lse = _attend(q, kc, vc, table, sl, ks, vs, cu_seqlens=cu, max_q=new)
    o, l, ob, lb = ref.attend(q, kc, vc, table, sl, lens, 64 ** -0.5, k_scale=ks, v_scale=vs)
    _within(out, o, ob)
    _within(lse, l, lb)
    for _ in range(30):
        again, l2 = _attend(q, kc, vc, table, sl, ks, vs, cu_seqlens=cu, max_q=new)
        assert torch.equal(out, again) and torch.equal(lse, l2)


@pytest.mark.parametrize("Hq,new", [(4, 1), (8, 4), (16, 4)])
@pytest.mark.parametrize("D", [64, 128])
def test_bf16_attention_is_the_formula_rounded_once(D, Hq, new):
    """Over a bf16 cache weights go into the product with the values in two parts, cut off to 8 bits and the
    rest rounded: 2^-16 of a weight (half a step of a rest below 2^-7 of it); the rest is taken 2^-19 of
    the weight larger.  Beside the bounds of scores and sums, one rounding of the output is left
    (2^-8 of it): not the 2^-8 of sum p |v| that weights of 8 bits would bring."""
    seq, lens = [700, 64 + new, 2100, new], [new] * 4
    q, kc, vc, table, sl, _ = _attend_inputs(BF16, BF16, D, Hq, 1, 32, "heads", seq, lens)
    out, lse = _attend(q, kc, vc, table, sl, cu_seqlens=_cu(lens), max_q=new)
    o, l, ob, lb = ref.attend(q, kc, vc, table, sl, lens, D ** -0.5)
    # sum p |v|: the attention of the values' sizes
    size = ref.attend(q, kc, vc.abs(), table, sl, lens, D ** -0.5)[0]
    # ob = (1 + h) (arithmetic + 2^-8 size) + h |o|, h = 2^-8, with the weights' rounding taken as 2^-8
    h = 2.0 ** -8
    arithmetic = (ob - h * o.abs()) / (1 + h) - h * size + (2.0 ** -16 + 2.0 ** -19) * size
    _within(out, o, (1 + h) * arithmetic + h * o.abs())
    _within(lse, l, lb)


@pytest.mark.parametrize("Hq,new", [(4, 1), (8, 4), (16, 4)])
def test_infinite_values_that_are_seen(Hq, new):
    """An infinity among the seen values is the sum, both signs are NaN, other channels keep their bits;
    keys of small weight (e^-60 of the largest) among them."""
    seq, lens, D = [300], [new], 64
    q, kc, vc, table, sl, _ = _attend_inputs(BF16, BF16, D, Hq, 1, 16, "heads", seq, lens)
    slopes = torch.full((Hq,), 0.25, device="cuda")   # key 17 lies about 280 keys back: e^-70
    opt = dict(cu_seqlens=_cu(lens), max_q=new, alibi_slopes=slopes)
    clean, _ = _attend(q, kc, vc, table, sl, **opt)
    inf = math.inf
    for j, c, x in ((17, 5, inf), (250, 6, -inf), (290, 7, inf), (100, 8, -inf), (90, 9, inf), (91, 9, -inf)):
        vc[int(table[0, j // 16]), :, j % 16, c] = x
    out, _ = _attend(q, kc, vc, table, sl, **opt)
    want = clean.clone()
    want[..., 5] = want[..., 7] = inf
    want[..., 6] = want[..., 8] = -inf
    want[..., 9] = math.nan
    assert torch.equal(out.isnan(), want.isnan())
    assert torch.equal(out.nan_to_num(nan=0.0), want.nan_to_num(nan=0.0))


BROKEN_CU = [   # entries, tokens in all
    ([0, 5, 3], 5), ([0, 4, 2, 2], 4), ([0, 0, 6, 4, 4], 6), ([0, 3, 7], 6), ([2, 4, 6], 6), ([-1, 3, 6], 6), ([0, 3, 2 ** 31 - 1, 6], 6),
    ([0, 3, -7, 6], 6), ([0, 0, 1, 0], 3), ([0, 2, 2, 1], 4),
    (list(range(0, 100, 2)) + [200, 102, 104, 106, 3], 106), ([0] * 40 + [5, 9, 7] + [7] * 40, 9),
    (list(range(70)) + [2 ** 31 - 1] + list(range(71, 80)), 79), (list(range(2000)) + [1990] * 3, 1999),
]


@pytest.mark.parametrize("cu,T", BROKEN_CU)
def test_append_reports_every_inconsistent_cu_seqlens(cu, T):
    """An entry that falls, also the last one, is reported whether a token comes to it or not; tokens of the
    sequences whose own entries are consistent are stored, no others are."""
    N = len(cu) - 1
    good = [n for n in range(N) if 0 <= cu[n] <= cu[n + 1] <= T and (n > 0 or cu[0] == 0)]
    assert len(good) < N
    ps = 16
    k = 1 + torch.arange(T, dtype=torch.float32)[:, None, None].expand(T, 1, 64).contiguous().cuda()
    kc, vc = _new_cache(N, 1, ps, 64, F32, fill=0.0)
    # sequence n has page n, its first new token row 0
    lens = [max(cu[n + 1] - cu[n], 0) if n in set(good) else 1 for n in range(N)]
    q = k.repeat(1, 2, 1)
    q_out = torch.zeros_like(q)
    kda.kda_kv_append(k, k, kc, vc, torch.arange(N, dtype=torch.int32)[:, None].contiguous().cuda(), _ints(lens), cu_seqlens=_ints(cu), q=q,
                      q_out=q_out)
    assert kda.kda_get_device_status() == kda.KDA_ERR_BAD_SEQLENS
    _ok()
    want, had = torch.zeros(N, ps), set()
    for n in good:
        for i, t in enumerate(range(cu[n], cu[n + 1])):
            assert t not in had   # no two of them share a token
            had.add(t)
            want[n, i] = t + 1
    assert torch.equal(kc[:, 0, :, 0].cpu(), want) and torch.equal(vc[:, 0, :, 63].cpu(), want)
    mine = torch.tensor([t in had for t in range(T)])
    assert torch.equal(q_out.cpu()[mine], q.cpu()[mine]) and (q_out.cpu()[~mine] == 0).all()


def test_steps_without_tokens():
    """No new token, with queries and positions of several axes: nothing is done, nothing is refused."""
    D, Hq, Hkv = 64, 4, 2
    kc, vc = _new_cache(3, Hkv, 16, D, BF16, fill=1.0)
    table, sl = _ints([[0], [1]]), _ints([5, 0])
    e = lambda h: torch.empty(0, h, D, dtype=BF16, device="cuda")
    inv = torch.ones(32, device="cuda")
    for kw in (dict(cu_seqlens=_ints([0, 0, 0])), dict(cu_seqlens=_ints([0, 0, 0]), positions=torch.empty(3, 0, dtype=torch.int32, device="cuda"),
                                                       axis_pairs=(16, 8, 8))):
        q_out = kda.kda_kv_append(e(Hkv), e(Hkv), kc, vc, table, sl, q=e(Hq), inv_freq=inv, **kw)
        assert q_out.shape == (0, Hq, D)
    kda.kda_kv_append(e(Hkv), e(Hkv), kc, vc, table[:0], sl[:0], q=e(Hq), inv_freq=inv)   # no sequence either
    kda.kda_kv_decode(e(Hq), kc, vc, table, sl, e(Hq), cu_seqlens=_ints([0, 0, 0]))
    pool = torch.ones(2, Hkv, D, D, device="cuda")
    kda.kda_decode_pool(e(Hkv), e(Hkv), e(Hkv), torch.empty(0, Hkv, D, device="cuda"), torch.empty(0, Hkv, device="cuda"), pool, _ints([0, 1]),
                        _ints([]), e(Hkv), cu_seqlens=_ints([0, 0, 0]))
    _ok()
    assert (kc == 1).all() and (vc == 1).all() and (pool == 1).all()


def test_append_divides_by_scales_of_any_size():
    """Scales from the least normal fp32 number to near the largest: the nearest e4m3 number to the fp32 quotient,
    held at 448.  That quotient is off from the 64-bit one by half its step, 2^-24 of it, and by a scale near
    2^-126 its remainder is rounded to 2^-149, so by 2^-24 more: so near a tie between two e4m3 numbers either
    may stand (17.5 / 0.7 is 25.0000004, in fp32 25, and goes to 24).  Below 2^-126, outside what a scale may
    be, zeros stay zeros all the same."""
    scales = [2.0 ** -126, 1.7e-38, 1.1e-30, 2.0 ** -101, 0.7, 1.0, 5e20, 2.0 ** 126, 3.3e38, 2.0 ** -130, 2.0 ** -149]
    H, D, T, normal = len(scales), 64, 5, len(scales) - 2
    s = torch.tensor(scales, device="cuda")
    gen = torch.Generator().manual_seed(60)
    x = torch.randn(T, H, D, generator=gen).mul(30).cuda().double() * s.double()[:, None]
    x[:, :, ::9] = 0.0
    x[:, 0, 3], x[:, 0, 4], x[:, 2, 5] = 1e30, -1e30, math.inf   # beyond 448 scales
    k = x.to(BF16)
    kc, vc = _new_cache(1, H, 16, D, E4M3, fill=0.0)
    kda.kda_kv_append(k, k, kc, vc, _ints([[0]]), _ints([T]), cu_seqlens=_ints([0, T]), k_scale=s, v_scale=s)
    _ok()
    exact = (k.double() / s.double()[:, None]).clamp(-448, 448)[:, :normal]
    ulp = 2.0 ** (torch.floor(torch.log2(exact.abs().clamp_min(2.0 ** -6))) - 3)   # of e4m3, subnormal below 2^-6
    for got in (kc, vc):
        y = got[0, :, :T].transpose(0, 1).double()
        assert torch.isfinite(y).all() and (y[:, :, ::9] == 0).all()
        assert ((y[:, :normal] - exact).abs() <= ulp / 2 + 2.0 ** -24 * exact.abs() + 2.0 ** -24).all()


@pytest.mark.parametrize("dtype,cdt", [(BF16, BF16), (BF16, E4M3), (F32, F32)])
@pytest.mark.parametrize("cap", [2.0 ** -100, 1e-20, 1e20, 2.0 ** 100])
def test_caps_of_the_extremes(dtype, cdt, cap):
    """The least caps leave scores of next to nothing, also those of a query of zeros; the largest none capped."""
    seq, lens = [70, 130], [2, 1]
    q, kc, vc, table, sl, (ks, vs) = _attend_inputs(dtype, cdt, 64, 4, 2, 16, "heads", seq, lens)
    q = q.contiguous()
    q[1, 2] = 0
    out, lse = _attend(q, kc, vc, table, sl, ks, vs, cu_seqlens=_cu(lens), max_q=2, softcap=cap)
    o, l, ob, lb = ref.attend(q, kc, vc, table, sl, lens, 0.125, softcap=cap if cap < 1 else 0.0, k_scale=ks, v_scale=vs)
    # A cap of 1e20 or more changes a score s by s (s / cap)^2 / 3, nothing here.  By s / cap times cap it is off by four
    # roundings more, 2^-22 |s|, |s| < 8: 2^-19 of a score, 2^-18 of a weight and of the weights' sum, values below 8.
    big = cap > 1
    _within(out, o, ob + big * 2 * 2.0 ** -18 * 8)
    _within(lse, l, lb + big * 2.0 ** -19)

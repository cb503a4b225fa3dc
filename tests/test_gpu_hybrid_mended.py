"""The hybrid step's operators in calls that they once answered wrongly, or that nothing had tested."""
import math

import pytest
import torch

from linear_attention_rule_b200 import kda
from tests import hybrid_reference as ref
from tests.test_gpu_hybrid_step import BF16, E4M3, F32, _Stack, _attend_inputs, _cu, _ints, _new_cache, _ok, _within

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


# ------------------------------------------------------------------------------- what was tested too loosely

U = 2.0 ** -24


@pytest.mark.parametrize("D,Hq,Hkv,new,opt", [(64, 4, 4, 1, {}), (128, 8, 2, 1, {}), (128, 6, 1, 3, dict(cap=5.0)), (64, 8, 1, 2, dict(bias=True)),
                                              (128, 2, 2, 1, dict(bias=True, cap=3.0))])
def test_fp32_attention_in_full_fp32(D, Hq, Hkv, new, opt):
    """The fp32 kernel multiplies fp32 numbers as they are.  A score is D products and sums (D U of sum |q k|), then
    scale, cap and bias (6 U of |s|, 2^-21 of a capped score for tanh, 2 U of bias and sum).  A weight is off by its
    score's error and by e^x's (2^-21 by ex2, 2^-21 for a score in units of log 2 below 2^3), so by 2^-20; the product with its
    value, the sum over the keys and the division add (keys + 4) U of sum p |v|.  Inputs in two parts of 11 bits would
    be 2^-20 of sum |q k| off, which this does not allow."""
    cap = opt.get("cap", 0.0)
    seq, lens = [600, 33 + new, new, 1200], [new] * 4
    q, kc, vc, table, sl, _ = _attend_inputs(F32, F32, D, Hq, Hkv, 16, "heads", seq, lens, seed=77)
    q = q.contiguous()
    slopes = 2.0 ** (-8.0 * torch.arange(1, Hq + 1, device="cuda") / Hq) if opt.get("bias") else None
    out, lse = _attend(q, kc, vc, table, sl, cu_seqlens=_cu(lens), max_q=new, softcap=cap, alibi_slopes=slopes)
    scale, t = D ** -0.5, 0
    for n, length in enumerate(lens):
        j = torch.arange(seq[n], device="cuda")
        K, V = (c[table[n].long()[j // 16], :, j % 16].double().repeat_interleave(Hq // Hkv, 1) for c in (kc, vc))
        for i in range(length):
            pos = seq[n] - length + i
            k, v, x = K[:pos + 1], V[:pos + 1], q[t].double()
            s = scale * torch.einsum("hd,jhd->hj", x, k)
            es = scale * torch.einsum("hd,jhd->hj", x.abs(), k.abs()) * D * U + 6 * U * s.abs()
            if cap:
                s = cap * torch.tanh(s / cap)
                es += 2.0 ** -21 * s.abs()
            if slopes is not None:
                b = slopes.double()[:, None] * (j[:pos + 1] - pos).double()
                s, es = s + b, es + 2 * U * (b.abs() + (s + b).abs())
            p = torch.softmax(s, -1)
            w = p * (es + 2.0 ** -20)                      # of each weight; a little more where a bias leaves nothing of it
            size = torch.einsum("hj,jhd->hd", p, v.abs())
            bound = torch.einsum("hj,jhd->hd", w, v.abs()) + (w.sum(-1)[:, None] + (pos + 5) * U) * size
            _within(out[t], torch.einsum("hj,jhd->hd", p, v).cpu(), bound.cpu() * (1 + 2.0 ** -10))
            l = torch.logsumexp(s, -1)
            _within(lse[t], l.cpu(), (w.sum(-1) * (1 + 2.0 ** -10) + 4 * U * l.abs() + (pos + 1) * U).cpu())
            t += 1


def test_two_stacks_at_once_leave_each_other_alone():
    """Steps of two stacks on two streams: outputs of every step, states and caches of both are those of
    the same steps alone."""
    N, steps = 3, 12
    one, two = [_Stack(N), _Stack(N)], [_Stack(N, seed=51), _Stack(N, seed=51)]
    ids = _ints(list(range(N)))
    xs = [[s.inputs(N, 100 * i + r) for r in range(steps)] for i, s in enumerate((one[0], two[0]))]
    lens = [_ints([r + 1] * N) for r in range(steps)]
    fresh = _ints([-1] * N)
    torch.cuda.synchronize()
    alone = [[s.step(x, None, l, fresh if r == 0 else ids, ids, 1) for r, (x, l) in enumerate(zip(xx, lens))]
             for s, xx in ((one[0], xs[0]), (two[0], xs[1]))]
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    got = [[], []]
    for r in range(steps):
        for i, (s, stream) in enumerate(((one[1], s1), (two[1], s2))):
            got[i].append(s.step(xs[i][r], None, lens[r], fresh if r == 0 else ids, ids, 1, stream=stream))
    torch.cuda.synchronize()
    _ok()
    for a, b in zip(alone, got):
        for (a1, a2), (b1, b2) in zip(a, b):
            assert torch.equal(a1, b1) and torch.equal(a2, b2)
    for a, b in (one, two):
        assert torch.equal(a.pool, b.pool)
        for x, y in ((a.kc, b.kc), (a.vc, b.vc)):   # rows that nothing was stored to are NaN in both
            assert torch.equal(x.view(torch.int16), y.view(torch.int16))
    assert not torch.equal(one[0].pool, two[0].pool)


@pytest.mark.parametrize("dtype,cdt", [(F32, F32), (BF16, BF16), (BF16, E4M3)])
def test_tokens_without_a_page_have_their_queries_turned(dtype, cdt):
    """A page outside the cache, positions behind the table and before 0: keys and values of those tokens are
    not stored anywhere, the others' are; the queries of all are turned."""
    H, D, ps, T = 2, 64, 16, 6
    gen = torch.Generator().manual_seed(61)
    q, k, v = (torch.randn(T, h, D, generator=gen).to(dtype).cuda() for h in (4, H, H))
    inv = (10000.0 ** (-torch.arange(32, dtype=torch.float64) / 32)).float()
    for table, length in (([[0, 3]], 20), ([[0, 2]], 34), ([[1, 2]], 4), ([[-1, 0]], 18)):
        kc, vc = _new_cache(3, H, ps, D, cdt, fill=0.0)
        q_out = torch.full_like(q, 9.0)
        kda.kda_kv_append(k, v, kc, vc, _ints(table), _ints([length]), cu_seqlens=_ints([0, T]), q=q, q_out=q_out, inv_freq=inv.cuda())
        assert kda.kda_get_device_status() == kda.KDA_ERR_BAD_PAGE
        place = torch.arange(length - T, length)
        y, size = ref.rotate(q, place[None], inv, [32], False)
        _within(q_out, y, ref.rotation_bound(y, size, dtype))
        y, size = ref.rotate(k, place[None], inv, [32], False)
        bound = ref.rotation_bound(y, size, cdt) + (2.0 ** -10 if cdt == E4M3 else 0.0)
        want_v = v.float().to(cdt).float()
        left_k, left_v = kc.clone().float(), vc.clone().float()
        stored = 0
        for t, j in enumerate(place.tolist()):
            page = table[0][j // ps] if 0 <= j < 2 * ps else -1
            if not 0 <= page < 3:
                continue
            stored += 1
            _within(kc[page, :, j % ps].float(), y[t], bound[t])
            assert torch.equal(vc[page, :, j % ps].float(), want_v[t])
            left_k[page, :, j % ps] = left_v[page, :, j % ps] = 0
        assert 0 < stored < T and (left_k == 0).all() and (left_v == 0).all()
    _ok()


def test_a_captured_step_behind_copies_and_beside_another():
    """A graph whose step stands behind copies and a fill (no kernels), and that forks into two stacks' steps and
    joins: replays follow new inputs, bit for bit as the steps one after another."""
    N = 3
    cap, ref_ = [_Stack(N), _Stack(N, seed=51)], [_Stack(N), _Stack(N, seed=51)]
    keys = ("q", "k", "v", "g", "beta", "aq", "ak", "av")
    src = [{k: v for k, v in s.inputs(N, 5).items() if k in keys} for s in cap]
    x = [{k: torch.empty_like(v) for k, v in xs.items()} for xs in src]
    ids, fresh = _ints(list(range(N))), _ints([-1] * N)
    slots, lens = fresh.clone(), _ints([1] * N)
    ws = [torch.empty(kda.kda_kv_decode_workspace_size(N, 4, 1, 128), dtype=torch.uint8, device="cuda") for _ in range(2)]

    def both(stacks, xs, fork):
        outs, main = [], torch.cuda.current_stream()
        side = torch.cuda.Stream() if fork else None
        for i, s in enumerate(stacks):
            for k in keys:
                xs[i][k].copy_(src[i][k])
        if fork:
            side.wait_stream(main)
        for i, s in enumerate(stacks):
            with torch.cuda.stream(side if fork and i else main):
                ws[i].zero_()
                outs.append(s.step(xs[i], None, lens, slots, ids, 1, ws[i]))
        if fork:
            main.wait_stream(side)
        outs.append(outs[0][1].clone())
        return outs

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        both(cap, x, False)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = both(cap, x, True)
    for s in cap:
        s.pool.zero_()
    y = [{k: torch.empty_like(v) for k, v in xs.items()} for xs in src]
    for r in range(4):
        for i, s in enumerate(cap):
            for k, v in s.inputs(N, 80 + 10 * i + r).items():
                if k in keys:
                    src[i][k].copy_(v)
        lens.fill_(r + 1)
        slots.copy_(fresh if r == 0 else ids)
        graph.replay()
        torch.cuda.synchronize()
        want = both(ref_, y, False)
        torch.cuda.synchronize()
        for (a1, a2), (b1, b2) in zip(outs[:2], want[:2]):
            assert torch.equal(a1, b1) and torch.equal(a2, b2)
        assert torch.equal(outs[2], want[2])
    _ok()
    for a, b in zip(cap, ref_):
        assert torch.equal(a.pool, b.pool)


@pytest.mark.parametrize("Hq", [4, 32, 64])
def test_e4m3_weights_hold_more_than_fp16(Hq):
    """Two keys with scores +-x and values +-1: the output is the difference of two weights, tanh x, and what a
    weight loses stands alone in it.  The larger one is 2^7 and exact; the other, in [2^6, 2^7), is off by 2^-8 from its
    third part and by 2^-10 from the first remainder's rounding to fp16, of a sum above 2^7.5: 1.25 2^-15.5 of the output's
    unit.  Scores are off by 64 2^-24 |x| and e^x by 2^-21, half of which reaches the difference; |tanh x| < 2^-7 is
    rounded by 2^-8 of itself.  A weight in fp16 would be off by 2^-5 of that sum, up to 2^-12.5."""
    N, D = 64, 64
    kc, vc = (torch.zeros(1, 1, 16, D, device="cuda") for _ in range(2))
    kc[0, 0, 0, 0], kc[0, 0, 1, 0] = 1.0, -1.0
    vc[0, 0, 0], vc[0, 0, 1] = 1.0, -1.0
    gen = torch.Generator().manual_seed(62)
    q = torch.zeros(N, Hq, D)
    q[:, :, 0] = (torch.rand(N, Hq, generator=gen) - 0.5) * 2.0 ** -6
    q = q.to(BF16).cuda()
    out, _ = _attend(q, kc.to(E4M3), vc.to(E4M3), _ints([[0]] * N), _ints([2] * N), scale=1.0)
    want = torch.tanh(q[:, :, :1].double()).expand(N, Hq, D).cpu()
    _within(out, want, 1.25 * 2.0 ** -15.5 + 2.0 ** -18 * want.abs() + 2.0 ** -22 + 2.0 ** -8 * want.abs())


@pytest.mark.parametrize("Hq,new", [(5, 4), (8, 4)])
def test_queries_of_short_items_wait_for_their_slot(Hq, new):
    """Rows of 17 to 32 by 128 channels have two slots for queries and three for tiles: items of one to four tiles,
    in orders that put one of each length behind each, with queries of very different size side by side."""
    gen = torch.Generator().manual_seed(63)
    N, D = 400, 128
    seq = (new + torch.randint(0, 4, (N,), generator=gen) * 128 + torch.randint(0, 100, (N,), generator=gen)).tolist()
    lens = [new] * N
    q, kc, vc, table, sl, _ = _attend_inputs(BF16, BF16, D, Hq, 1, 64, "heads", seq, lens)
    q = (q.contiguous().unflatten(0, (N, new)) * torch.tensor([4.0, 2.0 ** -6, 1.0, 0.0], device="cuda").repeat(N // 4)[:, None, None, None]).flatten(0, 1).to(BF16)
    cu = _cu(lens)
    out, lse = _attend(q, kc, vc, table, sl, cu_seqlens=cu, max_q=new)
    o, l, ob, lb = ref.attend(q, kc, vc, table, sl, lens, D ** -0.5)
    _within(out, o, ob)
    _within(lse, l, lb)
    for _ in range(40):
        again, l2 = _attend(q, kc, vc, table, sl, cu_seqlens=cu, max_q=new)
        assert torch.equal(out, again) and torch.equal(lse, l2)


@pytest.mark.parametrize("cu,T", [c for c in BROKEN_CU if len(c[0]) < 100])
def test_pool_and_attention_handle_the_consistent_sequences(cu, T):
    """Of an inconsistent cu_seqlens the consistent sequences come out as in calls of their own, and rows of no
    such sequence are left as they were."""
    N, D = len(cu) - 1, 64
    good = [n for n in range(N) if 0 <= cu[n] <= cu[n + 1] <= T and (n > 0 or cu[0] == 0)]
    gen = torch.Generator().manual_seed(64)
    q, k, v = (torch.randn(T, 2, D, generator=gen).mul(0.2).cuda() for _ in range(3))
    g, beta = -torch.rand(T, 2, D, generator=gen).cuda(), torch.rand(T, 2, generator=gen).cuda()
    pool = torch.randn(N, 2, D, D, generator=gen).cuda()
    kc, vc = (torch.randn(N, 2, 16, D, generator=gen).cuda() for _ in range(2))
    table = torch.arange(N, dtype=torch.int32)[:, None].contiguous().cuda()
    lens = _ints([12] * N)
    ids = torch.arange(N, dtype=torch.int32, device="cuda")
    out, att = (torch.full((T, 2, D), 7.0, device="cuda") for _ in range(2))
    kda.kda_decode_pool(q, k, v, g, beta, pool, ids, _ints([-1] * T), out, cu_seqlens=_ints(cu))
    assert kda.kda_get_device_status() == kda.KDA_ERR_BAD_SEQLENS
    kda.kda_kv_decode(q, kc, vc, table, lens, att, cu_seqlens=_ints(cu), max_q=16)
    assert kda.kda_get_device_status() == kda.KDA_ERR_BAD_SEQLENS
    want, w_att = (torch.full((T, 2, D), 7.0, device="cuda") for _ in range(2))
    for n in good:
        a, b = cu[n], cu[n + 1]
        if a == b:
            continue
        one = [x[a:b].contiguous() for x in (q, k, v, g, beta)]
        o = torch.empty(b - a, 2, D, device="cuda")
        kda.kda_decode_pool(*one, pool, ids[n:n + 1], _ints([-1] * (b - a)), o, cu_seqlens=_ints([0, b - a]))
        want[a:b] = o
        kda.kda_kv_decode(one[0], kc, vc, table[n:n + 1], lens[n:n + 1], o, cu_seqlens=_ints([0, b - a]), max_q=16)
        w_att[a:b] = o
    _ok()
    assert torch.equal(out, want)
    assert torch.allclose(att, w_att, rtol=0, atol=2.0 ** -18)   # sums of 12 weights and values of a few units, in another order
    assert torch.equal(att == 7.0, w_att == 7.0)

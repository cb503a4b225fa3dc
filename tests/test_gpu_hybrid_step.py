"""GPU parity of the hybrid step's operators against plain fp64 forms: the state pool, appending to
the paged cache and the attention over it; then the three together as a decode loop uses them."""
import math

import pytest
import torch

from linear_attention_rule_b200 import kda, synthetic
from tests import hybrid_reference as ref

pytestmark = pytest.mark.gpu

BF16, F32, E4M3 = torch.bfloat16, torch.float32, torch.float8_e4m3fn


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _cu(lens):
    return _ints([sum(lens[:n]) for n in range(len(lens) + 1)])


def _ok():
    status = kda.kda_get_device_status()
    assert status == kda.KDA_OK, kda.kda_status_string(status)


def _within(x, y, bound):
    x = x.double().cpu()
    assert torch.isfinite(x).all()
    d = (x - y).abs()
    worst = (d - bound).max()
    assert (d <= bound + 1e-300).all(), "off by %.3g over the bound (error %.3g)" % (worst, d.max())


# ------------------------------------------------------------------------------- the state pool

def _pool_inputs(lens, Hk, Hv, D, dtype, seed, raw=False, scalar=False, slots=None, pad=0):
    gen = torch.Generator().manual_seed(seed)
    T, N = sum(lens), len(lens)
    qkv = torch.randn(T + pad, (2 * Hk + Hv) * D, generator=gen)
    if not raw:
        for i in range(2 * Hk):
            x = qkv[:, i * D:(i + 1) * D]
            x /= x.norm(dim=-1, keepdim=True)
    qkv = qkv.to(dtype).cuda()
    q, k, v = (x.view(T + pad, -1, D) for x in qkv.split([Hk * D, Hk * D, Hv * D], 1))
    g = 3 + torch.randn(*((T + pad, Hv) if scalar else (T + pad, Hv, D)), generator=gen)
    b = torch.randn(T + pad, Hv, generator=gen)
    if not raw:
        g, b = torch.nn.functional.logsigmoid(g), torch.sigmoid(b)
    slots = slots or N + T + 3
    pool = 0.1 * torch.randn(slots, Hv, D, D, generator=gen)
    order = torch.randperm(slots, generator=gen).to(torch.int32)
    return q, k, v, g.cuda(), b.cuda(), pool.cuda(), order


POOL_CASES = [
    # dtype, D, Hk, Hv, lens, raw, scalar gate
    (BF16, 128, 3, 3, [1, 1, 1, 1, 1], False, False),
    (BF16, 128, 2, 4, [3, 0, 1, 5, 4, 0], False, False),
    (BF16, 128, 1, 5, [9, 2], True, True),
    (BF16, 64, 2, 2, [1, 4, 17], True, False),
    (F32, 128, 2, 2, [2, 1], False, True),
    (F32, 64, 1, 3, [0, 6, 33], True, False),
    (F32, 64, 1, 1, [1], False, False),
]


@pytest.mark.parametrize("dtype,D,Hk,Hv,lens,raw,scalar", POOL_CASES)
@pytest.mark.parametrize("keep", ["last", "all"])
def test_pool_matches_the_recurrence(dtype, D, Hk, Hv, lens, raw, scalar, keep):
    T, N, pad = sum(lens), len(lens), 2
    q, k, v, g, b, pool, order = _pool_inputs(lens, Hk, Hv, D, dtype, 5, raw, scalar, pad=pad)
    slots_in = order[:N].clone()
    slots_in[N - 1] = -1   # a fresh sequence
    slots_out = torch.full((T + pad,), -1, dtype=torch.int32)
    t = 0
    for n, length in enumerate(lens):
        for i in range(length):
            if keep == "all":
                slots_out[t] = order[N + t]
            elif i == length - 1:
                slots_out[t] = order[n]   # in place (the fresh one: a slot of its own)
            t += 1
    slots_out[T:] = 0   # padding is not read
    flags = (kda.KDA_IN_G_SCALAR if scalar else 0) | (
        kda.KDA_IN_NORMALIZE_QK | kda.KDA_IN_G_LOGITS | kda.KDA_IN_BETA_LOGITS if raw else 0)
    o_ref, pool_ref, bound = ref.pool_step(q[:T], k[:T], v[:T], g[:T], b[:T], pool, slots_in, slots_out, lens, raw, raw, raw)
    before = pool.clone()
    out = torch.full((T + pad, Hv, D), 7.0, dtype=dtype, device="cuda")
    kda.kda_decode_pool(q, k, v, g, b, pool, slots_in.cuda(), slots_out.cuda(), out, cu_seqlens=_cu(lens), in_flags=flags)
    _ok()
    assert (out[T:] == 7).all()
    _within(out[:T], o_ref, (1 + ref.HALF[dtype]) * bound + ref.HALF[dtype] * o_ref.abs())
    written = set(int(x) for x in slots_out[:T] if x >= 0)
    for s in range(pool.shape[0]):
        if s not in written:
            assert torch.equal(pool[s], before[s])
    # each token adds at most (D + 24) roundings of the terms of one product to a state
    scale = pool_ref.abs().amax()
    e = (pool.double().cpu() - pool_ref).abs().max() / scale
    assert e <= max(lens) * (D + 24) * 2.0 ** -24, e


def test_pool_one_token_without_cu_equals_the_dense_decode():
    N, H, D = 6, 3, 128
    q, k, v, g, b, pool, order = _pool_inputs([1] * N, H, H, D, BF16, 6)
    slots = order[:N].cuda()
    dense = pool[slots.long()].contiguous()
    o1, o2 = (torch.empty(N, H, D, dtype=BF16, device="cuda") for _ in range(2))
    kda.kda_decode(q.contiguous(), k.contiguous(), v.contiguous(), g, b, dense, o1)
    kda.kda_decode_pool(q, k, v, g, b, pool, slots, slots, o2)
    _ok()
    assert torch.allclose(pool[slots.long()], dense, rtol=0, atol=136 * 2.0 ** -24)
    assert torch.allclose(o1.float(), o2.float(), rtol=2.0 ** -7, atol=1e-5)   # two roundings to bf16


@pytest.mark.parametrize("dtype,D", [(BF16, 128), (F32, 64)])
def test_pool_roll_back_is_exact(dtype, D):
    """Going on from the state kept after token j gives the bits of a run that never saw the rest."""
    lens, Hv = [7], 2
    q, k, v, g, b, pool, order = _pool_inputs(lens, 1, Hv, D, dtype, 8)
    keep = order[1:8].cuda()
    out = torch.empty(7, Hv, D, dtype=dtype, device="cuda")
    kda.kda_decode_pool(q, k, v, g, b, pool, order[:1].cuda(), keep, out, cu_seqlens=_cu([7]))
    for j in (1, 4, 6):
        p2 = pool.clone()
        o2 = torch.empty(7 - j, Hv, D, dtype=dtype, device="cuda")
        kda.kda_decode_pool(q[j:], k[j:], v[j:], g[j:], b[j:], p2, keep[j - 1:j], keep[j:], o2, cu_seqlens=_cu([7 - j]))
        assert torch.equal(o2, out[j:]) and torch.equal(p2, pool)
    _ok()


def test_pool_shared_prefix_and_bad_slots():
    """Several sequences read one slot; a slot outside the pool is reported, the rest is done."""
    N, H, D = 4, 2, 64
    q, k, v, g, b, pool, _ = _pool_inputs([1] * N, H, H, D, F32, 9, slots=6)
    out = torch.full((N, H, D), 3.0, device="cuda")
    slots_in, slots_out = _ints([5, 5, 6, 5]), _ints([0, 1, 2, 9])
    o_ref, pool_ref, bound = ref.pool_step(q, k, v, g, b, pool, [5, 5, 5, 5], [0, 1, -1, -1], [1] * N)
    kda.kda_decode_pool(q, k, v, g, b, pool, slots_in, slots_out, out)
    assert kda.kda_get_device_status() == kda.KDA_ERR_BAD_SLOT
    _ok()
    assert (out[2] == 3).all()
    for n in (0, 1, 3):
        _within(out[n], o_ref[n], bound[n] + 2.0 ** -24 * o_ref[n].abs())
    assert torch.allclose(pool.double().cpu(), pool_ref, rtol=0, atol=1e-5)


def test_inconsistent_cu_seqlens_is_reported_by_each_operator():
    N, H, D = 3, 2, 64
    q, k, v, g, b, pool, order = _pool_inputs([1] * N, H, H, D, F32, 10)
    cache = torch.zeros(4, H, 16, D, device="cuda")
    table, lens = _ints([[0], [1], [2]]), _ints([1, 1, 1])
    for bad in ([0, 2, 1, 3], [1, 1, 2, 3], [0, 1, 2, 4], [0, -1, 2, 3]):
        out = torch.zeros(N, H, D, device="cuda")
        kda.kda_decode_pool(q, k, v, g, b, pool, order[:N].cuda(), _ints([-1] * N), out, cu_seqlens=_ints(bad))
        assert kda.kda_get_device_status() == kda.KDA_ERR_BAD_SEQLENS
        kda.kda_kv_append(k, v, cache, cache.clone(), table, lens, cu_seqlens=_ints(bad))
        assert kda.kda_get_device_status() in (kda.KDA_ERR_BAD_SEQLENS, kda.KDA_ERR_BAD_PAGE)
        kda.kda_kv_decode(q, cache, cache, table, lens, out, cu_seqlens=_ints(bad), max_q=3)
        assert kda.kda_get_device_status() == kda.KDA_ERR_BAD_SEQLENS
    kda.kda_kv_decode(q, cache, cache, table, lens, out, cu_seqlens=_ints([0, 2, 2, 3]), max_q=1)   # 2 > max_q
    assert kda.kda_get_device_status() == kda.KDA_ERR_BAD_SEQLENS
    _ok()


# ------------------------------------------------------------------------------- the paged cache

def _new_cache(pages, Hkv, ps, D, dtype, order="heads", fill=None, gen=None):
    """A cache view [pages, Hkv, ps, D]: heads before rows, rows before heads, or one array for both."""
    shape = {"heads": (2, pages, Hkv, ps, D), "rows": (2, pages, ps, Hkv, D), "both": (pages, 2, Hkv, ps, D)}[order]
    x = torch.randn(shape, generator=gen) if fill is None else torch.full(shape, fill)
    x = x.to(dtype).cuda()
    if order == "both":
        return x[:, 0], x[:, 1]
    return (x[0], x[1]) if order == "heads" else (x[0].transpose(1, 2), x[1].transpose(1, 2))


def _table(lens, ps, gen, extra=2):
    need = [-(-n // ps) for n in lens]
    pages = sum(need) + extra
    order = torch.randperm(pages, generator=gen)
    table = torch.full((len(lens), max(need + [1]) + 1), -7, dtype=torch.int32)
    at = 0
    for n, m in enumerate(need):
        table[n, :m] = order[at:at + m].to(torch.int32)
        at += m
    return table, pages


APPEND_CASES = [
    # dtype, cache, D, Hq, Hkv, ps, order, lens, rot, axes, adjacent
    (BF16, BF16, 128, 4, 2, 16, "heads", [1, 1, 1], 128, 1, False),
    (BF16, BF16, 128, 3, 1, 64, "rows", [5, 0, 130, 1], 64, 1, True),
    (BF16, E4M3, 128, 0, 2, 32, "both", [33, 70], 128, 3, False),
    (BF16, E4M3, 64, 6, 3, 16, "rows", [2, 0, 0, 40], 32, 3, True),
    (F32, F32, 64, 2, 2, 8, "heads", [19, 3], 64, 4, False),
    (F32, F32, 128, 5, 5, 1, "both", [4], 16, 1, True),
    (BF16, BF16, 64, 8, 1, 4096, "heads", [3, 2], 0, 1, False),
]


@pytest.mark.parametrize("dtype,cdt,D,Hq,Hkv,ps,order,lens,rot,axes,adjacent", APPEND_CASES)
def test_append_matches_the_rotation(dtype, cdt, D, Hq, Hkv, ps, order, lens, rot, axes, adjacent):
    gen = torch.Generator().manual_seed(21)
    T, N, pad = sum(lens), len(lens), 3
    past = [int(x) for x in torch.randint(0, 50, (N,), generator=gen)]
    seq = [p + n for p, n in zip(past, lens)]
    table, pages = _table(seq, ps, gen)
    kc, vc = _new_cache(pages, Hkv, ps, D, cdt, order, gen=gen)
    kb, vb = kc.clone(), vc.clone()
    qkv = torch.randn(T + pad, (Hq + 2 * Hkv) * D, generator=gen).to(dtype).cuda()
    q, k, v = (x.view(T + pad, -1, D) for x in qkv.split([Hq * D, Hkv * D, Hkv * D], 1))
    half = rot // 2
    inv = (10000.0 ** (-torch.arange(half, dtype=torch.float64) / max(half, 1))).float()
    per = [half - (axes - 1) * (half // axes)] + [half // axes] * (axes - 1)
    place = torch.tensor([p + i for p, n in zip(past, lens) for i in range(n)])
    positions = None
    if axes > 1:   # far positions on the first axis
        positions = torch.randint(0, 2 ** 31 - 1, (axes, T + pad), generator=gen, dtype=torch.int64).to(torch.int32)
    scales = [(0.02 + 0.01 * torch.rand(Hkv, generator=gen)).cuda() for _ in range(2)] if cdt == E4M3 else [None, None]
    q_out = torch.full((T + pad, Hq, D), 9.0, dtype=dtype, device="cuda") if Hq else None
    kda.kda_kv_append(k, v, kc, vc, table.cuda(), _ints(seq), cu_seqlens=_cu(lens), q=q if Hq else None, q_out=q_out,
                      inv_freq=inv.cuda() if rot else None, positions=None if positions is None else positions.cuda(),
                      axis_pairs=per if rot and axes > 1 else None, adjacent=adjacent, k_scale=scales[0], v_scale=scales[1])
    _ok()
    pos = place[None] if positions is None else positions[:, :T]
    if rot:
        kr, ksize = ref.rotate(k[:T], pos, inv, per, adjacent)
        qr, qsize = ref.rotate(q[:T], pos, inv, per, adjacent)
    else:
        kr, qr = k[:T].double().cpu(), q[:T].double().cpu()
        ksize, qsize = torch.zeros_like(kr), torch.zeros_like(qr)
    if Hq:
        _within(q_out[:T], qr, ref.rotation_bound(qr, qsize, dtype))
        assert (q_out[T:] == 9).all()
    seqs = torch.repeat_interleave(torch.arange(N), torch.tensor(lens))
    page, row = table[seqs, place // ps].long().cuda(), (place % ps).cuda()
    got_k, got_v = kc[page, :, row], vc[page, :, row]
    if cdt == E4M3:
        kr, ksize = kr / scales[0].double().cpu()[:, None], ksize / scales[0].double().cpu()[:, None]
        over = kr.abs() > 448
        kr = kr.clamp(-448, 448)
        bound = ref.rotation_bound(kr, ksize, E4M3) + 2.0 ** -10
        _within(got_k.float(), kr, bound)
        assert (got_k.float().cpu()[over].abs() == 448).all()
        want = (v[:T].float() / scales[1][:, None]).clamp(-448, 448).to(E4M3)
        assert torch.equal(got_v.float(), want.float())
    else:
        _within(got_k, kr, ref.rotation_bound(kr, ksize, cdt))
        assert torch.equal(got_v, v[:T])
    # everything else in the caches is as it was
    kb[page, :, row], vb[page, :, row] = got_k, got_v
    assert torch.equal(kc.float(), kb.float()) and torch.equal(vc.float(), vb.float())


def test_append_in_place_queries_and_default_positions():
    """q_out = q, and one token per sequence without cu_seqlens: the bits of the general call."""
    N, Hq, Hkv, D, ps = 5, 4, 2, 128, 16
    gen = torch.Generator().manual_seed(22)
    q, k, v = (torch.randn(N, h, D, generator=gen).to(BF16).cuda() for h in (Hq, Hkv, Hkv))
    seq = [1, 16, 17, 40, 3]
    table, pages = _table(seq, ps, gen)
    inv = (10000.0 ** (-torch.arange(64, dtype=torch.float64) / 64)).float().cuda()
    a = _new_cache(pages, Hkv, ps, D, BF16, fill=0.0)
    b = _new_cache(pages, Hkv, ps, D, BF16, fill=0.0)
    out = kda.kda_kv_append(k, v, *a, table.cuda(), _ints(seq), q=q, inv_freq=inv)
    q2 = q.clone()
    kda.kda_kv_append(k, v, *b, table.cuda(), _ints(seq), cu_seqlens=_cu([1] * N), q=q2, q_out=q2, inv_freq=inv,
                      positions=_ints([s - 1 for s in seq]))
    _ok()
    assert torch.equal(out, q2) and torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_append_drops_and_reports_tokens_without_a_page():
    H, D, ps = 2, 64, 16
    k, v = (torch.randn(6, H, D).cuda() for _ in range(2))
    kc, vc = _new_cache(3, H, ps, D, F32, fill=0.0)
    # a page id outside the cache, a position behind the table, a negative position
    for table, seq, stored in (([[0, 3]], [20], 2), ([[0, 2]], [34], 4), ([[1, 2]], [4], 4), ([[-1, 0]], [18], 2)):
        kc.zero_()
        q = torch.randn(6, H, D).cuda()
        kda.kda_kv_append(k, v, kc, vc, _ints(table), _ints(seq), cu_seqlens=_ints([0, 6]))
        assert kda.kda_get_device_status() == kda.KDA_ERR_BAD_PAGE
        assert int((kc != 0).any(-1).any(1).sum()) == stored
    _ok()


def test_append_finds_the_sequence_among_many():
    """Ragged sequences, most of them empty: every token lands in its own page."""
    gen = torch.Generator().manual_seed(23)
    N = 3001
    lens = [0] * N
    for i in torch.randint(0, N, (400,), generator=gen).tolist():
        lens[i] += 1
    lens[0] = lens[1] = lens[N - 1] = 0
    T = sum(lens)
    k = torch.arange(T, dtype=torch.float32)[:, None, None].expand(T, 1, 64).contiguous().cuda() + 1
    kc, vc = _new_cache(N, 1, 16, 64, F32, fill=0.0)
    kda.kda_kv_append(k, k, kc, vc, torch.arange(N, dtype=torch.int32)[:, None].contiguous().cuda(), _ints(lens),
                      cu_seqlens=_cu(lens))
    _ok()
    t = 0
    want = torch.zeros(N, 16)
    for n in range(N):
        for i in range(lens[n]):
            want[n, i] = t + 1
            t += 1
    assert torch.equal(kc[:, 0, :, 0].cpu(), want) and torch.equal(vc[:, 0, :, 63].cpu(), want)


# ------------------------------------------------------------------------------- attention

def _attend_inputs(dtype, cdt, D, Hq, Hkv, ps, order, seq, lens, seed=31, fill=float("nan"), pad=0):
    """Visible rows are drawn; every other row of the caches holds `fill`."""
    gen = torch.Generator().manual_seed(seed)
    table, pages = _table(seq, ps, gen)
    kc, vc = _new_cache(pages, Hkv, ps, D, cdt, order, fill=fill)
    for n, L in enumerate(seq):
        j = torch.arange(L)
        page, row = table[n].long()[j // ps].cuda(), (j % ps).cuda()
        kc[page, :, row] = torch.randn(L, Hkv, D, generator=gen).mul(40 if cdt == E4M3 else 1).to(cdt).cuda()
        vc[page, :, row] = torch.randn(L, Hkv, D, generator=gen).mul(40 if cdt == E4M3 else 1).to(cdt).cuda()
    q = torch.randn(sum(lens) + pad, Hq * D + 64, generator=gen).to(dtype).cuda()[:, :Hq * D].unflatten(1, (Hq, D))
    scales = [(0.02 + 0.01 * torch.rand(Hkv, generator=gen)).cuda() for _ in range(2)] if cdt == E4M3 else [None, None]
    return q, kc, vc, table.cuda(), _ints(seq), scales


ATTEND_CASES = [
    # dtype, cache, D, Hq, Hkv, ps, order, seq, lens, options
    (BF16, BF16, 128, 8, 2, 16, "heads", [1, 2, 15, 16, 17, 33, 257], [1] * 7, {}),
    (BF16, BF16, 128, 4, 4, 64, "rows", [700, 64, 63, 65], [1] * 4, dict(softcap=3.0)),
    (BF16, BF16, 64, 16, 1, 32, "both", [100, 1000, 31, 1], [1] * 4, dict(bias=True)),
    (BF16, BF16, 128, 5, 1, 8, "heads", [40, 7, 300, 0, 129], [3, 7, 1, 0, 4], {}),
    (BF16, BF16, 128, 8, 1, 16, "heads", [40, 200], [16, 9], dict(window=5)),
    (BF16, BF16, 64, 12, 4, 128, "rows", [500, 90, 260], [2, 3, 1], dict(window=100, softcap=20.0, bias=True)),
    (BF16, BF16, 128, 32, 1, 16, "heads", [70, 33], [1, 2], {}),
    (BF16, BF16, 64, 40, 2, 16, "heads", [150, 64], [4, 16], dict(bias=True)),
    (BF16, E4M3, 128, 8, 2, 16, "heads", [1, 2, 16, 33, 257], [1] * 5, {}),
    (BF16, E4M3, 128, 5, 1, 64, "rows", [300, 20], [6, 3], dict(window=30, softcap=10.0)),
    (BF16, E4M3, 64, 7, 7, 32, "both", [100, 1, 64], [1, 1, 2], dict(bias=True)),
    (F32, F32, 64, 4, 4, 16, "heads", [1, 17, 200], [1] * 3, {}),
    (F32, F32, 128, 6, 2, 32, "rows", [90, 33], [5, 2], dict(window=20, softcap=5.0)),
    (F32, F32, 128, 40, 2, 8, "both", [61], [2], dict(bias=True)),
]


@pytest.mark.parametrize("dtype,cdt,D,Hq,Hkv,ps,order,seq,lens,opt", ATTEND_CASES)
def test_attend_matches_the_softmax(dtype, cdt, D, Hq, Hkv, ps, order, seq, lens, opt):
    T, pad = sum(lens), 2
    q, kc, vc, table, sl, (ks, vs) = _attend_inputs(dtype, cdt, D, Hq, Hkv, ps, order, seq, lens, pad=pad)
    slopes = 2.0 ** (-8.0 * torch.arange(1, Hq + 1, device="cuda") / Hq) if opt.get("bias") else None
    cap, window, scale = opt.get("softcap", 0.0), opt.get("window", 0), D ** -0.5
    out = torch.full((T + pad, Hq, D), 7.0, dtype=dtype, device="cuda")
    lse = torch.full((T + pad, Hq), 7.0, device="cuda")
    kda.kda_kv_decode(q, kc, vc, table, sl, out, cu_seqlens=_cu(lens), max_q=max(lens), softcap=cap, window=window,
                      alibi_slopes=slopes, lse=lse, k_scale=ks, v_scale=vs)
    _ok()
    o, l, ob, lb = ref.attend(q[:T], kc, vc, table, sl, lens, scale, cap, window, slopes, None, ks, vs)
    _within(lse[:T], l, lb)
    _within(out[:T], o, ob)
    assert (out[T:] == 7).all() and (lse[T:] == 7).all()


@pytest.mark.parametrize("dtype,cdt", [(BF16, BF16), (BF16, E4M3), (F32, F32)])
def test_attend_rows_that_see_nothing(dtype, cdt):
    """Keys before kv_start are invisible; rows without any key give 0 and -infinity."""
    seq, lens = [100, 40, 0, 64, 70, 3], [1, 2, 1, 1, 3, 1]
    q, kc, vc, table, sl, (ks, vs) = _attend_inputs(dtype, cdt, 64, 4, 2, 16, "heads", seq, lens)
    start = [90, 39, 0, 64, 1000, -5]   # one key, one row of two without, none, none, none, all
    T = sum(lens)
    out = torch.full((T, 4, 64), 7.0, dtype=dtype, device="cuda")
    lse = torch.full((T, 4), 7.0, device="cuda")
    for n, s in enumerate(start):   # what a row does not see may be anything
        for j in range(min(max(s, 0), seq[n])):
            kc[int(table[n, j // 16]), :, j % 16] = float("nan")
            vc[int(table[n, j // 16]), :, j % 16] = float("nan")
    kda.kda_kv_decode(q, kc, vc, table, sl, out, cu_seqlens=_cu(lens), max_q=3, kv_start=_ints(start), lse=lse, k_scale=ks,
                      v_scale=vs)
    _ok()
    o, l, ob, lb = ref.attend(q, kc, vc, table, sl, lens, 64 ** -0.5, start=[max(s, 0) for s in start], k_scale=ks, v_scale=vs)
    empty = torch.isinf(l)
    assert int(empty.any(1).sum()) == 1 + 1 + 1 + 3
    assert (out.cpu()[empty] == 0).all() and (lse.cpu()[empty] == -math.inf).all()
    _within(out, o, ob)
    seen = ~empty
    _within(lse.cpu()[seen], l[seen], lb[seen])


@pytest.mark.parametrize("dtype,cdt", [(BF16, BF16), (BF16, E4M3), (F32, F32)])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_attend_later_drafts_do_not_reach_earlier_tokens(dtype, cdt, bad):
    """A NaN or infinity in the key and value of one new token: the tokens before it keep their bits,
    the ones that see it do not, and a window that has passed it is clean again."""
    if cdt == E4M3:
        bad = float("nan")   # e4m3 has no infinity
    seq, lens, D, Hq = [70], [8], 64, 4
    q, kc, vc, table, sl, (ks, vs) = _attend_inputs(dtype, cdt, D, Hq, 2, 16, "heads", seq, lens)

    def go(window):
        out = torch.zeros(8, Hq, D, dtype=dtype, device="cuda")
        kda.kda_kv_decode(q, kc, vc, table, sl, out, cu_seqlens=_cu(lens), max_q=8, window=window, k_scale=ks, v_scale=vs)
        _ok()
        return out

    clean, narrow = go(0), go(3)
    j = 62 + 3   # the fourth new token
    for c in (kc, vc):
        c[int(table[0, j // 16]), :, j % 16] = bad
    a, b = go(0), go(3)
    assert torch.equal(a[:3], clean[:3]) and torch.equal(b[:3], narrow[:3])
    assert torch.equal(b[6:], narrow[6:])
    assert not torch.isfinite(a[3:].float()).all(-1).any() and not torch.isfinite(b[3:6].float()).all(-1).any()


def test_attend_reads_no_page_outside_the_window_and_reports_bad_pages():
    seq, lens = [200, 200], [1, 1]
    q, kc, vc, table, sl, _ = _attend_inputs(BF16, BF16, 64, 2, 1, 16, "heads", seq, lens)
    t2 = table.clone()
    t2[:, :9] = 10 ** 6   # pages before the window of 50 (positions 150 .. 199 start on page 9)
    out, o2 = (torch.zeros(2, 2, 64, dtype=BF16, device="cuda") for _ in range(2))
    kda.kda_kv_decode(q, kc, vc, table, sl, out, window=50)
    kda.kda_kv_decode(q, kc, vc, t2, sl, o2, window=50)
    _ok()
    assert torch.equal(out, o2)
    for bad in (-1, kc.shape[0]):
        t2 = table.clone()
        t2[1, 10] = bad
        kda.kda_kv_decode(q, kc, vc, t2, sl, o2)
        assert kda.kda_get_device_status() == kda.KDA_ERR_BAD_PAGE
        o, _, ob, _ = ref.attend(q, kc, vc, t2, sl, lens, 64 ** -0.5)   # the page is left out
        _within(o2, o, ob)
    kda.kda_kv_decode(q, kc, vc, table[:, :10].contiguous(), sl, o2)   # positions behind the table
    assert kda.kda_get_device_status() == kda.KDA_ERR_BAD_PAGE
    o, _, ob, _ = ref.attend(q, kc, vc, table[:, :10], sl, lens, 64 ** -0.5)
    _within(o2, o, ob)
    kda.kda_kv_decode(q, kc, vc, table, _ints([2 ** 31 - 1, 200]), o2)   # a length far behind the table
    assert kda.kda_get_device_status() == kda.KDA_ERR_BAD_PAGE
    _ok()


@pytest.mark.parametrize("dtype,cdt,Hq,Hkv,new", [(BF16, BF16, 8, 2, 1), (BF16, E4M3, 4, 1, 4), (F32, F32, 2, 2, 1),
                                                 (BF16, BF16, 16, 1, 5)])
def test_attend_long_ragged_batches_split_and_joined(dtype, cdt, Hq, Hkv, new):
    """Lengths from 1 to thousands in one call, so that rows are split at every kind of place."""
    seq = [5000, max(1, new), 1024, 31 + new, 2047, 8191, 32, 100]
    lens = [min(new, s) for s in seq]
    q, kc, vc, table, sl, (ks, vs) = _attend_inputs(dtype, cdt, 128, Hq, Hkv, 64, "heads", seq, lens)
    T = sum(lens)
    out, lse = torch.zeros(T, Hq, 128, dtype=dtype, device="cuda"), torch.zeros(T, Hq, device="cuda")
    kda.kda_kv_decode(q, kc, vc, table, sl, out, cu_seqlens=_cu(lens), max_q=new, lse=lse, k_scale=ks, v_scale=vs)
    _ok()
    o, l, ob, lb = ref.attend(q, kc, vc, table, sl, lens, 128 ** -0.5, k_scale=ks, v_scale=vs)
    _within(out, o, ob)
    _within(lse, l, lb)
    again = torch.empty_like(out)
    kda.kda_kv_decode(q, kc, vc, table, sl, again, cu_seqlens=_cu(lens), max_q=new, k_scale=ks, v_scale=vs)
    assert torch.equal(out, again)


def test_attend_offsets_beyond_32_bits():
    """A cache whose last pages lie more than 2^32 bytes and 2^31 elements from its start."""
    pages, ps, D = 131080, 128, 128   # 2.1 G elements, one head
    c = torch.zeros(pages, 1, ps, D, dtype=E4M3, device="cuda")
    gen = torch.Generator().manual_seed(3)
    rows = torch.randn(2, 150, D, generator=gen).mul(40).to(E4M3).cuda()
    table = _ints([[pages - 1, pages - 7]])
    one = torch.ones(1, device="cuda")
    c2 = torch.zeros(2, 1, ps, D, dtype=E4M3, device="cuda")
    q = torch.randn(1, 2, D, generator=gen).to(BF16).cuda()
    outs = []
    for cache, tab in ((c, table), (c2, _ints([[1, 0]]))):
        for p in range(2):
            part = rows[0, p * ps:(p + 1) * ps]
            cache[int(tab[0, p]), 0, :part.shape[0]] = part
        out = torch.zeros(1, 2, D, dtype=BF16, device="cuda")
        kda.kda_kv_decode(q, cache, cache, tab, _ints([150]), out, k_scale=one * 0.02, v_scale=one * 0.02)
        outs.append(out)
    _ok()
    assert torch.equal(outs[0], outs[1]) and outs[0].abs().max() > 0
    # and appending there
    k = torch.randn(1, 1, D, generator=gen).to(BF16).cuda()
    kda.kda_kv_append(k, k, c, c, table, _ints([151]), k_scale=one, v_scale=one)
    _ok()
    assert torch.equal(c[pages - 7, 0, 22].float(), k[0, 0].float().clamp(-448, 448).to(E4M3).float())


# ------------------------------------------------------------------------------- as a stack uses them

class _Stack:
    """A KDA layer and an attention layer, with a state pool and a paged cache."""

    def __init__(self, N, D=128, H=2, Hq=4, ps=16, seed=50, max_pages=8):
        gen = torch.Generator().manual_seed(seed)
        self.N, self.D, self.H, self.Hq, self.ps = N, D, H, Hq, ps
        self.pool = torch.zeros(N * 6, H, D, D, device="cuda")
        self.kc, self.vc = (torch.full((N * max_pages, 1, ps, D), float("nan"), dtype=BF16, device="cuda") for _ in range(2))
        self.table = torch.randperm(N * max_pages, generator=gen).to(torch.int32).view(N, max_pages).cuda()
        self.inv = (10000.0 ** (-torch.arange(D // 2, dtype=torch.float64) / (D // 2))).float().cuda()

    def step(self, x, cu, seq_lens, slots_in, slots_out, max_q, ws=None, stream=None):
        T = x["q"].shape[0]
        o1 = torch.empty(T, self.H, self.D, dtype=BF16, device="cuda")
        o2 = torch.empty(T, self.Hq, self.D, dtype=BF16, device="cuda")
        kda.kda_decode_pool(x["q"], x["k"], x["v"], x["g"], x["beta"], self.pool, slots_in, slots_out, o1, cu_seqlens=cu,
                            stream=stream)
        qr = kda.kda_kv_append(x["ak"], x["av"], self.kc, self.vc, self.table, seq_lens, cu_seqlens=cu, q=x["aq"],
                               inv_freq=self.inv, stream=stream)
        kda.kda_kv_decode(qr, self.kc, self.vc, self.table, seq_lens, o2, cu_seqlens=cu, max_q=max_q, workspace=ws,
                          stream=stream)
        return o1, o2

    def inputs(self, T, seed):
        x = synthetic.make_prefill_inputs([T], self.H, self.D, self.D, BF16, 3.0, 0.0, seed)
        x = {k: v.cuda() for k, v in x.items() if v is not None}
        gen = torch.Generator().manual_seed(seed)
        for key, h in (("aq", self.Hq), ("ak", 1), ("av", 1)):
            x[key] = torch.randn(T, h, self.D, generator=gen).to(BF16).cuda()
        return x


def test_stack_prefill_then_drafts_with_roll_back_equal_token_by_token():
    """A prompt by kda_prefill into the pool, drafts of 4 tokens of which 2 are accepted, then more
    drafts from there: the outputs of a run that appends one token at a time."""
    N, prompt, D = 3, [70, 64, 5], 128
    a, b = _Stack(N), _Stack(N)
    x0 = a.inputs(sum(prompt), 1)
    out = torch.empty(sum(prompt), a.H, D, dtype=BF16, device="cuda")
    fin = torch.empty(N, a.H, D, D, device="cuda")
    kda.kda_prefill(x0["q"], x0["k"], x0["v"], x0["g"], x0["beta"], _cu(prompt), out, final_state=fin)
    for s in (a, b):
        s.pool[:N] = fin
        kda.kda_kv_append(x0["ak"], x0["av"], s.kc, s.vc, s.table, _ints(prompt), cu_seqlens=_cu(prompt), inv_freq=s.inv)
    draft, more = a.inputs(4 * N, 2), a.inputs(3 * N, 3)
    # drafts: token i of sequence n keeps its state in slot N + 4 n + i
    slots = _ints([N + 4 * n + i for n in range(N) for i in range(4)])
    o1, o2 = a.step(draft, _cu([4] * N), _ints([p + 4 for p in prompt]), _ints(list(range(N))), slots, 4)
    # two accepted; three more tokens from there, over the rejected ones' rows
    p1, p2 = a.step(more, _cu([3] * N), _ints([p + 5 for p in prompt]), _ints([N + 4 * n + 1 for n in range(N)]),
                    _ints([-1, -1, 0, -1, -1, 1, -1, -1, 2]), 3)
    # one token at a time
    seq = list(prompt)
    for i in range(5):
        src, j, width, w1, w2 = (draft, i, 4, o1, o2) if i < 2 else (more, i - 2, 3, p1, p2)
        rows = torch.tensor([width * n + j for n in range(N)], device="cuda")
        seq = [s + 1 for s in seq]
        ids = _ints(list(range(N)))
        r1, r2 = b.step({k: (v[rows].contiguous() if k != "cu_seqlens" else v) for k, v in src.items()}, None, _ints(seq), ids, ids, 1)
        assert torch.equal(r1, w1[rows])   # the recurrence: the same bits
        assert torch.allclose(r2.float(), w2[rows].float(), rtol=2.0 ** -6, atol=2.0 ** -7)   # both within 2^-8 of p and of o
    _ok()
    assert torch.equal(a.pool[:N], b.pool[:N])


def test_stack_step_captured_and_replayed_follows_new_lengths():
    """One captured step replayed on new contents (inputs, lengths, slots, fewer tokens) gives the
    bits of an eager step; a second graph with its own workspace does not disturb it."""
    N = 4
    eager, cap = _Stack(N), _Stack(N)
    T = 3 * N
    x = cap.inputs(T, 7)
    cu, seq = _cu([3] * N), _ints([3] * N)
    sin, sout = _ints([-1] * N), _ints([n for n in range(N) for _ in range(3)])
    need = kda.kda_kv_decode_workspace_size(N, 4, 1, 128, 3)
    ws, ws2 = (torch.empty(need, dtype=torch.uint8, device="cuda") for _ in range(2))
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        cap.step(x, cu, seq, sin, sout, 3, ws)
    torch.cuda.synchronize()
    cap.pool.zero_()
    graph, graph2 = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        g1, g2 = cap.step(x, cu, seq, sin, sout, 3, ws)
    with torch.cuda.graph(graph2):
        h1, h2 = cap.step(x, cu, seq, sin, sout, 3, ws2)
    base = [0] * N
    for r, lens in enumerate(([3, 3, 3, 3], [1, 3, 0, 2], [2, 2, 2, 2])):
        new = cap.inputs(T, 70 + r)
        for key in x:
            x[key].copy_(new[key])
        base = [b + n for b, n in zip(base, lens)]
        so = [n for n in range(N) for _ in range(lens[n])]
        so += [-1] * (T - len(so))
        cu.copy_(_cu(lens)); seq.copy_(_ints(base)); sout.copy_(_ints(so))
        sin.copy_(_ints([-1] * N if r == 0 else list(range(N))))
        g1.fill_(5); g2.fill_(5)
        before = cap.pool.clone()
        graph.replay()
        w1, w2 = eager.step(x, cu, seq, sin, sout, 3)
        torch.cuda.synchronize()
        m = sum(lens)
        assert torch.equal(g1[:m], w1[:m]) and torch.equal(g2[:m], w2[:m])
        assert (g1[m:] == 5).all() and (g2[m:] == 5).all()
        assert torch.equal(cap.pool, eager.pool)
        # the second graph on the state before gives the same
        after = cap.pool.clone()
        cap.pool.copy_(before)
        graph2.replay()
        torch.cuda.synchronize()
        assert torch.equal(h1[:m], w1[:m]) and torch.equal(h2[:m], w2[:m]) and torch.equal(cap.pool, after)
    _ok()


def test_stack_on_another_stream_and_two_at_once():
    """Work on a stream that is not the current one, workspaces allocated inside; two at once."""
    N = 3
    a, b, c = _Stack(N), _Stack(N), _Stack(N, seed=51)
    xs, xc = a.inputs(N, 11), c.inputs(N, 12)
    ids, seq = _ints(list(range(N))), _ints([1] * N)
    w1, w2 = b.step(xs, None, seq, _ints([-1] * N), ids, 1)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    fresh = _ints([-1] * N)
    torch.cuda.synchronize()
    for _ in range(20):
        r = a.step(xs, None, seq, fresh, ids, 1, stream=s1)
        c.step(xc, None, seq, fresh, ids, 1, stream=s2)
    torch.cuda.synchronize()
    _ok()
    assert torch.equal(r[0], w1) and torch.equal(r[1], w2)

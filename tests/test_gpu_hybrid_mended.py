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

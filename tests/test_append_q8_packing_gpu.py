"""The append into the 8-bit cache with a packing that does not rise: it is reported, and every page and every row of q_out is either as
it was or holds what a sequence that is in order puts there."""
import pytest
import torch

import q8_reference as R

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def S():
    from gqa_attention_learned_head_gb300 import sinkattn

    return sinkattn


@pytest.mark.parametrize("rot", [True, False])
@pytest.mark.parametrize("cu", [[0, 100, 50, 120], [0, 100, 10, 30], [0, 40, 39, 120], [-5, 40, 80, 120], [0, 40, 80, 121], [0, 2**31 - 1, 80, 120],
                                [120, 80, 40, 0], [0, 120, 0, 120]])
def test_pages_whole_or_as_they_were(S, rot, cu):
    Hq, Hkv, T, start = 4, 2, 120, [0, 5, 16]
    pp, cache = R.paged(Hq, Hkv, start, [120, 120, 120], seed=23)  # (pages for whatever length a sequence is given)
    cache = R.Cache(cache.k_wide, cache.v_wide)  # as the copies below are made (packing what was rounded may lower a scale)
    g = torch.Generator(device="cuda").manual_seed(4)
    qkv = torch.randn(T, (Hq + 2 * Hkv) * 64, device="cuda", generator=g).to(torch.bfloat16)
    kv = qkv.view(T, -1, 64)
    table = pp.page_table.cuda()
    q_out = torch.full((T, Hq, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731

    def call(a, b, offsets, starts, tab, c, out):
        if rot:
            S.sinkattn_qkv_prologue_q8(qkv[a:b], None, i32(offsets), i32(starts), tab, *c.args, Hq, q_out=out, **R.YARN)
        else:
            S.sinkattn_kv_append_q8(kv[a:b, Hq : Hq + Hkv].contiguous(), kv[a:b, Hq + Hkv :].contiguous(), i32(offsets), i32(starts), tab, *c.args)

    got = R.Cache(cache.k_wide, cache.v_wide)
    call(0, T, cu, start, table, got, q_out)
    assert S.sinkattn_get_error() == S.ERR_BAD_LENGTH
    state = lambda c, p: (c.k.view(torch.uint8)[p], c.v.view(torch.uint8)[p], c.scales[p])  # noqa: E731
    same = lambda x, y: all(torch.equal(a, b) for a, b in zip(x, y))  # noqa: E731
    may = {p: [] for p in range(cache.k_wide.shape[0])}
    rows = {t: [] for t in range(T)}
    for n in range(3):
        a, b = cu[n], cu[n + 1]
        if not 0 <= a <= b <= T or a == b:
            continue
        alone, q = R.Cache(cache.k_wide, cache.v_wide), torch.full((b - a, Hq, 64), 7.0, dtype=torch.bfloat16, device="cuda")
        call(a, b, [0, b - a], [start[n]], table[n : n + 1].contiguous(), alone, q)
        assert S.sinkattn_get_error() == 0
        for p in table[n].tolist():
            if p >= 0:
                may[p].append(state(alone, p))
        for t in range(a, b):
            rows[t].append(q[t - a])
    for p, choices in may.items():
        assert any(same(state(got, p), c) for c in [state(cache, p)] + choices), p
    for t, choices in rows.items():  # (a row that two sequences claim may hold pieces of either)
        was = torch.full_like(q_out[t], 7.0)
        for h in range(Hq):
            assert any(torch.equal(q_out[t, h], c[h]) for c in [was] + choices) or len(choices) > 1, t

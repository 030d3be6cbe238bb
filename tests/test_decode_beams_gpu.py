"""Decode of rows that share pages on the GPU against the fp64 oracle (which decodes every row on its own), through the
C ABI."""
import random

import pytest
import torch

import oracle
from gqa_attention_learned_head_gb300 import workloads as W
from parity_utils import assert_parity

pytestmark = pytest.mark.gpu

PS = 16


@pytest.fixture(scope="module")
def S():
    from gqa_attention_learned_head_gb300 import sinkattn

    return sinkattn


def make(Hq, Hkv, lens, seed=0, share="tree", garbage=True, max_pages=None):
    """N groups of K rows, lens [N][K].  share: "tree" (a common prefix, then pairs, then own pages), "all" (the longest
    row's pages), "none", "random" (any earlier row's page in the same column).  Slots past the last token of every
    holder, and pages that no row holds, are NaN where ``garbage``."""
    rng = random.Random(seed)
    N, K = len(lens), len(lens[0])
    longest = max(max(x) for x in lens)
    mp = max(1, (longest + PS - 1) // PS) if max_pages is None else max_pages
    table = torch.full((N, K, mp), -1, dtype=torch.int32)
    used, slots = 0, {}
    for n in range(N):
        for c in range(mp):
            seen = []
            for k in range(K):
                if c * PS >= lens[n][k]:
                    continue
                first = (max(lens[n]) // PS) // 2
                owner = {"all": 0, "none": k, "tree": 0 if c < first else (k // 2 * 2 if c < first + 2 else k),
                         "random": rng.randint(0, k)}[share]
                page = next((p for o, p in seen if o == owner), None)
                if page is None or (share == "random" and rng.random() < 0.3):
                    page, used = used, used + 1
                seen.append((owner, page))
                table[n, k, c] = page
                slots[page] = max(slots.get(page, 0), min(PS, lens[n][k] - c * PS))
    P = used + 3
    perm = torch.tensor(rng.sample(range(P), P), dtype=torch.int32)
    g = torch.Generator().manual_seed(seed)
    q = torch.randn(N, K, Hq, 64, generator=g).to(torch.bfloat16)
    k = torch.randn(P, Hkv, PS, 64, generator=g).to(torch.bfloat16)
    v = torch.randn(P, Hkv, PS, 64, generator=g).to(torch.bfloat16)
    if garbage:
        for p in range(P):
            s = slots.get(p, 0)
            k[perm[p], :, s:] = float("nan")
            v[perm[p], :, s:] = float("nan")
    table = torch.where(table >= 0, perm[table.clamp(min=0).long()], table)
    sinks = torch.randn(Hq, generator=g)
    return q, k, v, table, torch.tensor(lens, dtype=torch.int32), sinks


def run(S, q, k, v, table, lens, sinks, scale=0.125, **kw):
    out, lse = S.sinkattn_decode_beams(q.cuda(), k.cuda(), v.cuda(), table.cuda(), lens.cuda(), sinks.cuda(), scale, **kw)
    return out, lse, S.sinkattn_get_error()


def ref(q, k, v, table, lens, sinks, scale=0.125):
    N, K, Hq, D = q.shape
    out, lse = oracle.decode(q.view(N * K, Hq, D), torch.nan_to_num(k), torch.nan_to_num(v), table.view(N * K, -1),
                             lens.view(-1), sinks, scale)
    return out.reshape(N, K, Hq, D), lse.reshape(N, K, Hq)


def check(S, *inp, what="", **kw):
    out, lse, err = run(S, *inp, **kw)
    assert err == 0
    assert_parity(out.float().cpu().numpy(), lse.cpu().numpy(), *ref(*inp, **({"scale": kw["scale"]} if "scale" in kw else {})),
                  what)


# (Hq, Hkv, K): rows K * Hq / Hkv from 1 to 128
SHAPES = [(1, 1, 1), (8, 1, 1), (4, 4, 5), (8, 8, 32), (16, 2, 4), (5, 1, 6), (10, 2, 7), (64, 8, 8), (64, 8, 16),
          (16, 1, 8), (4, 1, 32), (128, 1, 1), (48, 1, 2), (33, 1, 3)]


@pytest.mark.parametrize("Hq,Hkv,K", SHAPES)
@pytest.mark.parametrize("share", ["tree", "random"])
def test_shapes(S, Hq, Hkv, K, share):
    rng = random.Random(Hq + K)
    lens = [[L] * K for L in (1, 16, 130)] + [[rng.randint(0, 200) for _ in range(K)]]
    check(S, *make(Hq, Hkv, lens, seed=Hq + K, share=share), what=f"{Hq} {Hkv} {K} {share}")


@pytest.mark.parametrize("share", ["all", "none", "tree", "random"])
@pytest.mark.parametrize("lens", [[[0, 0, 0], [5, 0, 33]], [[127, 128, 129], [1, 1, 1], [0, 0, 0], [700, 650, 3]],
                                  [[16, 16, 17]], [[15, 31, 47], [255, 256, 257]]])
def test_lengths(S, lens, share):
    check(S, *make(16, 2, lens, seed=len(lens), share=share), what=f"{lens} {share}")


@pytest.mark.parametrize("workers", [1, 2, 7, 50, 300, 2000])
def test_forced_splits(S, workers):
    """Equal shares cut groups anywhere: pieces of every size, merged by log-sum-exp."""
    inp = make(64, 8, [[300, 290, 310, 300], [20, 20, 20, 20], [900, 900, 901, 3]], seed=31)
    check(S, *inp, what=f"workers={workers}", num_workers=workers)


@pytest.mark.parametrize("sink", [float("-inf"), -30.0, 30.0])
def test_sink_values(S, sink):
    inp = make(16, 2, [[40, 0, 129], [0, 0, 0], [3, 3, 3]], seed=32)
    inp[5][:] = sink
    check(S, *inp, what=f"sink={sink}")


@pytest.mark.parametrize("scale", [0.0, -0.125, 1.0])
def test_scales(S, scale):
    check(S, *make(16, 2, [[40, 17, 129]], seed=33), what=f"scale={scale}", scale=scale)


@pytest.mark.parametrize("Hq,Hkv,K", [(8, 1, 3), (64, 8, 8), (64, 8, 16), (5, 1, 6)])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
@pytest.mark.parametrize("workers", [0, 7])
def test_poisoned_row(S, Hq, Hkv, K, value, workers):
    """A value that is not finite in a row's own pages stays that row's, whichever rows its tiles hold besides."""
    lens = [[300 - 7 * k for k in range(K)], [40] * K, [1200] * K]
    q, k, v, table, lens, sinks = make(Hq, Hkv, lens, seed=K, share="tree")
    ro, rl = ref(q, k, v, table, lens, sinks)
    hit = torch.zeros(3, K, dtype=torch.bool)
    for n in range(3):
        last = (int(lens[n, 1]) - 1) // PS  # row 1's last page: every column this late is a row's own
        page = int(table[n, 1, last])
        hit[n] = (table[n, :, last] == page)
        v[page, :, 0, 5] = value
        v[page, :, 1, 50] = value
    assert hit.any(1).all() and not hit.all(1).any()
    out, lse, err = run(S, q, k, v, table, lens, sinks, num_workers=workers)
    assert err == 0
    out, lse = out.float().cpu(), lse.cpu()
    assert not torch.isfinite(out[hit][..., 5]).any() and not torch.isfinite(out[hit][..., 50]).any()
    assert_parity(out[~hit].numpy(), lse[~hit].numpy(), torch.as_tensor(ro)[~hit].numpy(), torch.as_tensor(rl)[~hit].numpy(),
                  f"{Hq} {Hkv} {K} {value}")
    # ... and a key that is not finite: its row's scores only
    v[~torch.isfinite(v.float())] = 0
    for n in range(3):
        k[int(table[n, 1, (int(lens[n, 1]) - 1) // PS]), :, 0] = value
    ro, rl = ref(q, k, v, table, lens, sinks)
    out, lse, err = run(S, q, k, v, table, lens, sinks, num_workers=workers)
    assert err == 0
    assert_parity(out.float().cpu()[~hit].numpy(), lse.cpu()[~hit].numpy(), torch.as_tensor(ro)[~hit].numpy(),
                  torch.as_tensor(rl)[~hit].numpy(), f"key {Hq} {Hkv} {K} {value}")


def test_rising_scores(S):
    """Scores that grow along the cache: the running maximum is exceeded again and again, in whole and split groups."""
    q, k, v, table, lens, sinks = make(16, 2, [[2000, 1990, 2000, 1500]], seed=34, share="tree")
    q = (1 + 0.05 * torch.randn(q.shape)).to(torch.bfloat16)
    pos = torch.arange(table.shape[2] * PS).view(-1, PS)
    for b in range(4):
        for c in range((int(lens[0, b]) + PS - 1) // PS):
            ok = torch.isfinite(k[table[0, b, c]].float())
            rise = (5.0 * pos[c] / 2000)[None, :, None].expand(2, PS, 64).to(torch.bfloat16)
            k[table[0, b, c]] = torch.where(ok, rise, k[table[0, b, c]])
    for workers in (0, 1, 9):
        check(S, q, k, v, table, lens, sinks, what=f"rising, {workers} workers", num_workers=workers)


def test_long_table(S):
    """A table row of more than one step of columns, read by a cluster; groups of very different lengths."""
    lens = [[30000, 30000, 29990], [100, 100, 100], [17000, 3, 16500]]
    check(S, *make(8, 1, lens, seed=35, garbage=False), what="long")
    check(S, *make(8, 1, [[500, 500, 500]], seed=36, max_pages=5000), what="wide table")


def test_many_groups(S):
    """More groups than one step of the share search covers."""
    rng = random.Random(1)
    lens = [[rng.randint(0, 40) for _ in range(2)] for _ in range(700)]
    check(S, *make(4, 2, lens, seed=37), what="700 groups")


def test_most_groups(S):
    """The largest batch, a row or two each."""
    rng = random.Random(2)
    lens = [[rng.randint(0, 20)] for _ in range(32768)]
    check(S, *make(2, 1, lens, seed=44, garbage=False), what="32768 groups")


def test_equals_decode_on_the_rows(S):
    q, k, v, table, lens, sinks = (t.cuda() for t in make(64, 8, [[1000] * 8, [333] * 8], seed=38, garbage=False))
    out, lse = S.sinkattn_decode_beams(q, k, v, table, lens, sinks, 0.125)
    o2, l2 = S.sinkattn_decode(q.view(16, 64, 64), k, v, table.view(16, -1), lens.view(-1), sinks, 0.125)
    assert S.sinkattn_get_error() == 0
    assert_parity(out.view(16, 64, 64).float().cpu().numpy(), lse.view(16, 64).cpu().numpy(), o2.float().cpu().numpy(),
                  l2.cpu().numpy(), "against sinkattn_decode")


def test_repeats_give_the_same_bits(S):
    inp = [t.cuda() for t in make(64, 8, [[700] * 8, [333, 1, 0, 90, 333, 333, 333, 333]], seed=39)]
    first = S.sinkattn_decode_beams(*inp, 0.125)
    for _ in range(3):
        again = S.sinkattn_decode_beams(*inp, 0.125)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


def test_bad_pages_and_lengths_are_reported(S):
    q, k, v, table, lens, sinks = make(16, 2, [[200, 200, 200], [64, 64, 64]], seed=40, garbage=False)
    bad = table.clone()
    bad[0, 1, 3] = 10 ** 6
    bad[1, :, 0] = -9
    out, lse, err = run(S, q, k, v, bad, lens, sinks)
    assert err == S.ERR_BAD_PAGE
    keep = torch.ones(2, 3, table.shape[2], dtype=torch.bool)
    keep[0, 1, 3] = keep[1, :, 0] = False
    for n in range(2):
        for b in range(3):  # the row without the absent pages' tokens
            cols = [c for c in range(table.shape[2]) if keep[n, b, c] and c * PS < int(lens[n, b])]
            L = sum(min(PS, int(lens[n, b]) - c * PS) for c in cols)
            t = table[n, b, cols][None]
            o, l2 = oracle.decode(q[n, b][None], k, v, t, torch.tensor([L], dtype=torch.int32), sinks, 0.125)
            assert_parity(out[n, b].float().cpu().numpy()[None], lse[n, b].cpu().numpy()[None], o, l2, f"{n} {b}")
    lens2 = lens.clone()
    lens2[0, 2], lens2[1, 0] = 10 ** 6, -3
    table2 = table.clone()
    table2[0, 2] = table[0, 2]
    out, lse, err = run(S, q, k, v, table2, lens2, sinks)
    assert err == S.ERR_BAD_LENGTH
    clamped = lens2.clamp(0, table.shape[2] * PS)
    assert_parity(out.float().cpu().numpy(), lse.cpu().numpy(), *ref(q, k, v, table2, clamped, sinks), "clamped")


def test_empty_pool_and_no_groups(S):
    q, _, _, _, _, sinks = make(16, 2, [[5, 5]], seed=41)
    none = torch.empty(0, 2, PS, 64, dtype=torch.bfloat16)
    out, lse, err = run(S, q, none, none, torch.zeros(1, 2, 1, dtype=torch.int32), torch.zeros(1, 2, dtype=torch.int32), sinks)
    assert err == 0 and not out.any() and torch.equal(lse.cpu(), sinks.expand(1, 2, 16))
    out, lse, err = run(S, q, none, none, torch.zeros(1, 2, 1, dtype=torch.int32), torch.ones(1, 2, dtype=torch.int32), sinks)
    assert err == S.ERR_BAD_PAGE and not out.any()
    inp = make(16, 2, [[5, 5]], seed=41)
    out, lse, err = run(S, inp[0][:0], inp[1], inp[2], inp[3][:0], inp[4][:0], inp[5])
    assert err == 0 and out.shape == (0, 2, 16, 64)


def test_replayed_from_a_graph_with_new_tables(S):
    a = make(64, 8, [[400] * 8, [130] * 8], seed=42, garbage=False)
    q, k, v, table, lens, sinks = (t.cuda() for t in a)
    ws = torch.empty(S.sinkattn_decode_beams_workspace_size(q, k, table), dtype=torch.uint8, device="cuda")
    out, lse = torch.empty_like(q), torch.empty(2, 8, 64, device="cuda")
    S.sinkattn_decode_beams(q, k, v, table, lens, sinks, 0.125, out=out, lse=lse, workspace=ws)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        S.sinkattn_decode_beams(q, k, v, table, lens, sinks, 0.125, out=out, lse=lse, workspace=ws)
    table2 = a[3].clone()
    table2[:, 1:] = a[3][:, :1]  # every row now holds row 0's pages
    table2[1, 3, 5] = a[3][0, 0, 0]
    lens2 = a[4].clone()
    lens2[0, 5], lens2[1, 2] = 3, 0
    table.copy_(table2)
    lens.copy_(lens2)
    ws.fill_(0x7F)  # nothing in the workspace carries over
    for _ in range(2):
        g.replay()
    torch.cuda.synchronize()
    assert S.sinkattn_get_error() == 0
    assert_parity(out.float().cpu().numpy(), lse.cpu().numpy(), *ref(a[0], a[1], a[2], table2, lens2, a[5]), "replayed")


def test_refusals(S):
    inp = [t.cuda() for t in make(16, 2, [[5, 5]], seed=43)]
    q, k, v, table, lens, sinks = inp
    with pytest.raises(TypeError):
        S.sinkattn_decode_beams(q.float(), k, v, table, lens, sinks, 0.125)
    with pytest.raises(ValueError):
        S.sinkattn_decode_beams(q, k, v, table[:, :1].contiguous(), lens, sinks, 0.125)
    with pytest.raises(ValueError):
        S.sinkattn_decode_beams(q, k, v[:1], table, lens, sinks, 0.125)
    with pytest.raises(ValueError):
        S.sinkattn_decode_beams(q, k, v, table, lens, sinks[:3], 0.125)
    with pytest.raises(S.SinkAttnError) as e:
        S.sinkattn_decode_beams(q, k, v, table, lens, sinks, float("nan"))
    assert e.value.status == S.ERR_INVALID_ARG
    big = torch.zeros(1, 17, 16, 64, dtype=torch.bfloat16, device="cuda")  # 17 x 8 = 136 rows
    with pytest.raises(S.SinkAttnError) as e:
        S.sinkattn_decode_beams(big, k, v, torch.zeros(1, 17, 1, dtype=torch.int32, device="cuda"),
                                torch.zeros(1, 17, dtype=torch.int32, device="cuda"), sinks, 0.125)
    assert e.value.status == S.ERR_UNSUPPORTED
    with pytest.raises(S.SinkAttnError) as e:
        S.sinkattn_decode_beams(*inp, 0.125, workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))
    assert e.value.status == S.ERR_WORKSPACE


@pytest.mark.parametrize("width", [8, 32, 63, 65, 128])
def test_pools_of_another_head_size_are_refused(S, width):
    """The kernel takes a page as 64 values a token, whatever the pool was made for."""
    q, k, v, table, lens, sinks = [t.cuda() for t in make(16, 2, [[5, 5]], seed=45)]
    other = torch.zeros(*k.shape[:3], width, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ValueError):
        S.sinkattn_decode_beams(q, other, other, table, lens, sinks, 0.125)
    with pytest.raises(ValueError):
        S.sinkattn_decode_beams(q, k, other, table, lens, sinks, 0.125)
    assert S.sinkattn_get_error() == 0

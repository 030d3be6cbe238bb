"""Page-table forks, page copies and the compaction of accepted tokens on the GPU against plain Python, through the C
ABI.  Whole numbers and copies: everything has to be equal."""
import random

import pytest
import torch

pytestmark = pytest.mark.gpu

PS = 16


@pytest.fixture(scope="module")
def S():
    from gqa_attention_learned_head_gb300 import sinkattn

    return sinkattn


def cols(n):
    return (n + PS - 1) // PS


def fork_reference(table, held, parents, refs, keep=None, room=None, grow=0):
    """The definition, row by row; lists of ints.  None in place of the results where pages are short."""
    mp, R = len(table[0]) if table else 0, len(parents)
    keep = [held[p] if p >= 0 else 0 for p in parents] if keep is None else keep
    room = [k + grow if p >= 0 else 0 for k, p in zip(keep, parents)] if room is None else room
    writes = [m > k and k % PS != 0 for k, m in zip(keep, room)]
    free = [p for p, c in enumerate(refs) if c == 0]
    new_table, copies = [], []
    for r, p in enumerate(parents):
        kept = [table[p][c] for c in range(cols(keep[r]))] if p >= 0 else []
        copy = (-1, -1, 0)
        if writes[r]:
            mates = [q for q in range(R) if parents[q] == p]
            alone = refs[kept[-1]] == 1 and all(writes[q] and keep[q] == keep[r] for q in mates) and mates[0] == r
            if not alone:
                if not free:
                    return None
                page = free.pop(0)
                copy = (kept[-1], page, keep[r] % PS)
                kept[-1] = page
        while len(kept) < cols(room[r]):
            if not free:
                return None
            kept.append(free.pop(0))
        new_table.append(kept)
        copies.append(copy)
    counts = list(refs)
    for p in range(len(table)):
        for c in range(cols(held[p])):
            counts[table[p][c]] -= 1
    for row in new_table:
        for page in row:
            counts[page] += 1
    return new_table, room, counts, copies


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def call(S, table, mp, held, parents, refs, keep=None, room=None, grow=0, **kw):
    t = torch.full((len(table), mp), 123456789, dtype=torch.int32)  # columns that are not to be read
    for i, row in enumerate(table):
        t[i, :cols(held[i])] = torch.tensor(row[:cols(held[i])], dtype=torch.int32)
    return S.sinkattn_pages_fork(t.cuda(), ints(held), ints(parents), ints(refs), None if keep is None else ints(keep),
                                 None if room is None else ints(room), grow, **kw)


def same(got, ref, mp):
    new_table, room, counts, copies = ref
    want = torch.full((len(room), mp), -1, dtype=torch.int32)
    for i, row in enumerate(new_table):
        want[i, :len(row)] = torch.tensor(row, dtype=torch.int32)
    assert torch.equal(got[0].cpu(), want)
    assert got[1].tolist() == room
    assert got[2].tolist() == counts
    assert [tuple(c) for c in got[3].tolist()] == copies


def random_state(rng, rows, mp, P, sharing=0.5):
    """Rows of random lengths; a row may share the first pages of an earlier one."""
    order = list(range(P))
    rng.shuffle(order)
    table, held, refs = [], [], [0] * P
    for r in range(rows):
        n = rng.randint(0, mp * PS)
        row = []
        if table and rng.random() < sharing:
            row = rng.choice(table)[:]
            row = row[:min(len(row), rng.randint(0, cols(n)))]
        while len(row) < cols(n) and order:
            row.append(order.pop())
        n = min(n, len(row) * PS)
        table.append(row)
        held.append(n)
        for page in row:
            refs[page] += 1
    return table, held, refs


@pytest.mark.parametrize("seed", range(12))
def test_random_forks(S, seed):
    rng = random.Random(seed)
    rows, mp = rng.choice([1, 3, 40, 130]), rng.choice([1, 5, 33])
    P = rows * mp * 3 + rng.randint(0, 3000)
    table, held, refs = random_state(rng, rows, mp, P)
    R = rng.choice([1, rows, 2 * rows, 300])
    parents = [rng.randint(-1, rows - 1) for _ in range(R)]
    keep = [rng.randint(0, held[p]) if p >= 0 and rng.random() < 0.5 else (held[p] if p >= 0 else 0) for p in parents]
    room = [rng.randint(k, mp * PS) if rng.random() < 0.7 else k for k in keep]
    got = call(S, table, mp, held, parents, refs, keep, room)
    assert S.sinkattn_get_error() in ((0, S.ERR_NO_PAGES))
    ref = fork_reference(table, held, parents, refs, keep, room)
    if ref is None:
        assert got[2].tolist() == refs and (got[0] == -1).all() and (got[1] == 0).all()
    else:
        same(got, ref, mp)


@pytest.mark.parametrize("length", [1, 15, 16, 17, 160])
def test_beam_step(S, length):
    """Every row grows by a token: one child goes on in place, two children copy a partial page, none frees."""
    mp, K = 12, 4
    refs = [0] * 64
    table = [list(range(10 * k, 10 * k + cols(length))) for k in range(K)]
    for row in table:
        for page in row:
            refs[page] += 1
    for parents in ([0, 1, 2, 3], [3, 2, 1, 0], [1, 1, 1, 1], [2, 0, 2, 3]):
        got = call(S, table, mp, [length] * K, parents, refs, grow=1)
        assert S.sinkattn_get_error() == 0
        same(got, fork_reference(table, [length] * K, parents, refs, grow=1), mp)


def test_cases_by_hand(S):
    """A page with an outside holder, children that keep different lengths, a new request, a freed one, a fork that
    writes nothing."""
    table, held = [[4, 5], [4, 6], [7]], [20, 30, 16]
    refs = [0] * 12
    for row in table:
        for p in row:
            refs[p] += 1
    refs[6] += 1  # held outside the table as well
    for parents, keep, room in (([0], [20], [21]), ([1], [30], [31]), ([0, 0], [20, 17], [21, 18]),
                                ([0, 0], [20, 20], [20, 40]), ([0, 0], [20, 16], [20, 17]), ([-1, 2], [0, 16], [33, 17]),
                                ([0, 1, 2, -1], [20, 30, 16, 0], [20, 30, 16, 0]), ([2, 2, 2], [16, 8, 0], [16, 8, 16])):
        got = call(S, table, 4, held, parents, refs, keep, room)
        assert S.sinkattn_get_error() == 0
        same(got, fork_reference(table, held, parents, refs, keep, room), 4)


def test_in_place_counts_and_no_rows(S):
    table, held = [[0, 1], [0, 2]], [32, 20]
    refs = [2, 1, 1, 0, 0]
    r = ints(refs)
    t = ints([[0, 1, -1], [0, 2, -1]])
    out = S.sinkattn_pages_fork(t, ints(held), ints([1, 1]), r, grow=1, out_refs=r)
    assert out[2].data_ptr() == r.data_ptr() and S.sinkattn_get_error() == 0
    same(out, fork_reference(table, held, [1, 1], refs, grow=1), 3)
    none = torch.empty(0, dtype=torch.int32, device="cuda")
    out = S.sinkattn_pages_fork(t, ints(held), none, ints(refs))  # every row ends
    assert out[2].tolist() == [0] * 5 and out[0].shape == (0, 3)
    out = S.sinkattn_pages_fork(torch.empty(0, 3, dtype=torch.int32, device="cuda"), none, ints([-1, -1]), ints([1, 0, 0, 1, 0]),
                                room_lens=ints([17, 3]))  # the first requests
    assert out[0].tolist() == [[1, 2, -1], [4, -1, -1]] and out[2].tolist() == [1, 1, 1, 1, 1]
    assert S.sinkattn_get_error() == 0


def test_large_pool_and_table(S):
    """More pages, rows and columns than one step of the cluster covers."""
    rng = random.Random(5)
    rows, mp, P = 1500, 70, 100003
    table, held, refs = [], [], [1] * P  # the rest of the pool is held elsewhere, but for every seventh page
    ids = list(range(P))
    rng.shuffle(ids)
    for r in range(rows):
        n = rng.randint(1, 60 * PS)
        row = [ids.pop() for _ in range(cols(n))]
        table.append(row)
        held.append(n)
    for p in ids:
        refs[p] = 0 if p % 7 == 0 else 1
    parents = [rng.randrange(rows) for _ in range(2000)]
    room = [held[p] + rng.randint(0, 40) for p in parents]
    keep = [held[p] for p in parents]
    got = call(S, table, mp, held, parents, refs, keep, room)
    assert S.sinkattn_get_error() == 0
    same(got, fork_reference(table, held, parents, refs, keep, room), mp)


def test_no_pool(S):
    none = torch.empty(0, dtype=torch.int32, device="cuda")
    out = S.sinkattn_pages_fork(torch.empty(0, 2, dtype=torch.int32, device="cuda"), none, ints([-1]), none, room_lens=ints([5]))
    assert S.sinkattn_get_error() == S.ERR_NO_PAGES and out[0].tolist() == [[-1, -1]] and out[1].tolist() == [0]


@pytest.mark.parametrize("mp", [3, 4, 6, 9])
@pytest.mark.parametrize("shift", [0, 1])
def test_row_lengths_and_alignments(S, mp, shift):
    """Rows of every length modulo 16 bytes, tables and counts that start at any entry."""
    rng = random.Random(mp)
    table, held, refs = random_state(rng, 20, mp, 200)
    parents = [rng.randint(-1, 19) for _ in range(30)]
    room = [min(mp * PS, (held[p] if p >= 0 else 0) + rng.randint(0, 20)) for p in parents]
    keep = [held[p] if p >= 0 else 0 for p in parents]

    def off(x):  # the same values, starting `shift` entries into a buffer
        t = torch.as_tensor(x, dtype=torch.int32)
        buf = torch.zeros(t.numel() + shift, dtype=torch.int32, device="cuda")
        buf[shift:] = t.reshape(-1).cuda()
        return buf[shift:].view(t.shape)

    t = torch.zeros(20, mp, dtype=torch.int32)
    for i, row in enumerate(table):
        t[i, :len(row)] = torch.tensor(row, dtype=torch.int32)
    got = S.sinkattn_pages_fork(off(t), off(held), off(parents), off(refs), off(keep), off(room),
                                out_table=off(torch.zeros(30, mp)), out_refs=off(torch.zeros(200)))
    assert S.sinkattn_get_error() == 0
    same(got, fork_reference(table, held, parents, refs, keep, room), mp)


def test_short_of_pages(S):
    table, held, refs = [[0, 1]], [20], [1, 1, 0, 0]
    got = call(S, table, 8, held, [0, -1], refs, [20, 0], [20, 33])  # three new pages, two free
    assert S.sinkattn_get_error() == S.ERR_NO_PAGES
    assert (got[0] == -1).all() and (got[1] == 0).all() and got[2].tolist() == refs
    assert got[3].tolist() == [[-1, -1, 0]] * 2
    got = call(S, table, 8, held, [0, -1], refs, [20, 0], [20, 32])
    assert S.sinkattn_get_error() == 0
    same(got, fork_reference(table, held, [0, -1], refs, [20, 0], [20, 32]), 8)


def test_bad_fork_inputs_are_reported(S):
    table, held, refs = [[0, 1], [2]], [20, 10], [1, 1, 1, 0, 0, 0]
    got = call(S, table, 4, held, [7, -5, 1], refs, None, None, 1)  # parents out of range: empty rows
    assert S.sinkattn_get_error() == S.ERR_BAD_INDEX
    same(got, fork_reference(table, held, [-1, -1, 1], refs, grow=1), 4)
    got = call(S, table, 4, held, [0, 1], refs, [25, -3], [10, 1000])  # keep and room out of range: clamped to 20, 0
    assert S.sinkattn_get_error() == S.ERR_BAD_LENGTH  # (also ERR_NO_PAGES, four pages of three free: the lower code)
    assert got[1].tolist() == [0, 0]
    got = call(S, table, 3, held, [0, 1], refs, [25, -3], [10, 1000])
    assert S.sinkattn_get_error() == S.ERR_BAD_LENGTH
    same(got, fork_reference(table, held, [0, 1], refs, [20, 0], [20, 48]), 3)
    t = ints([[0, 1, -1, -1], [2, -1, -1, -1]])
    got = S.sinkattn_pages_fork(t, ints([-4, 10]), ints([0, 1]), ints(refs), grow=1)
    assert S.sinkattn_get_error() == S.ERR_BAD_LENGTH
    assert got[1].tolist() == [1, 11]
    t = ints([[0, 99, -1, -1], [-7, -1, -1, -1]])  # pages outside the pool: carried along, uncounted
    got = S.sinkattn_pages_fork(t, ints([20, 10]), ints([0, 0, 1]), ints(refs), grow=1)
    assert S.sinkattn_get_error() == S.ERR_BAD_PAGE
    assert got[0][:, :2].tolist() == [[0, 99], [0, 99], [-7, -1]]
    assert got[2].tolist() == [2, 1, 1, 0, 0, 0]


def test_fork_refusals(S):
    t, h, p, r = ints([[0, 1]]), ints([20]), ints([0]), ints([1, 1, 0])
    with pytest.raises(TypeError):
        S.sinkattn_pages_fork(t.long(), h, p, r)
    with pytest.raises(TypeError):
        S.sinkattn_pages_fork(t.cpu(), h, p, r)
    with pytest.raises(ValueError):
        S.sinkattn_pages_fork(t, ints([1, 2]), p, r)
    with pytest.raises(ValueError):
        S.sinkattn_pages_fork(t, h, p, r, keep_lens=ints([1, 2]))
    with pytest.raises(ValueError):
        S.sinkattn_pages_fork(t, h, p, r, out_lens=ints([1, 2]))
    for kw in (dict(grow=-1), dict(out_table=t)):
        with pytest.raises(S.SinkAttnError) as e:
            S.sinkattn_pages_fork(t, h, p, r, **kw)
        assert e.value.status == S.ERR_INVALID_ARG
    with pytest.raises(S.SinkAttnError) as e:
        S.sinkattn_pages_fork(t, h, p, r, workspace=torch.empty(8, dtype=torch.uint8, device="cuda"))
    assert e.value.status == S.ERR_WORKSPACE


# ------------------------------------------------------------------------------------- copies and compaction
def pools(shape, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return [torch.randn(shape, generator=g, device="cuda").to(torch.bfloat16) for _ in range(2)]


@pytest.mark.parametrize("layers,Hkv", [(None, 1), (None, 8), (1, 3), (3, 2)])
def test_copy(S, layers, Hkv):
    P = 60
    shape = (P, Hkv, PS, 64) if layers is None else (layers, P, Hkv, PS, 64)
    k, v = pools(shape, 1)
    k[..., 3, :] = float("nan")  # bits are copied, whatever they mean
    rng = random.Random(Hkv)
    ids = rng.sample(range(P), P)
    copies = [(ids[i], ids[30 + i], rng.randint(0, 16)) for i in range(25)] + [(-1, -1, 0), (-1, -1, 99), (ids[0], ids[58], 16)]
    rng.shuffle(copies)
    wk, wv = k.clone(), v.clone()
    for s, d, n in copies:
        if s >= 0:
            for w in (wk, wv):
                w[..., d, :, :n, :] = w[..., s, :, :n, :]
    S.sinkattn_kv_copy(k, v, ints(copies))
    assert S.sinkattn_get_error() == 0
    assert torch.equal(k.view(torch.int16), wk.view(torch.int16)) and torch.equal(v.view(torch.int16), wv.view(torch.int16))


def test_bad_copies_are_reported_and_skipped(S):
    for bad, code in (((60, 1, 4), "ERR_BAD_PAGE"), ((1, 60, 4), "ERR_BAD_PAGE"), ((-1, 2, 4), "ERR_BAD_PAGE"),
                      ((2, -2, 4), "ERR_BAD_PAGE"), ((0, 1, 17), "ERR_BAD_LENGTH"), ((0, 1, -1), "ERR_BAD_LENGTH")):
        k, v = pools((60, 2, PS, 64), 2)
        wk, wv = k.clone(), v.clone()
        for w in (wk, wv):
            w[41, :, :5] = w[40, :, :5]
            if bad[2] == 17:
                w[1] = w[0]
        S.sinkattn_kv_copy(k, v, ints([bad, (40, 41, 5)]))
        assert S.sinkattn_get_error() == getattr(S, code)
        assert torch.equal(k, wk) and torch.equal(v, wv)


@pytest.mark.parametrize("A", [1, 3, 8, 16])
@pytest.mark.parametrize("layers", [None, 2])
def test_compact(S, A, layers):
    """Any order and repeats of the accepted tokens: all are read before any is written."""
    B, Hkv, mp = 9, 3, 6
    P = B * mp
    k, v = pools((P, Hkv, PS, 64) if layers is None else (layers, P, Hkv, PS, 64), A)
    rng = random.Random(A)
    table = torch.tensor(rng.sample(range(P), P), dtype=torch.int32).view(B, mp)
    start = [rng.randint(0, mp * PS - 17) for _ in range(B)]
    start[0], start[1] = 0, 15
    accepted = [sorted(rng.sample(range(16), A)) if b % 3 else [rng.randrange(16) for _ in range(A)] for b in range(B)]
    count = [rng.randint(0, A) for _ in range(B)]
    count[0], count[1] = A, 0
    wk, wv = k.clone(), v.clone()
    for b in range(B):
        for w, x in ((wk, k), (wv, v)):
            for i in range(count[b]):
                ps, pd = start[b] + accepted[b][i], start[b] + i
                w[..., table[b, pd // PS], :, pd % PS, :] = x[..., table[b, ps // PS], :, ps % PS, :]
    S.sinkattn_kv_compact(k, v, table.cuda(), ints(start), ints(accepted), ints(count))
    assert S.sinkattn_get_error() == 0
    assert torch.equal(k, wk) and torch.equal(v, wv)


def test_bad_compactions_are_reported_and_skipped(S):
    table = ints([[0, 1], [2, 99]])
    for start, acc, n, code, moved in (
            ([0, 0], [[1, 2], [3, 4]], [3, 0], "ERR_BAD_LENGTH", [(0, 1), (1, 2)]),
            ([0, 0], [[1, 2], [3, 4]], [1, -1], "ERR_BAD_LENGTH", [(0, 1)]),
            ([30, 0], [[1, 2], [3, 4]], [2, 0], "ERR_BAD_LENGTH", [(30, 31)]),
            ([-1, 0], [[1, 2], [3, 4]], [2, 0], "ERR_BAD_LENGTH", [(0, 1)]),
            ([0, 0], [[-1, 2], [3, 4]], [2, 0], "ERR_BAD_INDEX", [(1, 2)]),
            ([0, 14], [[1, 2], [1, 4]], [1, 2], "ERR_BAD_PAGE", [(0, 1), (46, 47)])):
        k, v = pools((4, 2, PS, 64), 3)
        wk, wv = k.clone(), v.clone()
        for w, x in ((wk, k), (wv, v)):
            for d, s in moved:
                w[d // PS, :, d % PS] = x[s // PS, :, s % PS]
        S.sinkattn_kv_compact(k, v, table, ints(start), ints(acc), ints(n))
        assert S.sinkattn_get_error() == getattr(S, code), code
        assert torch.equal(k, wk) and torch.equal(v, wv), (start, acc, n)


def test_move_refusals(S):
    k, v = pools((4, 2, PS, 64), 4)
    with pytest.raises(ValueError):
        S.sinkattn_kv_copy(k, v[:2].contiguous(), ints([[0, 1, 2]]))
    with pytest.raises(ValueError):
        S.sinkattn_kv_copy(k, v, ints([[0, 1]]))
    with pytest.raises(TypeError):
        S.sinkattn_kv_copy(k.float(), v.float(), ints([[0, 1, 2]]))
    with pytest.raises(S.SinkAttnError) as e:
        S.sinkattn_kv_copy(torch.zeros(4, 2, 8, 64, dtype=torch.bfloat16, device="cuda"),
                           torch.zeros(4, 2, 8, 64, dtype=torch.bfloat16, device="cuda"), ints([[0, 1, 2]]))
    assert e.value.status == S.ERR_UNSUPPORTED
    with pytest.raises(S.SinkAttnError) as e:
        S.sinkattn_kv_compact(k, v, ints([[0]]), ints([0]), ints([list(range(17))]), ints([1]))
    assert e.value.status == S.ERR_UNSUPPORTED
    with pytest.raises(ValueError):
        S.sinkattn_kv_compact(k, v, ints([[0], [1]]), ints([0]), ints([[1]]), ints([1]))
    S.sinkattn_kv_copy(k, v, torch.empty(0, 3, dtype=torch.int32, device="cuda"))  # nothing to do


def test_more_rows_than_one_cta_keeps(S):
    """Over 4096 rows the plan is made by parts, with the parents' children in the workspace."""
    rng = random.Random(6)
    rows, mp, P = 9000, 3, 40001
    ids = rng.sample(range(P), P)
    held = [rng.randint(0, 40) for _ in range(rows)]
    table, refs = [], [0] * P
    for n in held:
        row = [ids.pop() for _ in range(cols(n))]
        if table and rng.random() < 0.3 and row and table[-1]:
            row[0] = table[-1][0]
        table.append(row)
        for p in row:
            refs[p] += 1
    for R in (4097, 12000):
        parents = [rng.randint(-1, rows - 1) for _ in range(R)]
        keep = [rng.randint(0, held[p]) if p >= 0 and rng.random() < 0.3 else (held[p] if p >= 0 else 0) for p in parents]
        room = [min(mp * PS, k + rng.randint(0, 3)) for k in keep]
        got = call(S, table, mp, held, parents, refs, keep, room)
        assert S.sinkattn_get_error() == 0
        same(got, fork_reference_fast(table, held, parents, refs, keep, room), mp)


def fork_reference_fast(table, held, parents, refs, keep, room):
    """fork_reference with every parent's children collected first (thousands of rows)."""
    kids = {}
    for r, p in enumerate(parents):
        kids.setdefault(p, []).append(r)
    writes = [m > k and k % PS != 0 for k, m in zip(keep, room)]
    free = iter([p for p, c in enumerate(refs) if c == 0])
    new_table, copies, counts = [], [], list(refs)
    for r, p in enumerate(parents):
        kept, copy = (table[p][:cols(keep[r])] if p >= 0 else []), (-1, -1, 0)
        if writes[r]:
            mates = kids[p]
            if not (refs[kept[-1]] == 1 and mates[0] == r and all(writes[q] and keep[q] == keep[r] for q in mates)):
                copy = (kept[-1], next(free), keep[r] % PS)
                kept = kept[:-1] + [copy[1]]
        kept = kept + [next(free) for _ in range(cols(room[r]) - len(kept))]
        new_table.append(kept)
        copies.append(copy)
    for p in range(len(table)):
        for c in range(cols(held[p])):
            counts[table[p][c]] -= 1
    for row in new_table:
        for page in row:
            counts[page] += 1
    return new_table, room, counts, copies

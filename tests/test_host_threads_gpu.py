"""Calls from several host threads."""
import threading
from concurrent.futures import ThreadPoolExecutor

import pytest
import torch

from gqa_attention_learned_head_gb300 import workloads as W

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def S():
    from gqa_attention_learned_head_gb300 import sinkattn

    return sinkattn


def in_new_thread(fn):
    """What fn returns, or raises, as the first thing that a thread does."""
    box = []

    def run():
        try:
            box.append((fn(), None))
        except Exception as e:  # noqa: BLE001
            box.append((None, e))

    t = threading.Thread(target=run)
    t.start()
    t.join()
    if box[0][1] is not None:
        raise box[0][1]
    return box[0][0]


def calls(S):
    """Every entry point with all of its outputs given, by name: (call, its outputs)."""
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    d = W.make_decode(3, 16, 2, [40, 1, 100], seed=1).to("cuda")
    v = W.make_decode(3, 16, 2, [40, 9, 100], seed=2, q_len=4).to("cuda")
    p = W.make_prefill(16, 2, [130, 5], seed=3).to("cuda")
    odd = W.make_prefill(6, 2, [130, 5], seed=4).to("cuda")
    c = W.make_paged_prefill(16, 2, [5, 30], [20, 7], seed=5).to("cuda")
    masks = torch.tensor([1, 3, 5, 15], dtype=torch.int64, device="cuda").expand(3, 4).contiguous()
    like = lambda q: dict(out=torch.zeros_like(q), lse=torch.zeros(q.shape[:-1], device="cuda"))  # noqa: E731
    ws = torch.empty(1 << 24, dtype=torch.uint8, device="cuda")
    out = {n: like(x) for n, x in (("decode", d.q), ("noalloc", d.q), ("verify", v.q), ("tree", v.q), ("prefill", p.q),
                                   ("prefill odd", odd.q), ("prefill shared", p.q), ("paged", c.q), ("beams", d.q.view(1, 3, 16, 64)))}
    qkv = torch.randn(27, 20 * 64, device="cuda").to(torch.bfloat16)
    q_out = torch.zeros(27, 16, 64, dtype=torch.bfloat16, device="cuda")
    pages = [(c.k_pages.clone(), c.v_pages.clone()) for _ in range(4)]
    part, part_lse = torch.randn(3, 4, 8, 64, device="cuda"), torch.randn(3, 4, 8, device="cuda")
    merged = dict(out=torch.zeros(4, 8, 64, dtype=torch.bfloat16, device="cuda"), lse=torch.zeros(4, 8, device="cuda"))
    z, s = torch.randn(2, 3, 500, device="cuda"), -torch.rand(2, 3, device="cuda")
    picks = dict(out_scores=torch.zeros(2, 4, device="cuda"), out_parents=i32([[0] * 4] * 2), out_tokens=i32([[0] * 4] * 2))
    fork = dict(out_table=i32([[0] * 3] * 2), out_lens=i32([0, 0]), out_refs=i32([0] * 6), copies=i32([[0] * 3] * 2))
    table, held, parents, refs = i32([[0, 1, -1], [2, -1, -1]]), i32([20, 10]), i32([0, 0]), i32([1, 1, 1, 0, 0, 0])
    dargs = (d.q, d.k_pages, d.v_pages, d.page_table, d.kv_lens, d.sinks, d.scale)
    vargs = (v.q, v.k_pages, v.v_pages, v.page_table, v.kv_lens)
    copies, start, acc, num, cargs = i32([[0, 1, 5]]), i32([3, 4]), i32([[1, 2], [0, 3]]), i32([2, 2]), (c.cu_seqlens, c.start_pos)
    odd_args, p_args = ((x.q, x.k, x.v, x.cu_seqlens, x.sinks, x.scale) for x in (odd, p))
    return {
        "decode": (lambda: S.sinkattn_decode(*dargs, workspace=ws, **out["decode"]), out["decode"].values()),
        "noalloc": (lambda: S.sinkattn_decode_noalloc(*dargs, **out["noalloc"]), out["noalloc"].values()),
        "verify": (lambda: S.sinkattn_verify(*vargs, v.sinks, v.scale, workspace=ws, **out["verify"]), out["verify"].values()),
        "tree": (lambda: S.sinkattn_verify_tree(*vargs, masks, v.sinks, v.scale, workspace=ws, **out["tree"]), out["tree"].values()),
        "prefill": (lambda: S.sinkattn_prefill(*p_args, max_seqlen=130, **out["prefill"]), out["prefill"].values()),
        "prefill odd": (lambda: S.sinkattn_prefill(*odd_args, max_seqlen=130, **out["prefill odd"]), out["prefill odd"].values()),
        "prefill shared": (lambda: S.sinkattn_prefill(*p_args, max_seqlen=130, share_sms=True, **out["prefill shared"]),
                           out["prefill shared"].values()),
        "paged": (lambda: S.sinkattn_prefill_paged(c.q, c.k_pages, c.v_pages, c.page_table, *cargs, c.sinks, c.scale, max_seqlen=20,
                                                   **out["paged"]), out["paged"].values()),
        "append": (lambda: S.sinkattn_kv_append(c.k_new, c.v_new, *cargs, c.page_table, *pages[0], max_seqlen=20), pages[0]),
        "prologue": (lambda: S.sinkattn_qkv_prologue(qkv, None, *cargs, c.page_table, *pages[1], 16, 1e4, 32.0, 4096, 32.0, 1.0,
                                                     q_out=q_out), (q_out, *pages[1])),
        "merge": (lambda: S.sinkattn_merge(part, part_lse, **merged), merged.values()),
        "select": (lambda: S.sinkattn_beam_select(z, s, 4, workspace=ws, **picks), picks.values()),
        "fork": (lambda: S.sinkattn_pages_fork(table, held, parents, refs, grow=1, workspace=ws, **fork), fork.values()),
        "copy": (lambda: S.sinkattn_kv_copy(*pages[2], copies), pages[2]),
        "compact": (lambda: S.sinkattn_kv_compact(*pages[3], c.page_table, start, acc, num), pages[3]),
        "beams": (lambda: S.sinkattn_decode_beams(d.q.view(1, 3, 16, 64), d.k_pages, d.v_pages, d.page_table.view(1, 3, -1),
                                                  d.kv_lens.view(1, 3), d.sinks, d.scale, workspace=ws, **out["beams"]),
                  out["beams"].values()),
    }


NAMES = ["decode", "noalloc", "verify", "tree", "prefill", "prefill odd", "prefill shared", "paged", "append", "prologue", "merge",
         "select", "fork", "copy", "compact", "beams"]


@pytest.mark.parametrize("name", NAMES)
def test_first_thing_a_thread_does(S, name):
    """A host thread whose first use of the GPU is a call: the same outputs as from the main thread."""
    call, outputs = calls(S)[name]
    if name == "compact":  # moves tokens: the same start for both
        outputs = list(outputs)
        start = [t.clone() for t in outputs]
    call()
    torch.cuda.synchronize()
    want = [t.clone() for t in outputs]
    for i, t in enumerate(outputs):
        t.copy_(start[i]) if name == "compact" else (t.zero_() if name not in ("append", "prologue", "copy") else None)
    torch.cuda.synchronize()
    in_new_thread(call)
    torch.cuda.synchronize()
    assert S.sinkattn_get_error() == 0
    for got, ref in zip(outputs, want):
        assert torch.equal(got, ref)
    assert S.sinkattn_get_error() == in_new_thread(S.sinkattn_get_error) == 0


def decode(S, n, Hq):
    g = W.make_decode(n, Hq, 2, (1, 40), seed=n).to("cuda")
    return lambda: S.sinkattn_decode(g.q, g.k_pages, g.v_pages, g.page_table, g.kv_lens, g.sinks, g.scale)


def prefill(S, n, Hq):
    g = W.make_prefill(Hq, 2, (n, 1, 20), seed=n).to("cuda")
    return lambda: S.sinkattn_prefill(g.q, g.k, g.v, g.cu_seqlens, g.sinks, g.scale, max_seqlen=20)


def prefill_paged(S, n, Hq):
    g = W.make_paged_prefill(Hq, 2, [5] * n, [7] * n, seed=n).to("cuda")
    return lambda: S.sinkattn_prefill_paged(g.q, g.k_pages, g.v_pages, g.page_table, g.cu_seqlens, g.start_pos, g.sinks,
                                            g.scale, max_seqlen=7)


@pytest.mark.parametrize("Hq", [16, 20, 6])  # 8, 10 and 3 query heads a KV head: the kernels' variants
@pytest.mark.parametrize("make", [decode, prefill, prefill_paged])
def test_a_small_batch_leaves_a_large_ones_limits(S, make, Hq):
    """A kernel's shared memory grows with the batch and its limit belongs to the process."""
    large, small = make(S, 3000, Hq), make(S, 2, Hq)
    torch.cuda.synchronize()

    def run(call):
        got = [t.clone() for t in call()]
        torch.cuda.synchronize()
        return got

    with ThreadPoolExecutor(1) as a, ThreadPoolExecutor(1) as b:
        first = a.submit(run, large).result()
        other = b.submit(run, small).result()
        again = a.submit(run, large).result()
        for x, y in zip(first, again):
            assert torch.equal(x, y)
        for x, y in zip(other, b.submit(run, small).result()):
            assert torch.equal(x, y)
    assert S.sinkattn_get_error() == 0


def test_beam_steps_at_once(S):
    """Threads with a stream each, all in selections, forks, copies and decodes of their own at the same time: the same bits as
    alone."""
    def state(seed):
        g = torch.Generator(device="cuda").manual_seed(seed)
        N, K, V, mp = 3 + seed, 4, 5001 + 700 * seed, 20
        P = N * K * mp + 50
        table = torch.randperm(N * K * mp, generator=g, device="cuda").to(torch.int32).view(N, K, mp)
        table[:, 1:, :12] = table[:, :1, :12]
        lens = torch.randint(mp * 16 - 30, mp * 16 - 1, (N, 1), generator=g, device="cuda", dtype=torch.int32).expand(N, K).contiguous()
        refs = torch.bincount(table.view(-1).long(), minlength=P).to(torch.int32)
        pool = [torch.randn(P, 2, 16, 64, generator=g, device="cuda").to(torch.bfloat16) for _ in range(2)]
        q = torch.randn(N, K, 16, 64, generator=g, device="cuda").to(torch.bfloat16)
        return (torch.randn(N, K, V, generator=g, device="cuda"), -torch.rand(N, K, generator=g, device="cuda"),
                table.view(N * K, mp), lens.view(-1), refs, pool, q, torch.randn(16, generator=g, device="cuda"))

    def step(s, stream):
        z, c, table, lens, refs, pool, q, sinks = s
        N, K = c.shape
        with torch.cuda.stream(stream):
            k, v = pool[0].clone(), pool[1].clone()
            scores, parents, tokens = S.sinkattn_beam_select(z, c, K)
            new, room, counts, copies = S.sinkattn_pages_fork(table, lens, parents.view(-1), refs, grow=1)
            S.sinkattn_kv_copy(k, v, copies)
            out, lse = S.sinkattn_decode_beams(q, k, v, new.view(N, K, -1), (room - 1).view(N, K), sinks, 0.125)
        return scores, parents, tokens, new, room, counts, copies, out, lse

    states = [state(i) for i in range(4)]
    main = torch.cuda.current_stream()
    alone = [[t.clone() for t in step(s, main)] for s in states]
    torch.cuda.synchronize()
    assert S.sinkattn_get_error() == 0

    def run(i):
        stream = torch.cuda.Stream()
        got = [step(states[i], stream) for _ in range(40)]
        stream.synchronize()
        return got

    with ThreadPoolExecutor(4) as pool:
        results = [f.result() for f in [pool.submit(run, i) for i in range(4)]]
    for got, want in zip(results, alone):
        for outs in got:
            assert all(torch.equal(a, b) for a, b in zip(outs, want))
    assert S.sinkattn_get_error() == 0

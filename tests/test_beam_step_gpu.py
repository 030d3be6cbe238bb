"""The beam step's calls together, as a search uses them: selection, page forks, page copies, appends and the decode over
shared pages, step after step, against attention over every row's own history in 64 bits; and a draft tree checked, its
accepted tokens moved together and decoded on."""
import math
import random

import numpy as np
import pytest
import torch

import oracle
from gqa_attention_learned_head_gb300 import workloads as W
from parity_utils import assert_parity

pytestmark = pytest.mark.gpu

PS, D = 16, 64


@pytest.fixture(scope="module")
def S():
    from gqa_attention_learned_head_gb300 import sinkattn

    return sinkattn


class Toy:
    """A "model" whose query, key and value of a token at a position are drawn from (token, position), and whose logits
    are a product of the attention's output: enough to drive a search."""

    def __init__(self, Hq, Hkv, V, seed):
        g = torch.Generator().manual_seed(seed)
        self.Hq, self.Hkv, self.V = Hq, Hkv, V
        self.tok = torch.randn(V, (Hq + 2 * Hkv) * D, generator=g)
        self.pos = torch.randn(200, (Hq + 2 * Hkv) * D, generator=g)
        self.head = (torch.randn(Hq * D, V, generator=g) * 0.2).cuda()
        self.sinks = torch.randn(Hq, generator=g)

    def qkv(self, tokens, positions):
        x = (0.7 * self.tok[tokens] + 0.7 * self.pos[positions]).to(torch.bfloat16)
        q, k, v = x.split([self.Hq * D, self.Hkv * D, self.Hkv * D], -1)
        return q.reshape(-1, self.Hq, D), k.reshape(-1, self.Hkv, D), v.reshape(-1, self.Hkv, D)

    def attention(self, history):
        """Of the last token of a history over all of it, in 64 bits: (out [Hq, 64], lse [Hq])."""
        q, k, v = (t.double().numpy() for t in self.qkv(torch.tensor(history), torch.arange(len(history))))
        G = self.Hq // self.Hkv
        out, lse = np.zeros((self.Hq, D)), np.zeros(self.Hq)
        for h in range(self.Hq):
            s = k[:, h // G] @ q[-1, h] * 0.125
            full = np.append(s, float(self.sinks[h]))
            m = full.max()
            p = np.exp(full - m)
            out[h], lse[h] = (p[:-1] / p.sum()) @ v[:, h // G], m + math.log(p.sum())
        return out, lse


def select_reference(logits, scores, M, finished, pad):
    """The M best of each group in 64 bits, from the very logits the call sees."""
    z, c = logits.double().cpu().numpy(), scores.double().cpu().numpy()
    N, K, V = z.shape
    picks = []
    for n in range(N):
        rows = np.full((K, V), -np.inf)
        for k in range(K):
            if np.isneginf(c[n, k]):
                continue
            if finished[n, k]:
                rows[k, pad] = c[n, k]
            else:
                m = z[n, k].max()
                rows[k] = c[n, k] + (z[n, k] - (m + np.log(np.exp(z[n, k] - m).sum())))
        flat = rows.reshape(-1)
        top = np.lexsort((np.arange(flat.size), -flat))[:M]
        picks.append((flat[top], n * K + top // V, top % V))
    return [np.stack(x) for x in zip(*picks)]


def check_counts(table, lens, refs):
    held = torch.zeros_like(refs)
    for row, n in zip(table.cpu(), lens.tolist()):
        for page in row[:(n + PS - 1) // PS].tolist():
            held[page] += 1
    assert torch.equal(held, refs)
    # a partial last page that a row alone may write is held by that row alone, or by rows that will not write it yet
    return int((refs > 0).sum())


@pytest.mark.parametrize("seed,Hq,Hkv,K,prompts", [(0, 16, 2, 4, [5, 33, 16]), (1, 8, 8, 3, [1, 47]), (2, 8, 1, 8, [31, 32])])
def test_search(S, seed, Hq, Hkv, K, prompts):
    rng = random.Random(seed)
    N, V, steps, eos = len(prompts), 97, 40, 3
    toy = Toy(Hq, Hkv, V, seed)
    mp = (max(prompts) + steps + PS) // PS + 1
    P = N * K * mp + 8
    kp, vp = (torch.full((P, Hkv, PS, D), float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    refs = torch.zeros(P, dtype=torch.int32, device="cuda")
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    sinks = toy.sinks.cuda()

    # the prompts' pages and tokens
    none = torch.empty(0, dtype=torch.int32, device="cuda")
    table, lens, refs, copies = S.sinkattn_pages_fork(torch.empty(0, mp, dtype=torch.int32, device="cuda"), none, i32([-1] * N),
                                                      refs, room_lens=i32(prompts))
    assert (copies == i32([-1, -1, 0])).all()
    hist = [[rng.randrange(V) for _ in range(L)] for L in prompts]
    q, k, v = toy.qkv(torch.tensor(sum(hist, [])), torch.cat([torch.arange(L) for L in prompts]))
    cu = i32([0] + np.cumsum(prompts).tolist())
    S.sinkattn_kv_append(k.cuda(), v.cuda(), cu, i32([0] * N), table, kp, vp)
    # every prompt forked to K beams, the first of them in use
    table, lens, refs, copies = S.sinkattn_pages_fork(table, lens, i32([n for n in range(N) for _ in range(K)]), refs)
    hist = [list(hist[n]) for n in range(N) for _ in range(K)]
    scores = torch.full((N, K), -math.inf, device="cuda")
    scores[:, 0] = 0.0
    done = torch.zeros(N, K, dtype=torch.bool, device="cuda")
    pages = [check_counts(table, lens, refs)]
    for step in range(steps):
        q, _, _ = toy.qkv(torch.tensor([h[-1] for h in hist]), torch.tensor([len(h) - 1 for h in hist]))
        out, lse = S.sinkattn_decode_beams(q.cuda().view(N, K, Hq, D), kp, vp, table.view(N, K, mp), lens.view(N, K), sinks, 0.125)
        ref = [toy.attention(h) for h in hist]
        assert_parity(out.view(N * K, Hq, D).float().cpu().numpy(), lse.view(N * K, Hq).cpu().numpy(),
                      np.stack([r[0] for r in ref]), np.stack([r[1] for r in ref]), f"step {step}")
        logits = (out.view(N, K, Hq * D).float() @ toy.head)
        want = select_reference(logits, scores, K, done.cpu().numpy(), eos)
        scores, parents, tokens = S.sinkattn_beam_select(logits, scores, K, finished=done, pad_token=eos)
        assert np.array_equal(parents.cpu().numpy(), want[1]) and np.array_equal(tokens.cpu().numpy(), want[2])
        assert np.allclose(scores.cpu().numpy(), want[0], rtol=2.0 ** -22, atol=1e-5)
        done = (tokens == eos) | done.view(-1)[parents.long()]
        table, lens, refs, copies = S.sinkattn_pages_fork(table, lens, parents.view(-1), refs, grow=1)
        S.sinkattn_kv_copy(kp, vp, copies)
        hist = [hist[p] + [t] for p, t in zip(parents.view(-1).tolist(), tokens.view(-1).tolist())]
        assert lens.tolist() == [len(h) for h in hist]
        _, k, v = toy.qkv(torch.tensor([h[-1] for h in hist]), torch.tensor([len(h) - 1 for h in hist]))
        S.sinkattn_kv_append(k.cuda(), v.cuda(), i32(list(range(N * K + 1))), lens - 1, table, kp, vp)
        pages.append(check_counts(table, lens, refs))
        assert S.sinkattn_get_error() == 0
    # shared pages: far fewer than the rows' own would be
    assert pages[-1] < sum((len(h) + PS - 1) // PS for h in hist)
    _, _, refs, _ = S.sinkattn_pages_fork(table, lens, none, refs)  # the search ends
    assert not refs.any() and S.sinkattn_get_error() == 0


def test_step_in_a_graph(S):
    """Fork, copies, append and decode captured once and replayed step after step, page counts in place: the same bits as
    the calls made one by one."""
    N, K, Hq, Hkv, steps, L0 = 2, 4, 16, 2, 20, 13
    mp = (L0 + steps) // PS + 2
    P, R = N * K * mp, N * K
    g = torch.Generator(device="cuda").manual_seed(1)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
    q, k, v = rnd(steps, N, K, Hq, D), rnd(steps, R, Hkv, D), rnd(steps, R, Hkv, D)
    parents = torch.randint(0, K, (steps, N, K), generator=g, device="cuda")
    parents = (parents + K * torch.arange(N, device="cuda")[:, None]).view(steps, R).to(torch.int32)
    sinks = torch.randn(Hq, generator=g, device="cuda")
    cu = torch.arange(R + 1, dtype=torch.int32, device="cuda")
    start = rnd(P, Hkv, PS, D), rnd(P, Hkv, PS, D)

    def fresh():
        table = torch.full((R, mp), -1, dtype=torch.int32, device="cuda")
        table[:, :1] = torch.arange(R, dtype=torch.int32, device="cuda")[:, None]
        refs = torch.zeros(P, dtype=torch.int32, device="cuda")
        refs[:R] = 1
        return dict(k=start[0].clone(), v=start[1].clone(), table=table, refs=refs, row=torch.empty(R, dtype=torch.int32, device="cuda"),
                    lens=torch.full((R,), L0, dtype=torch.int32, device="cuda"), qs=torch.empty_like(q[0]),
                    ks=torch.empty_like(k[0]), vs=torch.empty_like(v[0]), new=torch.empty_like(table),
                    new_lens=torch.empty(R, dtype=torch.int32, device="cuda"), out=torch.empty_like(q[0]),
                    copies=torch.empty(R, 3, dtype=torch.int32, device="cuda"))

    def step(s):
        S.sinkattn_pages_fork(s["table"], s["lens"], s["row"], s["refs"], grow=1, out_table=s["new"], out_lens=s["new_lens"],
                              out_refs=s["refs"], copies=s["copies"])
        S.sinkattn_kv_copy(s["k"], s["v"], s["copies"])
        S.sinkattn_kv_append(s["ks"], s["vs"], cu, s["lens_before"], s["new"], s["k"], s["v"])
        S.sinkattn_decode_beams(s["qs"], s["k"], s["v"], s["new"].view(N, K, mp), s["new_lens"].view(N, K), sinks, 0.125,
                                out=s["out"], return_lse=False)
        s["table"].copy_(s["new"])
        s["lens"].copy_(s["new_lens"])

    def run(graphed):
        s = fresh()
        s["lens_before"] = torch.empty(R, dtype=torch.int32, device="cuda")
        graph, outs = None, []
        for i in range(steps):
            for name, x in (("qs", q), ("ks", k), ("vs", v), ("row", parents)):
                s[name].copy_(x[i])
            s["lens_before"].copy_(s["lens"][parents[i].long()])
            if graphed and graph is None and i == 1:  # after one call outside, which sets up what a capture may not
                graph = torch.cuda.CUDAGraph()
                torch.cuda.synchronize()
                with torch.cuda.graph(graph):
                    step(s)
            if graph is not None:
                graph.replay()
            else:
                step(s)
            outs.append(s["out"].clone())
        torch.cuda.synchronize()
        assert S.sinkattn_get_error() == 0
        return outs, s

    a, sa = run(False)
    b, sb = run(True)
    for x, y in zip(a, b):
        assert torch.equal(x, y)
    for name in ("table", "refs", "lens"):
        assert torch.equal(sa[name], sb[name])
    # and the last step's attention over the tables as they stand
    ref = oracle.decode(sa["qs"].view(R, Hq, D), sa["k"], sa["v"], sa["table"], sa["lens"], sinks, 0.125)
    assert_parity(a[-1].view(R, Hq, D).float().cpu().numpy(), None, ref[0], ref[1], "last step")


def test_tree_accepted_and_decoded_on(S):
    """A draft tree is checked, the path that was accepted moves together, and the next token attends to it as if it had
    been written there in the first place."""
    B, Hq, Hkv, QL = 3, 16, 2, 8
    base = [20, 31, 5]
    inp = W.make_decode(B, Hq, Hkv, [L + QL for L in base], seed=50, q_len=QL, max_pages=4)
    masks = torch.tensor(W.tree_masks(W.DRAFT_TREE_PARENTS), dtype=torch.int64).expand(B, -1).contiguous()
    g = inp.to("cuda")
    S.sinkattn_verify_tree(g.q, g.k_pages, g.v_pages, g.page_table, g.kv_lens, masks.cuda(), g.sinks, g.scale)
    paths = [[0, 1, 3, 6], [0, 2, 5, 7], [0]]
    acc = torch.zeros(B, 4, dtype=torch.int32)
    for b, path in enumerate(paths):
        acc[b, :len(path)] = torch.tensor(path)
    # the same cache with the path's tokens where they belong
    k, v = inp.k_pages.clone(), inp.v_pages.clone()
    for b, path in enumerate(paths):
        for i, t in enumerate(path):
            s, d = base[b] + t, base[b] + i
            for w, x in ((k, inp.k_pages), (v, inp.v_pages)):
                w[inp.page_table[b, d // PS], :, d % PS] = x[inp.page_table[b, s // PS], :, s % PS]
    start = torch.tensor(base, dtype=torch.int32)
    S.sinkattn_kv_compact(g.k_pages, g.v_pages, g.page_table, start.cuda(), acc.cuda(),
                          torch.tensor([len(p) for p in paths], dtype=torch.int32).cuda())
    lens = start + torch.tensor([len(p) for p in paths], dtype=torch.int32)
    q = inp.q[:, 0].contiguous()
    out, lse = S.sinkattn_decode(q.cuda(), g.k_pages, g.v_pages, g.page_table, lens.cuda(), g.sinks, g.scale)
    assert S.sinkattn_get_error() == 0
    assert torch.equal(g.k_pages.cpu(), k) and torch.equal(g.v_pages.cpu(), v)
    assert_parity(out.float().cpu().numpy(), lse.cpu().numpy(),
                  *oracle.decode(q, k, v, inp.page_table, lens, inp.sinks, inp.scale), "after the tree")
    # the draft's pages past the accepted tokens go back to the pool
    P = inp.k_pages.shape[0]
    refs = torch.zeros(P, dtype=torch.int32)
    for b in range(B):
        for page in inp.page_table[b, :(base[b] + QL + PS - 1) // PS].tolist():
            refs[page] += 1
    table, held, refs, copies = S.sinkattn_pages_fork(g.page_table, g.kv_lens, torch.arange(B, dtype=torch.int32, device="cuda"),
                                                      refs.cuda(), keep_lens=lens.cuda(), room_lens=(lens + 1).cuda())
    assert S.sinkattn_get_error() == 0 and (copies[:, 0] == -1).all()
    assert int(refs.sum()) == sum((int(n) + 1 + PS - 1) // PS for n in lens)

"""A beam step over the paged KV cache: the operators, their plain forms and the sizes they are timed at.

One step of a beam search (or of several samples of one prompt) over a paged cache is
  beam_select   the best continuations over beams and vocabulary,
  pages_fork    the page tables follow the beams: pages shared, freed and taken from the pool,
  kv_copy       the pages that more than one beam is about to write are copied,
  decode_beams  one query token per beam attends to its own pages, shared pages read once per group,
and after a tree of drafted tokens was checked, kv_compact moves the accepted ones together.

``own`` False runs elementary torch operations in 32 bits or more; True calls the library.
"""
import math

import torch

own = False

DEVICE = "cuda"
D, PS = 64, 16  # head dimension and page size of the library's cache
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


# ------------------------------------------------------------------------------------- cases
def listed():
    return [
        # one user's beam search on a small vocabulary: latency counts
        dict(name="select 1x4 bf16 32k", op="select", N=1, K=4, V=32000, M=8, dtype="bf16", done=False),
        # a serving batch whose head computes in 32 bits, odd vocabulary (rows start at any 4 bytes), finished beams
        dict(name="select 32x8 f32 50021", op="select", N=32, K=8, V=50021, M=16, dtype="f32", done=True),
        # the largest: 64 requests of 8 beams, a large vocabulary
        dict(name="select 64x8 bf16 200k", op="select", N=64, K=8, V=200000, M=16, dtype="bf16", done=False),
        # one request's tables
        dict(name="fork 1x4", op="fork", N=1, K=4, lo=700, hi=700, own_tokens=90, extra=64, mode="beam"),
        # 256 requests of 8 beams with the mixed serving batch's lengths
        dict(name="fork 256x8 long", op="fork", N=256, K=8, lo=1024, hi=32768, own_tokens=128, extra=8192, mode="beam"),
        # the tail pages that the beams of a batch copy in one step
        dict(name="copy 256 tails", op="copy", R=256, Hkv=8, layers=1, P=2048, full=False),
        # whole pages of a forked or moved prompt
        dict(name="copy 4096 pages", op="copy", R=4096, Hkv=8, layers=1, P=12288, full=True),
        # accepted tokens of 32 draft trees of 8, one layer
        dict(name="compact 32 trees of 8", op="compact", B=32, A=8, Hkv=8, layers=1, lo=512, hi=4096),
        # accepted tokens of 256 draft trees of 16, a model's 24 layers at once
        dict(name="compact 256x16 24 layers", op="compact", B=256, A=16, Hkv=8, layers=24, lo=100, hi=400),
        # one request's beams
        dict(name="decode 1x4 len 1000", op="decode", N=1, K=4, Hq=64, Hkv=8, lo=1000, hi=1000, own_tokens=60, ragged=False),
        # the batched decode's lengths with 8 beams each
        dict(name="decode 32x8 512-4096", op="decode", N=32, K=8, Hq=64, Hkv=8, lo=512, hi=4096, own_tokens=128, ragged=False),
        # the long context with 8 samples of each prompt
        dict(name="decode 4x8 131072", op="decode", N=4, K=8, Hq=64, Hkv=8, lo=131072, hi=131072, own_tokens=512, ragged=False),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["select", "select", "fork", "copy", "compact", "decode", "decode"])
    if op == "select":
        K = rng.randint(1, 16)
        V = _log_int(rng, 1000, 200000)
        N = _log_int(rng, 1, max(1, min(64, 64 * 8 * 200000 // (K * V * 2))))
        return dict(op=op, N=N, K=K, V=V, M=rng.randint(1, 2 * K), dtype=rng.choice(["bf16", "f16", "f32"]),
                    done=rng.random() < 0.5)
    if op == "fork":
        K = rng.randint(1, 16)
        hi = _log_int(rng, 20, 32768)
        return dict(op=op, N=_log_int(rng, 1, 2048 // K), K=K, lo=rng.randint(1, hi), hi=hi,
                    own_tokens=_log_int(rng, 1, 500), extra=_log_int(rng, 8192, 40000), mode=rng.choice(["beam", "trim"]))
    if op == "copy":
        R, Hkv = _log_int(rng, 1, 4096), rng.choice([1, 2, 4, 8])
        layers = rng.randint(1, max(1, min(24, 4096 * 8 // (R * Hkv))))
        return dict(op=op, R=R, Hkv=Hkv, layers=layers, P=2 * R + rng.randint(1, 500), full=rng.random() < 0.3)
    if op == "compact":
        lo = rng.randint(1, 300)
        return dict(op=op, B=_log_int(rng, 1, 256), A=rng.randint(1, 16), Hkv=rng.choice([1, 2, 4, 8]),
                    layers=rng.randint(1, 24), lo=lo, hi=lo + rng.randint(0, 300))
    G, Hkv = rng.choice([1, 2, 4, 5, 8, 16]), rng.choice([1, 2, 4, 8])
    K = rng.randint(1, min(32, 128 // G))
    hi = _log_int(rng, 8, 32768)
    N = _log_int(rng, 1, max(1, min(64, 4 * 8 * 131072 * 8 // (K * hi * Hkv * 4))))
    return dict(op=op, N=N, K=K, Hq=G * Hkv, Hkv=Hkv, lo=rng.randint(1, hi), hi=hi, own_tokens=_log_int(rng, 1, 600),
                ragged=rng.random() < 0.5)


# ------------------------------------------------------------------------------------- inputs
def _lengths(n, lo, hi):
    """n lengths spread evenly over lo .. hi (the seed only orders them)."""
    return [lo + (i * (hi - lo)) // max(1, n - 1) for i in range(n)]


def _columns(tokens):
    return (tokens + PS - 1) // PS


def _shared_columns(L, own_tokens):
    """Columns that all beams share, and columns that pairs of beams share, of a group of length L."""
    return max(0, L - own_tokens) // PS, max(0, L - own_tokens // 2) // PS


def _group_pages(L, K, own_tokens):
    s1, s2 = _shared_columns(L, own_tokens)
    return s1 + (s2 - s1) * ((K + 1) // 2) + (_columns(L) - s2) * K


def _generator(seed):
    g = torch.Generator(device=DEVICE)
    g.manual_seed(seed)
    return g


def _tables(g, N, K, lens, own_tokens, P, max_pages):
    """Page tables [N, K, max_pages] of groups whose beams share their first pages, then pairwise, then not at all;
    unused entries -1.  lens: [N] int64 on the device."""
    c = torch.arange(max_pages, device=DEVICE)
    k = torch.arange(K, device=DEVICE)
    s1 = ((lens - own_tokens).clamp(min=0) // PS)[:, None, None]
    s2 = ((lens - own_tokens // 2).clamp(min=0) // PS)[:, None, None]
    owner = torch.where(c < s1, 0, torch.where(c < s2, (k // 2 * 2)[None, :, None], k[None, :, None]))  # [N, K, mp]
    held = (c < _columns(lens)[:, None, None]).expand(N, K, max_pages)
    first = held & (owner == k[None, :, None])
    ids = torch.cumsum(first.reshape(-1), 0).view(N, K, max_pages) - 1
    ids = torch.gather(ids, 1, owner)
    perm = torch.randperm(P, generator=g, device=DEVICE)
    return torch.where(held, perm[ids.clamp(min=0)], -1).to(torch.int32)


def _pool(g, shape):
    out = torch.empty(shape, dtype=torch.bfloat16, device=DEVICE)
    flat = out.view(-1)
    step = 1 << 28
    for lo in range(0, flat.numel(), step):
        part = flat[lo:lo + step]
        part.copy_(torch.randn(part.numel(), generator=g, device=DEVICE))
    return out


def prepare(case, seed):
    g = _generator(seed)
    c, op = case, case["op"]
    if op == "select":
        N, K, V = c["N"], c["K"], c["V"]
        logits = (torch.randn(N, K, V, generator=g, device=DEVICE) * 2.5).to(DTYPES[c["dtype"]])
        scores = -30 * torch.rand(N, K, generator=g, device=DEVICE)
        done = (torch.rand(N, K, generator=g, device=DEVICE) < 0.15) if c["done"] else None
        return dict(op=op, logits=logits, scores=scores, M=c["M"], done=done, pad=0)
    if op == "fork":
        N, K = c["N"], c["K"]
        lens = _lengths(N, c["lo"], c["hi"])
        P = sum(_group_pages(L, K, c["own_tokens"]) for L in lens) + c["extra"]
        max_pages = _columns(max(lens) + 2 * PS)
        L = torch.tensor(lens, device=DEVICE)[torch.randperm(N, generator=g, device=DEVICE)]
        table = _tables(g, N, K, L, c["own_tokens"], P, max_pages).view(N * K, max_pages)
        refs = torch.bincount(table[table >= 0].long(), minlength=P).to(torch.int32)
        held = L.to(torch.int32)[:, None].expand(N, K).reshape(-1).contiguous()
        pick = torch.randint(0, K, (N, K), generator=g, device=DEVICE)
        parents = (pick + K * torch.arange(N, device=DEVICE)[:, None]).to(torch.int32).view(-1).contiguous()
        keep = room = None
        if c["mode"] == "trim":  # drafted tokens were refused: up to 8 tokens go, up to 8 new ones need room
            keep = (held[parents.long()] - torch.randint(0, 9, (N * K,), generator=g, device=DEVICE)).clamp(min=0)
            keep = keep.to(torch.int32)
            room = keep + torch.randint(1, 9, (N * K,), generator=g, device=DEVICE, dtype=torch.int32)
        return dict(op=op, table=table, held=held, parents=parents, refs=refs, keep=keep, room=room)
    if op == "copy":
        R, P = c["R"], c["P"]
        shape = (c["layers"], P, c["Hkv"], PS, D)
        k, v = _pool(g, shape), _pool(g, shape)
        ids = torch.randperm(P, generator=g, device=DEVICE).to(torch.int32)
        if c["full"]:
            tokens = torch.full((R,), PS, dtype=torch.int32, device=DEVICE)
            live = torch.ones(R, dtype=torch.bool, device=DEVICE)
        else:  # a beam whose parent had one child copies nothing
            tokens = torch.randint(1, PS, (R,), generator=g, device=DEVICE, dtype=torch.int32)
            live = torch.arange(R, device=DEVICE)[torch.randperm(R, generator=g, device=DEVICE)] < max(1, (R * 5) // 8)
        copies = torch.stack([ids[:R], ids[R:2 * R], tokens], 1)
        copies = torch.where(live[:, None], copies, torch.tensor([-1, -1, 0], dtype=torch.int32, device=DEVICE))
        return dict(op=op, k=k, v=v, copies=copies.contiguous())
    if op == "compact":
        B, A = c["B"], c["A"]
        lens = _lengths(B, c["lo"], c["hi"])  # cached tokens before the draft
        max_pages = _columns(max(lens) + A)
        P = B * max_pages
        # the pages of the drafts are what the call touches: the pool holds them and no others
        first = torch.tensor(lens, device=DEVICE)[torch.randperm(B, generator=g, device=DEVICE)]
        per = _columns(A) + 1
        P = B * per
        shape = (c["layers"], P, c["Hkv"], PS, D)
        k, v = _pool(g, shape), _pool(g, shape)
        ids = torch.randperm(P, generator=g, device=DEVICE).view(B, per)
        col = torch.arange(max_pages, device=DEVICE)[None, :] - (first // PS)[:, None]
        table = torch.where((col >= 0) & (col < per), torch.gather(ids, 1, col.clamp(0, per - 1)), -1).to(torch.int32)
        # a path down the tree: rising node numbers, 1 .. A of them
        accepted = torch.rand(B, A, generator=g, device=DEVICE).argsort(1)
        count = _accepted(B, A)
        count = torch.tensor(count, device=DEVICE)[torch.randperm(B, generator=g, device=DEVICE)]
        accepted = torch.where(torch.arange(A, device=DEVICE) < count[:, None], accepted, A).sort(1).values
        return dict(op=op, k=k, v=v, table=table, start=first.to(torch.int32), accepted=accepted.to(torch.int32),
                    count=count.to(torch.int32))
    N, K, Hq, Hkv = c["N"], c["K"], c["Hq"], c["Hkv"]
    lens = _lengths(N, c["lo"], c["hi"])
    P = sum(_group_pages(L, K, c["own_tokens"]) for L in lens)
    max_pages = _columns(max(lens))
    L = torch.tensor(lens, device=DEVICE)[torch.randperm(N, generator=g, device=DEVICE)]
    table = _tables(g, N, K, L, c["own_tokens"], P, max_pages)
    kv_lens = L[:, None].expand(N, K) - (_ragged(K) if c["ragged"] else 0)
    kv_lens = kv_lens.clamp(min=0).to(torch.int32).contiguous()
    q = torch.randn(N, K, Hq, D, generator=g, device=DEVICE).to(torch.bfloat16)
    k, v = _pool(g, (P, Hkv, PS, D)), _pool(g, (P, Hkv, PS, D))
    sinks = torch.randn(Hq, generator=g, device=DEVICE)
    return dict(op=op, q=q, k=k, v=v, table=table, lens=kv_lens, sinks=sinks, scale=1 / math.sqrt(D))


def _accepted(B, A):
    """Accepted tokens of B drafts of A: half of a draft on average, at least one."""
    return [1 + (i * A) // B for i in range(B)]


def _ragged(K):
    """How much shorter the beams of a group are, where their lengths differ."""
    return torch.arange(K, device=DEVICE) * 7 % 23


def work(case):
    c, op = case, case["op"]
    if op == "select":
        n = c["N"] * c["K"] * c["V"]
        return {"bytes": n * DTYPES[c["dtype"]].itemsize + c["N"] * (4 * c["K"] + 12 * c["M"]), "flops": 4 * n}
    if op == "fork":
        lens = _lengths(c["N"], c["lo"], c["hi"])
        P = sum(_group_pages(L, c["K"], c["own_tokens"]) for L in lens) + c["extra"]
        R, mp = c["N"] * c["K"], _columns(max(lens) + 2 * PS)
        return {"bytes": 4 * c["K"] * sum(_columns(L) for L in lens) + 4 * R * mp + 8 * P + 24 * R, "flops": 0}
    if op == "copy":
        R = c["R"]
        tokens = R * PS if c["full"] else max(1, (R * 5) // 8) * PS / 2
        return {"bytes": tokens * c["layers"] * c["Hkv"] * D * 2 * 2 * 2 + 12 * R, "flops": 0}
    if op == "compact":
        # token i of the path stays where it is with a probability of about 1 / (i + 1): count them as moved
        return {"bytes": sum(_accepted(c["B"], c["A"])) * c["layers"] * c["Hkv"] * D * 2 * 2 * 2, "flops": 0}
    lens = _lengths(c["N"], c["lo"], c["hi"])
    pages = sum(_group_pages(L, c["K"], c["own_tokens"]) for L in lens)
    rows = c["N"] * c["K"] * c["Hq"]
    return {"bytes": pages * PS * c["Hkv"] * D * 2 * 2 + rows * (D * 4 + 4), "flops": 4 * c["K"] * c["Hq"] * D * sum(lens)}


# ------------------------------------------------------------------------------------- plain forms
def _select_plain(s):
    z, cum, M = s["logits"].float() + 0.0, s["scores"].double(), s["M"]
    N, K, V = z.shape
    m = z.amax(-1, keepdim=True)
    total = (z - m).double().exp().sum(-1)  # in 64 bits: scores of two beams may lie next to each other
    lse = m.squeeze(-1).double() + total.log()
    # a row's best, ties to the lowest token: the value's order and the token in one whole number
    bits = z.view(torch.int32).long()
    order = torch.where(bits >= 0, bits, bits ^ 0x7FFFFFFF)
    key = order * (1 << 32) + (0xFFFFFFFF - torch.arange(V, device=z.device))
    m_row = min(M, V)
    token = 0xFFFFFFFF - torch.topk(key, m_row, -1).values % (1 << 32)  # [N, K, m_row]
    score = cum[..., None] + (torch.gather(z, -1, token).double() - lse[..., None])
    if s["done"] is not None:  # a finished beam stays as it is, on the padding token
        only = torch.where(torch.arange(m_row, device=z.device) == 0, cum[..., None], -math.inf)
        score = torch.where(s["done"][..., None], only, score)
        token = torch.where(s["done"][..., None], s["pad"], token)
    row = torch.arange(N * K, device=z.device).view(N, K, 1).expand(N, K, m_row)
    score, at = torch.sort(score.reshape(N, -1), dim=-1, descending=True, stable=True)
    row, token = torch.gather(row.reshape(N, -1), 1, at), torch.gather(token.reshape(N, -1), 1, at)
    fill = max(0, M - score.shape[1])
    score = torch.nn.functional.pad(score[:, :M], (0, fill), value=-math.inf)
    row = torch.nn.functional.pad(row[:, :M], (0, fill), value=-1)
    token = torch.nn.functional.pad(token[:, :M], (0, fill), value=-1)
    none = score == -math.inf
    return dict(scores=score.float(), parents=row.masked_fill(none, -1).int(), tokens=token.masked_fill(none, -1).int())


def _fork_plain(s):
    table, held, parents, refs = s["table"], s["held"].long(), s["parents"].long(), s["refs"]
    (Rin, mp), R, P, dev = table.shape, parents.shape[0], refs.shape[0], table.device
    keep = held[parents] if s["keep"] is None else s["keep"].long()
    room = keep + 1 if s["room"] is None else s["room"].long()
    kc, rc, hc = _columns(keep), _columns(room), _columns(held)
    writes = (room > keep) & (keep % PS != 0)  # the last kept page will be written
    # the first child of a parent all of whose children keep the same, writes on in a page that the parent alone holds
    none = torch.zeros(Rin, dtype=torch.long, device=dev)
    mark = torch.where(writes, keep, -1)
    low = none.scatter_reduce(0, parents, mark, "amin", include_self=False)
    high = none.scatter_reduce(0, parents, mark, "amax", include_self=False)
    rows = torch.arange(R, device=dev)
    first = none.scatter_reduce(0, parents, rows, "amin", include_self=False)
    last = torch.gather(table[parents], 1, (kc - 1).clamp(min=0)[:, None]).squeeze(1).long()
    alone = (refs[last.clamp(min=0)] == 1) & (low == high)[parents] & (first[parents] == rows)
    copy = writes & ~alone
    need = rc - kc + copy.long()
    at = torch.cumsum(need, 0) - need
    free = refs == 0
    spot = torch.where(free, torch.cumsum(free, 0) - 1, P)
    free_ids = torch.zeros(P + 1, dtype=torch.long, device=dev).scatter(0, spot, torch.arange(P, device=dev))
    c = torch.arange(mp, device=dev)[None, :]
    fresh = ((c >= kc[:, None]) & (c < rc[:, None])) | (copy[:, None] & (c == kc[:, None] - 1))
    index = at[:, None] + c - kc[:, None] + copy.long()[:, None]
    new = free_ids[index.clamp(0, P - 1)]
    old = table[parents].long()
    kept = (c < kc[:, None]) & ~fresh
    out = torch.where(fresh, new, torch.where(kept, old, -1))
    count = torch.zeros(P + 1, dtype=torch.int32, device=dev)
    one = torch.ones((), dtype=torch.int32, device=dev)
    count.index_add_(0, torch.where(c < hc[:, None], table.long(), P).view(-1), -one.expand(Rin * mp))
    count.index_add_(0, torch.where(out >= 0, out, P).view(-1), one.expand(R * mp))
    page = torch.gather(out, 1, (kc - 1).clamp(min=0)[:, None]).squeeze(1)
    copies = torch.stack([torch.where(copy, last, -1), torch.where(copy, page, -1), torch.where(copy, keep % PS, 0)], 1)
    return dict(table=out.int(), lens=room.int(), refs=refs + count[:P], copies=copies.int())


def _copy_plain(s):
    src, dst, tokens = s["copies"].long().unbind(1)
    row, slot = ((torch.arange(PS, device=src.device) < tokens[:, None]) & (src >= 0)[:, None]).nonzero(as_tuple=True)
    a, b = src[row], dst[row]
    s["k"][:, b, :, slot] = s["k"][:, a, :, slot]
    s["v"][:, b, :, slot] = s["v"][:, a, :, slot]
    return dict(k=s["k"], v=s["v"])


def _compact_plain(s):
    A = s["accepted"].shape[1]
    step = torch.arange(A, device=s["k"].device)
    row, i = (step < s["count"][:, None]).nonzero(as_tuple=True)
    to = s["start"].long()[row] + i
    come = s["start"].long()[row] + s["accepted"].long()[row, i]
    b, a = s["table"][row, to // PS].long(), s["table"][row, come // PS].long()
    s["k"][:, b, :, to % PS] = s["k"][:, a, :, come % PS]
    s["v"][:, b, :, to % PS] = s["v"][:, a, :, come % PS]
    return dict(k=s["k"], v=s["v"])


def _decode_plain(s):
    q, table, lens = s["q"].float(), s["table"], s["lens"]
    N, K, Hq, _ = q.shape
    P, Hkv = s["k"].shape[:2]
    T = table.shape[2] * PS
    ids = table.clamp(min=0).long().view(N * K, -1)
    k = s["k"][ids].transpose(1, 2).reshape(N * K, Hkv, T, D).float()  # each beam's own keys, in order
    score = (q.view(N * K, Hkv, Hq // Hkv, D) @ k.transpose(2, 3)) * s["scale"]
    del k
    hidden = torch.arange(T, device=q.device) >= lens.view(-1, 1, 1, 1)
    score = score.masked_fill(hidden, -math.inf)
    sink = s["sinks"].view(1, Hkv, Hq // Hkv, 1)
    m = torch.maximum(score.amax(-1, keepdim=True), sink)
    p = (score - m).exp()
    z = p.sum(-1, keepdim=True) + (sink - m).exp()
    v = s["v"][ids].transpose(1, 2).reshape(N * K, Hkv, T, D).float()
    out = (p @ v) / z
    return dict(out=out.view(N, K, Hq, D).to(torch.bfloat16), lse=(m + z.log()).view(N, K, Hq))


_PLAIN = dict(select=_select_plain, fork=_fork_plain, copy=_copy_plain, compact=_compact_plain, decode=_decode_plain)


# ------------------------------------------------------------------------------------- the library's calls
def _own_calls(s):
    from gqa_attention_learned_head_gb300 import sinkattn as S

    op = s["op"]
    if op == "select":
        scores, parents, tokens = S.sinkattn_beam_select(s["logits"], s["scores"], s["M"], finished=s["done"],
                                                         pad_token=s["pad"])
        return dict(scores=scores, parents=parents, tokens=tokens)
    if op == "fork":
        table, lens, refs, copies = S.sinkattn_pages_fork(s["table"], s["held"], s["parents"], s["refs"],
                                                          keep_lens=s["keep"], room_lens=s["room"], grow=1)
        return dict(table=table, lens=lens, refs=refs, copies=copies)
    if op == "copy":
        S.sinkattn_kv_copy(s["k"], s["v"], s["copies"])
        return dict(k=s["k"], v=s["v"])
    if op == "compact":
        S.sinkattn_kv_compact(s["k"], s["v"], s["table"], s["start"], s["accepted"], s["count"])
        return dict(k=s["k"], v=s["v"])
    out, lse = S.sinkattn_decode_beams(s["q"], s["k"], s["v"], s["table"], s["lens"], s["sinks"], s["scale"])
    return dict(out=out, lse=lse)


def run(state):
    if own:
        return _own_calls(state)
    return _PLAIN[state["op"]](state)


# ------------------------------------------------------------------------------------- in 64 bits, from the definitions
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "select":
        z, cum, best = s["logits"], s["scores"].double(), []
        for n in range(z.shape[0]):
            logp = cum[n][:, None] + torch.log_softmax(z[n].double(), -1)
            if s["done"] is not None:
                stay = torch.full_like(logp, -math.inf)
                stay[:, s["pad"]] = cum[n]
                logp = torch.where(s["done"][n][:, None], stay, logp)
            best.append(logp.reshape(-1).topk(min(s["M"], logp.numel())).values)
        return dict(scores=torch.stack(best), parents=None, tokens=None)
    if case["op"] != "decode":
        return None  # whole numbers, and copies of what is there
    q, k, v, sinks = s["q"].double(), s["k"], s["v"], s["sinks"].double()
    N, K, Hq, _ = q.shape
    G = Hq // k.shape[1]
    out, lse = torch.zeros(N, K, Hq, D, dtype=torch.double, device=q.device), sinks.expand(N, K, Hq).clone()
    lens = s["lens"].tolist()
    for n in range(N):
        for b in range(K):
            if lens[n][b] == 0:
                continue
            ids = s["table"][n, b, :_columns(lens[n][b])].long()
            keys = k[ids].permute(1, 0, 2, 3).flatten(1, 2)[:, :lens[n][b]].double()  # [Hkv, tokens, D]
            vals = v[ids].permute(1, 0, 2, 3).flatten(1, 2)[:, :lens[n][b]].double()
            logit = torch.einsum("ghd,gtd->ght", q[n, b].view(-1, G, D), keys) * s["scale"]
            full = torch.cat([logit, sinks.view(-1, G, 1)], -1)
            prob = torch.softmax(full, -1)[..., :-1]
            out[n, b] = torch.einsum("ght,gtd->ghd", prob, vals).reshape(Hq, D)
            lse[n, b] = torch.logsumexp(full, -1).reshape(Hq)
    return dict(out=out, lse=lse)

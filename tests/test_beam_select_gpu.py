"""Beam search's selection on the GPU against numpy in 64 bits, through the C ABI.

Tolerance.  The largest share of a row here is 131104 tokens: each of 256 threads adds up to 528 exponentials into
four 32-bit sums, 132 additions each.  An addition is off by at most 2^-24 of the partial sum, which grows from 0 to the
whole, so for terms in no order 67 x 2^-24 = 4.0e-6 relative, were all 1024 sums to lean one way (shares of up to 65536
tokens, all other tests: 64 additions and 3.8e-6 even if each is off by 2^-24 of the whole).  An exponential is off by
2^-22 (the instruction's bound) plus 2^-24 times its argument, whose terms weigh e^argument (x e^-x <= 0.37); the groups'
order adds nothing.  Together the log-sum-exp is off by at most 5e-6, and a returned 32-bit score by that plus half a step
of its own.  Picks have to be the reference's wherever its next score is further away than twice that.
"""
import math
import random
from concurrent.futures import ThreadPoolExecutor
from fractions import Fraction

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

LSE_TOL = 5e-6


@pytest.fixture(scope="module")
def S():
    from gqa_attention_learned_head_gb300 import sinkattn

    return sinkattn


def reference(logits, scores, M, finished=None, pad=0):
    """(scores, parents, tokens) [N, M], and every group's sorted scores."""
    z = logits.double().cpu().numpy()
    c = scores.double().cpu().numpy()
    N, K, V = z.shape
    out_s, out_p, out_t = np.full((N, M), -np.inf), np.full((N, M), -1), np.full((N, M), -1)
    for n in range(N):
        rows = np.full((K, V), -np.inf)
        for k in range(K):
            if not np.isfinite(c[n, k]):
                continue
            if finished is not None and bool(finished[n, k]):
                rows[k, pad] = c[n, k]
                continue
            m = z[n, k].max()
            if not np.isfinite(m) or np.isnan(z[n, k]).any():
                continue
            lse = m + np.log(np.exp(z[n, k] - m).sum())
            rows[k] = c[n, k] + (z[n, k] - lse)
        flat = rows.reshape(-1)
        top = np.lexsort((np.arange(flat.size), -flat))[:M]
        top = top[flat[top] > -np.inf]
        out_s[n, :top.size] = flat[top]
        out_p[n, :top.size] = n * K + top // V
        out_t[n, :top.size] = top % V
    return out_s, out_p, out_t


def check(got, ref, exact=False):
    gs, gp, gt = (t.cpu().numpy() for t in got)
    rs, rp, rt = ref
    assert np.array_equal(np.isneginf(gs), np.isneginf(rs))
    live = ~np.isneginf(rs)
    err = np.abs(gs[live] - rs[live])
    assert np.all(err <= LSE_TOL + 2.0 ** -24 * np.abs(rs[live])), err.max()
    with np.errstate(invalid="ignore"):
        gap = np.minimum(np.abs(np.diff(rs, axis=1, prepend=np.inf)), np.abs(np.diff(rs, axis=1, append=-np.inf)))
    # (the last pick's rival is not in the list: its score was compared above)
    sure = np.ones_like(live) if exact else ~live | (np.nan_to_num(gap, nan=np.inf) > 2 * LSE_TOL)
    sure[:, -1] &= exact | ~live[:, -1]
    assert np.array_equal(gp[sure], rp[sure]) and np.array_equal(gt[sure], rt[sure])


def make(N, K, V, dtype, seed, std=2.5):
    g = torch.Generator().manual_seed(seed)
    z = (torch.randn(N, K, V, generator=g) * std).to(dtype).cuda()
    c = (-20 * torch.rand(N, K, generator=g)).cuda()
    return z, c


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("N,K,V,M", [(1, 1, 1, 1), (1, 1, 5, 3), (2, 3, 15, 8), (1, 4, 16, 64), (3, 2, 17, 5),
                                     (1, 32, 257, 64), (2, 8, 4099, 16), (1, 4, 32000, 8), (5, 3, 50021, 6),
                                     (1, 2, 200003, 4), (2, 1, 131072, 64)])
def test_sizes(S, dtype, N, K, V, M):
    z, c = make(N, K, V, dtype, seed=N + K + V + M)
    got = S.sinkattn_beam_select(z, c, M)
    assert S.sinkattn_get_error() == 0
    check(got, reference(z, c, M))


def test_more_rows_than_resident_shares(S):
    z, c = make(400, 4, 1003, torch.bfloat16, seed=5)
    got = S.sinkattn_beam_select(z, c, 8)
    assert S.sinkattn_get_error() == 0
    check(got, reference(z, c, 8))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("pad,first", [(1, 0), (3, 1), (24, 8), (0, 5)])
def test_padded_rows_and_odd_starts(S, dtype, pad, first):
    """Rows at any distance, starting at any element of the buffer: the same picks, and the padding is not read as
    logits (it holds the largest values)."""
    N, K, V, M = 2, 3, 5003, 7
    z, c = make(N, K, V, dtype, seed=9)
    buf = torch.full((first + N * K * (V + pad),), 1e4, dtype=dtype, device="cuda")
    view = torch.as_strided(buf, (N, K, V), (K * (V + pad), V + pad, 1), first)
    view.copy_(z)
    a, b = S.sinkattn_beam_select(z, c, M), S.sinkattn_beam_select(view, c, M)
    assert S.sinkattn_get_error() == 0
    check(b, reference(z, c, M))
    for x, y in zip(a, b):  # sums run in the tokens' order wherever a row starts: the same bits
        assert torch.equal(x, y)


def test_equal_beams_and_equal_logits_go_to_the_lowest(S):
    """Ties of every kind: identical beams (as at a search's first step), constant rows, long runs of one value."""
    N, K, V, M = 2, 4, 10007, 12
    z, c = make(N, 1, V, torch.float32, seed=3)
    z, c = z.expand(N, K, V).contiguous(), c[:, :1].expand(N, K).contiguous()
    check(S.sinkattn_beam_select(z, c, M), reference(z, c, M), exact=True)
    z = torch.full((N, K, V), -1.5, device="cuda", dtype=torch.bfloat16)
    s, p, t = S.sinkattn_beam_select(z, c, M)
    assert torch.equal(t.cpu(), torch.arange(M, dtype=torch.int32).expand(N, M))
    assert torch.equal(p.cpu(), (torch.arange(N, dtype=torch.int32) * K)[:, None].expand(N, M))
    z[:, 2, 7000:] = 4.0
    check(S.sinkattn_beam_select(z, c, 64), reference(z, c, 64), exact=True)


@pytest.mark.parametrize("order", [1, -1])
def test_sorted_logits(S, order):
    """Rising or falling logits: the best all lie in one thread's, or neighbouring, groups."""
    V = 70000
    z = (torch.arange(V, dtype=torch.float32) * order / 1000).expand(1, 2, V).contiguous().cuda()
    c = torch.tensor([[-1.0, -1.25]]).cuda()
    check(S.sinkattn_beam_select(z, c, 33), reference(z, c, 33))


def test_best_tokens_in_one_threads_groups(S):
    """The best tokens at a distance of 256 groups: one thread meets them all."""
    V = 65536
    z, c = make(1, 1, V, torch.float32, seed=8)
    z[0, 0, ::4096] += 40
    z[0, 0, 5::4096] += 41
    check(S.sinkattn_beam_select(z, c, 40), reference(z, c, 40))


def test_finished_and_unused_beams(S):
    N, K, V, M = 3, 5, 3001, 10
    z, c = make(N, K, V, torch.bfloat16, seed=4)
    c[0, 1:] = -math.inf  # the first step: one beam in use
    c[2, :] = -math.inf
    done = torch.zeros(N, K, dtype=torch.bool, device="cuda")
    done[1, 0] = done[1, 3] = done[0, 4] = True
    z[0, 1:] = float("nan")  # logits that are not to be read
    z[1, 3] = float("nan")
    got = S.sinkattn_beam_select(z, c, M, finished=done, pad_token=17)
    assert S.sinkattn_get_error() == 0
    check(got, reference(z, c, M, done, 17))
    everyone = torch.ones(N, K, dtype=torch.uint8, device="cuda")
    s, p, t = S.sinkattn_beam_select(z, c, M, finished=everyone, pad_token=3000)
    assert S.sinkattn_get_error() == 0
    check((s, p, t), reference(z, c, M, everyone, 3000), exact=True)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
def test_masked_tokens(S, dtype):
    """-inf tokens are no continuations; masks of the type's lowest value are very unlikely ones."""
    N, K, V, M = 2, 3, 9001, 20
    z, c = make(N, K, V, dtype, seed=6)
    z[0, 0, :] = -math.inf           # a row without a token
    z[0, 1, 5:] = -math.inf          # five tokens left
    z[0, 2, 100:8990] = -math.inf
    lowest = torch.finfo(dtype).min
    z[1, 0, 7:] = lowest
    z[1, 1, :] = lowest              # uniform, at the bottom of the type's range
    z[1, 2, :] = -math.inf
    got = S.sinkattn_beam_select(z, c, M)
    assert S.sinkattn_get_error() == 0
    rs, rp, rt = reference(z, c, M)
    gs, gp, gt = (t.cpu().numpy() for t in got)
    assert np.allclose(gs, rs, rtol=2.0 ** -22, atol=LSE_TOL)
    assert np.array_equal(gp, rp) and np.array_equal(gt, rt)


@pytest.mark.parametrize("value", [3e5, 2e6, 1e30, -2e6, -3e38])
def test_large_logits(S, value):
    """Rows around a value whose product with log2 e has no fraction left, or overflows."""
    V, M = 5000, 6
    z = torch.full((1, 2, V), value, device="cuda")
    z[0, 0, 3000] = value + abs(value) * 1e-5
    z[0, 1, 17] = -math.inf
    c = torch.tensor([[-2.0, -1.0]]).cuda()
    got = S.sinkattn_beam_select(z, c, M)
    assert S.sinkattn_get_error() == 0
    rs, rp, rt = reference(z, c, M)
    gs, gp, gt = (t.cpu().numpy() for t in got)
    assert np.allclose(gs, rs, rtol=2.0 ** -22, atol=LSE_TOL)
    assert np.array_equal(gp, rp) and np.array_equal(gt, rt)


@pytest.mark.parametrize("where", ["nan", "inf", "nan score", "inf score", "nan among masked"])
def test_bad_values_are_reported_and_their_beam_left_out(S, where):
    N, K, V, M = 2, 3, 20011, 5
    z, c = make(N, K, V, torch.float32, seed=7)
    if where == "nan":
        z[1, 1, 19999] = float("nan")
    elif where == "inf":
        z[1, 1, 3] = math.inf
    elif where == "nan among masked":
        z[1, 1, :] = -math.inf
        z[1, 1, 12345] = float("nan")
    else:
        c[1, 1] = float("nan") if where == "nan score" else math.inf
    got = S.sinkattn_beam_select(z, c, M)
    assert S.sinkattn_get_error() == S.ERR_BAD_VALUE
    c2 = c.clone()
    c2[1, 1] = -math.inf
    check(got, reference(torch.nan_to_num(z, posinf=0.0), c2, M))
    assert S.sinkattn_get_error() == 0


@pytest.mark.parametrize("fill", ["random", "equal", "one quad"])
def test_largest_shares(S, fill):
    """Rows of more than one full share of 262144 tokens, the most picks: the lists at their capacity."""
    V, M = 2 * 262144 + 77, 64
    z, c = make(1, 2, V, torch.float32, seed=21)
    if fill == "equal":
        z[:] = 0.25
    elif fill == "one quad":  # the best tokens of all of a quad of threads' groups: two groups of every 128
        z = z.view(-1)
        lead = torch.arange(2 * V, device="cuda") % V % 4096 < 64
        z = torch.where(lead, z + 50, z).view(1, 2, V)
    got = S.sinkattn_beam_select(z, c, M)
    assert S.sinkattn_get_error() == 0
    if fill == "equal":
        best = 0 if float(c[0, 0]) >= float(c[0, 1]) else 1
        assert torch.equal(got[2].cpu(), torch.arange(M, dtype=torch.int32)[None]) and (got[1] == best).all()
    else:
        check(got, reference(z, c, M))


def test_groups_and_empty_call(S):
    z, c = make(1, 2, 100, torch.float32, seed=1)
    s, p, t = S.sinkattn_beam_select(z[:0], c[:0], 4)
    assert s.shape == (0, 4) and p.shape == (0, 4) and t.shape == (0, 4)


def test_replayed_from_a_graph_and_on_another_stream(S):
    z, c = make(3, 4, 8009, torch.bfloat16, seed=11)
    out = [torch.empty(3, 8, dtype=d, device="cuda") for d in (torch.float32, torch.int32, torch.int32)]
    ws = torch.empty(S.sinkattn_beam_select_workspace_size(z, 8), dtype=torch.uint8, device="cuda")
    call = lambda **kw: S.sinkattn_beam_select(z, c, 8, out_scores=out[0], out_parents=out[1],  # noqa: E731
                                               out_tokens=out[2], workspace=ws, **kw)
    call()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    z2, c2 = make(3, 4, 8009, torch.bfloat16, seed=12)
    z.copy_(z2)
    c.copy_(c2)
    g.replay()
    torch.cuda.synchronize()
    check(out, reference(z2, c2, 8))
    other = torch.cuda.Stream()
    other.wait_stream(torch.cuda.current_stream())
    got = S.sinkattn_beam_select(z, c, 8, stream=other)
    other.synchronize()
    for x, y in zip(got, out):
        assert torch.equal(x, y)


def test_refusals(S):
    z, c = make(2, 3, 100, torch.float32, seed=2)
    with pytest.raises(TypeError):
        S.sinkattn_beam_select(z.double(), c, 4)
    with pytest.raises(TypeError):
        S.sinkattn_beam_select(z.cpu(), c, 4)
    with pytest.raises(TypeError):
        S.sinkattn_beam_select(z, c.half(), 4)
    with pytest.raises(ValueError):
        S.sinkattn_beam_select(z, c[:1], 4)
    with pytest.raises(ValueError):
        S.sinkattn_beam_select(z.transpose(1, 2), c, 4)
    with pytest.raises(ValueError):
        S.sinkattn_beam_select(z, c, 4, finished=torch.zeros(2, 2, dtype=torch.bool, device="cuda"))
    for M, pad in ((0, 0), (65, 0), (4, 100), (4, -1)):
        with pytest.raises(S.SinkAttnError):
            S.sinkattn_beam_select(z, c, M, pad_token=pad)
    with pytest.raises(S.SinkAttnError) as e:
        S.sinkattn_beam_select(z, c, 4, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    assert e.value.status == S.ERR_WORKSPACE


@pytest.mark.parametrize("V,M", [(300, 20), (1125, 20), (1125, 64), (2047, 64), (2048, 63), (2100, 64), (4232, 24)])
@pytest.mark.parametrize("fill", ["random", "levels", "equal"])
def test_few_groups(S, V, M, fill):
    """Short rows, where the picks reach into most groups of tokens: hundreds of candidates a row, or equal ones."""
    z, c = make(3, 4, V, torch.bfloat16, seed=V + M)
    if fill == "levels":  # four values only: ties everywhere
        z = (z * 0.4).round().clamp(-2, 1)
    elif fill == "equal":
        z = torch.full_like(z, 0.25)
    got = S.sinkattn_beam_select(z, c, M)
    assert S.sinkattn_get_error() == 0
    check(got, reference(z, c, M))
    if fill == "equal":  # the first tokens of the best beam
        best = c.argmax(1)
        assert torch.equal(got[1].long(), (torch.arange(3, device="cuda") * 4 + best)[:, None].expand(3, M))
        assert torch.equal(got[2].long(), torch.arange(M, device="cuda").expand(3, M))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("V,M", [(40009, 64), (777, 64), (33, 64)])
def test_every_start_of_a_row(S, dtype, V, M):
    """One row's logits 32 times, at every distance from a sector's start: the same scores to the last bit, so that the
    beams come in their order at every token."""
    z, _ = make(1, 1, V, dtype, seed=V)
    stride = V + 1 + V % 2  # odd
    buf = torch.full((32 * stride,), 50.0, dtype=dtype, device="cuda")
    rows = buf.as_strided((1, 32, V), (32 * stride, stride, 1))
    rows.copy_(z.expand(1, 32, V))
    c = torch.full((1, 32), -3.0, device="cuda")
    got = S.sinkattn_beam_select(rows, c, M)
    assert S.sinkattn_get_error() == 0
    assert torch.equal(got[1][0].long(), torch.arange(M, device="cuda") % 32)
    order = torch.sort(z.view(-1).float(), descending=True, stable=True)[1]
    assert torch.equal(got[2][0].long(), order[:2].repeat_interleave(32))
    check(got, reference(rows, c, M))


def test_scores_in_place(S):
    """The running scores of the next step over those of this one."""
    z, c = make(70, 6, 9001, torch.bfloat16, seed=23)
    want = S.sinkattn_beam_select(z, c, 6)
    kept = c.clone()
    got = S.sinkattn_beam_select(z, kept, 6, out_scores=kept)
    assert got[0].data_ptr() == kept.data_ptr()
    assert all(torch.equal(x, y) for x, y in zip(want, got))
    assert S.sinkattn_get_error() == 0


def levels(N, K, V, dtype, seed):
    """Logits of four values (whole-number draws, the same on every machine) and scores that keep the beams apart."""
    g = torch.Generator().manual_seed(seed)
    z = (torch.randint(0, 4, (N, K, V), generator=g) - 2).to(dtype)
    c = -(0.37 * torch.arange(K) + 0.053 * torch.arange(N)[:, None]).float()
    return z.cuda(), c.cuda()


def in_order(z, c, M):
    """The reference's picks where scores of different beams are so far apart that every pick is certain."""
    ref = reference(z, c, M + 1 if M < z.shape[1] * z.shape[2] else M)
    step = -np.diff(ref[0], axis=1)
    assert np.all((step == 0) | (step > 4 * LSE_TOL))  # equal ones are of one beam: the draw's, not the call's
    return tuple(x[:, :M] for x in ref)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("V,M,fill", [(2100, 64, "levels"), (1125, 40, "levels"), (400, 20, "equal")])
def test_second_threshold_again_and_again(S, dtype, V, M, fill):
    """More than 256 equal tokens in the best groups of every row, in every resident block at once: the tokens that the second
    threshold leaves are the same, and the reference's, each time."""
    z, c = levels(64, 8, V, dtype, seed=V)
    if fill == "equal":
        z = torch.full_like(z, 0.25)
    first = S.sinkattn_beam_select(z, c, M)
    check(first, in_order(z, c, M), exact=True)
    for _ in range(200):
        again = S.sinkattn_beam_select(z, c, M)
        assert all(torch.equal(x, y) for x, y in zip(first, again))
    assert S.sinkattn_get_error() == 0


def exact_picks(logits, scores, M):
    """(scores f32, parents, tokens) [N, M] of finite logits and scores from rational numbers, the logarithm alone in 64 bits."""
    z, c = logits.double().cpu().numpy(), scores.double().cpu().numpy()
    N, K, V = z.shape
    out = np.full((N, M), -np.inf, np.float32), np.full((N, M), -1), np.full((N, M), -1)
    for n in range(N):
        rows = []
        for k in range(K):
            m = z[n, k].max()
            log = Fraction(float(np.log(np.exp(z[n, k] - m).sum())))
            rows += [(-(Fraction(c[n, k]) + (Fraction(x) - Fraction(m) - log)), k, v) for v, x in enumerate(z[n, k])]
        for i, (s, k, v) in enumerate(sorted(rows)[:M]):
            with np.errstate(over="ignore"):
                out[0][n, i], out[1][n, i], out[2][n, i] = np.float32(float(-s)), n * K + k, v
    return out


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("V", [40, 4500])
def test_scores_below_the_range(S, dtype, V):
    """Beams marked by the lowest f32 score whose tokens are masked by the type's lowest value: what falls below f32's range is
    -inf, comes after everything within it, and in its order."""
    low, masked = torch.finfo(torch.float32).min, torch.finfo(dtype).min
    K, M = 4, 30
    z = torch.full((3, K, V), masked, dtype=dtype)
    ramp = (torch.arange(6) * -0.5).to(dtype)
    z[0, 0, :6] = ramp                 # six tokens of a beam in use, behind them a beam out of use
    z[0, 1, 3:9] = ramp
    z[1, :, 5:11] = ramp               # every beam out of use, two as far down as can be
    z[2, 0, :4] = ramp[:4]
    z[2, 1, :] = 0                     # all of the same logit
    z[2, 2, 7] = 3.0
    z[2, 3, :2] = ramp[:2]
    c = torch.tensor([[-1.0, low, low / 2, low], [low, low / 2, low, low / 4], [low / 8, low, low / 2, -3.0]])
    got = [t.cpu().numpy() for t in S.sinkattn_beam_select(z.cuda(), c.cuda(), M)]
    assert S.sinkattn_get_error() == 0
    want = exact_picks(z, c, M)
    assert not np.isnan(got[0]).any()
    with np.errstate(invalid="ignore"):
        assert np.all((got[0] == want[0]) | (np.abs(got[0] - want[0]) <= LSE_TOL + 2.0 ** -23 * np.abs(want[0])))
    assert np.array_equal(got[1], want[1]) and np.array_equal(got[2], want[2])


def test_wide_logits_below_the_range(S):
    """Logits further apart than f32 reaches: z - lse alone falls below the range, and comes back where the score is large."""
    z = torch.full((2, 1, 50), -3.0e38)
    z[:, 0, 7] = 3.0e38
    z[:, 0, 9] = 2.0e38
    z[:, 0, 20:] = -1.0e38
    c = torch.tensor([[-2.0], [3.0e38]])
    got = [t.cpu().numpy() for t in S.sinkattn_beam_select(z.cuda(), c.cuda(), 45)]
    assert S.sinkattn_get_error() == 0
    want = exact_picks(z, c, 45)
    assert np.isneginf(want[0][0]).any() and not np.isneginf(want[0][1]).any()
    assert np.array_equal(got[1], want[1]) and np.array_equal(got[2], want[2])
    assert np.allclose(got[0], want[0], rtol=2.0 ** -22, atol=LSE_TOL)


@pytest.mark.parametrize("shape,large,small", [((40, 8, 200000), 64, 32), ((3, 32, 257), 64, 48)])
def test_two_host_threads(S, shape, large, small):
    """A thread's call that needs little shared memory leaves the kernels' limits to another thread's that needs much."""
    z = torch.randn(shape, device="cuda")
    c = -torch.rand(shape[:2], device="cuda")
    torch.cuda.synchronize()

    def call(M):
        stream = torch.cuda.Stream()
        got = S.sinkattn_beam_select(z, c, M, stream=stream)
        stream.synchronize()
        return got

    with ThreadPoolExecutor(1) as a, ThreadPoolExecutor(1) as b:
        first = a.submit(call, large).result()
        other = b.submit(call, small).result()
        again = a.submit(call, large).result()
        both = [x.submit(call, m) for _ in range(20) for x, m in ((a, large), (b, small))]
        both = [x.result() for x in both]
    for x, y, o in zip(first, again, other):
        assert torch.equal(x, y) and torch.equal(x[:, :small], o)
    for got, want in zip(both, [first, other] * 20):
        assert all(torch.equal(x, y) for x, y in zip(got, want))
    assert S.sinkattn_get_error() == 0


def check_picks(got, z, c):
    """Every pick is another continuation, of the score that it has in 64 bits, and runs of equal scores of one beam are in their
    tokens' order."""
    gs, gp, gt = (t.cpu().numpy() for t in got)
    z, c = z.double().cpu().numpy(), c.double().cpu().numpy()
    N, K, V = z.shape
    m = z.max(-1, keepdims=True)
    score = c[..., None] + (z - m - np.log(np.exp(z - m).sum(-1, keepdims=True)))
    for n in range(N):
        live = gp[n] >= 0
        assert live.sum() == min(gp.shape[1], K * V)
        k, v, s = gp[n, live] - n * K, gt[n, live], gs[n, live]
        assert len(set(zip(k.tolist(), v.tolist()))) == live.sum()
        assert np.all((0 <= k) & (k < K) & (0 <= v) & (v < V))
        want = score[n, k, v]
        assert np.all(np.abs(s - want) <= LSE_TOL + 2.0 ** -24 * np.abs(want))
        assert np.all(np.diff(s) <= 0)
        same = (np.diff(k) == 0) & (z[n, k[1:], v[1:]] == z[n, k[:-1], v[:-1]])
        assert np.all(np.diff(v)[same] > 0)
        for q in range(K):  # no continuation of a beam is left out for a later one of it
            mine = v[k == q]
            order = np.lexsort((np.arange(V), -z[n, q]))[:mine.size]
            assert np.array_equal(mine, order)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("V,M", [(31, 64), (300, 20), (1125, 20), (1125, 64), (2047, 64), (2048, 63), (2100, 64), (4232, 24),
                                 (40009, 40)])
@pytest.mark.parametrize("fill", ["random", "levels", "coarse"])
def test_every_pick(S, dtype, V, M, fill):
    """Pick by pick, ties among them: flat, coarsely rounded and ordinary logits."""
    z, c = levels(3, 4, V, dtype, seed=V + M)
    if fill != "levels":
        z, _ = make(3, 4, V, dtype, seed=V + M)
    if fill == "coarse":
        z = (z * 4).round() / 4
    got = S.sinkattn_beam_select(z, c, M)
    assert S.sinkattn_get_error() == 0
    check_picks(got, z, c)
    if fill == "levels":
        check(got, in_order(z, c, M), exact=True)


def test_logarithm_between_two_beams(S):
    """Rows of n zeros and nothing else, whose sums are whole numbers: the beams' order hangs on the logarithms alone.

    The logarithm is off by at most 1.6e-9 (series and roundings), and by its base's rounding, 1.34e-8 of the entropy ln n: between
    two beams 2 x 1.6e-9 + 1.34e-8 x 0.17 = 5.5e-9 here, under half of the 1.2e-8 by which the scores differ at least."""
    rng, V, N = random.Random(4), 70000, 96
    z = torch.full((N, 2, V), -math.inf)
    c, best = torch.empty(N, 2), []
    while len(best) < N:
        n0 = int(math.exp(rng.uniform(math.log(20), math.log(60000))))
        n1 = n0 + rng.randint(-n0 // 7, n0 // 7)
        c0 = np.float32(rng.uniform(-0.08, -0.01))
        c1 = np.float32(float(c0) - math.log(n0) + math.log(n1) + rng.uniform(-1e-7, 1e-7))
        gap = (float(c0) - math.log(n0)) - (float(c1) - math.log(n1))
        if abs(gap) < 1.2e-8 or abs(math.log(n0 / n1)) > 0.17:
            continue
        i = len(best)
        z[i, 0, :n0], z[i, 1, :n1], c[i, 0], c[i, 1] = 0, 0, float(c0), float(c1)
        best.append(2 * i + (0 if gap > 0 else 1))
    s, p, t = S.sinkattn_beam_select(z.cuda(), c.cuda(), 2)
    assert S.sinkattn_get_error() == 0
    assert p.cpu().tolist() == [[b, b] for b in best]
    assert t.cpu().tolist() == [[0, 1]] * N

"""Sampling where the random number falls into a run of tokens so light that none of its steps raises the sum before them: every row gets
a token that has weight, next to where exact arithmetic ends."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def S():
    from gqa_attention_learned_head_gb300 import sinkattn

    return sinkattn


def test_every_row_gets_a_token(S):
    gen = np.random.default_rng(17)
    N, V, a, b = 64, 200000, 100000, 103128  # a row is eight chunks of eight runs of 3128 tokens: a..b is one run
    half = V - b
    z = np.full((N, V), -np.inf, np.float32)
    for n in range(N):
        x = gen.uniform(-2, 0, half).astype(np.float32)
        x[0] = 0
        z[n, :half], z[n, b:] = x, gen.permutation(x)  # as much before the run as behind it
    z[:, a:b] = -42 * np.log(2)
    tokens, logprobs = torch.full((N,), -7, dtype=torch.int32, device="cuda"), torch.full((N,), 7.0, device="cuda")
    S.sinkattn_sample(torch.from_numpy(z).cuda(), torch.full((N,), 0.5, device="cuda"), out_tokens=tokens, out_logprobs=logprobs)
    assert S.sinkattn_get_error() == 0
    inside = 0
    for n, (token, lp) in enumerate(zip(tokens.tolist(), logprobs.tolist())):
        w = np.exp(z[n].astype(np.longdouble))
        line = np.cumsum(w)
        assert 0 <= token < V and w[token] > 0, n
        inside += a <= token < b
        # sums in 46 bits, some 16 of them one in the other; the weights on both sides are the same
        assert line[token] - w[token] - line[-1] * 2.0**-42 <= line[-1] / 2 <= line[token] + line[-1] * 2.0**-42, n
        want = float(z[n, token].astype(np.longdouble) - np.log(line[-1]))
        assert abs(lp - want) <= 2.0**-24 * abs(want) + 3e-9, n  # 2^-28.5 of the weights
    assert inside > 0


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_tokens_without_weight_between(S, dtype):
    """Weights below 2^-110 of the largest are nothing: with equal weights around them, numbers at the very border pick the next token that
    has some."""
    V = 4096
    logits = torch.full((5, V), -200.0, dtype=dtype, device="cuda")
    logits[:, [100, 101, 900, 4000]] = 3.0
    u = torch.tensor([0.0, 0.25, 0.5, 0.75, 1 - 2.0**-24], device="cuda")
    token, logprob = S.sinkattn_sample(logits, u)
    assert S.sinkattn_get_error() == 0
    assert token.tolist() == [100, 101, 900, 4000, 4000]
    assert torch.allclose(logprob, torch.full_like(logprob, -np.log(4.0)), atol=1e-6)
    low = torch.full((2, V), -200.0, dtype=dtype, device="cuda")  # top-k's last tokens have no weight
    low[:, 4000] = 3.0
    token, logprob = S.sinkattn_sample(low, u[[0, 4]], top_k=torch.full((2,), 50, dtype=torch.int32, device="cuda"))
    assert token.tolist() == [4000, 4000] and logprob.abs().max() <= 2.0**-28


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
def test_a_sure_token_has_log_probability_zero(S, dtype):
    """The only kept token, whatever the size of its logit and the temperature, by each filter and by itself."""
    logits = torch.full((8, 999), -torch.inf, dtype=dtype, device="cuda")
    logits[:, 500] = torch.tensor([3.0, -7.25, 0.3, 1e-4, 900.0, -31000.0, 0.0, 17.0]).to(dtype).cuda()
    u = torch.rand(8, device="cuda")
    t = torch.tensor([1.0, 0.7, 2.3, 0.01, 0.1, 1e-3, 5.0, 0.33], device="cuda")
    for more in (False, True):
        if more:
            logits[:, 100:400] = (logits[:, 500:501].float() - 90 * t[:, None] - 0.02 * logits[:, 500:501].float().abs()).to(dtype)  # next to nothing
        p, q = torch.full((8,), 0.5, device="cuda"), torch.full((8,), 0.5, device="cuda")
        for kw in ((dict(top_p=p), dict(min_p=q), dict(top_k=torch.ones(8, dtype=torch.int32, device="cuda"))) if more else ({}, dict(top_p=p))):
            token, logprob = S.sinkattn_sample(logits, u, t, **kw)
            assert S.sinkattn_get_error() == 0
            assert token.tolist() == [500] * 8 and not logprob.any(), kw

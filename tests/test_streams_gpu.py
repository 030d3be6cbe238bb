"""Calls on a stream of the caller's: what they allocate belongs to that stream."""
import pytest
import torch

from gqa_attention_learned_head_gb300 import workloads as W

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def S():
    from gqa_attention_learned_head_gb300 import sinkattn

    return sinkattn


def call(S, name, **kw):
    if name in ("decode", "beams"):
        g = W.make_decode(4, 16, 2, [300, 1, 40, 77], seed=1).to("cuda")
        if name == "beams":
            return S.sinkattn_decode_beams(g.q.view(2, 2, 16, 64), g.k_pages, g.v_pages, g.page_table.view(2, 2, -1),
                                           g.kv_lens.view(2, 2), g.sinks, g.scale, **kw)
        return S.sinkattn_decode(g.q, g.k_pages, g.v_pages, g.page_table, g.kv_lens, g.sinks, g.scale, **kw)
    if name in ("verify", "tree"):
        g = W.make_decode(3, 16, 2, [40, 9, 100], seed=2, q_len=4).to("cuda")
        args = (g.q, g.k_pages, g.v_pages, g.page_table, g.kv_lens)
        if name == "tree":
            masks = torch.tensor([1, 3, 5, 15], dtype=torch.int64, device="cuda").expand(3, 4).contiguous()
            return S.sinkattn_verify_tree(*args, masks, g.sinks, g.scale, **kw)
        return S.sinkattn_verify(*args, g.sinks, g.scale, **kw)
    if name == "prefill":
        g = W.make_prefill(16, 2, [130, 5], seed=3).to("cuda")
        return S.sinkattn_prefill(g.q, g.k, g.v, g.cu_seqlens, g.sinks, g.scale, max_seqlen=130, **kw)
    if name == "merge":
        g = torch.Generator(device="cuda").manual_seed(4)
        return S.sinkattn_merge(torch.randn(3, 4, 8, 64, generator=g, device="cuda"), torch.randn(3, 4, 8, generator=g, device="cuda"),
                                **kw)
    if name == "select":
        g = torch.Generator(device="cuda").manual_seed(5)
        return S.sinkattn_beam_select(torch.randn(2, 3, 500, generator=g, device="cuda"), torch.zeros(2, 3, device="cuda"), 4, **kw)
    g = W.make_paged_prefill(16, 2, [5, 30], [20, 7], seed=5).to("cuda")
    if name == "paged":
        return S.sinkattn_prefill_paged(g.q, g.k_pages, g.v_pages, g.page_table, g.cu_seqlens, g.start_pos, g.sinks, g.scale,
                                        max_seqlen=20, **kw)
    qkv = torch.randn(27, 20 * 64, generator=torch.Generator(device="cuda").manual_seed(6), device="cuda").to(torch.bfloat16)
    return (S.sinkattn_qkv_prologue(qkv, None, g.cu_seqlens, g.start_pos, g.page_table, g.k_pages, g.v_pages, 16, 1e4, 32.0, 4096, 32.0,
                                    1.0, **kw),)


@pytest.mark.parametrize("name", ["decode", "verify", "tree", "prefill", "paged", "prologue", "merge", "select", "beams"])
def test_outputs_and_workspace_belong_to_the_calls_stream(S, name, monkeypatch):
    want = [t.clone() for t in call(S, name)]
    torch.cuda.synchronize()
    side, seen = torch.cuda.Stream(), []
    call(S, name)  # the inputs' allocations come from the caller's stream in both runs
    torch.cuda.synchronize()

    def watched(fn):
        def alloc(*a, **kw):
            seen.append(torch.cuda.current_stream().cuda_stream)
            return fn(*a, **kw)
        return alloc

    class Torch:  # what the binding sees of torch
        empty, empty_like = staticmethod(watched(torch.empty)), staticmethod(watched(torch.empty_like))

        def __getattr__(self, attr):
            return getattr(torch, attr)

    monkeypatch.setattr(S, "torch", Torch())
    side.wait_stream(torch.cuda.current_stream())
    torch.cuda.synchronize()
    got = call(S, name, stream=side)
    monkeypatch.undo()
    side.synchronize()
    assert seen and all(x == side.cuda_stream for x in seen)
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    assert S.sinkattn_get_error() == 0

"""The beam step's entry points refuse malformed calls on the host, before they touch a device (no GPU needed)."""
import ctypes

import pytest


@pytest.fixture(scope="module")
def S():
    from gqa_attention_learned_head_gb300 import build

    build.build()
    from gqa_attention_learned_head_gb300 import sinkattn

    return sinkattn


def test_new_status_strings(S):
    assert "pages" in S.status_string(S.ERR_NO_PAGES)
    assert "NaN" in S.status_string(S.ERR_BAD_VALUE)
    assert "index" in S.status_string(S.ERR_BAD_INDEX)


def test_beam_select_dims(S):
    ok = dict(num_groups=2, num_beams=4, vocab=1000, num_select=8, dtype=S.DTYPE_BF16, pad_token=0, row_stride=1000)

    def call(**kw):
        d = S.BeamDims(**{**ok, **kw})
        st = S._lib.sinkattn_beam_select(None, None, None, None, None, None, ctypes.byref(d), None, 0, None)
        if st != S.ERR_INVALID_ARG or kw:
            assert kw.get("num_groups") == 0 or S._lib.sinkattn_beam_select_workspace_size(ctypes.byref(d)) == 0
        return st

    assert call() == S.ERR_INVALID_ARG  # null buffers
    for kw in (dict(num_groups=-1), dict(num_beams=0), dict(vocab=0), dict(num_select=0), dict(row_stride=999),
               dict(pad_token=1000), dict(pad_token=-1)):
        assert call(**kw) == S.ERR_INVALID_ARG, kw
    for kw in (dict(dtype=3), dict(dtype=-1), dict(num_beams=33), dict(num_select=65), dict(num_groups=65536),
               dict(vocab=(1 << 30) + 1, row_stride=1 << 31), dict(row_stride=(1 << 40) + 1),
               dict(num_beams=32, num_select=64, vocab=1 << 20, row_stride=1 << 20)):
        assert call(**kw) == S.ERR_UNSUPPORTED, kw
    assert call(num_groups=0) == S.OK  # nothing to do
    assert S._lib.sinkattn_beam_select(None, None, None, None, None, None, None, None, 0, None) == S.ERR_INVALID_ARG


def test_pages_fork_dims(S):
    ok = dict(num_rows_in=2, num_rows_out=2, num_pages=8, max_pages=4, page_size=16, grow=1)

    def call(**kw):
        d = S.ForkDims(**{**ok, **kw})
        if kw:
            assert S._lib.sinkattn_pages_fork_workspace_size(ctypes.byref(d)) == 0
        return S._lib.sinkattn_pages_fork(*[None] * 10, ctypes.byref(d), None, 0, None)

    assert call() == S.ERR_INVALID_ARG  # null buffers
    for kw in (dict(num_rows_in=-1), dict(num_rows_out=-1), dict(num_pages=-1), dict(max_pages=0), dict(grow=-1)):
        assert call(**kw) == S.ERR_INVALID_ARG, kw
    for kw in (dict(page_size=8), dict(num_rows_in=(1 << 20) + 1), dict(num_rows_out=(1 << 20) + 1),
               dict(max_pages=1 << 27)):
        assert call(**kw) == S.ERR_UNSUPPORTED, kw
    d = S.ForkDims(**ok)
    # more words than the rows and pages need themselves, and a whole number of them
    assert S._lib.sinkattn_pages_fork_workspace_size(ctypes.byref(d)) >= 4 * (3 * 2 + 2 + 8)
    # the new table may not overlap the present one
    buf = (ctypes.c_int32 * 64)()
    at = lambda i: ctypes.c_void_p(ctypes.addressof(buf) + 4 * i)  # noqa: E731
    args = [at(0), at(20), at(22), None, None, at(24), at(4), at(32), at(34), at(42)]
    assert S._lib.sinkattn_pages_fork(*args, ctypes.byref(d), None, 0, None) == S.ERR_INVALID_ARG


def test_move_dims(S):
    ok = dict(num_layers=1, num_rows=2, num_kv_heads=2, head_dim=64, page_size=16, num_pages=8, max_pages=4, max_accepted=4)

    def copy(**kw):
        return S._lib.sinkattn_kv_copy(None, None, None, ctypes.byref(S.MoveDims(**{**ok, **kw})), None)

    def compact(**kw):
        return S._lib.sinkattn_kv_compact(*[None] * 6, ctypes.byref(S.MoveDims(**{**ok, **kw})), None)

    for call in (copy, compact):
        assert call() == S.ERR_INVALID_ARG
        for kw in (dict(num_layers=0), dict(num_rows=-1), dict(num_kv_heads=0), dict(num_pages=-1)):
            assert call(**kw) == S.ERR_INVALID_ARG, kw
        for kw in (dict(head_dim=128), dict(page_size=32), dict(num_rows=(1 << 20) + 1), dict(num_pages=1 << 27),
                   dict(num_layers=1 << 20, num_rows=1 << 20)):
            assert call(**kw) == S.ERR_UNSUPPORTED, kw
        assert call(num_rows=0) == S.OK
    assert compact(max_pages=0) == S.ERR_INVALID_ARG and compact(max_accepted=0) == S.ERR_INVALID_ARG
    assert compact(max_accepted=17) == S.ERR_UNSUPPORTED and compact(max_pages=1 << 27) == S.ERR_UNSUPPORTED


def test_decode_beams_dims(S):
    ok = dict(num_groups=2, num_beams=4, num_q_heads=8, num_kv_heads=2, head_dim=64, page_size=16, num_pages=8, max_pages=4,
              num_workers=0)

    def call(scale=0.125, **kw):
        d = S.BeamsDims(**{**ok, **kw})
        if kw and kw != dict(num_groups=0):
            assert S._lib.sinkattn_decode_beams_workspace_size(ctypes.byref(d)) == 0
        return S._lib.sinkattn_decode_beams(*[None] * 6, scale, None, None, ctypes.byref(d), None, 0, None)

    assert call() == S.ERR_INVALID_ARG
    for kw in (dict(num_groups=-1), dict(num_beams=0), dict(num_q_heads=0), dict(num_q_heads=9), dict(num_pages=-1),
               dict(max_pages=0), dict(num_workers=-1)):
        assert call(**kw) == S.ERR_INVALID_ARG, kw
    for kw in (dict(head_dim=128), dict(page_size=32), dict(num_groups=32769), dict(num_beams=33), dict(num_q_heads=66),
               dict(num_pages=1 << 27), dict(max_pages=1 << 27)):
        assert call(**kw) == S.ERR_UNSUPPORTED, kw
    assert call(num_groups=0) == S.OK

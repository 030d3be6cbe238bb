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


SANITIZED_CHILD = r"""
import ctypes, sys
sys.path.insert(0, sys.argv[1])
from gqa_attention_learned_head_gb300 import abi
lib = abi.declare(ctypes.CDLL(sys.argv[2]))
big = 2 ** 31 - 1
n = 0
for d in (abi.BeamDims(-1, 4, 10, 4, 1, 0, 10), abi.BeamDims(1, 33, 10, 4, 1, 0, 10), abi.BeamDims(big, 32, big, 64, 2, 0, 2 ** 62),
          abi.BeamDims(1, 4, 10, 4, 7, 0, 10), abi.BeamDims(1, 4, 10, 65, 1, 0, 10), abi.BeamDims(65535, 32, 2 ** 30, 64, 0, 0, 2 ** 40)):
    assert lib.sinkattn_beam_select(*[None] * 6, ctypes.byref(d), None, 0, None) != 0
    assert lib.sinkattn_beam_select_workspace_size(ctypes.byref(d)) == 0
    n += 1
for d in (abi.ForkDims(big, 1, 1, 1, 16, 0), abi.ForkDims(1, big, 1, 1, 16, 0), abi.ForkDims(1, 1, big, 1, 16, 0),
          abi.ForkDims(1, 1, 1, big, 16, 0), abi.ForkDims(1, 1, 1, 1, 16, -big), abi.ForkDims(1, 1, 1, 1, 8, 0)):
    assert lib.sinkattn_pages_fork(*[None] * 10, ctypes.byref(d), None, 0, None) != 0
    assert lib.sinkattn_pages_fork_workspace_size(ctypes.byref(d)) == 0
    n += 1
assert lib.sinkattn_pages_fork_workspace_size(ctypes.byref(abi.ForkDims(1 << 20, 1 << 20, 1 << 30, (1 << 27) - 1, 16, big))) > 0
for d in (abi.MoveDims(big, big, big, 64, 16, big, big, 16), abi.MoveDims(0, 1, 1, 64, 16, 1, 1, 1), abi.MoveDims(big, 1 << 20, 8, 64, 16, 1, 1, 1),
          abi.MoveDims(1, 1, big, 64, 16, big, 1, 1)):
    assert lib.sinkattn_kv_copy(None, None, None, ctypes.byref(d), None) != 0
    assert lib.sinkattn_kv_compact(*[None] * 6, ctypes.byref(d), None) != 0
    n += 1
for d in (abi.BeamsDims(big, 32, big, 1, 64, 16, big, big, big), abi.BeamsDims(1, 32, 8, 1, 64, 16, 1, 1, 0),
          abi.BeamsDims(1, 1, 8, 1, 64, 16, 1, 1 << 27, 0), abi.BeamsDims(1, 1, 0, 1, 64, 16, 1, 1, 0)):
    assert lib.sinkattn_decode_beams(*[None] * 6, 0.125, None, None, ctypes.byref(d), None, 0, None) != 0
    assert lib.sinkattn_decode_beams_workspace_size(ctypes.byref(d)) == 0
    n += 1
print("ok", n)
"""


def test_beam_validation_under_sanitizers():
    """The host code of the beam step's entry points, built with AddressSanitizer and UndefinedBehaviorSanitizer, refuses
    dims at the ends of their types without a sanitizer report."""
    import os
    import subprocess
    import sys
    from pathlib import Path

    from gqa_attention_learned_head_gb300 import build

    asan = subprocess.run(["gcc", "-print-file-name=libasan.so"], capture_output=True, text=True).stdout.strip()
    if not asan or not os.path.isabs(asan) or not os.path.exists(asan):
        pytest.skip("the AddressSanitizer runtime is not installed")
    lib = build.build_sanitized()
    env = dict(os.environ, LD_PRELOAD=asan, ASAN_OPTIONS="detect_leaks=0:abort_on_error=1",
               UBSAN_OPTIONS="halt_on_error=1:print_stacktrace=1")
    r = subprocess.run([sys.executable, "-c", SANITIZED_CHILD, str(Path(__file__).resolve().parents[1]), str(lib)], env=env,
                       capture_output=True, text=True, timeout=600)
    assert r.returncode == 0 and r.stdout.startswith("ok"), r.stdout[-2000:] + r.stderr[-4000:]
    assert "AddressSanitizer" not in r.stderr and "runtime error" not in r.stderr, r.stderr[-4000:]


@pytest.mark.parametrize("width", [8, 32, 63, 65, 128])
def test_pools_of_another_head_size_never_reach_the_library(S, monkeypatch, width):
    """sinkattn_decode_beams refuses pools whose tokens are not as wide as the queries (CPU tensors, with the test for a GPU
    left out and a library that must not be called)."""
    import torch

    class NoLibrary:
        def __getattr__(self, name):
            raise AssertionError(f"{name} called")

    monkeypatch.setattr(S, "_arg", lambda *a: None)
    monkeypatch.setattr(S, "_lib", NoLibrary())
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    q = torch.zeros(1, 2, 16, 64, dtype=torch.bfloat16)
    pool = torch.zeros(4, 2, 16, width, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        S.sinkattn_decode_beams(q, pool, pool, torch.zeros(1, 2, 3, dtype=torch.int32), torch.zeros(1, 2, dtype=torch.int32),
                                torch.zeros(16), 0.125)

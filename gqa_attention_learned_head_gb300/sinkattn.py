"""Python binding of libsinkattn: argument marshalling only.

Each function takes torch tensors already on the GPU, checks dtypes and
shapes, allocates missing outputs with ``torch.empty`` and calls the C ABI
(``include/sinkattn.h``) with raw device pointers and the current CUDA stream.
Every arithmetic step runs in the library's kernels; there is no fallback:
if ``libsinkattn.so`` is absent, importing this module raises.
"""
from __future__ import annotations

import ctypes
import functools
from pathlib import Path

import torch

from .abi import (DTYPE_BF16, DTYPE_F16, DTYPE_F32, EXPORTS, ERR_BAD_INDEX, ERR_BAD_LENGTH, ERR_BAD_PAGE,  # noqa: F401
                  ERR_BAD_VALUE, ERR_CUDA, ERR_INVALID_ARG, ERR_NO_PAGES, ERR_TIMEOUT, ERR_UNSUPPORTED, ERR_WORKSPACE,
                  OK, BeamDims, BeamsDims, DecodeDims, ForkDims, MergeDims, MoveDims, PagedDims, PrefillDims, RopeParams,
                  VerifyDims, declare)

_LIB_PATH = Path(__file__).resolve().parent / "_build" / "libsinkattn.so"


class SinkAttnError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {status_string(status)} (status {status})")


def _load():
    if not _LIB_PATH.exists():
        raise ImportError(f"libsinkattn is not built ({_LIB_PATH} missing); run "
                          "`python -m gqa_attention_learned_head_gb300.build` (needs nvcc)")
    return declare(ctypes.CDLL(str(_LIB_PATH)))


_lib = _load()
library_path = str(_LIB_PATH)


def status_string(status: int) -> str:
    return _lib.sinkattn_status_string(int(status)).decode()


def version() -> int:
    return int(_lib.sinkattn_version())


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _raw_stream(device):
    """The current stream of device number ``device``, as an integer."""
    return torch._C._cuda_getCurrentRawStream(device)


def _empty(shape, device, dtype, stream):
    """An output or workspace of a call on ``stream`` (None: the current one), of that stream's memory: freed, it goes back to the
    stream that uses it."""
    if stream is None:
        return torch.empty(shape, device=device, dtype=dtype)
    with torch.cuda.stream(stream):
        return torch.empty(shape, device=device, dtype=dtype)


def _need(t, name, dtype, ndim):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.dim() != ndim or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {ndim}-d tensor, got shape {tuple(t.shape)}")


def _pools_match(k_pages, v_pages, head_dim):
    """Refuses pools of two shapes, or whose tokens are not as wide as the call's queries or keys."""
    if v_pages.shape != k_pages.shape:
        raise ValueError("k_pages and v_pages must have the same shape")
    if k_pages.shape[3] != head_dim:
        raise ValueError(f"k_pages must have {head_dim} values a token, got shape {tuple(k_pages.shape)}")


def _check(status, what):
    if status != OK:
        raise SinkAttnError(status, what)


def decode_dims(q, k_pages, page_table, num_workers=0) -> DecodeDims:
    B, Hq, D = q.shape
    P, Hkv, PS, _ = k_pages.shape
    return DecodeDims(B, Hq, Hkv, D, PS, P, page_table.shape[1], num_workers)


def sinkattn_decode_workspace_size(q, k_pages, page_table, num_workers=0) -> int:
    return int(_lib.sinkattn_decode_workspace_size(ctypes.byref(decode_dims(q, k_pages, page_table, num_workers))))


def sinkattn_decode(q, k_pages, v_pages, page_table, kv_lens, sinks, scale, out=None, lse=None, workspace=None,
                    num_workers=0, return_lse=True, stream=None):
    """Paged split-KV decode.  Shapes: see ``include/sinkattn.h``.  Returns (out, lse)."""
    _need(q, "q", torch.bfloat16, 3)
    _need(k_pages, "k_pages", torch.bfloat16, 4)
    _need(v_pages, "v_pages", torch.bfloat16, 4)
    _need(page_table, "page_table", torch.int32, 2)
    _need(kv_lens, "kv_lens", torch.int32, 1)
    _need(sinks, "sinks", torch.float32, 1)
    B, Hq, D = q.shape
    _pools_match(k_pages, v_pages, D)
    if page_table.shape[0] != B or kv_lens.shape[0] != B or sinks.shape[0] != Hq or k_pages.shape[1] == 0:
        raise ValueError("inconsistent decode shapes")
    dims = decode_dims(q, k_pages, page_table, num_workers)
    if out is None:
        out = _empty(q.shape, q.device, q.dtype, stream)
    if lse is None and return_lse:
        lse = _empty((B, Hq), q.device, torch.float32, stream)
    if workspace is None:
        nbytes = int(_lib.sinkattn_decode_workspace_size(ctypes.byref(dims)))
        if nbytes == 0:
            raise SinkAttnError(ERR_INVALID_ARG, "sinkattn_decode_workspace_size")
        workspace = _empty(nbytes, q.device, torch.uint8, stream)
    st = _lib.sinkattn_decode(_ptr(q), _ptr(k_pages), _ptr(v_pages), _ptr(page_table), _ptr(kv_lens), _ptr(sinks),
                              float(scale), _ptr(out), _ptr(lse), ctypes.byref(dims), _ptr(workspace),
                              workspace.numel() * workspace.element_size(), _stream(stream))
    _check(st, "sinkattn_decode")
    return out, lse


def verify_dims(q, k_pages, page_table, num_workers=0) -> VerifyDims:
    B, QL, Hq, D = q.shape
    P, Hkv, PS, _ = k_pages.shape
    return VerifyDims(B, QL, Hq, Hkv, D, PS, P, page_table.shape[1], num_workers)


def sinkattn_verify_workspace_size(q, k_pages, page_table, num_workers=0) -> int:
    return int(_lib.sinkattn_verify_workspace_size(ctypes.byref(verify_dims(q, k_pages, page_table, num_workers))))


def sinkattn_verify(q, k_pages, v_pages, page_table, kv_lens, sinks, scale, out=None, lse=None, workspace=None,
                    num_workers=0, return_lse=True, stream=None):
    """Attention of q_len drafted tokens per request over the paged cache (their K/V already in it).

    q [B, q_len, Hq, 64]; kv_lens counts the drafted tokens.  Shapes: see ``include/sinkattn.h``.
    Returns (out [B, q_len, Hq, 64], lse [B, q_len, Hq]).
    """
    _need(q, "q", torch.bfloat16, 4)
    _need(k_pages, "k_pages", torch.bfloat16, 4)
    _need(v_pages, "v_pages", torch.bfloat16, 4)
    _need(page_table, "page_table", torch.int32, 2)
    _need(kv_lens, "kv_lens", torch.int32, 1)
    _need(sinks, "sinks", torch.float32, 1)
    B, QL, Hq, D = q.shape
    _pools_match(k_pages, v_pages, D)
    if page_table.shape[0] != B or kv_lens.shape[0] != B or sinks.shape[0] != Hq or k_pages.shape[1] == 0:
        raise ValueError("inconsistent verify shapes")
    dims = verify_dims(q, k_pages, page_table, num_workers)
    if out is None:
        out = _empty(q.shape, q.device, q.dtype, stream)
    if lse is None and return_lse:
        lse = _empty((B, QL, Hq), q.device, torch.float32, stream)
    if workspace is None:
        nbytes = int(_lib.sinkattn_verify_workspace_size(ctypes.byref(dims)))
        if nbytes == 0:
            raise SinkAttnError(ERR_INVALID_ARG, "sinkattn_verify_workspace_size")
        workspace = _empty(nbytes, q.device, torch.uint8, stream)
    st = _lib.sinkattn_verify(_ptr(q), _ptr(k_pages), _ptr(v_pages), _ptr(page_table), _ptr(kv_lens), _ptr(sinks),
                              float(scale), _ptr(out), _ptr(lse), ctypes.byref(dims), _ptr(workspace),
                              workspace.numel() * workspace.element_size(), _stream(stream))
    _check(st, "sinkattn_verify")
    return out, lse


def sinkattn_verify_tree(q, k_pages, v_pages, page_table, kv_lens, tree_mask, sinks, scale, out=None, lse=None,
                         workspace=None, num_workers=0, return_lse=True, stream=None):
    """sinkattn_verify for a draft tree: tree_mask [B, q_len] int64 on the device, bit j of mask i = drafted
    token i sees drafted token j (its ancestors and itself).  Returns (out, lse)."""
    _need(tree_mask, "tree_mask", torch.int64, 2)
    B, QL = q.shape[0], q.shape[1]
    if tuple(tree_mask.shape) != (B, QL):
        raise ValueError("tree_mask must be [batch, q_len]")
    _need(q, "q", torch.bfloat16, 4)
    _need(k_pages, "k_pages", torch.bfloat16, 4)
    _need(v_pages, "v_pages", torch.bfloat16, 4)
    _need(page_table, "page_table", torch.int32, 2)
    _need(kv_lens, "kv_lens", torch.int32, 1)
    _need(sinks, "sinks", torch.float32, 1)
    _pools_match(k_pages, v_pages, q.shape[3])
    Hq = q.shape[2]
    dims = verify_dims(q, k_pages, page_table, num_workers)
    if out is None:
        out = _empty(q.shape, q.device, q.dtype, stream)
    if lse is None and return_lse:
        lse = _empty((B, QL, Hq), q.device, torch.float32, stream)
    if workspace is None:
        nbytes = int(_lib.sinkattn_verify_workspace_size(ctypes.byref(dims)))
        if nbytes == 0:
            raise SinkAttnError(ERR_INVALID_ARG, "sinkattn_verify_workspace_size")
        workspace = _empty(nbytes, q.device, torch.uint8, stream)
    st = _lib.sinkattn_verify_tree(_ptr(q), _ptr(k_pages), _ptr(v_pages), _ptr(page_table), _ptr(kv_lens),
                                   _ptr(tree_mask), _ptr(sinks), float(scale), _ptr(out), _ptr(lse), ctypes.byref(dims),
                                   _ptr(workspace), workspace.numel() * workspace.element_size(), _stream(stream))
    _check(st, "sinkattn_verify_tree")
    return out, lse


def paged_dims(k_pages, page_table, cu_seqlens, total_tokens, max_seqlen, num_q_heads=0, share_sms=False) -> PagedDims:
    P, Hkv, PS, D = k_pages.shape
    return PagedDims(cu_seqlens.shape[0] - 1, total_tokens, max_seqlen, num_q_heads, Hkv, D, PS, P,
                     page_table.shape[1], int(bool(share_sms)))


def sinkattn_kv_append(k, v, cu_seqlens, start_pos, page_table, k_pages, v_pages, max_seqlen=0, stream=None):
    """Writes new tokens' k / v [T, Hkv, 64] into the pages, in place, at cache positions start_pos[n] + i."""
    _need(k, "k", torch.bfloat16, 3)
    _need(v, "v", torch.bfloat16, 3)
    _need(cu_seqlens, "cu_seqlens", torch.int32, 1)
    _need(start_pos, "start_pos", torch.int32, 1)
    _need(page_table, "page_table", torch.int32, 2)
    _need(k_pages, "k_pages", torch.bfloat16, 4)
    _need(v_pages, "v_pages", torch.bfloat16, 4)
    if v.shape != k.shape or v_pages.shape != k_pages.shape or k.shape[1] != k_pages.shape[1]:
        raise ValueError("inconsistent append shapes")
    _pools_match(k_pages, v_pages, k.shape[2])
    dims = paged_dims(k_pages, page_table, cu_seqlens, k.shape[0], max_seqlen)
    st = _lib.sinkattn_kv_append(_ptr(k), _ptr(v), _ptr(cu_seqlens), _ptr(start_pos), _ptr(page_table),
                                 _ptr(k_pages), _ptr(v_pages), ctypes.byref(dims), _stream(stream))
    _check(st, "sinkattn_kv_append")


def sinkattn_qkv_prologue(qkv, bias, cu_seqlens, start_pos, page_table, k_pages, v_pages, num_q_heads, theta,
                          factor, original_max_position, beta_fast, beta_slow, attn_factor=0.0, interleaved=False,
                          q_out=None, stream=None):
    """QKV bias + YaRN rotary embedding of new tokens qkv [T, (Hq + 2 Hkv) * 64]; returns q [T, Hq, 64] and
    writes the rotated k and the v into the pages at positions start_pos[n] + i (in place)."""
    _need(qkv, "qkv", torch.bfloat16, 2)
    if bias is not None:
        _need(bias, "bias", torch.bfloat16, 1)
    _need(cu_seqlens, "cu_seqlens", torch.int32, 1)
    _need(start_pos, "start_pos", torch.int32, 1)
    _need(page_table, "page_table", torch.int32, 2)
    _need(k_pages, "k_pages", torch.bfloat16, 4)
    _need(v_pages, "v_pages", torch.bfloat16, 4)
    T = qkv.shape[0]
    Hkv = k_pages.shape[1]
    _pools_match(k_pages, v_pages, k_pages.shape[3])  # (the library refuses widths other than 64)
    if qkv.shape[1] != (num_q_heads + 2 * Hkv) * 64 or (bias is not None and bias.shape[0] != qkv.shape[1]):
        raise ValueError("qkv must be [T, (Hq + 2 Hkv) * 64] and bias [(Hq + 2 Hkv) * 64]")
    if q_out is None:
        q_out = _empty((T, num_q_heads, 64), qkv.device, torch.bfloat16, stream)
    dims = paged_dims(k_pages, page_table, cu_seqlens, T, 0, num_q_heads)
    rope = RopeParams(theta, factor, original_max_position, beta_fast, beta_slow, attn_factor, int(bool(interleaved)))
    st = _lib.sinkattn_qkv_prologue(_ptr(qkv), _ptr(bias), _ptr(cu_seqlens), _ptr(start_pos), _ptr(page_table),
                                    ctypes.byref(rope), _ptr(q_out), _ptr(k_pages), _ptr(v_pages), ctypes.byref(dims),
                                    _stream(stream))
    _check(st, "sinkattn_qkv_prologue")
    return q_out


def sinkattn_prefill_paged(q, k_pages, v_pages, page_table, cu_seqlens, start_pos, sinks, scale, max_seqlen=None,
                           out=None, lse=None, return_lse=True, stream=None, share_sms=False):
    """Chunked prefill of new tokens q [T, Hq, 64] over the paged cache (their K/V already appended):
    new token i of sequence n sees cache tokens 0 .. start_pos[n] + i.  Returns (out, lse).
    ``share_sms`` as in sinkattn_prefill."""
    _need(q, "q", torch.bfloat16, 3)
    _need(k_pages, "k_pages", torch.bfloat16, 4)
    _need(v_pages, "v_pages", torch.bfloat16, 4)
    _need(page_table, "page_table", torch.int32, 2)
    _need(cu_seqlens, "cu_seqlens", torch.int32, 1)
    _need(start_pos, "start_pos", torch.int32, 1)
    _need(sinks, "sinks", torch.float32, 1)
    if max_seqlen is None:
        raise ValueError("max_seqlen is required (an upper bound of the new tokens per sequence)")
    T, Hq, D = q.shape
    _pools_match(k_pages, v_pages, D)
    dims = paged_dims(k_pages, page_table, cu_seqlens, T, max_seqlen, Hq, share_sms)
    if out is None:
        out = _empty(q.shape, q.device, q.dtype, stream)
    if lse is None and return_lse:
        lse = _empty((T, Hq), q.device, torch.float32, stream)
    st = _lib.sinkattn_prefill_paged(_ptr(q), _ptr(k_pages), _ptr(v_pages), _ptr(page_table), _ptr(cu_seqlens),
                                     _ptr(start_pos), _ptr(sinks), float(scale), _ptr(out), _ptr(lse),
                                     ctypes.byref(dims), _stream(stream))
    _check(st, "sinkattn_prefill_paged")
    return out, lse


def sinkattn_prefill(q, k, v, cu_seqlens, sinks, scale, causal=True, max_seqlen=None, out=None, lse=None,
                     return_lse=True, stream=None, share_sms=False):
    """Packed varlen prefill.  ``max_seqlen`` (an upper bound of the lengths) is required.  ``share_sms``
    picks the kernel that leaves room on every SM for a decode launched just before it on another
    stream with two shares per SM."""
    _need(q, "q", torch.bfloat16, 3)
    _need(k, "k", torch.bfloat16, 3)
    _need(v, "v", torch.bfloat16, 3)
    _need(cu_seqlens, "cu_seqlens", torch.int32, 1)
    _need(sinks, "sinks", torch.float32, 1)
    if max_seqlen is None:
        raise ValueError("max_seqlen is required (an upper bound of the sequence lengths)")
    T, Hq, D = q.shape
    if k.shape != v.shape or k.shape[0] != T or k.shape[2] != D or sinks.shape[0] != Hq:
        raise ValueError("inconsistent prefill shapes")
    dims = PrefillDims(cu_seqlens.shape[0] - 1, T, int(max_seqlen), Hq, k.shape[1], D, int(bool(share_sms)))
    if out is None:
        out = _empty(q.shape, q.device, q.dtype, stream)
    if lse is None and return_lse:
        lse = _empty((T, Hq), q.device, torch.float32, stream)
    st = _lib.sinkattn_prefill(_ptr(q), _ptr(k), _ptr(v), _ptr(cu_seqlens), _ptr(sinks), float(scale),
                               int(bool(causal)), _ptr(out), _ptr(lse), ctypes.byref(dims), _stream(stream))
    _check(st, "sinkattn_prefill")
    return out, lse


def sinkattn_merge(partial_o, partial_lse, sinks=None, out=None, lse=None, return_lse=True, stream=None):
    """LSE merge of partials [S,R,H,64] / [S,R,H]; ``sinks`` adds the sink once."""
    _need(partial_o, "partial_o", torch.float32, 4)
    _need(partial_lse, "partial_lse", torch.float32, 3)
    if sinks is not None:
        _need(sinks, "sinks", torch.float32, 1)
    S, R, H, D = partial_o.shape
    if partial_lse.shape != (S, R, H):
        raise ValueError("partial_lse must be [S, R, H]")
    dims = MergeDims(S, R, H, D)
    if out is None:
        out = _empty((R, H, D), partial_o.device, torch.bfloat16, stream)
    if lse is None and return_lse:
        lse = _empty((R, H), partial_o.device, torch.float32, stream)
    st = _lib.sinkattn_merge(_ptr(partial_o), _ptr(partial_lse), _ptr(sinks), _ptr(out), _ptr(lse),
                             ctypes.byref(dims), _stream(stream))
    _check(st, "sinkattn_merge")
    return out, lse


NOALLOC_SCRATCH_BYTES = 16 << 20  # SINKATTN_DECODE_NOALLOC_SCRATCH_BYTES


def sinkattn_decode_noalloc(q, k_pages, v_pages, page_table, kv_lens, sinks, scale, out, lse=None, stream=None):
    """Decode with the library's built-in scratch instead of a workspace.

    For callers that cannot allocate device memory on this path (a framework
    owning the whole device through its own pool, a plugin interface that
    passes only inputs and outputs, a loop that must avoid cudaMalloc's
    device synchronisation).  ``out`` (and ``lse`` if wanted) must be given:
    this function allocates nothing.  Problems needing more than 16 MiB of
    scratch raise SinkAttnError(ERR_WORKSPACE); calls must not overlap on the GPU.
    """
    for t, name, dt, nd in ((q, "q", torch.bfloat16, 3), (k_pages, "k_pages", torch.bfloat16, 4),
                            (v_pages, "v_pages", torch.bfloat16, 4), (page_table, "page_table", torch.int32, 2),
                            (kv_lens, "kv_lens", torch.int32, 1), (sinks, "sinks", torch.float32, 1),
                            (out, "out", torch.bfloat16, 3)):
        _need(t, name, dt, nd)
    if lse is not None:
        _need(lse, "lse", torch.float32, 2)
    _pools_match(k_pages, v_pages, q.shape[2])
    dims = decode_dims(q, k_pages, page_table)
    st = _lib.sinkattn_decode_noalloc(_ptr(q), _ptr(k_pages), _ptr(v_pages), _ptr(page_table), _ptr(kv_lens),
                                      _ptr(sinks), float(scale), _ptr(out), _ptr(lse), ctypes.byref(dims),
                                      _stream(stream))
    _check(st, "sinkattn_decode_noalloc")
    return out, lse


# ---- a beam step over the paged cache -------------------------------------------------------------
# These calls are short on the GPU, so their host path is kept short: plain integers instead of pointer objects, the raw
# handle of the current stream, and one test per tensor where nothing is wrong.

_Tensor, _f32, _bf16, _i32 = torch.Tensor, torch.float32, torch.bfloat16, torch.int32
_LOGIT_DTYPES = {torch.float32: DTYPE_F32, torch.bfloat16: DTYPE_BF16, torch.float16: DTYPE_F16}


def _on_stream(fn):
    """Runs a call with its ``stream`` argument current, so that what it allocates (outputs, workspace) belongs to the
    stream that uses it."""
    @functools.wraps(fn)
    def call(*args, stream=None, **kw):
        if stream is None:
            return fn(*args, **kw)
        with torch.cuda.stream(stream):
            return fn(*args, **kw)
    return call


def _here(t, device):
    """Refuses a tensor on another device than the current one, ``device``, to which the call's stream belongs."""
    if t.get_device() != device:
        raise ValueError(f"tensor on {t.device}, but the current device is cuda:{device}")


def _arg(t, name, dtype, ndim, device):
    """A contiguous tensor of this type and rank on ``device``, or an error."""
    if (type(t) is _Tensor and t.get_device() == device and t.dtype is dtype and t.dim() == ndim and t.is_contiguous()):
        return
    _need(t, name, dtype, ndim)
    _here(t, device)


def _at(t):
    """A tensor's address for a void pointer argument."""
    return None if t is None else t.data_ptr()


def _out(t, name, dtype, shape, like, device):
    """An output: the given tensor, checked, or a new one."""
    if t is None:
        return torch.empty(shape, device=like.device, dtype=dtype)
    _arg(t, name, dtype, len(shape), device)
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {shape}, got {tuple(t.shape)}")
    return t


def _room(workspace, nbytes, like, device):
    """(workspace, its bytes): the caller's, or a new one of ``nbytes``."""
    if workspace is None:
        return torch.empty(nbytes, device=like.device, dtype=torch.uint8), nbytes
    if not workspace.is_cuda or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous CUDA tensor")
    _here(workspace, device)
    return workspace, workspace.numel() * workspace.element_size()


def beam_dims(logits, num_select, pad_token=0) -> BeamDims:
    N, K, V = logits.shape
    stride = logits.stride(1) if K > 1 else (logits.stride(0) if N > 1 else V)
    return BeamDims(N, K, V, num_select, _LOGIT_DTYPES[logits.dtype], pad_token, stride)


def sinkattn_beam_select_workspace_size(logits, num_select) -> int:
    return int(_lib.sinkattn_beam_select_workspace_size(ctypes.byref(beam_dims(logits, num_select))))


@_on_stream
def sinkattn_beam_select(logits, scores, num_select, finished=None, pad_token=0, out_scores=None, out_parents=None,
                         out_tokens=None, workspace=None):
    """The num_select best continuations of each group over its beams and the vocabulary.

    logits [N, K, V] (f32, bf16 or f16; rows may be padded: any stride between them, tokens contiguous), scores
    [N, K] f32 running log-probabilities, finished [N, K] bool or uint8.  Returns (scores [N, M] f32, parents [N, M]
    int32 rows n * K + k, tokens [N, M] int32), best first.
    """
    device = torch._C._cuda_getDevice()
    if not isinstance(logits, _Tensor) or not logits.is_cuda:
        raise TypeError("logits must be a CUDA tensor")
    dtype = _LOGIT_DTYPES.get(logits.dtype)
    if dtype is None:
        raise TypeError(f"logits must be float32, bfloat16 or float16, got {logits.dtype}")
    if logits.dim() != 3 or 0 in logits.shape[1:]:
        raise ValueError(f"logits must be [N, K, V], got shape {tuple(logits.shape)}")
    N, K, V = shape = logits.shape
    if logits.is_contiguous():
        stride = V
    else:
        stride = logits.stride(1) if K > 1 else (logits.stride(0) if N > 1 else V)
        if (V > 1 and logits.stride(2) != 1) or (N > 1 and K > 1 and logits.stride(0) != K * stride):
            raise ValueError("logits must have contiguous tokens and rows at one distance from each other")
    _here(logits, device)
    _arg(scores, "scores", _f32, 2, device)
    if scores.shape != shape[:2]:
        raise ValueError("scores must be [N, K]")
    if finished is not None:
        _arg(finished, "finished", torch.bool if finished.dtype is torch.bool else torch.uint8, 2, device)
        if finished.shape != shape[:2]:
            raise ValueError("finished must be [N, K]")
    M = int(num_select)
    dims = BeamDims(N, K, V, M, dtype, int(pad_token), stride)
    nbytes = _lib.sinkattn_beam_select_workspace_size(dims)
    if nbytes == 0:  # invalid dims: the call says why
        st = _lib.sinkattn_beam_select(None, None, None, None, None, None, dims, None, 0, None)
        raise SinkAttnError(st if st != OK else ERR_CUDA, "sinkattn_beam_select")
    out_scores = _out(out_scores, "out_scores", _f32, (N, M), scores, device)
    out_parents = _out(out_parents, "out_parents", _i32, (N, M), scores, device)
    out_tokens = _out(out_tokens, "out_tokens", _i32, (N, M), scores, device)
    workspace, nbytes = _room(workspace, nbytes, scores, device)
    st = _lib.sinkattn_beam_select(logits.data_ptr(), scores.data_ptr(), _at(finished), out_scores.data_ptr(),
                                   out_parents.data_ptr(), out_tokens.data_ptr(), dims, workspace.data_ptr(), nbytes,
                                   _raw_stream(device))
    if st != OK:
        raise SinkAttnError(st, "sinkattn_beam_select")
    return out_scores, out_parents, out_tokens


@_on_stream
def sinkattn_pages_fork(page_table, held_lens, parents, page_refs, keep_lens=None, room_lens=None, grow=0,
                        out_table=None, out_lens=None, out_refs=None, copies=None, workspace=None):
    """Page tables and page counts after rows were forked, dropped, trimmed and grown.

    Row r of the new table continues row parents[r] (-1: none) with its first keep_lens[r] tokens (None: all) and has
    pages for room_lens[r] tokens (None: keep + grow).  ``out_refs`` may be ``page_refs`` itself.  Returns (table [R_out,
    max_pages], lens [R_out], refs [P], copies [R_out, 3]); ``copies`` goes to sinkattn_kv_copy before the new tokens
    are written.
    """
    device = torch._C._cuda_getDevice()
    _arg(page_table, "page_table", _i32, 2, device)
    _arg(held_lens, "held_lens", _i32, 1, device)
    _arg(parents, "parents", _i32, 1, device)
    _arg(page_refs, "page_refs", _i32, 1, device)
    Rin, mp = page_table.shape
    (R,), (P,) = parents.shape, page_refs.shape
    if held_lens.shape[0] != Rin:
        raise ValueError("held_lens must have one entry per row of page_table")
    if keep_lens is not None:
        _arg(keep_lens, "keep_lens", _i32, 1, device)
    if room_lens is not None:
        _arg(room_lens, "room_lens", _i32, 1, device)
    if (keep_lens is not None and keep_lens.shape[0] != R) or (room_lens is not None and room_lens.shape[0] != R):
        raise ValueError("keep_lens and room_lens must have one entry per new row")
    dims = ForkDims(Rin, R, P, mp, 16, int(grow))
    nbytes = _lib.sinkattn_pages_fork_workspace_size(dims)
    if nbytes == 0:  # invalid dims: the call says why
        st = _lib.sinkattn_pages_fork(*[None] * 10, dims, None, 0, None)
        raise SinkAttnError(st if st != OK else ERR_CUDA, "sinkattn_pages_fork")
    out_table = _out(out_table, "out_table", _i32, (R, mp), page_table, device)
    out_lens = _out(out_lens, "out_lens", _i32, (R,), page_table, device)
    out_refs = _out(out_refs, "out_refs", _i32, (P,), page_table, device)
    copies = _out(copies, "copies", _i32, (R, 3), page_table, device)
    workspace, nbytes = _room(workspace, nbytes, page_table, device)
    st = _lib.sinkattn_pages_fork(page_table.data_ptr(), held_lens.data_ptr(), parents.data_ptr(), _at(keep_lens),
                                  _at(room_lens), page_refs.data_ptr(), out_table.data_ptr(), out_lens.data_ptr(),
                                  out_refs.data_ptr(), copies.data_ptr(), dims, workspace.data_ptr(), nbytes,
                                  _raw_stream(device))
    if st != OK:
        raise SinkAttnError(st, "sinkattn_pages_fork")
    return out_table, out_lens, out_refs, copies


def _pools(k_pages, v_pages, device):
    """The pools as [L, P, Hkv, 16, 64]; one layer's pool may come without its first dimension."""
    ndim = 5 if k_pages.dim() == 5 else 4
    _arg(k_pages, "k_pages", _bf16, ndim, device)
    _arg(v_pages, "v_pages", _bf16, ndim, device)
    shape = k_pages.shape
    if v_pages.shape != shape:
        raise ValueError("k_pages and v_pages must have the same shape")
    return shape if ndim == 5 else (1, *shape)


@_on_stream
def sinkattn_kv_copy(k_pages, v_pages, copies):
    """Copies the first ``tokens`` slots of page src to page dst for every (src, dst, tokens) of copies [n, 3] int32,
    in place; k_pages / v_pages [P, Hkv, 16, 64] or, for several layers, [L, P, Hkv, 16, 64]."""
    device = torch._C._cuda_getDevice()
    L, P, Hkv, PS, D = _pools(k_pages, v_pages, device)
    _arg(copies, "copies", _i32, 2, device)
    n, three = copies.shape
    if three != 3:
        raise ValueError("copies must be [n, 3]")
    st = _lib.sinkattn_kv_copy(k_pages.data_ptr(), v_pages.data_ptr(), copies.data_ptr(),
                               MoveDims(L, n, Hkv, D, PS, P, 0, 0), _raw_stream(device))
    if st != OK:
        raise SinkAttnError(st, "sinkattn_kv_copy")


@_on_stream
def sinkattn_kv_compact(k_pages, v_pages, page_table, start_pos, accepted, num_accepted):
    """Moves the accepted drafted tokens together, in place: cache position start_pos[b] + accepted[b][i] to
    start_pos[b] + i for i < num_accepted[b].  Pools as in sinkattn_kv_copy; accepted [B, <= 16] int32."""
    device = torch._C._cuda_getDevice()
    L, P, Hkv, PS, D = _pools(k_pages, v_pages, device)
    _arg(page_table, "page_table", _i32, 2, device)
    _arg(start_pos, "start_pos", _i32, 1, device)
    _arg(accepted, "accepted", _i32, 2, device)
    _arg(num_accepted, "num_accepted", _i32, 1, device)
    (B, A), (rows, mp) = accepted.shape, page_table.shape
    if rows != B or start_pos.shape[0] != B or num_accepted.shape[0] != B:
        raise ValueError("inconsistent compact shapes")
    st = _lib.sinkattn_kv_compact(k_pages.data_ptr(), v_pages.data_ptr(), page_table.data_ptr(), start_pos.data_ptr(),
                                  accepted.data_ptr(), num_accepted.data_ptr(), MoveDims(L, B, Hkv, D, PS, P, mp, A),
                                  _raw_stream(device))
    if st != OK:
        raise SinkAttnError(st, "sinkattn_kv_compact")


def beams_dims(q, k_pages, page_table, num_workers=0) -> BeamsDims:
    N, K, Hq, D = q.shape
    P, Hkv, PS, _ = k_pages.shape
    return BeamsDims(N, K, Hq, Hkv, D, PS, P, page_table.shape[2], num_workers)


def sinkattn_decode_beams_workspace_size(q, k_pages, page_table, num_workers=0) -> int:
    return int(_lib.sinkattn_decode_beams_workspace_size(ctypes.byref(beams_dims(q, k_pages, page_table, num_workers))))


@_on_stream
def sinkattn_decode_beams(q, k_pages, v_pages, page_table, kv_lens, sinks, scale, out=None, lse=None, workspace=None,
                          num_workers=0, return_lse=True):
    """Decode of N groups of K rows whose page tables share pages; a shared page is read once per group.

    q [N, K, Hq, 64]; page_table [N, K, max_pages]; kv_lens [N, K].  Returns (out [N, K, Hq, 64], lse [N, K, Hq]).
    """
    device = torch._C._cuda_getDevice()
    _arg(q, "q", _bf16, 4, device)
    _arg(k_pages, "k_pages", _bf16, 4, device)
    _arg(v_pages, "v_pages", _bf16, 4, device)
    _arg(page_table, "page_table", _i32, 3, device)
    _arg(kv_lens, "kv_lens", _i32, 2, device)
    _arg(sinks, "sinks", _f32, 1, device)
    P, Hkv, PS, Dk = pool = k_pages.shape
    if v_pages.shape != pool:
        raise ValueError("k_pages and v_pages must have the same shape")
    N, K, Hq, D = shape = q.shape
    rows, beams, mp = page_table.shape
    if rows != N or beams != K or kv_lens.shape != shape[:2] or sinks.shape[0] != Hq or Dk != D:
        raise ValueError("inconsistent decode_beams shapes")
    dims = BeamsDims(N, K, Hq, Hkv, D, PS, P, mp, num_workers)
    nbytes = _lib.sinkattn_decode_beams_workspace_size(dims)
    scale = float(scale)
    if nbytes == 0:  # invalid dims: the call says why
        st = _lib.sinkattn_decode_beams(None, None, None, None, None, None, scale, None, None, dims, None, 0, None)
        raise SinkAttnError(st if st != OK else ERR_CUDA, "sinkattn_decode_beams")
    out = _out(out, "out", _bf16, shape, q, device)
    if lse is not None or return_lse:
        lse = _out(lse, "lse", _f32, (N, K, Hq), q, device)
    workspace, nbytes = _room(workspace, nbytes, q, device)
    st = _lib.sinkattn_decode_beams(q.data_ptr(), k_pages.data_ptr(), v_pages.data_ptr(), page_table.data_ptr(),
                                    kv_lens.data_ptr(), sinks.data_ptr(), scale, out.data_ptr(), _at(lse), dims,
                                    workspace.data_ptr(), nbytes, _raw_stream(device))
    if st != OK:
        raise SinkAttnError(st, "sinkattn_decode_beams")
    return out, lse


def sinkattn_selftest_wait_timeout(stream=None) -> None:
    """Enqueues the bounded-wait failure path (one thread waiting on an mbarrier nothing completes);
    the device error word then holds ERR_TIMEOUT (see include/sinkattn.h)."""
    _check(_lib.sinkattn_selftest_wait_timeout(_stream(stream)), "sinkattn_selftest_wait_timeout")


def sinkattn_get_error(stream=None) -> int:
    """Synchronises the stream; returns and clears the device error word (0 = no problem)."""
    return int(_lib.sinkattn_get_error(_stream(stream)))

// api_beam.cu -- the C ABI of the beam step over the paged cache (declared in include/sinkattn.h): host-side
// validation and launch of the beam selection, the page-table fork, the moves of cached tokens and the decode
// over shared pages.
#include <sinkattn.h>

#include <cstring>

#include "args_beam.h"
#include "args_beams.h"
#include "args_pages.h"
#include "args_verify.h"
#include "call_range.h"
#include "host.h"

namespace sinkattn {
namespace {

sinkattn_status_t check_beam_dims(const sinkattn_beam_dims_t* d) {
    if (!d) return SINKATTN_ERR_INVALID_ARG;
    if (d->num_groups < 0 || d->num_beams < 1 || d->vocab < 1 || d->num_select < 1 || d->row_stride < d->vocab ||
        d->pad_token < 0 || d->pad_token >= d->vocab)
        return SINKATTN_ERR_INVALID_ARG;
    if (d->dtype != SINKATTN_DTYPE_F32 && d->dtype != SINKATTN_DTYPE_BF16 && d->dtype != SINKATTN_DTYPE_F16)
        return SINKATTN_ERR_UNSUPPORTED;
    if (d->num_groups > 65535 || d->num_beams > kBeamMaxBeams || d->num_select > kBeamMaxSelect ||
        d->vocab > (1 << 30) || d->row_stride > (1ll << 40))
        return SINKATTN_ERR_UNSUPPORTED;
    const long long shares = ((long long)d->vocab + kBeamMaxPart - 1) / kBeamMaxPart;
    if (d->num_beams * shares * d->num_select > kBeamMaxCands) return SINKATTN_ERR_UNSUPPORTED;
    if ((long long)d->num_groups * d->num_beams * shares > 0x7fffffffll) return SINKATTN_ERR_UNSUPPORTED;
    return SINKATTN_OK;
}

sinkattn_status_t check_fork_dims(const sinkattn_fork_dims_t* d) {
    if (!d) return SINKATTN_ERR_INVALID_ARG;
    if (d->num_rows_in < 0 || d->num_rows_out < 0 || d->num_pages < 0 || d->max_pages < 1 || d->grow < 0)
        return SINKATTN_ERR_INVALID_ARG;
    if (d->page_size != kPageSize || d->num_rows_in > (1 << 20) || d->num_rows_out > (1 << 20) ||
        d->num_pages > (1 << 30))
        return SINKATTN_ERR_UNSUPPORTED;
    if ((long long)d->max_pages * kPageSize >= (1ll << 31)) return SINKATTN_ERR_UNSUPPORTED;
    return SINKATTN_OK;
}

sinkattn_status_t check_move_dims(const sinkattn_move_dims_t* d, bool compact) {
    if (!d) return SINKATTN_ERR_INVALID_ARG;
    if (d->num_layers < 1 || d->num_rows < 0 || d->num_kv_heads < 1 || d->num_pages < 0) return SINKATTN_ERR_INVALID_ARG;
    if (compact && (d->max_pages < 1 || d->max_accepted < 1)) return SINKATTN_ERR_INVALID_ARG;
    if (d->head_dim != kHeadDim || d->page_size != kPageSize || d->num_rows > (1 << 20)) return SINKATTN_ERR_UNSUPPORTED;
    if (compact && (d->max_accepted > kMaxAccepted || (long long)d->max_pages * kPageSize >= (1ll << 31)))
        return SINKATTN_ERR_UNSUPPORTED;
    // the kernel's units (warps) and a layer's rows
    if ((long long)d->num_pages * d->num_kv_heads >= (1ll << 31) / kPageSize ||
        (double)d->num_layers * d->num_rows * d->num_kv_heads > 8e9)
        return SINKATTN_ERR_UNSUPPORTED;
    return SINKATTN_OK;
}

sinkattn_status_t check_beams_dims(const sinkattn_beams_dims_t* d) {
    if (!d) return SINKATTN_ERR_INVALID_ARG;
    if (d->num_groups < 0 || d->num_beams < 1 || d->num_q_heads <= 0 || d->num_kv_heads <= 0 || d->num_pages < 0 ||
        d->max_pages < 1 || d->num_workers < 0 || d->num_workers > (1 << 22) || d->num_q_heads % d->num_kv_heads)
        return SINKATTN_ERR_INVALID_ARG;
    if (d->head_dim != kHeadDim || d->page_size != kPageSize || d->num_groups > 32768 || d->num_beams > kBeamsMaxBeams ||
        (long long)d->num_beams * (d->num_q_heads / d->num_kv_heads) > kBeamsMaxRows)
        return SINKATTN_ERR_UNSUPPORTED;
    // TMA row coordinates are 32-bit, and so are a row's tokens and a group's page entries
    if ((long long)d->num_pages * d->num_kv_heads >= (1ll << 31) / kPageSize ||
        (long long)d->max_pages * (d->num_beams > kPageSize ? d->num_beams : kPageSize) >= (1ll << 31))
        return SINKATTN_ERR_UNSUPPORTED;
    return SINKATTN_OK;
}

sinkattn_status_t from_cuda(cudaError_t e) { return e == cudaSuccess ? SINKATTN_OK : SINKATTN_ERR_CUDA; }

}  // namespace
}  // namespace sinkattn

using namespace sinkattn;

extern "C" {

size_t sinkattn_beam_select_workspace_size(const sinkattn_beam_dims_t* dims) {
    if (check_beam_dims(dims) != SINKATTN_OK) return 0;
    BeamPlan plan;
    if (beam_plan(dims->num_groups, dims->num_beams, dims->vocab, dims->num_select, &plan) != cudaSuccess) return 0;
    return plan.ws_bytes > 0 ? plan.ws_bytes : 256;
}

sinkattn_status_t sinkattn_beam_select(const void* logits, const float* scores, const uint8_t* finished,
                                       float* out_scores, int32_t* out_parents, int32_t* out_tokens,
                                       const sinkattn_beam_dims_t* dims, void* workspace, size_t workspace_bytes,
                                       void* stream) {
    CallRange range("sinkattn_beam_select");
    sinkattn_status_t st = check_beam_dims(dims);
    if (st != SINKATTN_OK) return st;
    if (dims->num_groups == 0) return SINKATTN_OK;
    if (!logits || !scores || !out_scores || !out_parents || !out_tokens) return SINKATTN_ERR_INVALID_ARG;
    if (!aligned(logits, dims->dtype == SINKATTN_DTYPE_F32 ? 4 : 2) || !aligned(scores, 4) || !aligned(out_scores, 4) ||
        !aligned(out_parents, 4) || !aligned(out_tokens, 4))
        return SINKATTN_ERR_INVALID_ARG;
    DeviceState* ds = nullptr;
    if ((st = device_state(&ds)) != SINKATTN_OK) return st;
    BeamPlan plan;
    if (beam_plan(dims->num_groups, dims->num_beams, dims->vocab, dims->num_select, &plan) != cudaSuccess)
        return SINKATTN_ERR_CUDA;
    if (!workspace || workspace_bytes < plan.ws_bytes || !aligned(workspace, 256)) return SINKATTN_ERR_WORKSPACE;
    BeamArgs a;
    a.logits = logits;
    a.scores = scores;
    a.finished = finished;
    a.out_scores = out_scores;
    a.out_parents = out_parents;
    a.out_tokens = out_tokens;
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    a.part = reinterpret_cast<BeamPart*>(ws);
    a.best = reinterpret_cast<unsigned long long*>(ws + plan.best_offset);
    a.err = ds->err;
    a.row_stride = dims->row_stride;
    a.N = dims->num_groups;
    a.K = dims->num_beams;
    a.V = dims->vocab;
    a.M = dims->num_select;
    a.pad_token = dims->pad_token;
    a.dtype = dims->dtype;
    a.parts = plan.parts;
    a.part_len = plan.part_len;
    return from_cuda(beam_select_launch(a, static_cast<cudaStream_t>(stream)));
}

size_t sinkattn_pages_fork_workspace_size(const sinkattn_fork_dims_t* dims) {
    if (check_fork_dims(dims) != SINKATTN_OK) return 0;
    ForkPlan plan;
    fork_plan(dims->num_rows_in, dims->num_rows_out, dims->num_pages, &plan);
    return plan.ws_bytes;
}

sinkattn_status_t sinkattn_pages_fork(const int32_t* page_table, const int32_t* held_lens, const int32_t* parents,
                                      const int32_t* keep_lens, const int32_t* room_lens, const int32_t* page_refs,
                                      int32_t* out_table, int32_t* out_lens, int32_t* out_refs, int32_t* copies,
                                      const sinkattn_fork_dims_t* dims, void* workspace, size_t workspace_bytes,
                                      void* stream) {
    CallRange range("sinkattn_pages_fork");
    sinkattn_status_t st = check_fork_dims(dims);
    if (st != SINKATTN_OK) return st;
    const sinkattn_fork_dims_t& d = *dims;
    if (d.num_rows_in > 0 && (!page_table || !held_lens)) return SINKATTN_ERR_INVALID_ARG;
    if (d.num_rows_out > 0 && (!parents || !out_table || !out_lens || !copies)) return SINKATTN_ERR_INVALID_ARG;
    if (d.num_pages > 0 && (!page_refs || !out_refs)) return SINKATTN_ERR_INVALID_ARG;
    if (!aligned(page_table, 4) || !aligned(held_lens, 4) || !aligned(parents, 4) || !aligned(keep_lens, 4) ||
        !aligned(room_lens, 4) || !aligned(page_refs, 4) || !aligned(out_table, 4) || !aligned(out_lens, 4) ||
        !aligned(out_refs, 4) || !aligned(copies, 4))
        return SINKATTN_ERR_INVALID_ARG;
    // the new table is written while the present one is read
    if (out_table && page_table) {
        const uintptr_t in0 = reinterpret_cast<uintptr_t>(page_table), out0 = reinterpret_cast<uintptr_t>(out_table);
        const uintptr_t in1 = in0 + (uintptr_t)d.num_rows_in * d.max_pages * 4;
        const uintptr_t out1 = out0 + (uintptr_t)d.num_rows_out * d.max_pages * 4;
        if (in0 < out1 && out0 < in1) return SINKATTN_ERR_INVALID_ARG;
    }
    DeviceState* ds = nullptr;
    if ((st = device_state(&ds)) != SINKATTN_OK) return st;
    ForkPlan plan;
    fork_plan(d.num_rows_in, d.num_rows_out, d.num_pages, &plan);
    if (!workspace || workspace_bytes < plan.ws_bytes || !aligned(workspace, 256)) return SINKATTN_ERR_WORKSPACE;
    ForkArgs a;
    a.page_table = page_table;
    a.held_lens = held_lens;
    a.parents = parents;
    a.keep_lens = keep_lens;
    a.room_lens = room_lens;
    a.refs_in = page_refs;
    a.out_table = out_table;
    a.out_lens = out_lens;
    a.refs_out = out_refs;
    a.copies = copies;
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    a.rows = reinterpret_cast<int4*>(ws);
    a.drops = reinterpret_cast<int2*>(ws + plan.drops);
    a.first = reinterpret_cast<int32_t*>(ws + plan.first);
    a.low = reinterpret_cast<int32_t*>(ws + plan.low);
    a.high = reinterpret_cast<int32_t*>(ws + plan.high);
    a.free_ids = reinterpret_cast<int32_t*>(ws + plan.free_ids);
    a.ok = reinterpret_cast<int32_t*>(ws + plan.ok);
    a.err = ds->err;
    a.Rin = d.num_rows_in;
    a.Rout = d.num_rows_out;
    a.P = d.num_pages;
    a.max_pages = d.max_pages;
    a.grow = d.grow;
    return from_cuda(pages_fork_launch(a, static_cast<cudaStream_t>(stream)));
}

sinkattn_status_t sinkattn_kv_copy(void* k_pages, void* v_pages, const int32_t* copies, const sinkattn_move_dims_t* dims,
                                   void* stream) {
    CallRange range("sinkattn_kv_copy");
    sinkattn_status_t st = check_move_dims(dims, false);
    if (st != SINKATTN_OK) return st;
    if (dims->num_rows == 0) return SINKATTN_OK;
    if (!copies || (dims->num_pages > 0 && (!k_pages || !v_pages))) return SINKATTN_ERR_INVALID_ARG;
    if (!aligned(k_pages, 16) || !aligned(v_pages, 16) || !aligned(copies, 4)) return SINKATTN_ERR_INVALID_ARG;
    DeviceState* ds = nullptr;
    if ((st = device_state(&ds)) != SINKATTN_OK) return st;
    CopyArgs a;
    a.k_pages = static_cast<__nv_bfloat16*>(k_pages);
    a.v_pages = static_cast<__nv_bfloat16*>(v_pages);
    a.copies = copies;
    a.err = ds->err;
    a.L = dims->num_layers;
    a.n = dims->num_rows;
    a.Hkv = dims->num_kv_heads;
    a.P = dims->num_pages;
    return from_cuda(kv_copy_launch(a, static_cast<cudaStream_t>(stream)));
}

sinkattn_status_t sinkattn_kv_compact(void* k_pages, void* v_pages, const int32_t* page_table, const int32_t* start_pos,
                                      const int32_t* accepted, const int32_t* num_accepted,
                                      const sinkattn_move_dims_t* dims, void* stream) {
    CallRange range("sinkattn_kv_compact");
    sinkattn_status_t st = check_move_dims(dims, true);
    if (st != SINKATTN_OK) return st;
    if (dims->num_rows == 0) return SINKATTN_OK;
    if (!page_table || !start_pos || !accepted || !num_accepted || (dims->num_pages > 0 && (!k_pages || !v_pages)))
        return SINKATTN_ERR_INVALID_ARG;
    if (!aligned(k_pages, 16) || !aligned(v_pages, 16) || !aligned(page_table, 4) || !aligned(start_pos, 4) ||
        !aligned(accepted, 4) || !aligned(num_accepted, 4))
        return SINKATTN_ERR_INVALID_ARG;
    DeviceState* ds = nullptr;
    if ((st = device_state(&ds)) != SINKATTN_OK) return st;
    CompactArgs a;
    a.k_pages = static_cast<__nv_bfloat16*>(k_pages);
    a.v_pages = static_cast<__nv_bfloat16*>(v_pages);
    a.page_table = page_table;
    a.start_pos = start_pos;
    a.accepted = accepted;
    a.num_accepted = num_accepted;
    a.err = ds->err;
    a.L = dims->num_layers;
    a.B = dims->num_rows;
    a.A = dims->max_accepted;
    a.Hkv = dims->num_kv_heads;
    a.P = dims->num_pages;
    a.max_pages = dims->max_pages;
    return from_cuda(kv_compact_launch(a, static_cast<cudaStream_t>(stream)));
}

size_t sinkattn_decode_beams_workspace_size(const sinkattn_beams_dims_t* dims) {
    if (check_beams_dims(dims) != SINKATTN_OK) return 0;
    BeamsPlan plan;
    if (beams_plan(dims->num_groups, dims->num_beams, dims->num_q_heads, dims->num_kv_heads, dims->max_pages,
                   dims->num_workers, &plan) != cudaSuccess)
        return 0;
    return plan.ws_bytes;
}

sinkattn_status_t sinkattn_decode_beams(const void* q, const void* k_pages, const void* v_pages,
                                        const int32_t* page_table, const int32_t* kv_lens, const float* sinks,
                                        float scale, void* out, float* lse, const sinkattn_beams_dims_t* dims,
                                        void* workspace, size_t workspace_bytes, void* stream) {
    CallRange range("sinkattn_decode_beams");
    sinkattn_status_t st = check_beams_dims(dims);
    if (st != SINKATTN_OK) return st;
    const sinkattn_beams_dims_t& d = *dims;
    if (d.num_groups == 0) return SINKATTN_OK;
    if (!q || !page_table || !kv_lens || !sinks || !out) return SINKATTN_ERR_INVALID_ARG;
    if (d.num_pages > 0 && (!k_pages || !v_pages)) return SINKATTN_ERR_INVALID_ARG;
    if (!aligned(q, 16) || !aligned(k_pages, 16) || !aligned(v_pages, 16) || !aligned(out, 16) ||
        !aligned(page_table, 4) || !aligned(kv_lens, 4) || !aligned(sinks, 4) || (lse && !aligned(lse, 4)))
        return SINKATTN_ERR_INVALID_ARG;
    if (!(scale == scale)) return SINKATTN_ERR_INVALID_ARG;
    DeviceState* ds = nullptr;
    if ((st = device_state(&ds)) != SINKATTN_OK) return st;
    BeamsPlan plan;
    if (beams_plan(d.num_groups, d.num_beams, d.num_q_heads, d.num_kv_heads, d.max_pages, d.num_workers, &plan) !=
        cudaSuccess)
        return SINKATTN_ERR_CUDA;
    if (!workspace || workspace_bytes < plan.ws_bytes || !aligned(workspace, 256)) return SINKATTN_ERR_WORKSPACE;
    const int Hkv = d.num_kv_heads, G = d.num_q_heads / Hkv;
    const unsigned long long rows = (unsigned long long)d.num_pages * Hkv * kPageSize;
    if (rows == 0) {
        // an empty pool has no page to copy: every cached token is absent, so every row is the sink's alone
        VerifyArgs v;
        std::memset(&v, 0, sizeof v);
        v.kv_lens = kv_lens;
        v.sinks = sinks;
        v.out = static_cast<__nv_bfloat16*>(out);
        v.lse = lse;
        v.err = ds->err;
        v.B = d.num_groups * d.num_beams;
        v.QL = 1;
        v.Hq = d.num_q_heads;
        v.max_pages = d.max_pages;
        return from_cuda(verify_empty_pool_launch(v, static_cast<cudaStream_t>(stream)));
    }
    CUtensorMap tq, tk, tv;
    if (!encode_rows(&tk, k_pages, rows, 128, kPageSize) || !encode_rows(&tv, v_pages, rows, 128, kPageSize) ||
        !encode_token_groups(&tq, q, (long long)d.num_groups * d.num_beams, d.num_q_heads, (unsigned)G,
                             (unsigned)d.num_beams))
        return SINKATTN_ERR_INVALID_ARG;
    BeamsArgs a;
    a.q = static_cast<const __nv_bfloat16*>(q);
    a.k_pages = static_cast<const __nv_bfloat16*>(k_pages);
    a.v_pages = static_cast<const __nv_bfloat16*>(v_pages);
    a.page_table = page_table;
    a.kv_lens = kv_lens;
    a.sinks = sinks;
    a.out = static_cast<__nv_bfloat16*>(out);
    a.lse = lse;
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    a.part_o = reinterpret_cast<float*>(ws);
    a.part_lse = reinterpret_cast<float*>(ws + plan.part_lse_offset);
    a.merge_list = reinterpret_cast<int2*>(ws + plan.merge_list_offset);
    a.counts = reinterpret_cast<int32_t*>(ws + plan.counts_offset);
    a.entries = reinterpret_cast<PageEntry*>(ws + plan.entries_offset);
    a.err = ds->err;
    a.N = d.num_groups;
    a.K = d.num_beams;
    a.Hq = d.num_q_heads;
    a.Hkv = Hkv;
    a.G = G;
    a.R = d.num_beams * G;
    a.num_pages = d.num_pages;
    a.max_pages = d.max_pages;
    a.fixed_workers = d.num_workers > 0 ? 1 : 0;
    a.tc_grid = plan.tc_grid;
    a.scale_log2 = scale * 1.4426950408889634f;
    // one share (a fixed single worker, or an automatic split whose largest possible work stays under the
    // minimum share) cuts no segment
    const long long max_tiles = (long long)d.num_groups * Hkv * (((long long)d.num_beams * d.max_pages + 7) / 8);
    const bool may_split = plan.tc_grid > 1 && (a.fixed_workers || max_tiles > kBeamsMinTiles);
    return from_cuda(decode_beams_launch(a, tq, tk, tv, may_split, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"

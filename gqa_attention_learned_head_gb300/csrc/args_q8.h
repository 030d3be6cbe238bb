// args_q8.h -- launch interfaces of the calls over a cache held in 8 bits: append (with or without the pre-attention step),
// unpack, decode and the widening that a prefill over it begins with (between the C ABI layer, api_q8.cu, and the kernel translation
// units).  Internal to libsinkattn.
#pragma once
#include "args_common.h"

namespace sinkattn {

// Exponents that a scale 2^e may have, and the largest code (e4m3).  2^40 x 448 is 4.9e14; the step at the least scale is 2^-49.
// The range is this narrow on purpose: value scales of one sequence are at most 2^80 apart, so that sums of weighted values relative to
// any one of them stay within 32 bits (decode_q8.cu).
constexpr int kScaleExpMin = -40, kScaleExpMax = 40;
constexpr int kScaleBias = 127;  // a scale's byte is its exponent + 127 (E8M0)

// ------------------------------------------------------------------ append, with or without bias and rotation
struct AppendQ8Args {
    const __nv_bfloat16* qkv;   // [T, (Hq + 2 Hkv) * 64], or null: k and v are ready
    const __nv_bfloat16* bias;  // [(Hq + 2 Hkv) * 64] or null
    const __nv_bfloat16* k;     // [T, Hkv, 64] ready keys and values (qkv null)
    const __nv_bfloat16* v;
    const int32_t* cu_seqlens;  // [N+1]
    const int32_t* start_pos;   // [N]
    const int32_t* page_table;  // [N, max_pages]
    __nv_bfloat16* q_out;       // [T, Hq, 64]
    uint8_t* k_pages;           // [P, Hkv, 16, 64] e4m3 codes
    uint8_t* v_pages;
    uint8_t* kv_scales;         // [P, Hkv, 2]
    unsigned* err;
    int N, T, Hq, Hkv, num_pages, max_pages, interleaved;
    float mscale;
    double inv_freq[kHeadDim / 2];
};
cudaError_t append_q8_launch(const AppendQ8Args& args, cudaStream_t stream);

// ------------------------------------------------------------------ unpack
struct UnpackQ8Args {
    const uint8_t* k_pages;    // [P, Hkv, 16, 64]
    const uint8_t* v_pages;
    const uint8_t* kv_scales;  // [P, Hkv, 2]
    const int32_t* copies;     // [n, 3]
    __nv_bfloat16* k_out;      // [P_out, Hkv, 16, 64]
    __nv_bfloat16* v_out;
    unsigned* err;
    int n, Hkv, P, P_out;
};
cudaError_t unpack_q8_launch(const UnpackQ8Args& args, cudaStream_t stream);

// Widens the pages that N sequences hold into a bf16 pool, for the prefill: page j of sequence n goes to page `id` (its own number)
// where remap is null, else to page n * max_pages + j, which is written into remap [N, max_pages] (-1: no such page).
struct WidenQ8Args {
    const uint8_t* k_pages;
    const uint8_t* v_pages;
    const uint8_t* kv_scales;
    const int32_t* page_table;  // [N, max_pages]
    const int32_t* cu_seqlens;  // [N+1]
    const int32_t* start_pos;   // [N]
    __nv_bfloat16* k_out;
    __nv_bfloat16* v_out;
    int32_t* remap;
    unsigned* err;
    int N, T, max_seqlen, Hkv, num_pages, max_pages;
};
cudaError_t widen_q8_launch(const WidenQ8Args& args, cudaStream_t stream);

// ------------------------------------------------------------------ decode
struct DecodeQ8Args {
    const __nv_bfloat16* q;     // [B, Hq, 64]
    const uint8_t* k_pages;     // [P, Hkv, 16, 64]
    const uint8_t* v_pages;
    const uint8_t* kv_scales;   // [P, Hkv, 2]
    const int32_t* page_table;  // [B, max_pages]
    const int32_t* kv_lens;     // [B]
    const float* sinks;         // [Hq]
    __nv_bfloat16* out;         // [B, Hq, 64]
    float* lse;                 // [B, Hq] or null
    float* part_o;              // [slots, G, 64]
    float* part_lse;            // [slots, G], base-2 log-sum-exp
    int2* merge_list;           // [grid], or null when no segment can be split (no merge kernel then)
    unsigned* err;
    int B, Hq, Hkv, G, num_pages, max_pages;
    int workers;                // CTAs sharing the work
    int min_pages_per_worker;   // automatic mode: never cut shares finer than this
    int fixed_workers;          // 1: `workers` shares exactly (capped at the page count)
    float scale_log2;           // scale * log2(e)
};
struct DecodeQ8Plan {
    int grid, workers, min_pages;
    size_t smem, slots, merge_list_offset, ws_bytes;
};
cudaError_t decode_q8_plan(int B, int Hq, int Hkv, int num_workers, DecodeQ8Plan* plan);
cudaError_t decode_q8_launch(const DecodeQ8Args& args, const DecodeQ8Plan& plan, bool may_split, cudaStream_t stream);

}  // namespace sinkattn

// args_beams.h -- launch interface of the decode of rows that share pages (between the C ABI layer,
// api_beam.cu, and the kernel translation unit).  Internal to libsinkattn.
#pragma once
#include "args_common.h"

namespace sinkattn {

constexpr int kBeamsMaxBeams = 32;  // K
constexpr int kBeamsMaxRows = 128;  // K * G query rows of one (group, KV head)
constexpr int kBeamsMinTiles = 4;   // automatic split: never cut shares finer than this many key tiles

// A distinct (column, page) of a group: which of its rows hold it, and how many of its slots hold a token of any.
struct PageEntry {
    int page;        // page id
    int col;         // column: the page's tokens are 16 col .. 16 col + 15 of every row that holds it
    unsigned beams;  // bit k: row k of the group holds it
    int slots;       // 1..16, plus kAllSee if all K rows see all 16 slots
};
constexpr int kAllSee = 32;

struct BeamsArgs {
    const __nv_bfloat16* q;     // [N, K, Hq, 64]
    const __nv_bfloat16* k_pages;  // [P, Hkv, 16, 64]
    const __nv_bfloat16* v_pages;
    const int32_t* page_table;  // [N, K, max_pages]
    const int32_t* kv_lens;     // [N, K]
    const float* sinks;         // [Hq]
    __nv_bfloat16* out;         // [N, K, Hq, 64]
    float* lse;                 // [N, K, Hq] or null
    PageEntry* entries;         // [N, K * max_pages] the groups' distinct pages, by column
    int32_t* counts;            // [N] how many
    float* part_o;              // [slots, R, 64]
    float* part_lse;            // [slots, R], base-2 log-sum-exp
    int2* merge_list;           // [grid]: (segment, pieces) whose first piece the CTA holds without
                                // completing it, or (-1, 0); null when no segment can be split
    unsigned* err;
    int N, K, Hq, Hkv, G, R, num_pages, max_pages;  // R = K * G rows per segment
    int fixed_workers;  // 1: exactly tc_grid shares (the caller's num_workers)
    long long tc_grid;  // shares of the (group, KV head, tile of 8 distinct pages) units, one CTA each
    float scale_log2;
};
struct BeamsPlan {
    long long tc_grid;
    size_t slots, part_lse_offset, merge_list_offset, counts_offset, entries_offset, ws_bytes;
};
cudaError_t beams_plan(int N, int K, int Hq, int Hkv, int max_pages, int num_workers, BeamsPlan* plan);
// may_split = false: one share, so no segment is cut and no merge kernel is launched.
cudaError_t decode_beams_launch(const BeamsArgs& args, const CUtensorMap& tmap_q, const CUtensorMap& tmap_k,
                                const CUtensorMap& tmap_v, bool may_split, cudaStream_t stream);

}  // namespace sinkattn

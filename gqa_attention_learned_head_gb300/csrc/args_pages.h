// args_pages.h -- launch interface of the page-table fork and of the calls that move cached tokens (between
// the C ABI layer, api_beam.cu, and the kernel translation units).  Internal to libsinkattn.
#pragma once
#include "args_common.h"

namespace sinkattn {

// ------------------------------------------------------------------ fork of page tables
struct ForkArgs {
    const int32_t* page_table;  // [Rin, max_pages]
    const int32_t* held_lens;   // [Rin]
    const int32_t* parents;     // [Rout]
    const int32_t* keep_lens;   // [Rout] or null
    const int32_t* room_lens;   // [Rout] or null
    const int32_t* refs_in;     // [P]
    int32_t* out_table;         // [Rout, max_pages]
    int32_t* out_lens;          // [Rout]
    int32_t* refs_out;          // [P], may be refs_in
    int32_t* copies;            // [Rout, 3]
    // workspace
    int4* rows;                 // [Rout] parent, keep, room (top bit: the parent's first child), where its new pages
                                //        start in free_ids (top bit: the first replaces its last kept page)
    int2* drops;                // [Rin] the columns that this row holds and its first child does not keep
    int32_t* first;             // [Rin] lowest row that continues this one, INT_MAX: none
    int32_t* low;               // [Rin] least and greatest keep of the rows that continue this one and will
    int32_t* high;              //       write their last page (-1 for one that will not)
    int32_t* free_ids;          // [P] free pages, lowest first (as many as are needed)
    int32_t* ok;                // [1] 1: there are enough of them
    unsigned* err;
    int Rin, Rout, P, max_pages, grow;
};
struct ForkPlan {
    size_t drops, first, low, high, free_ids, ok, ws_bytes;  // offsets in the workspace (rows at 0)
};
void fork_plan(int Rin, int Rout, int P, ForkPlan* plan);
cudaError_t pages_fork_launch(const ForkArgs& args, cudaStream_t stream);

// ------------------------------------------------------------------ moves of cached tokens
struct CopyArgs {
    __nv_bfloat16* k_pages;  // [L, P, Hkv, 16, 64]
    __nv_bfloat16* v_pages;
    const int32_t* copies;   // [n, 3]: source page, destination page, tokens
    unsigned* err;
    int L, n, Hkv, P;
};
cudaError_t kv_copy_launch(const CopyArgs& args, cudaStream_t stream);

constexpr int kMaxAccepted = 16;
struct CompactArgs {
    __nv_bfloat16* k_pages;       // [L, P, Hkv, 16, 64]
    __nv_bfloat16* v_pages;
    const int32_t* page_table;    // [B, max_pages]
    const int32_t* start_pos;     // [B]
    const int32_t* accepted;      // [B, A]
    const int32_t* num_accepted;  // [B]
    unsigned* err;
    int L, B, A, Hkv, P, max_pages;
};
cudaError_t kv_compact_launch(const CompactArgs& args, cudaStream_t stream);

}  // namespace sinkattn

// host.h -- what the C ABI translation units share on the host side: the per-device error word, pointer
// alignment and the encoding of tensor maps (all defined in api.cu).  Internal to libsinkattn.
#pragma once
#include <sinkattn.h>

#include <cstddef>
#include <cstdint>
#include <cuda.h>

namespace sinkattn {

struct DeviceState {
    bool ready = false;
    unsigned* err = nullptr;    // device address of the error word
    unsigned* taken = nullptr;  // device address where sinkattn_get_error's exchange leaves what it took
};
// The state of the device that is current for the calling thread (set up by its first use).
sinkattn_status_t device_state(DeviceState** out);

inline bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// 3-D map over q [tokens, H, 64] whose box is 64 x box_heads heads x box_tokens tokens.
bool encode_token_groups(CUtensorMap* map, const void* base, long long tokens, int H, unsigned box_heads,
                         unsigned box_tokens);
// 2-D map over rows of 64 elements (128 B), box = box_rows x 64.
bool encode_rows(CUtensorMap* map, const void* base, unsigned long long rows, unsigned long long row_stride_bytes,
                 unsigned box_rows);

}  // namespace sinkattn

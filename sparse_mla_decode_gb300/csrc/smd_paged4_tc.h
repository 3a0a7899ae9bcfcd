// The decode of a 4-bit cache on the tcgen05 tensor cores (128 columns).
#pragma once

#include "smd_paged_decode.cuh"

namespace smd {

// One launch: p with what is of the call, tiles of 128 tokens at most, units of up to `rows` (8, 16 or 32)
// query rows; the maps' boxes hold `box` tokens (16, 32, 64 or 128).
int paged4_tc(const PagedParams& p, const Maps<4>& maps, int box, int rows, int sms, int64_t tiles,
              smd_stream_t stream);

}  // namespace smd

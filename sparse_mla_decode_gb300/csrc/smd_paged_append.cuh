// What the appends of both caches share: bf16 pairs, the bounds of a page's keys, lanes.
#pragma once

#include <cstdint>

namespace smd {
namespace {

__device__ __forceinline__ uint32_t bmax2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

__device__ __forceinline__ uint32_t bmin2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("min.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// Infinities as the largest finite bf16.
__device__ __forceinline__ uint32_t finite2(uint32_t a) {
    return bmin2(bmax2(a, 0xff7fff7fu), 0x7f7f7f7fu);
}

__device__ __forceinline__ float lo_f(uint32_t v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ float hi_f(uint32_t v) { return __uint_as_float(v & 0xffff0000u); }

// The largest and smallest key of 8 channels, as bf16 pairs; nothing met: -infinity, infinity.
struct Extremes {
    uint4 hi = make_uint4(0xff80ff80u, 0xff80ff80u, 0xff80ff80u, 0xff80ff80u);
    uint4 lo = make_uint4(0x7f807f80u, 0x7f807f80u, 0x7f807f80u, 0x7f807f80u);

    // Those that a page's bounds hold, from column `col` on.
    __device__ __forceinline__ void read(const uint16_t* bounds, int D, int col) {
        const uint4* const w = reinterpret_cast<const uint4*>(bounds + col);
        hi = w[0];
        lo = w[D / 8];
    }
};

// The largest and smallest of a run's keys, joined with the bounds before and
// written: 8 columns from `col` on.
__device__ __forceinline__ void write_bounds(uint16_t* bounds, int D, int col, const Extremes& was,
                                             uint32_t (&hi)[4], uint32_t (&lo)[4]) {
    uint4* const b = reinterpret_cast<uint4*>(bounds + col);
    const uint4 h = was.hi, l = was.lo;
    b[0] = make_uint4(finite2(bmax2(hi[0], h.x)), finite2(bmax2(hi[1], h.y)), finite2(bmax2(hi[2], h.z)),
                      finite2(bmax2(hi[3], h.w)));
    b[D / 8] = make_uint4(finite2(bmin2(lo[0], l.x)), finite2(bmin2(lo[1], l.y)), finite2(bmin2(lo[2], l.z)),
                          finite2(bmin2(lo[3], l.w)));
}

// Takes 8 values into the extremes.
__device__ __forceinline__ void take(const uint4& v, uint32_t (&hi)[4], uint32_t (&lo)[4]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        hi[j] = bmax2(hi[j], w[j]);
        lo[j] = bmin2(lo[j], w[j]);
    }
}

// The lanes of this lane's group of N.
template <int N>
__device__ __forceinline__ unsigned group_mask(int lane) {
    return N == 32 ? 0xffffffffu : ((1u << (N & 31)) - 1u) << (lane / N * N);
}

}  // namespace
}  // namespace smd

// New keys and values into the pages of an E4M3 cache (smd_paged_append).
//
// A run: tokens whose slots continue one another inside one page. For each run,
// head and side (K or V), over the run's values x:
//   e = ceil(log2(max|x| / 448)), scale = max(2^e, the kept tokens' scale),
//   code = E4M3(x / scale); kept codes are re-encoded if the scale grew.
// A power of two divides exactly, so codes never depend on how the quotient is
// computed, and a kept code that is re-encoded later moves by an exponent.
//
// What bounds it: 4 D bytes read and 2 D written for each token and head, and a
// page's bounds (8 D bytes) where it is touched: HBM for prompts, and the
// dependent loads slot -> x -> scale -> (kept codes) for a decode step.
//
// D / 8 lanes hold a token, 8 columns (16 bytes of bf16) each. Few tokens: one such
// group of lanes takes a run of one head and side. Many: a block of four warps
// looks up the runs that start in its chunk of tokens and writes them for one head:
// long ones together (two warps the keys, two the values), shorter ones by a warp
// or a group of lanes each. A warp keeps its values in registers between the
// maximum and the encoding (of a run, 32 tokens of 256 columns, 64 of 128, 128
// of 64; what is longer is read again, from L2), so that 8 KB a warp and 160
// KB an SM are on their way at a time.
//
// Measured (GB300): 96 tokens of as many requests, 8 heads of 128 columns, 2.5 us; 28
// thousand tokens of 23 requests 37 us (68% of the copy rate for the 173 MB: the
// slots, a run's loads, its maximum and its stores follow one another, and 20 warps
// an SM do not quite cover that), 16 thousand of one 21 us (69%).
#include "smd_internal.h"
#include "smd_paged.h"
#include "smd_ptx.cuh"

namespace smd {
namespace {

constexpr int kMinExponent = -120;

struct AppendParams {
    const uint16_t* x[2];
    int64_t x_stride[2];
    const int32_t* slots;
    int32_t T;
    uint8_t* pool[2];
    int64_t stride[2][3];
    float* scale[2];
    uint16_t* bounds;
    int32_t pages, heads, P;
};

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

// The least power of two at which a / 2^e is at most 448 = 1.75 * 2^8.
__device__ __forceinline__ float power_of(float a) {
    const uint32_t u = __float_as_uint(a);
    int e = static_cast<int>(u >> 23) - 127 - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
    e = max(e, kMinExponent);
    return __uint_as_float(static_cast<uint32_t>(e + 127) << 23);
}

__device__ __forceinline__ bool is_power(float scale) { return (__float_as_uint(scale) & 0x7fffffu) == 0; }

__device__ __forceinline__ uint32_t encode4(float a, float b, float c, float d) {
    return static_cast<uint32_t>(e4m3x2(a, b)) | static_cast<uint32_t>(e4m3x2(c, d)) << 16;
}

// Four kept codes at a new scale, which is a power of two.
__device__ __forceinline__ uint32_t reencode(uint32_t w, float was, float inv) {
    uint32_t lo, hi;
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(w));
    float f[4];
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}"
        : "=f"(f[0]), "=f"(f[1])
        : "r"(lo));
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}"
        : "=f"(f[2]), "=f"(f[3])
        : "r"(hi));
#pragma unroll
    for (int j = 0; j < 4; ++j) f[j] = f[j] * was * inv;
    return encode4(f[0], f[1], f[2], f[3]);
}

// Whether a run starts at token t: its slot is in the pool and does not continue
// the token before it in one page.
__device__ __forceinline__ bool starts_run(const AppendParams& p, int t, int slot) {
    if (slot < 0 || slot / p.P >= p.pages) return false;
    return t == 0 || slot % p.P == 0 || p.slots[t - 1] != slot - 1;
}

// What a page holds before a run: its scale and, of 8 columns from `col` on, its bounds
// (loaded ahead of the run's values, so that nothing waits for them afterwards).
struct Before {
    float scale;
    uint4 hi, lo;
};

template <int D>
__device__ __forceinline__ Before before(const AppendParams& p, int64_t at, int side, int o, int col) {
    Before b;
    b.scale = o > 0 ? p.scale[side][at] : __uint_as_float(static_cast<uint32_t>(kMinExponent + 127) << 23);
    b.hi = make_uint4(0xff80ff80u, 0xff80ff80u, 0xff80ff80u, 0xff80ff80u);  // -infinity
    b.lo = make_uint4(0x7f807f80u, 0x7f807f80u, 0x7f807f80u, 0x7f807f80u);
    if (side == 0 && o > 0 && p.bounds != nullptr) {
        const uint4* const w = reinterpret_cast<const uint4*>(p.bounds + at * 2 * D + col);
        b.hi = w[0];
        b.lo = w[D / 8];
    }
    return b;
}

// The largest and smallest of a run's keys, joined with the bounds before and
// written: 8 columns from `col` on.
__device__ __forceinline__ void write_bounds(uint16_t* bounds, int D, int col, const Before& was,
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

// The largest size: the largest of hi and -lo, or 0 where nothing but NaN was met
// (hi is then -infinity, lo infinity).
__device__ __forceinline__ float largest(const uint32_t (&hi)[4], const uint32_t (&lo)[4]) {
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) m = bmax2(m, finite2(bmax2(hi[j], lo[j] ^ 0x80008000u)));
    return fmaxf(lo_f(m), hi_f(m));
}

// Eight values over the scale. A product where the scale is a power of two (kExact: the
// quotient has no rounding either way); the branch between the two is taken once for
// a run.
template <bool kExact>
__device__ __forceinline__ uint2 encode8(const uint4& v, float scale, float inv) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    uint32_t c[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        float x = lo_f(w[j]), y = hi_f(w[j]);
        if (kExact) {  // both products at once
            asm("{\n\t.reg .b64 a, b;\n\tmov.b64 a, {%0, %1};\n\tmov.b64 b, {%2, %2};\n\t"
                "mul.rn.f32x2 a, a, b;\n\tmov.b64 {%0, %1}, a;\n\t}"
                : "+f"(x), "+f"(y)
                : "f"(inv));
        } else {
            x = __fdiv_rn(x, scale);
            y = __fdiv_rn(y, scale);
        }
        c[j] = e4m3x2(x, y);
    }
    return make_uint2(c[0] | c[1] << 16, c[2] | c[3] << 16);
}

// Writes the first o tokens of a page again at a larger scale: lane i of N.
template <int N, int D>
__device__ __forceinline__ void reencode_kept(uint8_t* pool, int64_t ts, int o, float old, float inv, int i) {
    constexpr int kCols = D / 16;
#pragma unroll 2
    for (int m = i / kCols; m < o; m += N / kCols) {
        uint4* const w = reinterpret_cast<uint4*>(pool + m * ts + i % kCols * 16);
        uint4 v = *w;
        v.x = reencode(v.x, old, inv);
        v.y = reencode(v.y, old, inv);
        v.z = reencode(v.z, old, inv);
        v.w = reencode(v.w, old, inv);
        *w = v;
    }
}

// A run: its first token, length and slot.
struct Run {
    int64_t t;
    int n, slot;
};

// One run of one head and side by N lanes (i: this one; N = D / 8 or 32; `mask`: the
// lanes that run together). The first kKept values of a lane stay in registers.
template <int N, int kKept, int D>
__device__ __forceinline__ void write_run(const AppendParams& p, const Run& r, int head, int side,
                                          int i, unsigned mask, const Before* given = nullptr,
                                          const uint4* first = nullptr) {
    constexpr int kCols = D / 8, kStep = N / kCols;  // lanes of a token; tokens at once
    const int col = (i % kCols) * 8, t_in = i / kCols;
    const int page = r.slot / p.P, o = r.slot - page * p.P;
    const int64_t xs = p.x_stride[side], at = static_cast<int64_t>(page) * p.heads + head;
    const uint16_t* const x = p.x[side] + r.t * xs + head * D + col;
    float* const scale = p.scale[side] + at;
    const Before was = given != nullptr ? *given : before<D>(p, at, side, o, col);
    const float old = was.scale;
    uint4 v[kKept];
#pragma unroll
    for (int k = 0; k < kKept; ++k) {
        const int m = t_in + k * kStep;
        v[k] = make_uint4(0, 0, 0, 0);
        if (k == 0 && first != nullptr) v[k] = *first;
        else if (m < r.n) v[k] = __ldcs(reinterpret_cast<const uint4*>(x + m * xs));
    }
    uint32_t hi[4], lo[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        hi[j] = 0xff80ff80u;  // -infinity
        lo[j] = 0x7f807f80u;
    }
#pragma unroll
    for (int k = 0; k < kKept; ++k)
        if (t_in + k * kStep < r.n) take(v[k], hi, lo);
#pragma unroll 8
    for (int m = t_in + kKept * kStep; m < r.n; m += kStep)
        take(*reinterpret_cast<const uint4*>(x + m * xs), hi, lo);
    float a = largest(hi, lo);
#pragma unroll
    for (int s = 1; s < N; s <<= 1) a = fmaxf(a, __shfl_xor_sync(mask, a, s));
    if (side == 0 && p.bounds != nullptr) {
#pragma unroll
        for (int s = kCols; s < N; s <<= 1)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                hi[j] = bmax2(hi[j], __shfl_xor_sync(mask, hi[j], s));
                lo[j] = bmin2(lo[j], __shfl_xor_sync(mask, lo[j], s));
            }
        if (i < kCols) write_bounds(p.bounds + at * 2 * D, D, col, was, hi, lo);
    }
    const float now = fmaxf(power_of(a), old);
    __syncwarp(mask);  // every lane has read the old scale
    if (i == 0) *scale = now;
    const float inv = 1.0f / now;
    uint8_t* const pool = p.pool[side] + page * p.stride[side][0] + head * p.stride[side][1];
    const int64_t ts = p.stride[side][2];
    if (is_power(now)) {
        if (o > 0 && now > old) reencode_kept<N, D>(pool, ts, o, old, inv, i);
#pragma unroll
        for (int k = 0; k < kKept; ++k) {
            const int m = t_in + k * kStep;
            if (m < r.n)
                *reinterpret_cast<uint2*>(pool + (o + m) * ts + col) = encode8<true>(v[k], now, inv);
        }
#pragma unroll 8
        for (int m = t_in + kKept * kStep; m < r.n; m += kStep)
            *reinterpret_cast<uint2*>(pool + (o + m) * ts + col) =
                encode8<true>(*reinterpret_cast<const uint4*>(x + m * xs), now, inv);
    } else {  // a kept scale that the caller has set: larger than the run's own, nothing is re-encoded
#pragma unroll 1
        for (int m = t_in; m < r.n; m += kStep)
            *reinterpret_cast<uint2*>(pool + (o + m) * ts + col) =
                encode8<false>(*reinterpret_cast<const uint4*>(x + m * xs), now, inv);
    }
}

// What the warps of a block tell one another of a run.
template <int D>
struct RunShared {
    float a[4];
    uint4 hi[D / 8], lo[D / 8];
};

// One run of one head by a block of four warps: two for the keys and two for the
// values, each every second step of tokens. The first kKept values of a lane
// stay in registers.
template <int kKept, int D>
__device__ __forceinline__ void write_run_block(const AppendParams& p, const Run& r, int head, int warp,
                                                int lane, RunShared<D>& shared) {
    constexpr int kCols = D / 8, kStep = 32 / kCols;
    const int side = warp >> 1, half = warp & 1;
    const int col = (lane % kCols) * 8, t_in = lane / kCols + half * kStep;
    const int page = r.slot / p.P, o = r.slot - page * p.P;
    const int64_t xs = p.x_stride[side], at = static_cast<int64_t>(page) * p.heads + head;
    const uint16_t* const x = p.x[side] + r.t * xs + head * D + col;
    float* const scale = p.scale[side] + at;
    uint4 v[kKept];
    constexpr int kSpan = 2 * kKept * kStep;  // tokens that the two warps hold
    const auto load = [&](int m0) {
#pragma unroll
        for (int k = 0; k < kKept; ++k) {
            const int m = m0 + t_in + 2 * k * kStep;
            v[k] = make_uint4(0, 0, 0, 0);
            if (m < r.n) v[k] = __ldcg(reinterpret_cast<const uint4*>(x + m * xs));
        }
    };
    const float old = before<D>(p, at, side, o, col).scale;  // the bounds later: registers
    uint32_t hi[4], lo[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        hi[j] = 0xff80ff80u;  // -infinity
        lo[j] = 0x7f807f80u;
    }
    // What is not kept comes first and is read again, from L2, when the scale is known. (32
    // thousand tokens in pages of 128: 44 us; four loads at a time 53.)
#pragma unroll 1
    for (int m0 = (r.n - 1) / kSpan * kSpan; m0 >= 0; m0 -= kSpan) {
        load(m0);
#pragma unroll
        for (int k = 0; k < kKept; ++k)
            if (m0 + t_in + 2 * k * kStep < r.n) take(v[k], hi, lo);
    }
    const float a = warp_max(largest(hi, lo));
    const bool bounds = side == 0 && p.bounds != nullptr;
    if (bounds) {
#pragma unroll
        for (int s = kCols; s < 32; s <<= 1)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                hi[j] = bmax2(hi[j], __shfl_xor_sync(0xffffffffu, hi[j], s));
                lo[j] = bmin2(lo[j], __shfl_xor_sync(0xffffffffu, lo[j], s));
            }
        if (half == 1 && lane < kCols) {
            shared.hi[lane] = make_uint4(hi[0], hi[1], hi[2], hi[3]);
            shared.lo[lane] = make_uint4(lo[0], lo[1], lo[2], lo[3]);
        }
    }
    if (lane == 0) shared.a[warp] = a;
    __syncthreads();
    const float now = fmaxf(power_of(fmaxf(a, shared.a[warp ^ 1])), old);
    if (bounds && half == 0 && lane < kCols) {
        const uint4 h = shared.hi[lane], l = shared.lo[lane];
        hi[0] = bmax2(hi[0], h.x), hi[1] = bmax2(hi[1], h.y);
        hi[2] = bmax2(hi[2], h.z), hi[3] = bmax2(hi[3], h.w);
        lo[0] = bmin2(lo[0], l.x), lo[1] = bmin2(lo[1], l.y);
        lo[2] = bmin2(lo[2], l.z), lo[3] = bmin2(lo[3], l.w);
        write_bounds(p.bounds + at * 2 * D, D, col, before<D>(p, at, 0, o, col), hi, lo);
    }
    __syncthreads();  // shared is free again, and every thread has read the old scale
    if (half == 0 && lane == 0) *scale = now;
    const float inv = 1.0f / now;
    uint8_t* const pool = p.pool[side] + page * p.stride[side][0] + head * p.stride[side][1];
    const int64_t ts = p.stride[side][2];
    if (is_power(now)) {
        if (o > 0 && now > old) reencode_kept<64, D>(pool, ts, o, old, inv, half * 32 + lane);
#pragma unroll 1
        for (int m0 = 0; m0 < r.n; m0 += kSpan) {
            if (m0 > 0) load(m0);
#pragma unroll
            for (int k = 0; k < kKept; ++k) {
                const int m = m0 + t_in + 2 * k * kStep;
                if (m < r.n)
                    *reinterpret_cast<uint2*>(pool + (o + m) * ts + col) = encode8<true>(v[k], now, inv);
            }
        }
    } else {  // a kept scale that the caller has set: larger than the run's own, nothing is re-encoded
#pragma unroll 1
        for (int m = t_in; m < r.n; m += 2 * kStep)
            *reinterpret_cast<uint2*>(pool + (o + m) * ts + col) =
                encode8<false>(*reinterpret_cast<const uint4*>(x + m * xs), now, inv);
    }
}

// The lanes of this lane's group of N.
template <int N>
__device__ __forceinline__ unsigned group_mask(int lane) {
    return N == 32 ? 0xffffffffu : ((1u << (N & 31)) - 1u) << (lane / N * N);
}

constexpr int kThreads = 128;

// D / 8 lanes for each (token, head, side); those whose token starts no run leave.
template <int D>
__global__ void __launch_bounds__(kThreads) append_few_kernel(const AppendParams p) {
    constexpr int N = D / 8;
    pdl_entry();
    const int lane = threadIdx.x & 31, i = threadIdx.x % N;
    const unsigned mask = group_mask<N>(lane);
    const int64_t unit = (static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x) / N;
    const int t = static_cast<int>(unit / (2 * p.heads)), hs = static_cast<int>(unit % (2 * p.heads));
    if (t >= p.T) return;
    const int slot = p.slots[t];
    if (!starts_run(p, t, slot)) return;
    // The first token's values and the page's state are on their way meanwhile.
    const int side = hs & 1, head = hs >> 1, page = slot / p.P, o = slot - page * p.P;
    const uint4 first = __ldcs(reinterpret_cast<const uint4*>(p.x[side] + t * p.x_stride[side] + head * D + 8 * i));
    const Before was = before<D>(p, static_cast<int64_t>(page) * p.heads + head, side, o, 8 * i);
    // Tokens that continue it, up to the page's end.
    const int most = min(p.P - slot % p.P, p.T - t);
    int n = 1;
    while (n < most) {
        const bool on = n + i < most && p.slots[t + n + i] == slot + n + i;
        const unsigned off = ~__ballot_sync(mask, on) & mask;
        const int c = off == 0 ? N : (__ffs(off) - 1) % N;
        n += c;
        if (c < N) break;
    }
    write_run<N, 1, D>(p, Run{t, n, slot}, head, side, i, mask, &was, &first);
}

constexpr int kChunk = 64;      // tokens of a block
constexpr int kMostPage = 256;  // tokens of a page

constexpr int kShort = 4;       // runs up to this length go to D / 8 lanes each

// A block for each chunk of tokens and head: it takes the runs that start in its
// chunk.
template <int D>
__global__ void __launch_bounds__(kThreads, 5) append_many_kernel(const AppendParams p) {
    constexpr int N = D / 8, kWarps = kThreads / 32;
    // Runs up to kHalf tokens go to half a warp each, up to kMedium to a warp: 8 values a lane.
    // (30 thousand tokens in pages of 16 of 64 columns: 33 us, by whole warps 41; in pages of 32,
    // whose runs take a warp each, 33 and 32.)
    constexpr int kHalf = D == 64 ? 16 : 0, kMedium = 8 * (32 / N);
    __shared__ int s_slot[kChunk];
    __shared__ int2 s_runs[kChunk];  // first token and length: short runs from the front, long from the back
    __shared__ uint32_t s_goes[(kChunk + kMostPage) / 32], s_lead[kChunk / 32];
    __shared__ int s_short, s_long;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int head = blockIdx.y;
    if (tid == 0) s_short = s_long = 0;
    pdl_entry();
    const int64_t t0 = static_cast<int64_t>(blockIdx.x) * kChunk;
    const int span = static_cast<int>(min(static_cast<int64_t>(p.T) - t0, static_cast<int64_t>(kChunk)));
    const int seen = static_cast<int>(min(static_cast<int64_t>(p.T) - t0, static_cast<int64_t>(kChunk) + p.P));
    // A token goes on with the run of the one before it, or it leads one; a run of this
    // chunk may go on into the next chunks.
    for (int j0 = 0; j0 < kChunk + p.P; j0 += kThreads) {
        const int j = j0 + tid;
        bool goes = false, lead = false;
        if (j < seen) {
            const int slot = p.slots[t0 + j], before = t0 + j > 0 ? p.slots[t0 + j - 1] : -2;
            if (slot >= 0 && slot / p.P < p.pages) {
                goes = slot % p.P != 0 && before == slot - 1;
                lead = !goes && j < span;
            }
            if (j < kChunk) s_slot[j] = slot;
        }
        const uint32_t g = __ballot_sync(0xffffffffu, goes), l = __ballot_sync(0xffffffffu, lead);
        if (lane == 0 && j < kChunk + kMostPage) {
            s_goes[j >> 5] = g;
            if (j < kChunk) s_lead[j >> 5] = l;
        }
    }
    __syncthreads();
    if (tid < kChunk && (s_lead[tid >> 5] >> (tid & 31) & 1) != 0) {
        int end = tid + 1;  // the first token after this one that does not go on
        while (end < kChunk + p.P) {
            const uint32_t stop = ~s_goes[end >> 5] >> (end & 31);
            if (stop != 0) {
                end += __ffs(stop) - 1;
                break;
            }
            end = (end | 31) + 1;
        }
        const int n = min(end, seen) - tid;
        const int at = n <= kShort ? atomicAdd(&s_short, 1) : kChunk - 1 - atomicAdd(&s_long, 1);
        s_runs[at] = make_int2(tid, n);
    }
    __syncthreads();
    __shared__ RunShared<D> s_run;
#pragma unroll 1
    for (int u = 0; u < s_long; ++u) {
        const int2 r = s_runs[kChunk - 1 - u];
        if (r.y > kMedium) write_run_block<16, D>(p, Run{t0 + r.x, r.y, s_slot[r.x]}, head, warp, lane, s_run);
    }
#pragma unroll 1
    for (int u = warp; u < 2 * s_long; u += kWarps) {
        const int2 r = s_runs[kChunk - 1 - (u >> 1)];
        if ((kHalf == 0 || r.y > kHalf) && r.y <= kMedium)
            write_run<32, 8, D>(p, Run{t0 + r.x, r.y, s_slot[r.x]}, head, u & 1, lane, 0xffffffffu);
    }
    if constexpr (kHalf > 0) {
#pragma unroll 1
        for (int u = tid / 16; u < 2 * s_long; u += kThreads / 16) {
            const int2 r = s_runs[kChunk - 1 - (u >> 1)];
            if (r.y <= kHalf)
                write_run<16, 8, D>(p, Run{t0 + r.x, r.y, s_slot[r.x]}, head, u & 1, tid % 16,
                                                   group_mask<16>(lane));
        }
    }
    const unsigned mask = group_mask<N>(lane);
#pragma unroll 1
    for (int u = tid / N; u < 2 * s_short; u += kThreads / N) {
        const int2 r = s_runs[u >> 1];
        write_run<N, 1, D>(p, Run{t0 + r.x, r.y, s_slot[r.x]}, head, u & 1, tid % N, mask);
    }
}

template <int D>
int launch_append(const AppendParams& p, int sms, smd_stream_t stream) {
    // Few tokens: lanes for each token. Many: blocks by chunks of tokens. The rule is set for
    // runs of a token or a few, which is what a step writes; it does not know the runs' length,
    // and a prompt below the limit (2432 tokens at 8 heads, 19456 at one) takes the slower form.
    // Pages of 64 tokens of 128 columns, few / many in us, * where the rule takes the slower:
    //                                      1 head         2 heads        4 heads        8 heads
    //   96 tokens of as many requests      2.3 / 14.0     2.3 / 14.5     2.4 / 14.9     2.5 / 15.2
    //   1000 of as many                    2.6 / 15.5     3.2 / 16.3     3.3 / 17.3     5.2 / 18.0
    //   2400 of as many                    2.8 / 16.3     3.4 / 18.1     6.1 / 18.0    10.6 / 21.4
    //   900 of 30                          6.1 /  7.8     6.4 /  7.9     7.7 /  8.1     9.5 /  8.4 *
    //   4000 of 30                        10.6 /  5.7 *  13.9 /  5.8 *  21.3 /  6.3 *  29.6 /  8.3
    //   16000 of 30                       18.4 /  6.7 *  27.8 /  8.6    43.7 / 15.3    62.3 / 23.2
    //   500 of one                        10.1 /  4.2 *  10.2 /  4.2 *  12.4 /  4.2 *  15.8 /  4.3 *
    //   1000 of one                        9.9 /  4.1 *  10.4 /  4.2 *  15.2 /  4.3 *  18.6 /  4.5 *
    //   4000 of one                       10.7 /  4.3 *  14.8 /  4.7 *  21.3 /  5.5 *  29.8 /  6.6
    //   16000 of one                      19.1 /  5.8 *  28.3 /  6.6    44.1 / 13.3    62.2 / 21.2
    const int64_t units = static_cast<int64_t>(p.T) * p.heads * 2;
    if (units <= static_cast<int64_t>(sms) * 256)
        return launch_pdl(append_few_kernel<D>,
                          dim3(static_cast<unsigned>((units * (D / 8) + kThreads - 1) / kThreads)),
                          kThreads, 0, stream, p);
    return launch_pdl(append_many_kernel<D>,
                      dim3(static_cast<unsigned>((p.T + kChunk - 1) / kChunk),
                           static_cast<unsigned>(p.heads)),
                      kThreads, 0, stream, p);
}

}  // namespace
}  // namespace smd

extern "C" int smd_paged_append(const smd_paged_cache_t* cache, const uint16_t* k, int64_t k_stride,
                                const uint16_t* v, int64_t v_stride, const int32_t* slots, int32_t T,
                                smd_stream_t stream) {
    using namespace smd;
    if (cache == nullptr) return SMD_ERR_NULL;
    if (!paged_ready(cache)) return SMD_ERR_PLAN;
    if (cache->k == nullptr) return SMD_ERR_NULL;
    const int64_t row = static_cast<int64_t>(cache->heads) * cache->head_dim;
    if (T < 0 || k_stride < row || v_stride < row || k_stride % 8 != 0 || v_stride % 8 != 0)
        return SMD_ERR_SHAPE;
    if (T == 0) return SMD_OK;
    if (k == nullptr || v == nullptr || slots == nullptr) return SMD_ERR_NULL;
    if (!aligned(k, 16) || !aligned(v, 16) || !aligned(slots, 4)) return SMD_ERR_ALIGN;
    const int sms = device_sms();
    if (sms <= 0) return SMD_ERR_DEVICE;
    AppendParams p{};
    p.x[0] = k;
    p.x[1] = v;
    p.x_stride[0] = k_stride;
    p.x_stride[1] = v_stride;
    p.slots = slots;
    p.T = T;
    p.pool[0] = cache->k;
    p.pool[1] = cache->v;
    for (int i = 0; i < 3; ++i) {
        p.stride[0][i] = cache->k_stride[i];
        p.stride[1][i] = cache->v_stride[i];
    }
    p.scale[0] = cache->k_scale;
    p.scale[1] = cache->v_scale;
    p.bounds = cache->bounds;
    p.pages = cache->pages;
    p.heads = cache->heads;
    p.P = cache->page_size;
    return cache->head_dim == 64    ? launch_append<64>(p, sms, stream)
           : cache->head_dim == 128 ? launch_append<128>(p, sms, stream)
                                    : launch_append<256>(p, sms, stream);
}

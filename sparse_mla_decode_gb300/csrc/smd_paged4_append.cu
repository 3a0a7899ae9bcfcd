// New keys and values into the pages of an E2M1 cache, and values out of them
// (smd_paged4_append, smd_paged4_read).
//
// For each token, head, side and block of 16 columns, with y = x 2^-e:
//   s = E4M3(max|y| / 6),  code = E2M1(y / s);  read: code s 2^e
// Quotients before rounding are exact where it matters, without a division a value. x is a
// bf16 (8 bits), s has 4 bits and a border between codes (0.25, 0.75, 1.25, .. 5) 3, so y / s
// is on a border or at least 2^-8 of it away: at least 2^-10. So y times the rounded 1 / s,
// off by 2^-22 of itself (at most 2^-19), is rounded to a multiple of 2^-13 by adding 1024 and
// taking it off again: borders come out as themselves, nothing crosses one. max|y| / 6 is
// corrected by its remainder, which gives the quotient to nearest (Markstein 1990).
//
// What bounds it: 2 D bytes read and 0.5625 D written for each token, head and side, and a
// page's bounds (8 D bytes) where it is touched: HBM for prompts, the dependent
// loads slot -> x for a decode step.
//
// A lane holds a block of 16 columns, D / 16 lanes a token of one head and side. A token's
// codes depend on nothing else, so the lanes are dealt out without regard to pages. Bounds are of
// runs (tokens whose slots continue one another inside a page), D / 8 lanes of 8 columns: few
// tokens: the lanes whose token begins a run read its keys too; many: a block takes the runs that
// begin in its chunk of tokens.
//
// Measured (GB300, device time): 96 tokens of as many requests, 8 heads of 128 columns, 2.4 to 2.6 us (1.8
// without bounds); 28 thousand tokens of 23 requests 35 us, 63% of the copy rate for the 146 MB (27
// without bounds, 80%: the bounds read the keys again from L2 and follow the codes), 256 columns 62 (71%),
// 64 columns in pages of 16 29 (38%). Read: 96 tokens 2.1 us, 28 thousand 24.9 (88%;
// 256 columns 94%; stores of 16 bytes, two a lane, 30.7, so too where rows are 16 bytes off). Tried for
// the append: loads of 32 bytes (36). For its bounds: blocks of their own beside those of the codes 36 us, behind them
// 44 (the keys have left L2), keys kept in shared memory 41.
#include "smd_internal.h"
#include "smd_paged.h"
#include "smd_paged_append.cuh"
#include "smd_ptx.cuh"

namespace smd {
namespace {

constexpr int kThreads = 128;
constexpr int kChunk = 64;      // tokens of a block, where they are many
constexpr int kMostPage = 256;  // tokens of a page
constexpr int kFewUnits = 384;  // (token, head) pairs an SM up to which tokens count as few
constexpr int kAtOnce = 4;      // loads of a lane in flight (append)
constexpr int kHeads = 8;       // heads of a lane in flight (read; 4: 5 to 10% slower up to 4000 tokens)

struct Append4Params {
    const uint16_t* x[2];
    int64_t x_stride[2];
    const int32_t* slots;
    int32_t T;
    uint8_t* pool[2];
    int64_t stride[2][3];
    uint8_t* scales[2];
    const int32_t* exps[2];
    uint16_t* bounds;
    int32_t pages, heads, P;
};

// max, a NaN wherever one of the two is.
__device__ __forceinline__ uint32_t bmax2_nan(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// 2^-e or 2^e of a head (sign -1 or 1).
__device__ __forceinline__ float power(const int32_t* exps, int head, int sign) {
    const int e = exps != nullptr ? max(min(__ldg(exps + head), 100), -100) : 0;
    return __uint_as_float(static_cast<uint32_t>(127 + sign * e) << 23);
}

// Eight codes of the nearest values to x `by`, the low nibble first.
__device__ __forceinline__ uint32_t codes_of(const uint4& v, float by) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    float q[8];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        float x = lo_f(w[j]), y = hi_f(w[j]);
        asm("{\n\t.reg .b64 a, b, c;\n\tmov.b64 a, {%0, %1};\n\tmov.b64 b, {%2, %2};\n\tmov.b64 c, {%3, %3};\n\t"
            "fma.rn.f32x2 a, a, b, c;\n\tmov.b64 c, {%4, %4};\n\tadd.rn.f32x2 a, a, c;\n\tmov.b64 {%0, %1}, a;\n\t}"
            : "+f"(x), "+f"(y)
            : "f"(by), "f"(1024.0f), "f"(-1024.0f));
        q[2 * j] = x;
        q[2 * j + 1] = y;
    }
    uint32_t r;
    asm("{\n\t.reg .b8 a, b, c, d;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\tcvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\tcvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
        "mov.b32 %0, {a, b, c, d};\n\t}"
        : "=r"(r)
        : "f"(q[0]), "f"(q[1]), "f"(q[2]), "f"(q[3]), "f"(q[4]), "f"(q[5]), "f"(q[6]), "f"(q[7]));
    return r;
}

// A block of 16 values: their codes, and the scale as E4M3.
__device__ __forceinline__ uint2 quantise(const uint4 (&v)[2], float down, uint32_t& scale) {
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        m = bmax2_nan(m, bmax2_nan(v[j].x & 0x7fff7fffu, v[j].y & 0x7fff7fffu));
        m = bmax2_nan(m, bmax2_nan(v[j].z & 0x7fff7fffu, v[j].w & 0x7fff7fffu));
    }
    float a;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(a) : "f"(lo_f(m)), "f"(hi_f(m)));
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(a) : "f"(a * down), "f"(65536.0f));  // far above 6 * 448
    constexpr float kSixth = 1.0f / 6.0f;
    float s = a * kSixth;
    s = fmaf(fmaf(-6.0f, s, a), kSixth, s);
    scale = e4m3x2(s, 0.0f) & 0xffu;
    asm("{\n\t.reg .b16 l, h;\n\t.reg .b32 t;\n\tcvt.u16.u32 l, %1;\n\tcvt.rn.f16x2.e4m3x2 t, l;\n\t"
        "mov.b32 {l, h}, t;\n\tcvt.f32.f16 %0, l;\n\t}"
        : "=f"(s)
        : "r"(scale));
    float by;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(by) : "f"(s));
    by = s > 0.0f ? by * down : 0.0f;
    return make_uint2(codes_of(v[0], by), codes_of(v[1], by));
}

// Whether the slot is in the pool.
__device__ __forceinline__ bool in_pool(const Append4Params& p, int slot) {
    return slot >= 0 && slot / p.P < p.pages;
}

// Block i of a token.
template <int D>
__device__ __forceinline__ void store(const Append4Params& p, int side, int head, int slot, int i,
                                      const uint2& codes, uint32_t scale) {
    const int page = slot / p.P, o = slot - page * p.P;
    const int64_t* const st = p.stride[side];
    *reinterpret_cast<uint2*>(p.pool[side] + page * st[0] + head * st[1] + o * st[2] + 8 * i) = codes;
    p.scales[side][((static_cast<int64_t>(page) * p.heads + head) * p.P + o) * (D / 16) + i] =
        static_cast<uint8_t>(scale);
}

// The extremes of n keys: 8 columns, every `step`-th token, kLoads of them in flight.
template <int kLoads>
__device__ __forceinline__ void scan_keys(const uint16_t* x, int64_t xs, int n, int step, uint32_t (&hi)[4],
                                          uint32_t (&lo)[4]) {
#pragma unroll 1
    for (int m0 = 0; m0 < n; m0 += kLoads * step) {
        uint4 v[kLoads];
#pragma unroll
        for (int j = 0; j < kLoads; ++j)
            if (m0 + j * step < n) v[j] = __ldg(reinterpret_cast<const uint4*>(x + (m0 + j * step) * xs));
#pragma unroll
        for (int j = 0; j < kLoads; ++j)
            if (m0 + j * step < n) take(v[j], hi, lo);
    }
}

__device__ __forceinline__ void nothing_met(uint32_t (&hi)[4], uint32_t (&lo)[4]) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        hi[j] = 0xff80ff80u;  // -infinity
        lo[j] = 0x7f807f80u;
    }
}

// The bounds of the page that a run of n tokens from t on is in, by D / 8 lanes.
template <int D>
__device__ __forceinline__ void run_bounds(const Append4Params& p, int64_t t, int n, int slot, int head, int i) {
    const int page = slot / p.P, o = slot - page * p.P;
    uint16_t* const bounds = p.bounds + (static_cast<int64_t>(page) * p.heads + head) * 2 * D;
    Extremes was;
    if (o > 0) was.read(bounds, D, 8 * i);
    uint32_t hi[4], lo[4];
    nothing_met(hi, lo);
    const uint16_t* const x = p.x[0] + t * p.x_stride[0] + head * D + 8 * i;
    // Of a page's 64 keys 8 at a time; 4: 500 tokens of a request 8.0 us instead of 6.9.
    if (n <= 2) scan_keys<2>(x, p.x_stride[0], n, 1, hi, lo);
    else scan_keys<8>(x, p.x_stride[0], n, 1, hi, lo);
    write_bounds(bounds, D, 8 * i, was, hi, lo);
}

// D / 8 lanes for each (token, head): one half the keys, the other the values.
template <int D>
__global__ void __launch_bounds__(kThreads) append4_few_kernel(const Append4Params p) {
    constexpr int N = D / 8;
    pdl_entry();
    const int lane = threadIdx.x & 31, i = threadIdx.x % N, side = i / (N / 2), b = i % (N / 2);
    const unsigned mask = group_mask<N>(lane);
    const int64_t unit = (static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x) / N;
    const int t = static_cast<int>(unit / p.heads), head = static_cast<int>(unit % p.heads);
    if (t >= p.T) return;
    const uint4* const x =
        reinterpret_cast<const uint4*>(p.x[side] + t * p.x_stride[side] + head * D + 16 * b);
    const uint4 v[2] = {__ldg(x), __ldg(x + 1)};
    const int slot = p.slots[t];
    const int before = p.bounds != nullptr && t > 0 ? p.slots[t - 1] : -2;
    if (!in_pool(p, slot)) return;
    uint32_t scale;
    const uint2 codes = quantise(v, power(p.exps[side], head, -1), scale);
    store<D>(p, side, head, slot, b, codes, scale);
    if (p.bounds == nullptr || (slot % p.P != 0 && before == slot - 1)) return;  // not a run's first
    const int most = min(p.P - slot % p.P, p.T - t);
    int n = 1;
    while (n < most) {
        const bool on = n + i < most && p.slots[t + n + i] == slot + n + i;
        const unsigned off = ~__ballot_sync(mask, on) & mask;
        const int c = off == 0 ? N : (__ffs(off) - 1) % N;
        n += c;
        if (c < N) break;
    }
    run_bounds<D>(p, t, n, slot, head, i);
}

// A block for each chunk of tokens and head. kBounds: then the bounds of the runs that begin in the
// chunk, whose keys are read again, from L1 or L2.
template <int D, bool kBounds>
__global__ void __launch_bounds__(kThreads, 8) append4_many_kernel(const Append4Params p) {
    constexpr int N = D / 8, kGroups = kThreads / N;
    __shared__ int s_slot[kChunk];
    __shared__ int2 s_runs[kChunk];  // first token and length: short runs from the front, long from the back
    __shared__ uint32_t s_goes[(kChunk + kMostPage) / 32], s_lead[kChunk / 32];
    __shared__ int s_short, s_long;
    __shared__ uint4 s_hi[kGroups][N], s_lo[kGroups][N];
    const int tid = threadIdx.x, lane = tid & 31, head = blockIdx.y;
    pdl_entry();
    const int64_t t0 = static_cast<int64_t>(blockIdx.x) * kChunk;
    const int span = static_cast<int>(min(static_cast<int64_t>(p.T) - t0, static_cast<int64_t>(kChunk)));
    if (tid < span) s_slot[tid] = p.slots[t0 + tid];
    if constexpr (kBounds) {
        // A token goes on with the run of the one before it, or it leads one; a run of this chunk may go
        // on into the next chunks.
        if (tid == 0) s_short = s_long = 0;
        const int seen = static_cast<int>(min(static_cast<int64_t>(p.T) - t0, static_cast<int64_t>(kChunk) + p.P));
        for (int j0 = 0; j0 < kChunk + p.P; j0 += kThreads) {
            const int j = j0 + tid;
            bool goes = false, lead = false;
            if (j < seen) {
                const int slot = p.slots[t0 + j], before = t0 + j > 0 ? p.slots[t0 + j - 1] : -2;
                if (in_pool(p, slot)) {
                    goes = slot % p.P != 0 && before == slot - 1;
                    lead = !goes && j < span;
                }
            }
            const uint32_t g = __ballot_sync(0xffffffffu, goes), l = __ballot_sync(0xffffffffu, lead);
            if (lane == 0 && j < kChunk + kMostPage) {
                s_goes[j >> 5] = g;
                if (j < kChunk) s_lead[j >> 5] = l;
            }
        }
        __syncthreads();
        constexpr int kShort = 4;  // runs up to this length go to D / 8 lanes each
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
    }
    __syncthreads();
    {
        // Codes: a unit of D / 16 lanes is a token and a side.
        constexpr int NB = D / 16, kUnits = kThreads / NB;  // units at a time: as many of each side
        const int i = tid % NB, unit = tid / NB, side = unit & 1;
        const float by = power(p.exps[side], head, -1);
        const uint16_t* const x = p.x[side] + t0 * p.x_stride[side] + head * D + 16 * i;
#pragma unroll 1
        for (int m0 = unit >> 1; m0 < span; m0 += kAtOnce * (kUnits / 2)) {
            uint4 v[kAtOnce][2];
#pragma unroll
            for (int j = 0; j < kAtOnce; ++j) {
                const int m = m0 + j * (kUnits / 2);
                if (m < span) {
                    const uint4* const at = reinterpret_cast<const uint4*>(x + m * p.x_stride[side]);
                    v[j][0] = __ldg(at);
                    v[j][1] = __ldg(at + 1);
                }
            }
#pragma unroll
            for (int j = 0; j < kAtOnce; ++j) {
                const int m = m0 + j * (kUnits / 2);
                if (m >= span) break;
                uint32_t scale;
                const uint2 codes = quantise(v[j], by, scale);
                if (in_pool(p, s_slot[m])) store<D>(p, side, head, s_slot[m], i, codes, scale);
            }
        }
    }
    if constexpr (!kBounds) return;
    const int i = tid % N, group = tid / N;
    __syncthreads();
    const uint16_t* const x = p.x[0] + t0 * p.x_stride[0] + head * D + 8 * i;
    const auto extremes = [&](const int2& r, int first, int step, uint32_t (&hi)[4], uint32_t (&lo)[4]) {
        nothing_met(hi, lo);
#pragma unroll 4
        for (int m = r.x + first; m < r.x + r.y; m += step)
            take(__ldg(reinterpret_cast<const uint4*>(x + m * p.x_stride[0])), hi, lo);
    };
    const auto bounds_of = [&](int slot) {
        return p.bounds + (static_cast<int64_t>(slot / p.P) * p.heads + head) * 2 * D;
    };
    constexpr int kRuns = 4;  // short runs of a group whose pages' bounds are on their way together
#pragma unroll 1
    for (int u0 = group; u0 < s_short; u0 += kRuns * kGroups) {
        Extremes was[kRuns];
#pragma unroll
        for (int j = 0; j < kRuns; ++j)
            if (u0 + j * kGroups < s_short) {
                const int slot = s_slot[s_runs[u0 + j * kGroups].x];
                if (slot % p.P != 0) was[j].read(bounds_of(slot), D, 8 * i);
            }
#pragma unroll
        for (int j = 0; j < kRuns; ++j)
            if (u0 + j * kGroups < s_short) {
                const int2 r = s_runs[u0 + j * kGroups];
                uint32_t hi[4], lo[4];
                extremes(r, 0, 1, hi, lo);
                write_bounds(bounds_of(s_slot[r.x]), D, 8 * i, was[j], hi, lo);
            }
    }
#pragma unroll 1
    for (int u = 0; u < s_long; ++u) {
        const int2 r = s_runs[kChunk - 1 - u];
        const int slot = s_slot[r.x];
        Extremes was;
        if (group == 0 && slot % p.P != 0) was.read(bounds_of(slot), D, 8 * i);
        uint32_t hi[4], lo[4];
        extremes(r, group, kGroups, hi, lo);
        s_hi[group][i] = make_uint4(hi[0], hi[1], hi[2], hi[3]);
        s_lo[group][i] = make_uint4(lo[0], lo[1], lo[2], lo[3]);
        __syncthreads();
        if (group == 0) {
#pragma unroll
            for (int g = 1; g < kGroups; ++g) {
                const uint4 h = s_hi[g][i], l = s_lo[g][i];
                hi[0] = bmax2(hi[0], h.x), hi[1] = bmax2(hi[1], h.y);
                hi[2] = bmax2(hi[2], h.z), hi[3] = bmax2(hi[3], h.w);
                lo[0] = bmin2(lo[0], l.x), lo[1] = bmin2(lo[1], l.y);
                lo[2] = bmin2(lo[2], l.z), lo[3] = bmin2(lo[3], l.w);
            }
            write_bounds(bounds_of(slot), D, 8 * i, was, hi, lo);
        }
        __syncthreads();
    }
}

struct Read4Params {
    const int32_t* slots;
    int32_t T;
    const uint8_t* pool[2];
    int64_t stride[2][3];
    const uint8_t* scales[2];
    const int32_t* exps[2];
    uint16_t* out[2];
    int64_t out_stride[2];
    int32_t pages, heads, P;
    int32_t first, sides;  // the first side that is read, and how many
    int32_t shares;        // units that share a token's heads
    bool wide;             // rows are 32-byte aligned
};

// 32 bytes in one store (wide: 32-byte aligned) or two, each of which is half a sector a lane.
__device__ __forceinline__ void store32(uint16_t* to, bool wide, const uint32_t (&w)[8]) {
    if (wide) {
        asm volatile("st.global.cs.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(to), "r"(w[0]),
                     "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                     : "memory");
    } else {
        __stcs(reinterpret_cast<uint4*>(to), make_uint4(w[0], w[1], w[2], w[3]));
        __stcs(reinterpret_cast<uint4*>(to) + 1, make_uint4(w[4], w[5], w[6], w[7]));
    }
}

// D / 16 lanes for each (token, side) and share of the heads: a block of 16 columns each.
template <int D>
__global__ void __launch_bounds__(kThreads) read4_kernel(const Read4Params p) {
    constexpr int N = D / 16;
    pdl_entry();
    const int i = threadIdx.x % N;
    const int64_t unit = (static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x) / N;
    const int64_t ts = unit / p.shares, t = ts / p.sides;
    const int side = p.first + static_cast<int>(ts % p.sides);
    if (t >= p.T) return;
    const int slot = p.slots[t], page = slot / p.P, o = slot - page * p.P;
    if (slot < 0 || page >= p.pages) return;
    const int64_t* const st = p.stride[side];
    const uint8_t* const pool = p.pool[side] + page * st[0] + o * st[2] + 8 * i;
    const uint8_t* const scales =
        p.scales[side] + (static_cast<int64_t>(page) * p.heads * p.P + o) * (D / 16) + i;
    uint16_t* const out = p.out[side] + t * p.out_stride[side] + 16 * i;
#pragma unroll 1
    for (int h0 = static_cast<int>(unit % p.shares); h0 < p.heads; h0 += kHeads * p.shares) {
        uint2 codes[kHeads];
        uint32_t scale[kHeads];
#pragma unroll
        for (int j = 0; j < kHeads; ++j) {
            const int h = h0 + j * p.shares;
            if (h < p.heads) {
                codes[j] = __ldg(reinterpret_cast<const uint2*>(pool + h * st[1]));
                scale[j] = __ldg(scales + static_cast<int64_t>(h) * p.P * (D / 16));
            }
        }
#pragma unroll
        for (int j = 0; j < kHeads; ++j) {
            const int h = h0 + j * p.shares;
            if (h >= p.heads) break;
            const float up = power(p.exps[side], h, 1);
            uint32_t w[8];
#pragma unroll
            for (int z = 0; z < 2; ++z)
                asm("{\n\t.reg .b8 a, b, c, d;\n\t.reg .b16 s;\n\t.reg .b32 t;\n\t"
                    "cvt.u16.u32 s, %5;\n\tcvt.rn.f16x2.e4m3x2 t, s;\n\tmov.b32 {a, b, c, d}, %4;\n\t"
                    "cvt.rn.f16x2.e2m1x2 %0, a;\n\tcvt.rn.f16x2.e2m1x2 %1, b;\n\t"
                    "cvt.rn.f16x2.e2m1x2 %2, c;\n\tcvt.rn.f16x2.e2m1x2 %3, d;\n\t"
                    "mul.rn.f16x2 %0, %0, t;\n\tmul.rn.f16x2 %1, %1, t;\n\t"
                    "mul.rn.f16x2 %2, %2, t;\n\tmul.rn.f16x2 %3, %3, t;\n\t}"
                    : "=&r"(w[4 * z]), "=&r"(w[4 * z + 1]), "=&r"(w[4 * z + 2]), "=&r"(w[4 * z + 3])
                    : "r"(z == 0 ? codes[j].x : codes[j].y), "r"(scale[j] * 0x101u));
#pragma unroll
            for (int z = 0; z < 8; ++z) {
                float a, b;
                asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.f32.f16 %0, l;\n\tcvt.f32.f16 %1, h;\n\t}"
                    : "=f"(a), "=f"(b)
                    : "r"(w[z]));
                w[z] = bf16x2(a * up, b * up);
            }
            store32(out + h * D, p.wide, w);
        }
    }
}

template <int D>
int launch_append(const Append4Params& p, int sms, smd_stream_t stream) {
    // Few tokens: lanes for each. Many: blocks by chunks of tokens. The limit is one of units: which tokens
    // continue one another is known to the GPU only. Just below it tokens of as many requests gain and prompts lose.
    // Few / many in us, 8 heads of 128 columns, pages of 64 (in brackets without bounds):
    //   96 tokens of as many requests   2.4 /  7.8  ( 1.8 /  4.3)
    //   3000 of as many                 8.4 / 14.2  ( 5.3 /  7.1)
    //   7000 of as many                18.5 / 22.2  (13.0 / 12.1)
    //   8000 of as many                21.0 / 24.6  (14.5 / 13.5)
    //   500 of one                      6.8 /  5.3  ( 2.2 /  4.3)
    //   4000 of one                    11.9 / 10.3  ( 6.3 /  8.4)
    //   7000 of one, of 30             18.0 / 12.8, 13.7  (11.6 / 10.6)
    //   16000 of one                   33.8 / 20.7  (25.9 / 17.1)
    const int64_t units = static_cast<int64_t>(p.T) * p.heads;
    if (units <= static_cast<int64_t>(sms) * kFewUnits)
        return launch_pdl(append4_few_kernel<D>,
                          dim3(static_cast<unsigned>((units * (D / 8) + kThreads - 1) / kThreads)),
                          kThreads, 0, stream, p);
    const dim3 grid(static_cast<unsigned>((static_cast<int64_t>(p.T) + kChunk - 1) / kChunk),
                    static_cast<unsigned>(p.heads));
    return p.bounds != nullptr ? launch_pdl(append4_many_kernel<D, true>, grid, kThreads, 0, stream, p)
                               : launch_pdl(append4_many_kernel<D, false>, grid, kThreads, 0, stream, p);
}

template <int D>
int launch_read(Read4Params p, int sms, smd_stream_t stream) {
    // A token's heads go to one unit, kHeads at a time, unless that leaves SMs without work (96
    // tokens of 8 heads: 2.6 us by one unit or two, 1.8 by eight).
    const int64_t units = static_cast<int64_t>(p.T) * p.sides, want = static_cast<int64_t>(sms) * 2 * kThreads / (D / 16);
    const int64_t shares = (want + units - 1) / units;
    p.shares = static_cast<int32_t>(shares < 1 ? 1 : shares < p.heads ? shares : p.heads);
    const int64_t blocks = (units * p.shares * (D / 16) + kThreads - 1) / kThreads;
    if (blocks >= (1ll << 31)) return SMD_ERR_SHAPE;
    return launch_pdl(read4_kernel<D>, dim3(static_cast<unsigned>(blocks)), kThreads, 0, stream, p);
}

}  // namespace
}  // namespace smd

extern "C" int smd_paged4_append(const smd_paged4_cache_t* cache, const uint16_t* k, int64_t k_stride,
                                 const uint16_t* v, int64_t v_stride, const int32_t* slots, int32_t T,
                                 smd_stream_t stream) {
    using namespace smd;
    if (cache == nullptr) return SMD_ERR_NULL;
    if (!paged_ready(cache)) return SMD_ERR_PLAN;
    const int64_t row = static_cast<int64_t>(cache->heads) * cache->head_dim;
    if (T < 0 || k_stride < row || v_stride < row || k_stride % 8 != 0 || v_stride % 8 != 0)
        return SMD_ERR_SHAPE;
    if (T == 0) return SMD_OK;
    if (k == nullptr || v == nullptr || slots == nullptr) return SMD_ERR_NULL;
    if (!aligned(k, 16) || !aligned(v, 16) || !aligned(slots, 4)) return SMD_ERR_ALIGN;
    const int sms = device_sms();
    if (sms <= 0) return SMD_ERR_DEVICE;
    Append4Params p{};
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
    p.scales[0] = cache->k_scales;
    p.scales[1] = cache->v_scales;
    p.exps[0] = cache->k_exp;
    p.exps[1] = cache->v_exp;
    p.bounds = cache->bounds;
    p.pages = cache->pages;
    p.heads = cache->heads;
    p.P = cache->page_size;
    return cache->head_dim == 64    ? launch_append<64>(p, sms, stream)
           : cache->head_dim == 128 ? launch_append<128>(p, sms, stream)
                                    : launch_append<256>(p, sms, stream);
}

extern "C" int smd_paged4_read(const smd_paged4_cache_t* cache, const int32_t* slots, int32_t T,
                               uint16_t* k, int64_t k_stride, uint16_t* v, int64_t v_stride,
                               smd_stream_t stream) {
    using namespace smd;
    if (cache == nullptr) return SMD_ERR_NULL;
    if (!paged_ready(cache)) return SMD_ERR_PLAN;
    const int64_t row = static_cast<int64_t>(cache->heads) * cache->head_dim;
    if (T < 0 || (k != nullptr && (k_stride < row || k_stride % 8 != 0)) ||
        (v != nullptr && (v_stride < row || v_stride % 8 != 0)))
        return SMD_ERR_SHAPE;
    if (T == 0 || (k == nullptr && v == nullptr)) return SMD_OK;
    if (slots == nullptr) return SMD_ERR_NULL;
    if (!aligned(k, 16) || !aligned(v, 16) || !aligned(slots, 4)) return SMD_ERR_ALIGN;
    Read4Params p{};
    p.slots = slots;
    p.T = T;
    p.pool[0] = cache->k;
    p.pool[1] = cache->v;
    for (int i = 0; i < 3; ++i) {
        p.stride[0][i] = cache->k_stride[i];
        p.stride[1][i] = cache->v_stride[i];
    }
    p.scales[0] = cache->k_scales;
    p.scales[1] = cache->v_scales;
    p.exps[0] = cache->k_exp;
    p.exps[1] = cache->v_exp;
    p.out[0] = k;
    p.out[1] = v;
    p.out_stride[0] = k_stride;
    p.out_stride[1] = v_stride;
    p.wide = (k == nullptr || (aligned(k, 32) && k_stride % 16 == 0)) &&
             (v == nullptr || (aligned(v, 32) && v_stride % 16 == 0));
    p.pages = cache->pages;
    p.heads = cache->heads;
    p.P = cache->page_size;
    p.first = k != nullptr ? 0 : 1;
    p.sides = (k != nullptr ? 1 : 0) + (v != nullptr ? 1 : 0);
    const int sms = device_sms();
    if (sms <= 0) return SMD_ERR_DEVICE;
    return cache->head_dim == 64    ? launch_read<64>(p, sms, stream)
           : cache->head_dim == 128 ? launch_read<128>(p, sms, stream)
                                    : launch_read<256>(p, sms, stream);
}

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
// D / 8 lanes hold a token of one head and side, 8 columns (16 bytes of bf16) each; two
// neighbours share a block's scale. A token's codes depend on nothing else, so the lanes are
// dealt out without regard to pages. Bounds are of runs (tokens whose slots continue one
// another inside a page): few tokens: the lanes whose token begins a run read its
// other keys too; many: a block takes the runs that begin in its chunk of tokens.
#include "smd_internal.h"
#include "smd_paged.h"
#include "smd_paged_append.cuh"
#include "smd_ptx.cuh"

namespace smd {
namespace {

constexpr int kThreads = 128;
constexpr int kChunk = 64;      // tokens of a block, where they are many
constexpr int kMostPage = 256;  // tokens of a page
constexpr int kAtOnce = 4;      // loads of a lane in flight

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

// Two values' codes in a byte, from their quotients.
__device__ __forceinline__ uint32_t codes_of(const float (&q)[8]) {
    uint32_t r;
    asm("{\n\t.reg .b8 a, b, c, d;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\tcvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\tcvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
        "mov.b32 %0, {a, b, c, d};\n\t}"
        : "=r"(r)
        : "f"(q[0]), "f"(q[1]), "f"(q[2]), "f"(q[3]), "f"(q[4]), "f"(q[5]), "f"(q[6]), "f"(q[7]));
    return r;
}

// Eight values (half a block: the lane beside has the other half; `mask`: the lanes that run
// together): their codes, and the block's scale as E4M3.
__device__ __forceinline__ uint32_t quantise(const uint4& v, float down, unsigned mask, uint32_t& scale) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    uint32_t m = w[0] & 0x7fff7fffu;
#pragma unroll
    for (int j = 1; j < 4; ++j) m = bmax2_nan(m, w[j] & 0x7fff7fffu);
    m = bmax2_nan(m, __shfl_xor_sync(mask, m, 1));
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
    float q[8];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        q[2 * j] = fmaf(lo_f(w[j]), by, 1024.0f) - 1024.0f;
        q[2 * j + 1] = fmaf(hi_f(w[j]), by, 1024.0f) - 1024.0f;
    }
    return codes_of(q);
}

// Whether the slot is in the pool.
__device__ __forceinline__ bool in_pool(const Append4Params& p, int slot) {
    return slot >= 0 && slot / p.P < p.pages;
}

template <int D>
__device__ __forceinline__ void store(const Append4Params& p, int side, int head, int slot, int i,
                                      uint32_t codes, uint32_t scale) {
    const int page = slot / p.P, o = slot - page * p.P;
    const int64_t* const st = p.stride[side];
    *reinterpret_cast<uint32_t*>(p.pool[side] + page * st[0] + head * st[1] + o * st[2] + 4 * i) = codes;
    if ((i & 1) == 0)
        p.scales[side][((static_cast<int64_t>(page) * p.heads + head) * p.P + o) * (D / 16) + (i >> 1)] =
            static_cast<uint8_t>(scale);
}

// The extremes of n keys from token t on: 8 columns, every `step`-th token.
__device__ __forceinline__ void scan_keys(const uint16_t* x, int64_t xs, int n, int step, uint32_t (&hi)[4],
                                          uint32_t (&lo)[4]) {
#pragma unroll 4
    for (int m = 0; m < n; m += step) take(*reinterpret_cast<const uint4*>(x + m * xs), hi, lo);
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
    scan_keys(p.x[0] + t * p.x_stride[0] + head * D + 8 * i, p.x_stride[0], n, 1, hi, lo);
    write_bounds(bounds, D, 8 * i, was, hi, lo);
}

// D / 8 lanes for each (token, head, side).
template <int D>
__global__ void __launch_bounds__(kThreads) append4_few_kernel(const Append4Params p) {
    constexpr int N = D / 8;
    pdl_entry();
    const int lane = threadIdx.x & 31, i = threadIdx.x % N;
    const unsigned mask = group_mask<N>(lane);
    const int64_t unit = (static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x) / N;
    const int t = static_cast<int>(unit / (2 * p.heads)), hs = static_cast<int>(unit % (2 * p.heads));
    if (t >= p.T) return;
    const int side = hs & 1, head = hs >> 1;
    const uint4 v = __ldcs(reinterpret_cast<const uint4*>(p.x[side] + t * p.x_stride[side] + head * D + 8 * i));
    const int slot = p.slots[t];
    if (!in_pool(p, slot)) return;
    uint32_t scale;
    const uint32_t codes = quantise(v, power(p.exps[side], head, -1), mask, scale);
    store<D>(p, side, head, slot, i, codes, scale);
    if (p.bounds == nullptr || side != 0) return;
    if (t > 0 && slot % p.P != 0 && p.slots[t - 1] == slot - 1) return;  // not a run's first
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

// A block for each chunk of tokens and head.
template <int D>
__global__ void __launch_bounds__(kThreads) append4_many_kernel(const Append4Params p) {
    constexpr int N = D / 8, kGroups = kThreads / N;
    __shared__ int s_slot[kChunk];
    __shared__ int2 s_runs[kChunk];  // first token and length: short runs from the front, long from the back
    __shared__ uint32_t s_goes[(kChunk + kMostPage) / 32], s_lead[kChunk / 32];
    __shared__ int s_short, s_long;
    __shared__ uint4 s_hi[kGroups][N], s_lo[kGroups][N];
    const int tid = threadIdx.x, lane = tid & 31, i = tid % N, group = tid / N;
    const unsigned mask = group_mask<N>(lane);
    const int head = blockIdx.y;
    if (tid == 0) s_short = s_long = 0;
    pdl_entry();
    const int64_t t0 = static_cast<int64_t>(blockIdx.x) * kChunk;
    const int span = static_cast<int>(min(static_cast<int64_t>(p.T) - t0, static_cast<int64_t>(kChunk)));
    const float down[2] = {power(p.exps[0], head, -1), power(p.exps[1], head, -1)};
    if (tid < span) s_slot[tid] = p.slots[t0 + tid];
    __syncthreads();
    // Codes: a group's unit is a token and a side.
#pragma unroll 1
    for (int u0 = group; u0 < 2 * span; u0 += kAtOnce * kGroups) {
        uint4 v[kAtOnce];
#pragma unroll
        for (int j = 0; j < kAtOnce; ++j) {
            const int u = u0 + j * kGroups, t = u >> 1, side = u & 1;
            v[j] = make_uint4(0, 0, 0, 0);
            if (u < 2 * span)
                v[j] = *reinterpret_cast<const uint4*>(p.x[side] + (t0 + t) * p.x_stride[side] + head * D + 8 * i);
        }
#pragma unroll
        for (int j = 0; j < kAtOnce; ++j) {
            const int u = u0 + j * kGroups, t = u >> 1, side = u & 1;
            if (u >= 2 * span) break;  // the same in a group's lanes
            uint32_t scale;
            const uint32_t codes = quantise(v[j], down[side], mask, scale);
            if (in_pool(p, s_slot[t])) store<D>(p, side, head, s_slot[t], i, codes, scale);
        }
    }
    if (p.bounds == nullptr) return;

    // Bounds. A token goes on with the run of the one before it, or it leads one; a run of this
    // chunk may go on into the next chunks.
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
    constexpr int kShort = 8;  // runs up to this length go to a group of lanes each
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
#pragma unroll 1
    for (int u = group; u < s_short; u += kGroups) {
        const int2 r = s_runs[u];
        run_bounds<D>(p, t0 + r.x, r.y, s_slot[r.x], head, i);
    }
#pragma unroll 1
    for (int u = 0; u < s_long; ++u) {
        const int2 r = s_runs[kChunk - 1 - u];
        uint32_t hi[4], lo[4];
        nothing_met(hi, lo);
        scan_keys(p.x[0] + (t0 + r.x + group) * p.x_stride[0] + head * D + 8 * i, p.x_stride[0], r.y - group,
                  kGroups, hi, lo);
        s_hi[group][i] = make_uint4(hi[0], hi[1], hi[2], hi[3]);
        s_lo[group][i] = make_uint4(lo[0], lo[1], lo[2], lo[3]);
        __syncthreads();
        if (group == 0) {
            const int slot = s_slot[r.x], page = slot / p.P, o = slot - page * p.P;
            uint16_t* const bounds = p.bounds + (static_cast<int64_t>(page) * p.heads + head) * 2 * D;
            Extremes was;
            if (o > 0) was.read(bounds, D, 8 * i);
#pragma unroll
            for (int g = 1; g < kGroups; ++g) {
                const uint4 h = s_hi[g][i], l = s_lo[g][i];
                hi[0] = bmax2(hi[0], h.x), hi[1] = bmax2(hi[1], h.y);
                hi[2] = bmax2(hi[2], h.z), hi[3] = bmax2(hi[3], h.w);
                lo[0] = bmin2(lo[0], l.x), lo[1] = bmin2(lo[1], l.y);
                lo[2] = bmin2(lo[2], l.z), lo[3] = bmin2(lo[3], l.w);
            }
            write_bounds(bounds, D, 8 * i, was, hi, lo);
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
};

// D / 8 lanes for each (token, side, head): 8 columns each.
template <int D>
__global__ void __launch_bounds__(kThreads) read4_kernel(const Read4Params p) {
    constexpr int N = D / 8;
    pdl_entry();
    const int i = threadIdx.x % N;
    const int64_t unit = (static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x) / N;
    const int head = static_cast<int>(unit % p.heads);
    const int64_t ts = unit / p.heads;
    const int64_t t = ts / p.sides;
    const int side = p.first + static_cast<int>(ts % p.sides);
    if (t >= p.T) return;
    const int slot = p.slots[t], page = slot / p.P, o = slot - page * p.P;
    if (slot < 0 || page >= p.pages) return;
    const int64_t* const st = p.stride[side];
    const uint32_t codes =
        *reinterpret_cast<const uint32_t*>(p.pool[side] + page * st[0] + head * st[1] + o * st[2] + 4 * i);
    const uint32_t scale =
        p.scales[side][((static_cast<int64_t>(page) * p.heads + head) * p.P + o) * (D / 16) + (i >> 1)];
    const float up = power(p.exps[side], head, 1);
    uint32_t w[4];
    asm("{\n\t.reg .b8 a, b, c, d;\n\t.reg .b16 s;\n\t.reg .b32 t;\n\t"
        "cvt.u16.u32 s, %5;\n\tcvt.rn.f16x2.e4m3x2 t, s;\n\tmov.b32 {a, b, c, d}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, a;\n\tcvt.rn.f16x2.e2m1x2 %1, b;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, c;\n\tcvt.rn.f16x2.e2m1x2 %3, d;\n\t"
        "mul.rn.f16x2 %0, %0, t;\n\tmul.rn.f16x2 %1, %1, t;\n\t"
        "mul.rn.f16x2 %2, %2, t;\n\tmul.rn.f16x2 %3, %3, t;\n\t}"
        : "=&r"(w[0]), "=&r"(w[1]), "=&r"(w[2]), "=&r"(w[3])
        : "r"(codes), "r"(scale * 0x101u));
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        float a, b;
        asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.f32.f16 %0, l;\n\tcvt.f32.f16 %1, h;\n\t}"
            : "=f"(a), "=f"(b)
            : "r"(w[j]));
        w[j] = bf16x2(a * up, b * up);
    }
    *reinterpret_cast<uint4*>(p.out[side] + t * p.out_stride[side] + head * D + 8 * i) =
        make_uint4(w[0], w[1], w[2], w[3]);
}

template <int D>
int launch_append(const Append4Params& p, int sms, smd_stream_t stream) {
    const int64_t units = static_cast<int64_t>(p.T) * p.heads * 2;
    if (units <= static_cast<int64_t>(sms) * 256)
        return launch_pdl(append4_few_kernel<D>,
                          dim3(static_cast<unsigned>((units * (D / 8) + kThreads - 1) / kThreads)),
                          kThreads, 0, stream, p);
    return launch_pdl(append4_many_kernel<D>,
                      dim3(static_cast<unsigned>((static_cast<int64_t>(p.T) + kChunk - 1) / kChunk),
                           static_cast<unsigned>(p.heads)),
                      kThreads, 0, stream, p);
}

template <int D>
int launch_read(const Read4Params& p, smd_stream_t stream) {
    const int64_t blocks = (static_cast<int64_t>(p.T) * p.heads * p.sides * (D / 8) + kThreads - 1) / kThreads;
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
    p.pages = cache->pages;
    p.heads = cache->heads;
    p.P = cache->page_size;
    p.first = k != nullptr ? 0 : 1;
    p.sides = (k != nullptr ? 1 : 0) + (v != nullptr ? 1 : 0);
    return cache->head_dim == 64    ? launch_read<64>(p, stream)
           : cache->head_dim == 128 ? launch_read<128>(p, stream)
                                    : launch_read<256>(p, stream);
}

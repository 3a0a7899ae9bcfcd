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
// A group of threads (a warp, or a block of 256) takes one run of one head and
// side: a thread holds 8 columns (16 bytes of bf16) of every TPG-th token. The
// maximum of the run comes first, then the run is read again (from L1 or L2)
// to be encoded.
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
    int32_t chunk;  // tokens of a block (block-wide groups)
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

// x / scale for any positive scale; a product where that is exact.
struct Quotient {
    float s, inv;
    bool exact;
    __device__ __forceinline__ float operator()(float x) const { return exact ? x * inv : __fdiv_rn(x, s); }
};

__device__ __forceinline__ Quotient quotient(float scale) {
    return Quotient{scale, 1.0f / scale, (__float_as_uint(scale) & 0x7fffffu) == 0};
}

__device__ __forceinline__ uint32_t encode4(float a, float b, float c, float d) {
    return static_cast<uint32_t>(e4m3x2(a, b)) | static_cast<uint32_t>(e4m3x2(c, d)) << 16;
}

__device__ __forceinline__ uint32_t reencode(uint32_t w, float was, const Quotient& q) {
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
    return encode4(q(f[0] * was), q(f[1] * was), q(f[2] * was), q(f[3] * was));
}

// Whether a run starts at token t: its slot is in the pool and does not continue
// the token before it in one page.
__device__ __forceinline__ bool starts_run(const AppendParams& p, int t, int slot) {
    if (slot < 0 || slot / p.P >= p.pages) return false;
    return t == 0 || slot % p.P == 0 || p.slots[t - 1] != slot - 1;
}

// One run of n tokens from token t on, at `slot`, for one head and side, by a
// group of NT threads (thread `i` of it). smem: NT / 32 x (4 D + 4) bytes, for
// groups wider than a warp.
template <int NT, int D>
__device__ __forceinline__ void write_run(const AppendParams& p, int t, int n, int slot, int head,
                                          int side, int i, uint8_t* smem) {
    constexpr int kCols = D / 8;         // threads of a token
    constexpr int kStep = NT / kCols;    // tokens at once
    const int col = (i % kCols) * 8, t_in = i / kCols;
    const int page = slot / p.P, o = slot - page * p.P;
    const uint16_t* const x = p.x[side] + static_cast<int64_t>(t) * p.x_stride[side] + head * D + col;
    const int64_t at = static_cast<int64_t>(page) * p.heads + head;
    float* const scale = p.scale[side] + at;
    const float old = o > 0 ? *scale : __uint_as_float(static_cast<uint32_t>(kMinExponent + 127) << 23);
    const bool keep_bounds = side == 0 && p.bounds != nullptr;

    uint32_t hi[4], lo[4], big = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        hi[j] = 0xff80ff80u;  // -infinity
        lo[j] = 0x7f807f80u;
    }
#pragma unroll 4
    for (int m = t_in; m < n; m += kStep) {
        const uint4 v = *reinterpret_cast<const uint4*>(x + m * p.x_stride[side]);
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            hi[j] = bmax2(hi[j], w[j]);
            lo[j] = bmin2(lo[j], w[j]);
            big = bmax2(big, w[j] & 0x7fff7fffu);
        }
    }
    float a = fmaxf(lo_f(finite2(big)), hi_f(finite2(big)));
    a = warp_max(a);
    if (keep_bounds) {
#pragma unroll
        for (int s = kCols; s < 32; s <<= 1)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                hi[j] = bmax2(hi[j], __shfl_xor_sync(0xffffffffu, hi[j], s));
                lo[j] = bmin2(lo[j], __shfl_xor_sync(0xffffffffu, lo[j], s));
            }
    }
    bool writes_bounds = keep_bounds && i < kCols;
    if (NT > 32) {
        constexpr int kWarps = NT / 32;
        uint4* const s_hi = reinterpret_cast<uint4*>(smem);
        uint4* const s_lo = s_hi + kWarps * kCols;
        float* const s_a = reinterpret_cast<float*>(s_lo + kWarps * kCols);
        const int warp = i >> 5, lane = i & 31;
        if (keep_bounds && lane < kCols) {
            s_hi[warp * kCols + lane] = make_uint4(hi[0], hi[1], hi[2], hi[3]);
            s_lo[warp * kCols + lane] = make_uint4(lo[0], lo[1], lo[2], lo[3]);
        }
        if (lane == 0) s_a[warp] = a;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < kWarps; ++w) a = fmaxf(a, s_a[w]);
        if (writes_bounds)
            for (int w = 1; w < kWarps; ++w) {
                const uint4 h = s_hi[w * kCols + i], l = s_lo[w * kCols + i];
                hi[0] = bmax2(hi[0], h.x), hi[1] = bmax2(hi[1], h.y);
                hi[2] = bmax2(hi[2], h.z), hi[3] = bmax2(hi[3], h.w);
                lo[0] = bmin2(lo[0], l.x), lo[1] = bmin2(lo[1], l.y);
                lo[2] = bmin2(lo[2], l.z), lo[3] = bmin2(lo[3], l.w);
            }
    }
    if (writes_bounds) {
        uint4* const b = reinterpret_cast<uint4*>(p.bounds + at * 2 * D + col);
        if (o > 0) {
            const uint4 h = b[0], l = b[D / 8];
            hi[0] = bmax2(hi[0], h.x), hi[1] = bmax2(hi[1], h.y);
            hi[2] = bmax2(hi[2], h.z), hi[3] = bmax2(hi[3], h.w);
            lo[0] = bmin2(lo[0], l.x), lo[1] = bmin2(lo[1], l.y);
            lo[2] = bmin2(lo[2], l.z), lo[3] = bmin2(lo[3], l.w);
        }
        b[0] = make_uint4(finite2(hi[0]), finite2(hi[1]), finite2(hi[2]), finite2(hi[3]));
        b[D / 8] = make_uint4(finite2(lo[0]), finite2(lo[1]), finite2(lo[2]), finite2(lo[3]));
    }
    const float now = fmaxf(power_of(a), old);
    // Every thread has read the old scale: the shuffles or the barrier above ordered them.
    if (i == 0) *scale = now;
    const Quotient q = quotient(now);
    uint8_t* const pool = p.pool[side] + page * p.stride[side][0] + head * p.stride[side][1];
    const int64_t ts = p.stride[side][2];
    if (o > 0 && now > old) {
        constexpr int kOldCols = D / 16;
        const int c16 = (i % kOldCols) * 16;
#pragma unroll 2
        for (int m = i / kOldCols; m < o; m += NT / kOldCols) {
            uint4* const w = reinterpret_cast<uint4*>(pool + m * ts + c16);
            uint4 v = *w;
            v.x = reencode(v.x, old, q);
            v.y = reencode(v.y, old, q);
            v.z = reencode(v.z, old, q);
            v.w = reencode(v.w, old, q);
            *w = v;
        }
    }
#pragma unroll 4
    for (int m = t_in; m < n; m += kStep) {
        const uint4 v = *reinterpret_cast<const uint4*>(x + m * p.x_stride[side]);
        *reinterpret_cast<uint2*>(pool + (o + m) * ts + col) =
            make_uint2(encode4(q(lo_f(v.x)), q(hi_f(v.x)), q(lo_f(v.y)), q(hi_f(v.y))),
                       encode4(q(lo_f(v.z)), q(hi_f(v.z)), q(lo_f(v.w)), q(hi_f(v.w))));
    }
}

constexpr int kWarpsPerBlock = 4;

// A warp for each (token, head, side); those whose token starts no run leave.
template <int D>
__global__ void __launch_bounds__(32 * kWarpsPerBlock) append_warp_kernel(const AppendParams p) {
    pdl_entry();
    const int lane = threadIdx.x & 31;
    const int64_t unit = static_cast<int64_t>(blockIdx.x) * kWarpsPerBlock + (threadIdx.x >> 5);
    const int t = static_cast<int>(unit / (2 * p.heads)), hs = static_cast<int>(unit % (2 * p.heads));
    if (t >= p.T) return;
    const int slot = p.slots[t];
    if (!starts_run(p, t, slot)) return;
    // Tokens that continue it, up to the page's end (P <= 256: eight at most).
    const int most = min(p.P - slot % p.P, p.T - t);
    int n = 1;
    while (n < most) {
        const int m = n + lane;
        const bool on = m < most && p.slots[t + m] == slot + m;
        const unsigned ballot = __ballot_sync(0xffffffffu, on);
        const int c = ballot == 0xffffffffu ? 32 : __ffs(~ballot) - 1;
        n += c;
        if (c < 32) break;
    }
    write_run<32, D>(p, t, n, slot, hs >> 1, hs & 1, lane, nullptr);
}

constexpr int kBlock = 256;

// A block for each chunk of tokens, head and side: it takes the runs that start
// in its chunk, one after another.
template <int D>
__global__ void __launch_bounds__(kBlock) append_block_kernel(const AppendParams p) {
    __shared__ __align__(16) uint8_t smem[kBlock / 32 * (4 * D + 4)];
    __shared__ int s_slot[512 + 1];
    pdl_entry();
    const int tid = threadIdx.x, head = blockIdx.y, side = blockIdx.z;
    const int64_t t0 = static_cast<int64_t>(blockIdx.x) * p.chunk;
    const int span = static_cast<int>(min(static_cast<int64_t>(p.T) - t0, static_cast<int64_t>(p.chunk)));
    const int seen = static_cast<int>(min(static_cast<int64_t>(p.T) - t0, static_cast<int64_t>(p.chunk) + p.P));
    // s_slot[j + 1]: the slot of token t0 + j; a run of this chunk may go on into the next.
    for (int j = tid; j <= seen; j += kBlock) s_slot[j] = t0 + j > 0 ? p.slots[t0 + j - 1] : -2;
    __syncthreads();
    int j = 0;
    while (j < span) {
        const int slot = s_slot[j + 1];
        if (slot < 0 || slot / p.P >= p.pages || (slot % p.P != 0 && s_slot[j] == slot - 1)) {
            ++j;
            continue;
        }
        const int most = min(p.P - slot % p.P, seen - j);
        int n = 1;
        while (n < most && s_slot[j + 1 + n] == slot + n) ++n;
        write_run<kBlock, D>(p, static_cast<int>(t0) + j, n, slot, head, side, tid, smem);
        __syncthreads();
        j += n;
    }
}

template <int D>
int launch_append(const AppendParams& p, int sms, smd_stream_t stream) {
    // Few tokens: a warp each. Many: blocks by chunks of about a page.
    const int64_t units = static_cast<int64_t>(p.T) * p.heads * 2;
    if (units <= static_cast<int64_t>(sms) * 256)
        return launch_pdl(append_warp_kernel<D>,
                          dim3(static_cast<unsigned>((units + kWarpsPerBlock - 1) / kWarpsPerBlock)),
                          32 * kWarpsPerBlock, 0, stream, p);
    return launch_pdl(append_block_kernel<D>,
                      dim3(static_cast<unsigned>((p.T + p.chunk - 1) / p.chunk),
                           static_cast<unsigned>(p.heads), 2),
                      kBlock, 0, stream, p);
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
    p.chunk = cache->page_size < 64 ? 64 : cache->page_size;
    return cache->head_dim == 64    ? launch_append<64>(p, sms, stream)
           : cache->head_dim == 128 ? launch_append<128>(p, sms, stream)
                                    : launch_append<256>(p, sms, stream);
}

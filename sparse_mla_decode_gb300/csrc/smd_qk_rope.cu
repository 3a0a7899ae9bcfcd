// The norm of query and key heads and the position rotation in one pass (smd_qk_norm_rope).
//
//   y = x w / sqrt(mean x^2 + eps),  (y_u, y_v) -> (y_u cos - y_v sin, y_u sin + y_v cos)
// with the angle of pair j at a token the sum over axes of position times frequency.
//
// Angles. A position up to 2^31 times a frequency has to be known modulo a turn. Frequencies
// are turned into turns a position in 64-bit fixed point (2^64 is a turn): an integer
// product with the first 64 bits of 1 / (2 pi); the product with a position then wraps as the
// angle does, in integer arithmetic, and the axes' products are added the same way. No fp64
// (a few lanes an SM on this GPU), no reduction of large arguments.
//
// What bounds it: 2 D bytes read and 2 D written for each token and head: HBM for
// prompts; launch and two round trips (position and frequency, beside the values) for a step.
//
// D / 16 lanes hold a head of a token, 16 columns each: chunks c and c + rot / 16 of 8
// columns, so that both columns of a pair are in one lane in either order of pairs, and loads
// and stores are 16 bytes. A block takes a few tokens: its threads compute a sine and cosine
// each, into shared memory; a group of lanes then keeps those of its token in
// registers over its heads, three heads on their way at a time. Weights are in shared memory too, in fp32.
//
// Measured (GB300, device time): 28 thousand tokens, 64 + 8 heads of 128 columns, three axes 165 us, 93% of the
// copy rate (159 without norm; 256 columns 92%, 64 89%, 16 of 128 columns turning 89%); 1000 tokens 8.4
// (66%: start); 96 tokens 3.3; 28 thousand tokens of 5 heads 28 (38%: angles and the phases around them). With 80 registers a thread
// the kernel spills and takes 204.
#include "smd_internal.h"
#include "smd_paged.h"
#include "smd_ptx.cuh"

namespace smd {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxAxes = 4;

struct RopeParams {
    const uint16_t* x[2];  // queries, keys
    int64_t x_stride[2];
    uint16_t* y[2];
    int64_t y_stride[2];
    const uint16_t* w[2];
    int32_t T, Hq, H;      // tokens, query heads, heads in all
    const int32_t* positions;
    int64_t positions_stride;
    int32_t axes;
    const float* freqs;
    int32_t rot;
    float eps;
    int32_t slices;        // blocks that share a token's heads
};

// A frequency (radians) as turns in units of 2^-64; 0 beyond 1024 and for what is not finite.
__device__ __forceinline__ uint64_t turns(float f) {
    constexpr uint64_t kInv2Pi = 0x28be60db9391054aull;  // floor(2^64 / (2 pi))
    const uint32_t u = __float_as_uint(f), e = (u >> 23) & 255u;
    if (!(fabsf(f) <= 1024.0f) || e == 0) return 0;
    const uint64_t m = (u & 0x7fffffu) | 0x800000u;  // f = m 2^(e - 150)
    const uint64_t hi = __umul64hi(m, kInv2Pi), lo = m * kInv2Pi;
    const uint32_t shift = 150u - e;  // 13 at least
    const uint64_t t = shift < 64 ? hi << (64 - shift) | lo >> shift : shift < 128 ? hi >> (shift - 64) : 0;
    return (u >> 31) != 0 ? 0 - t : t;
}

// Two fp32 values in a register pair, and operations on both.
__device__ __forceinline__ uint64_t pack2(float a, float b) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ void unpack2(uint64_t v, float& a, float& b) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

__device__ __forceinline__ float lo_f(uint32_t v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ float hi_f(uint32_t v) { return __uint_as_float(v & 0xffff0000u); }

// A lane's 16 columns as the first and second columns of 8 pairs that turn together: chunk 0 with
// chunk 1, or (kInter) even columns with odd ones.
template <bool kInter>
__device__ __forceinline__ void widen(const uint4& c0, const uint4& c1, uint64_t (&x)[4], uint64_t (&y)[4]) {
    const uint32_t a[4] = {c0.x, c0.y, c0.z, c0.w}, b[4] = {c1.x, c1.y, c1.z, c1.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        if (kInter) {
            const uint32_t u = j < 2 ? a[2 * j] : b[2 * j - 4], v = j < 2 ? a[2 * j + 1] : b[2 * j - 3];
            x[j] = pack2(lo_f(u), lo_f(v));
            y[j] = pack2(hi_f(u), hi_f(v));
        } else {
            x[j] = pack2(lo_f(a[j]), hi_f(a[j]));
            y[j] = pack2(lo_f(b[j]), hi_f(b[j]));
        }
    }
}

template <bool kInter>
__device__ __forceinline__ void narrow(const uint64_t (&x)[4], const uint64_t (&y)[4], uint4& c0, uint4& c1) {
    uint32_t a[4], b[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        float x0, x1, y0, y1;
        unpack2(x[j], x0, x1);
        unpack2(y[j], y0, y1);
        if (kInter) {
            (j < 2 ? a[2 * j] : b[2 * j - 4]) = bf16x2(x0, y0);
            (j < 2 ? a[2 * j + 1] : b[2 * j - 3]) = bf16x2(x1, y1);
        } else {
            a[j] = bf16x2(x0, x1);
            b[j] = bf16x2(y0, y1);
        }
    }
    c0 = make_uint4(a[0], a[1], a[2], a[3]);
    c1 = make_uint4(b[0], b[1], b[2], b[3]);
}

// TB tokens of a block; kInter: pairs (2 j, 2 j + 1); kNorm: a weight is given.
template <int D, int TB, bool kInter, bool kNorm>
__global__ void __launch_bounds__(kThreads, TB == 512 / D ? 2 : 3) qk_rope_kernel(const RopeParams p) {
    constexpr int kAtOnce = TB == 512 / D ? 3 : 1;          // heads of a group in flight
    constexpr int N = D / 16, kGroups = kThreads / N / TB;  // lanes of a head; groups of a token
    static_assert(kGroups >= 1, "a group for each token");
    __shared__ uint64_t s_freq[kMaxAxes][D / 2];
    __shared__ __align__(16) float s_cos[TB][D / 2], s_sin[TB][D / 2], s_w[2][kNorm ? D : 4];  // [2][D / 8] four columns
    const int tid = threadIdx.x, half = p.rot / 2, turning = p.rot / 16;
    pdl_entry();
    for (int i = tid; i < p.axes * half; i += kThreads) s_freq[i / half][i % half] = turns(__ldg(p.freqs + i));
    if (kNorm)  // in the order of widen(): the first four columns of each chunk, then the others
        for (int u = tid; u < 2 * D; u += kThreads) {
            const int side = u / D, c = u % D, k = kInter ? (c & 1) * 4 + (c & 7) / 2 : c & 7;
            s_w[side][(k >> 2) * (D / 2) + c / 8 * 4 + (k & 3)] =
                p.w[side] == nullptr ? 1.0f : lo_f(__ldg(p.w[side] + c));
        }
    const bool normed[2] = {p.w[0] != nullptr, p.w[1] != nullptr};
    const int i = tid % N, group = tid / N, tl = group / kGroups, g = group % kGroups;
    // The lane's chunks of 8 columns.
    const bool turns_here = i < turning;
    const int c0 = turns_here ? i : i + turning, c1 = turns_here ? i + turning : i + N;
    const int slice = static_cast<int>(blockIdx.x) % p.slices, step = kGroups * p.slices;
    const int chunks = (p.T + TB - 1) / TB, stride = static_cast<int>(gridDim.x) / p.slices;
    const unsigned mask = N == 32 ? 0xffffffffu : ((1u << N) - 1u) << ((tid & 31) / N * N);
#pragma unroll 1
    for (int chunk = static_cast<int>(blockIdx.x) / p.slices; chunk < chunks; chunk += stride) {
        const int t0 = chunk * TB, t = t0 + tl;
        const bool live = t < p.T && (p.positions == nullptr || __ldg(p.positions + t) >= 0);
        uint4 v[kAtOnce][2] = {};
        const auto load = [&](int h0) {
#pragma unroll
            for (int j = 0; j < kAtOnce; ++j) {
                const int h = h0 + j * step, side = h >= p.Hq ? 1 : 0;
                if (live && h < p.H) {
                    const uint4* const x = reinterpret_cast<const uint4*>(
                        p.x[side] + t * p.x_stride[side] + static_cast<int64_t>(h - side * p.Hq) * D);
                    v[j][0] = __ldcs(x + c0);
                    v[j][1] = __ldcs(x + c1);
                }
            }
        };
        int h0 = slice * kGroups + g;
        load(h0);
        __syncthreads();  // the frequencies are there; the last chunk's angles have been read
        for (int u = tid; u < TB * half; u += kThreads) {
            const int tt = u / half, j = u % half;
            if (t0 + tt >= p.T) break;
            uint64_t phase = 0;
            for (int a = 0; a < p.axes; ++a)
                phase += static_cast<uint64_t>(static_cast<int64_t>(
                             __ldg(p.positions + a * p.positions_stride + t0 + tt))) * s_freq[a][j];
            // Half turns in [-1, 1).
            const float x = static_cast<float>(static_cast<int32_t>(phase >> 32)) * 4.656612873077393e-10f;
            sincospif(x, &s_sin[tt][j], &s_cos[tt][j]);
        }
        __syncthreads();
        if (!live) continue;
        // Pairs of the lane: 8 i .. 8 i + 7; interleaved: 4 c0 .., 4 c1 ..
        uint64_t cs[4], sn[4];
#pragma unroll
        for (int z = 0; z < 2; ++z) {
            const int at = !turns_here ? 0 : kInter ? 4 * (z == 0 ? c0 : c1) : 8 * i + 4 * z;
            const float4 c = *reinterpret_cast<const float4*>(&s_cos[tl][at]);
            const float4 s = *reinterpret_cast<const float4*>(&s_sin[tl][at]);
            cs[2 * z] = pack2(c.x, c.y), cs[2 * z + 1] = pack2(c.z, c.w);
            sn[2 * z] = pack2(s.x, s.y), sn[2 * z + 1] = pack2(s.z, s.w);
        }
#pragma unroll 1
        while (h0 < p.H) {
            uint64_t x[kAtOnce][4], y[kAtOnce][4];
#pragma unroll
            for (int j = 0; j < kAtOnce; ++j) widen<kInter>(v[j][0], v[j][1], x[j], y[j]);
            const int h1 = h0;
            h0 += kAtOnce * step;
            load(h0);
            if (kNorm) {
                float sum[kAtOnce];
#pragma unroll
                for (int j = 0; j < kAtOnce; ++j) {
                    uint64_t s = mul2(x[j][0], x[j][0]);
#pragma unroll
                    for (int z = 1; z < 4; ++z) s = fma2(x[j][z], x[j][z], s);
#pragma unroll
                    for (int z = 0; z < 4; ++z) s = fma2(y[j][z], y[j][z], s);
                    float a, b;
                    unpack2(s, a, b);
                    sum[j] = a + b;
                }
#pragma unroll
                for (int o = 1; o < N; o <<= 1)
#pragma unroll
                    for (int j = 0; j < kAtOnce; ++j) sum[j] += __shfl_xor_sync(mask, sum[j], o);
#pragma unroll
                for (int j = 0; j < kAtOnce; ++j) {
                    const int side = h1 + j * step >= p.Hq ? 1 : 0;
                    const float r = normed[side] ? rsqrtf(fmaf(sum[j], 1.0f / D, p.eps)) : 1.0f;
                    const uint64_t rr = pack2(r, r);
#pragma unroll
                    for (int z = 0; z < 4; ++z) {
                        // Four weights: pairs 2 (z & 1) and the next of x or y, out of chunk 0 or 1.
                        const bool of_y = kInter ? (z & 1) != 0 : z >= 2;
                        const int first = kInter ? 2 * (z >> 1) : 2 * (z & 1);
                        const int at = (z & 1) * (D / 2) + 4 * (z < 2 ? c0 : c1);
                        const float4 w = *reinterpret_cast<const float4*>(&s_w[side][at]);
                        uint64_t (&to)[4] = of_y ? y[j] : x[j];
                        to[first] = mul2(mul2(to[first], rr), pack2(w.x, w.y));
                        to[first + 1] = mul2(mul2(to[first + 1], rr), pack2(w.z, w.w));
                    }
                }
            }
#pragma unroll
            for (int j = 0; j < kAtOnce; ++j) {
                const int h = h1 + j * step, side = h >= p.Hq ? 1 : 0;
                if (turns_here) {
#pragma unroll
                    for (int z = 0; z < 4; ++z) {
                        const uint64_t u = mul2(y[j][z], sn[z]), w = mul2(y[j][z], cs[z]);
                        y[j][z] = fma2(x[j][z], sn[z], w);
                        x[j][z] = fma2(x[j][z], cs[z], u ^ 0x8000000080000000ull);
                    }
                }
                if (h < p.H) {
                    uint4* const out = reinterpret_cast<uint4*>(
                        p.y[side] + t * p.y_stride[side] + static_cast<int64_t>(h - side * p.Hq) * D);
                    uint4 o0, o1;
                    narrow<kInter>(x[j], y[j], o0, o1);
                    out[c0] = o0;
                    out[c1] = o1;
                }
            }
        }
    }
}

template <int D, int TB>
int launch_rope(RopeParams p, bool inter, int sms, smd_stream_t stream) {
    if (TB > 1) {
        p.slices = 1;
    } else {  // heads over blocks while SMs are idle
        constexpr int kUnits = kThreads / (D / 16);
        const int most = (p.H + kUnits - 1) / kUnits, want = 2 * sms / p.T;
        p.slices = want < 1 ? 1 : want < most ? want : most;
    }
    const int64_t chunks = (p.T + TB - 1) / TB, most = static_cast<int64_t>(sms) * 6 / p.slices;
    const unsigned grid = static_cast<unsigned>((chunks < most ? chunks : most) * p.slices);
    const bool norm = p.w[0] != nullptr || p.w[1] != nullptr;
    auto kernel = norm ? (inter ? qk_rope_kernel<D, TB, true, true> : qk_rope_kernel<D, TB, false, true>)
                       : (inter ? qk_rope_kernel<D, TB, true, false> : qk_rope_kernel<D, TB, false, false>);
    return launch_pdl(kernel, dim3(grid), kThreads, 0, stream, p);
}

template <int D>
int launch_rope(const RopeParams& p, bool inter, int sms, smd_stream_t stream) {
    constexpr int kMany = 512 / D;  // tokens whose angles are one a thread
    // Tokens of a block: one while SMs would idle, and, for few heads, four times as many once there are
    // enough for all SMs (the angles are most of the work then). 128 columns, 1 / kMany / 4 kMany in us:
    //   72 heads, 300 / 600 / 14000 tokens     4.4 / 5.1 / 18.8     7.0 / 6.3 / 23.1     104 / 81 / 99
    //   24 heads, 300 / 600 / 14000            3.1 / 3.1 /  8.2     4.8 / 3.7 /  8.2      47 / 35 / 37
    //   16 heads, 300 / 600 / 14000            2.7 / 3.1 /  6.4     4.4 / 3.6 /  6.4      41 / 31 / 27
    //    5 heads, 300 / 2000 / 14000           2.6 / 2.9 /  4.2     7.1 / 6.0 /  5.3      35 / 27 / 12
    if (p.T < 2 * sms) return launch_rope<D, 1>(p, inter, sms, stream);
    return p.H >= 20 || p.T < 8 * kMany * sms ? launch_rope<D, kMany>(p, inter, sms, stream)
                                              : launch_rope<D, 4 * kMany>(p, inter, sms, stream);
}

}  // namespace
}  // namespace smd

extern "C" int smd_qk_norm_rope(const uint16_t* q, int64_t q_stride, const uint16_t* k, int64_t k_stride,
                                int32_t T, int32_t Hq, int32_t Hk, int32_t head_dim,
                                const int32_t* positions, int64_t positions_stride, int32_t axes,
                                const float* freqs, int32_t rot, int32_t interleaved,
                                const uint16_t* q_weight, const uint16_t* k_weight, float eps,
                                uint16_t* q_out, int64_t q_out_stride, uint16_t* k_out,
                                int64_t k_out_stride, smd_stream_t stream) {
    using namespace smd;
    const int64_t q_row = static_cast<int64_t>(Hq) * head_dim, k_row = static_cast<int64_t>(Hk) * head_dim;
    if (T < 0 || T >= (1 << 30) || (head_dim != 64 && head_dim != 128 && head_dim != 256) || Hq < 1 || Hk < 0 ||
        static_cast<int64_t>(Hq) + Hk > 65535 || rot < 0 || rot > head_dim || rot % 16 != 0 || axes < 1 ||
        axes > kMaxAxes || !(eps >= 0.0f) || eps > 3.402823466e38f || q_stride < q_row ||
        q_out_stride < q_row || q_stride % 8 != 0 || q_out_stride % 8 != 0 ||
        (Hk > 0 && (k_stride < k_row || k_out_stride < k_row || k_stride % 8 != 0 || k_out_stride % 8 != 0)) ||
        (positions != nullptr && positions_stride < T))
        return SMD_ERR_SHAPE;
    if (T == 0) return SMD_OK;
    if (q == nullptr || q_out == nullptr || (Hk > 0 && (k == nullptr || k_out == nullptr)) ||
        (rot > 0 && (positions == nullptr || freqs == nullptr)))
        return SMD_ERR_NULL;
    for (const void* a : {static_cast<const void*>(q), static_cast<const void*>(k),
                          static_cast<const void*>(q_out), static_cast<const void*>(k_out),
                          static_cast<const void*>(q_weight), static_cast<const void*>(k_weight)})
        if (!aligned(a, 16)) return SMD_ERR_ALIGN;
    if (!aligned(positions, 4) || !aligned(freqs, 4)) return SMD_ERR_ALIGN;
    const int sms = device_sms();
    if (sms <= 0) return SMD_ERR_DEVICE;
    RopeParams p{};
    p.x[0] = q;
    p.x[1] = k;
    p.x_stride[0] = q_stride;
    p.x_stride[1] = k_stride;
    p.y[0] = q_out;
    p.y[1] = k_out;
    p.y_stride[0] = q_out_stride;
    p.y_stride[1] = k_out_stride;
    p.w[0] = q_weight;
    p.w[1] = k_weight;
    p.T = T;
    p.Hq = Hq;
    p.H = Hq + Hk;
    p.positions = positions;
    p.positions_stride = positions_stride;
    p.axes = axes;
    p.freqs = freqs;
    p.rot = rot;
    p.eps = eps;
    return head_dim == 64    ? launch_rope<64>(p, interleaved != 0, sms, stream)
           : head_dim == 128 ? launch_rope<128>(p, interleaved != 0, sms, stream)
                             : launch_rope<256>(p, interleaved != 0, sms, stream);
}

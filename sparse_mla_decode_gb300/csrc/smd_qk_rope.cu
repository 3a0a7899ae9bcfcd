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
// registers over its heads.
#include "smd_internal.h"
#include "smd_paged.h"
#include "smd_ptx.cuh"

namespace smd {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxAxes = 4;
constexpr int kAtOnce = 3;  // heads of a group in flight

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

__device__ __forceinline__ float lo_f(uint32_t v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ float hi_f(uint32_t v) { return __uint_as_float(v & 0xffff0000u); }

__device__ __forceinline__ void widen(const uint4& v, float* f) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        f[2 * j] = lo_f(w[j]);
        f[2 * j + 1] = hi_f(w[j]);
    }
}

__device__ __forceinline__ uint4 narrow(const float* f) {
    return make_uint4(bf16x2(f[0], f[1]), bf16x2(f[2], f[3]), bf16x2(f[4], f[5]), bf16x2(f[6], f[7]));
}

// TB tokens of a block; kInter: pairs (2 j, 2 j + 1).
template <int D, int TB, bool kInter>
__global__ void __launch_bounds__(kThreads) qk_rope_kernel(const RopeParams p) {
    constexpr int N = D / 16, kGroups = kThreads / N / TB;  // lanes of a head; groups of a token
    __shared__ uint64_t s_freq[kMaxAxes][D / 2];
    __shared__ __align__(16) float s_cos[TB][D / 2], s_sin[TB][D / 2];
    const int tid = threadIdx.x, half = p.rot / 2, turning = p.rot / 16;
    pdl_entry();
    for (int i = tid; i < p.axes * half; i += kThreads) s_freq[i / half][i % half] = turns(__ldg(p.freqs + i));
    const int i = tid % N, group = tid / N, tl = group / kGroups, g = group % kGroups;
    // The lane's chunks of 8 columns.
    const bool turns_here = i < turning;
    const int c0 = turns_here ? i : 2 * i, c1 = turns_here ? i + turning : 2 * i + 1;
    const int slice = static_cast<int>(blockIdx.x) % p.slices, step = kGroups * p.slices;
    const int chunks = (p.T + TB - 1) / TB, stride = static_cast<int>(gridDim.x) / p.slices;
#pragma unroll 1
    for (int chunk = static_cast<int>(blockIdx.x) / p.slices; chunk < chunks; chunk += stride) {
        const int t0 = chunk * TB, t = t0 + tl;
        const bool live = t < p.T && (p.positions == nullptr || __ldg(p.positions + t) >= 0);
        const auto row = [&](int h) {  // a head's first column
            const int side = h >= p.Hq ? 1 : 0;
            return p.x[side] + t * p.x_stride[side] + static_cast<int64_t>(h - side * p.Hq) * D;
        };
        uint4 v[kAtOnce][2];
        const auto load = [&](int h0) {
#pragma unroll
            for (int j = 0; j < kAtOnce; ++j) {
                const int h = h0 + j * step;
                if (live && h < p.H) {
                    const uint4* const x = reinterpret_cast<const uint4*>(row(h));
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
        if (live) {
            // Pairs of the lane: 8 i .. 8 i + 7; interleaved: 4 c0 .., 4 c1 ..
            float cs[8], sn[8];
            if (turns_here) {
#pragma unroll
                for (int z = 0; z < 2; ++z) {
                    const int at = kInter ? 4 * (z == 0 ? c0 : c1) : 8 * i + 4 * z;
                    const float4 c = *reinterpret_cast<const float4*>(&s_cos[tl][at]);
                    const float4 s = *reinterpret_cast<const float4*>(&s_sin[tl][at]);
                    cs[4 * z] = c.x, cs[4 * z + 1] = c.y, cs[4 * z + 2] = c.z, cs[4 * z + 3] = c.w;
                    sn[4 * z] = s.x, sn[4 * z + 1] = s.y, sn[4 * z + 2] = s.z, sn[4 * z + 3] = s.w;
                }
            }
            uint4 w[2];
            int w_side = -1;
            const unsigned mask = N == 32 ? 0xffffffffu : ((1u << N) - 1u) << ((tid & 31) / N * N);
#pragma unroll 1
            while (h0 < p.H) {
#pragma unroll
                for (int j = 0; j < kAtOnce; ++j) {
                    const int h = h0 + j * step;
                    if (h >= p.H) break;  // the same in a head's lanes
                    const int side = h >= p.Hq ? 1 : 0;
                    float f[16];
                    widen(v[j][0], f);
                    widen(v[j][1], f + 8);
                    if (p.w[side] != nullptr) {
                        if (w_side != side) {
                            const uint4* const at = reinterpret_cast<const uint4*>(p.w[side]);
                            w[0] = __ldg(at + c0);
                            w[1] = __ldg(at + c1);
                            w_side = side;
                        }
                        float sum = 0.0f;
#pragma unroll
                        for (int z = 0; z < 16; ++z) sum = fmaf(f[z], f[z], sum);
#pragma unroll
                        for (int s = 1; s < N; s <<= 1) sum += __shfl_xor_sync(mask, sum, s);
                        const float r = rsqrtf(fmaf(sum, 1.0f / D, p.eps));
                        float by[16];
                        widen(w[0], by);
                        widen(w[1], by + 8);
#pragma unroll
                        for (int z = 0; z < 16; ++z) f[z] *= r * by[z];
                    }
                    if (turns_here) {
#pragma unroll
                        for (int z = 0; z < 8; ++z) {
                            const int a = kInter ? 2 * z : z, b = kInter ? 2 * z + 1 : z + 8;
                            const float x = f[a], y = f[b];
                            f[a] = fmaf(x, cs[z], -y * sn[z]);
                            f[b] = fmaf(x, sn[z], y * cs[z]);
                        }
                    }
                    uint4* const out = reinterpret_cast<uint4*>(
                        p.y[side] + t * p.y_stride[side] + static_cast<int64_t>(h - side * p.Hq) * D);
                    out[c0] = narrow(f);
                    out[c1] = narrow(f + 8);
                }
                h0 += kAtOnce * step;
                load(h0);
            }
        }
    }
}

template <int D>
int launch_rope(RopeParams p, bool inter, int sms, smd_stream_t stream) {
    constexpr int kMany = 512 / D;  // tokens of a block whose angles are one a thread
    const bool many = p.T >= 2 * sms * kMany;
    const int groups = kThreads / (D / 16);
    if (many) {
        p.slices = 1;
    } else {  // heads over blocks while SMs are idle
        const int most = (p.H + groups - 1) / groups, want = 2 * sms / p.T;
        p.slices = want < 1 ? 1 : want < most ? want : most;
    }
    const int64_t chunks = many ? (p.T + kMany - 1) / kMany : p.T;
    const int64_t most = static_cast<int64_t>(sms) * 8 / p.slices;
    const unsigned grid = static_cast<unsigned>((chunks < most ? chunks : most) * p.slices);
    auto kernel = many ? (inter ? qk_rope_kernel<D, kMany, true> : qk_rope_kernel<D, kMany, false>)
                       : (inter ? qk_rope_kernel<D, 1, true> : qk_rope_kernel<D, 1, false>);
    return launch_pdl(kernel, dim3(grid), kThreads, 0, stream, p);
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

// Which drafted tokens stay, and the token after them (smd_verify_drafts).
//
//   d_i stays while u_i q_i(d_i) < p_i(d_i); then the first v at which the sum of
//   w = floor(2^40 max(p - q, 0)) exceeds floor(U sum w / 2^31)
// The products of the test are exact in fp64 (24 bits times 24). The weights are whole
// numbers, so sums over threads, warps and CTAs give the same token in any order: among 10^5
// borders a sum in fp32 would put some draws on the other side.
//
// What bounds it: one row of p and one of q are read for each request, HBM for a
// batch; for one request the latency of the chain: drafted tokens, their probabilities,
// the row, the sums of the others, the place.
//
// A cluster of CTAs takes a request, each a contiguous part of the vocabulary and each warp a
// contiguous part of that. Every CTA finds the row for itself, sums its part and writes the sum
// into its peers' shared memory; after one cluster barrier each knows whether the
// draw falls into its part. The one where it does looks again at the part of the warp
// that holds it (from L2), a few entries a thread.
//
// floor(2^40 x) of x in [0, 1] without conversions: x 2^22 + 2^23, rounded towards zero,
// holds floor(x 2^22) in its last bits; the remainder (exact) times 2^18 gives the rest the
// same way. Both are added up in 32 bits over a few hundred entries, then in 64.
//
// Measured (GB300, device time): 96 requests of 131072 entries with drafts' distributions 19.5 us, 77% of the
// copy rate (65536 entries of 512 requests: 97%): start, drafted tokens and their probabilities are 3
// us, the place at the end 2. One request of 100003 entries 6.7 us (rows off 16 bytes: loads of 4 bytes, 12 in
// flight; 8: 9.2; 100000 entries 5.8).
#include "smd_internal.h"
#include "smd_paged.h"
#include "smd_ptx.cuh"

namespace smd {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kMaxDrafts = 63;
constexpr int kMaxCluster = 8;
constexpr int kMaxVocab = 1 << 22;

struct VerifyParams {
    const float* target;
    int64_t target_stride;
    const float* draft;
    int64_t draft_stride;
    const int32_t* tokens;
    const float* accept;
    const float* sample;
    int32_t R, G, V;
    int32_t part;       // entries of a CTA, a multiple of kWarps * 128
    int32_t* out_tokens;
    int32_t* accepted;
    int32_t* rejected;
};

// Entries of a row taken in: sums of floor(x 2^22) and of the 18 bits below, as added bits.
struct Share {
    uint32_t hi = 0, lo = 0;
    uint64_t sum = 0;  // in units of 2^-40

    __device__ __forceinline__ void add(float x) {  // x within [0, 1]
        constexpr uint32_t kBias = 0x4b000000u;  // of 2^23
        const float a = __fmaf_rz(x, 4194304.0f, 8388608.0f);
        const float rest = fmaf(x, 4194304.0f, -(a - 8388608.0f));
        hi += __float_as_uint(a) - kBias;
        lo += __float_as_uint(__fmaf_rz(rest, 262144.0f, 8388608.0f)) - kBias;
    }
    // At least every 1023 entries.
    __device__ __forceinline__ void flush() {
        sum += (static_cast<uint64_t>(hi) << 18) + lo;
        hi = lo = 0;
    }
};

// A row of weights: max(p - q, 0) within [0, 1], NaN as 0 (q NULL: p), and nothing at `gone`.
struct Row {
    const float* p;
    const float* q;
    int gone;
    __device__ __forceinline__ float at(int v) const {
        const float x = __saturatef(q != nullptr ? __ldg(p + v) - __ldg(q + v) : __ldg(p + v));
        return v == gone ? 0.0f : x;
    }
};

__device__ __forceinline__ uint64_t warp_sum(uint64_t v) {
#pragma unroll
    for (int s = 16; s > 0; s >>= 1) v += __shfl_xor_sync(0xffffffffu, v, s);
    return v;
}

// Sum of the row's entries [v0, v1) by a warp, the same in every lane. kWide: 16-byte loads
// (v0 a multiple of 4, rows 16-byte aligned).
template <bool kWide>
__device__ __forceinline__ uint64_t sum_part(const Row& row, int v0, int v1, int lane) {
    constexpr int kAtOnce = kWide ? 4 : 12;
    Share s;
    if constexpr (kWide) {
#pragma unroll 1
        for (int v = v0 + 4 * lane; v < v1; v += 128 * kAtOnce) {
            float4 p[kAtOnce], q[kAtOnce];
#pragma unroll
            for (int j = 0; j < kAtOnce; ++j) {
                const int at = v + 128 * j;
                p[j] = q[j] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                if (at + 3 < v1) {
                    p[j] = __ldg(reinterpret_cast<const float4*>(row.p + at));
                    if (row.q != nullptr) q[j] = __ldg(reinterpret_cast<const float4*>(row.q + at));
                } else {
                    if (at < v1) p[j].x = row.at(at);
                    if (at + 1 < v1) p[j].y = row.at(at + 1);
                    if (at + 2 < v1) p[j].z = row.at(at + 2);
                }
            }
#pragma unroll
            for (int j = 0; j < kAtOnce; ++j) {
                const int g = row.gone - (v + 128 * j);
                s.add(g == 0 ? 0.0f : __saturatef(p[j].x - q[j].x));
                s.add(g == 1 ? 0.0f : __saturatef(p[j].y - q[j].y));
                s.add(g == 2 ? 0.0f : __saturatef(p[j].z - q[j].z));
                s.add(g == 3 ? 0.0f : __saturatef(p[j].w - q[j].w));
            }
            s.flush();
        }
    } else {
#pragma unroll 1
        for (int v = v0 + lane; v < v1; v += 32 * kAtOnce) {
            float p[kAtOnce], q[kAtOnce];
#pragma unroll
            for (int j = 0; j < kAtOnce; ++j) {
                const int at = v + 32 * j;
                p[j] = q[j] = 0.0f;
                if (at < v1) {
                    p[j] = __ldg(row.p + at);
                    if (row.q != nullptr) q[j] = __ldg(row.q + at);
                }
            }
#pragma unroll
            for (int j = 0; j < kAtOnce; ++j) s.add(v + 32 * j == row.gone ? 0.0f : __saturatef(p[j] - q[j]));
            s.flush();
        }
    }
    return warp_sum(s.sum);
}

// A word into the same place of a peer CTA's shared memory.
__device__ __forceinline__ void st_peer_u64(uint64_t* at, int rank, uint64_t v) {
    asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(mapa(smem_addr(at), rank)), "l"(v) : "memory");
}

template <bool kWide>
__global__ void __launch_bounds__(kThreads, 5) verify_kernel(const VerifyParams p) {
    __shared__ uint64_t s_warp[kWarps], s_all[kMaxCluster], s_scan[kWarps];
    __shared__ int s_stay, s_refused;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int rank = static_cast<int>(cluster_ctarank()), C = static_cast<int>(gridDim.x);
    const int r = static_cast<int>(blockIdx.y), D = p.G - 1;
    cluster_arrive_relaxed();  // a peer is written to once it runs
    pdl_entry();

    // Drafts of two rounds of 32: the first that does not stay.
    if (warp == 0) {
        int stay = 0, refused = 0;
#pragma unroll 1
        for (int i0 = 0; i0 < D; i0 += 32) {
            const int i = i0 + lane;
            bool ok = false, drafted = false;
            if (i < D) {
                const int64_t at = static_cast<int64_t>(r) * D + i;
                const int d = p.tokens[at];
                drafted = d >= 0 && d < p.V;
                if (drafted) {
                    const float pd = p.target[(static_cast<int64_t>(r) * p.G + i) * p.target_stride + d];
                    const float qd = p.draft != nullptr ? p.draft[at * p.draft_stride + d] : 1.0f;
                    ok = static_cast<double>(p.accept[at]) * static_cast<double>(qd) < static_cast<double>(pd);
                }
            }
            const uint32_t out = ~__ballot_sync(0xffffffffu, ok), given = __ballot_sync(0xffffffffu, drafted);
            const int first = out == 0 ? 32 : __ffs(out) - 1;
            stay = i0 + first;
            refused = first < 32 && (given >> first & 1u) != 0;
            if (first < 32) break;
        }
        if (lane == 0) {
            s_stay = min(stay, D);
            s_refused = refused;
        }
    }
    __syncthreads();
    const int stay = s_stay;
    const bool refused = s_refused != 0;
    if (rank == 0) {
        const int64_t at = static_cast<int64_t>(r) * p.G;
        for (int i = tid; i < p.G; i += kThreads)
            if (i != stay) p.out_tokens[at + i] = i < stay ? p.tokens[static_cast<int64_t>(r) * D + i] : -1;
        if (tid == 0) {
            if (p.accepted != nullptr) p.accepted[r] = stay;
            if (p.rejected != nullptr) p.rejected[r] = D - stay;
        }
    }
    Row row;
    row.p = p.target + (static_cast<int64_t>(r) * p.G + stay) * p.target_stride;
    row.q = refused && p.draft != nullptr ? p.draft + (static_cast<int64_t>(r) * D + stay) * p.draft_stride : nullptr;
    row.gone = refused && p.draft == nullptr ? p.tokens[static_cast<int64_t>(r) * D + stay] : -1;
    const float u = p.sample[r];
    const uint64_t U = u >= 1.0f ? 0x7fffffffu : u > 0.0f ? static_cast<uint32_t>(u * 2147483648.0f) : 0u;

    // The residual, then (all of it 0) the target itself.
#pragma unroll 1
    for (int turn = 0; turn < 2; ++turn) {
        const int per = p.part / kWarps, v0 = min(rank * p.part + warp * per, p.V), v1 = min(v0 + per, p.V);
        const uint64_t mine = sum_part<kWide>(row, v0, v1, lane);
        if (lane == 0) s_warp[warp] = mine;
        __syncthreads();
        uint64_t part = 0;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) part += s_warp[w];
        cluster_wait();
        if (tid < C) st_peer_u64(&s_all[rank], tid, part);
        cluster_arrive_release();
        cluster_wait();
        uint64_t total = 0, before = 0;
        for (int c = 0; c < C; ++c) {
            if (c < rank) before += s_all[c];
            total += s_all[c];
        }
        if (total == 0) {
            if (turn == 0 && (row.q != nullptr || row.gone >= 0)) {
                row.q = nullptr;
                row.gone = -1;
                cluster_arrive_relaxed();  // waited for before they are written again: every CTA has read them
                continue;
            }
            if (rank == 0 && tid == 0) p.out_tokens[static_cast<int64_t>(r) * p.G + stay] = -1;
            return;
        }
        // floor(U total / 2^31) is below total: one CTA holds it.
        uint64_t t = __umul64hi(total, U) << 33 | (total * U) >> 31;
        if (t < before || t - before >= part) return;
        t -= before;
        int w = 0;
        while (t >= s_warp[w]) t -= s_warp[w++];
        // That warp's part, contiguous entries to a thread.
        const int a0 = min(rank * p.part + w * per, p.V), a1 = min(a0 + per, p.V);
        const int each = (a1 - a0 + kThreads - 1) / kThreads;
        const int b0 = min(a0 + tid * each, a1), b1 = min(b0 + each, a1);
        Share s;
#pragma unroll 4
        for (int v = b0; v < b1; ++v) {
            s.add(row.at(v));
            s.flush();
        }
        uint64_t inc = s.sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint64_t up = __shfl_up_sync(0xffffffffu, inc, o);
            if (lane >= o) inc += up;
        }
        if (lane == 31) s_scan[warp] = inc;
        __syncthreads();
        for (int z = 0; z < warp; ++z) inc += s_scan[z];
        if (t >= inc || t < inc - s.sum) return;
        t -= inc - s.sum;
        for (int v = b0; v < b1; ++v) {
            Share one;
            one.add(row.at(v));
            one.flush();
            if (t < one.sum) {
                p.out_tokens[static_cast<int64_t>(r) * p.G + stay] = v;
                return;
            }
            t -= one.sum;
        }
        return;
    }
}

}  // namespace
}  // namespace smd

extern "C" int smd_verify_drafts(const float* target, int64_t target_stride, const float* draft,
                                 int64_t draft_stride, const int32_t* tokens, const float* accept,
                                 const float* sample, int32_t R, int32_t G, int32_t V,
                                 int32_t* out_tokens, int32_t* accepted, int32_t* rejected,
                                 smd_stream_t stream) {
    using namespace smd;
    if (R < 0 || G < 1 || G > kMaxDrafts + 1 || V < 1 || V > kMaxVocab || target_stride < V ||
        (draft != nullptr && G > 1 && draft_stride < V) || static_cast<int64_t>(R) * G >= (1ll << 31))
        return SMD_ERR_SHAPE;
    if (R == 0) return SMD_OK;
    if (target == nullptr || sample == nullptr || out_tokens == nullptr ||
        (G > 1 && (tokens == nullptr || accept == nullptr)))
        return SMD_ERR_NULL;
    for (const void* a : {static_cast<const void*>(target), static_cast<const void*>(draft),
                          static_cast<const void*>(tokens), static_cast<const void*>(accept),
                          static_cast<const void*>(sample), static_cast<const void*>(out_tokens),
                          static_cast<const void*>(accepted), static_cast<const void*>(rejected)})
        if (!aligned(a, 4)) return SMD_ERR_ALIGN;
    VerifyParams p{target, target_stride, G > 1 ? draft : nullptr, draft_stride, tokens, accept, sample,
                   R, G, V, 0, out_tokens, accepted, rejected};
    // CTAs of a request, of a few thousand entries at least: as many as a cluster takes, or, where it is
    // the memory that bounds the call, as many as load the SMs most evenly (96 requests of 131072 entries,
    // 6 a request 4 on an SM: 19.5 us; 8, 5 or 6 on an SM: 20.5. 64 of 32768: 8 a request 6.3, 7 7.6).
    const int sms = device_sms();
    if (sms <= 0) return SMD_ERR_DEVICE;
    int C = 1;
    double best = 0.0;
    for (int c = 1; c <= kMaxCluster && (c == 1 || V > 4096 * (c - 1)); ++c) {
        const int64_t ctas = static_cast<int64_t>(R) * c, rounds = (ctas + sms - 1) / sms;
        const double share = static_cast<int64_t>(R) * V < (1 << 23)
                                 ? 1.0 : static_cast<double>(ctas) / static_cast<double>(rounds * sms);
        if (share >= best) best = share, C = c;
    }
    const int unit = kWarps * 128;
    p.part = ((V + C - 1) / C + unit - 1) / unit * unit;
    const bool wide = aligned(target, 16) && target_stride % 4 == 0 &&
                      (p.draft == nullptr || (aligned(draft, 16) && draft_stride % 4 == 0));
    auto kernel = wide ? verify_kernel<true> : verify_kernel<false>;
    // Requests go along grid.y, which holds 65535.
    for (int64_t r = 0; r < R; r += 65535) {
        const int n = static_cast<int>(R - r < 65535 ? R - r : 65535);
        p.R = n;
        p.target = target + r * G * target_stride;
        p.draft = G > 1 && draft != nullptr ? draft + r * (G - 1) * draft_stride : nullptr;
        p.tokens = tokens != nullptr ? tokens + r * (G - 1) : nullptr;
        p.accept = accept != nullptr ? accept + r * (G - 1) : nullptr;
        p.sample = sample + r;
        p.out_tokens = out_tokens + r * G;
        p.accepted = accepted != nullptr ? accepted + r : nullptr;
        p.rejected = rejected != nullptr ? rejected + r : nullptr;
        const int rc = launch_cluster(kernel, dim3(static_cast<unsigned>(C), static_cast<unsigned>(n)), kThreads,
                                  stream, C, p);
        if (rc != SMD_OK) return rc;
    }
    return SMD_OK;
}

// Tokens off the end of requests, and their pages back to the ring (smd_block_trim).
//
// back_r = ceil(len_r / P) - ceil((len_r - drop_r) / P); request r's last back_r pages go to
// ring[(given + sum_{q<r} back_q + j) mod pages].
//
// What bounds it: 12 bytes a request and 8 bytes a page: the latency of lengths, sum, table entry and
// store. One launch, as smd_block_tables: every block sums for itself (at most 8192
// requests, from L2) and moves its share of the pages; a page's request is found by a
// binary search in the sums, so that one long request and a thousand short ones load the grid alike.
//
// Measured (GB300, device time): 96 requests 2.1 us, 2000 that give 350 thousand pages back 7.3, 8000
// 13.2 (the sums: 16 requests a thread).
#include "smd_internal.h"
#include "smd_paged.h"
#include "smd_ptx.cuh"

namespace smd {
namespace {

constexpr int kMaxRequests = 8192;
constexpr int kSmall = 128, kThreadsMost = 512;  // threads of a block
constexpr int kAtOnce = 4;                       // pages of a thread in flight

struct TrimParams {
    const int32_t* lengths;
    const int32_t* drop;
    int32_t R;
    const int32_t* table;
    int64_t table_stride;
    int32_t width;
    int32_t* ring;
    int32_t pages;
    const int64_t* state;
    int32_t P, shift;  // tokens of a page; its logarithm, or -1
    int32_t* new_lengths;
    int64_t* new_state;
};

__device__ __forceinline__ int pages_of(const TrimParams& p, int tokens) {
    return p.shift >= 0 ? static_cast<int>((static_cast<uint32_t>(tokens) + static_cast<uint32_t>(p.P) - 1) >> p.shift)
                        : smd::pages_of(tokens, p.P);
}

// A request's place in shared memory: a thread's requests follow one another, and a word more for
// every 16 keeps the threads' places in different banks (8000 requests: 18.8 us without).
__host__ __device__ constexpr int place(int r) { return r + (r >> 4); }

// s_back: pages that go back before request r's; s_keep: pages that it keeps.
template <int kThreads>
__global__ void __launch_bounds__(kThreads) trim_kernel(const TrimParams p) {
    constexpr int kWarps = kThreads / 32;
    extern __shared__ int32_t smem[];
    int32_t* const s_back = smem;
    int32_t* const s_keep = smem + place(p.R) + 1;
    __shared__ int64_t s_sum[kWarps];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    pdl_entry();
    const int64_t taken = p.state[0], given = p.state[1];
    const int per = (p.R + kThreads - 1) / kThreads;
    const int r0 = min(tid * per, p.R), r1 = min(r0 + per, p.R), room = p.width * p.P;
    int64_t back = 0;
    constexpr int kLoads = 8;  // requests of a thread in flight
#pragma unroll 1
    for (int q = r0; q < r1; q += kLoads) {
        int len[kLoads], drop[kLoads];
#pragma unroll
        for (int j = 0; j < kLoads; ++j) {
            len[j] = drop[j] = 0;
            if (q + j < r1) {
                len[j] = p.lengths[q + j];
                drop[j] = p.drop[q + j];
            }
        }
#pragma unroll
        for (int j = 0; j < kLoads; ++j) {
            if (q + j >= r1) break;
            const int n = max(min(len[j], room), 0), left = max(n - max(drop[j], 0), 0);
            const int keep = pages_of(p, left), goes = pages_of(p, n) - keep;
            s_keep[place(q + j)] = keep;
            s_back[place(q + j)] = goes;
            back += goes;
            if (blockIdx.x == 0) p.new_lengths[q + j] = left;
        }
    }
    int64_t inc = back;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t up = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += up;
    }
    if (lane == 31) s_sum[warp] = inc;
    __syncthreads();
    int64_t before = inc - back, total64 = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        if (w < warp) before += s_sum[w];
        total64 += s_sum[w];
    }
    if (blockIdx.x == 0 && tid == 0) {
        p.new_state[0] = taken;
        p.new_state[1] = given + total64;
    }
    // More pages than the ring holds are none of this pool's: the ring is written once around.
    const int total = static_cast<int>(min(total64, static_cast<int64_t>(p.pages)));
    for (int r = r0; r < r1; ++r) {
        const int goes = s_back[place(r)];
        s_back[place(r)] = static_cast<int32_t>(min(before, static_cast<int64_t>(p.pages)));
        before += goes;
    }
    if (tid == 0) s_back[place(p.R)] = total;
    __syncthreads();
    int64_t g0 = given % p.pages;
    if (g0 < 0) g0 += p.pages;
    const int step = static_cast<int>(gridDim.x) * kThreads;
    for (int64_t i0 = static_cast<int64_t>(blockIdx.x) * kThreads + tid; i0 < total; i0 += static_cast<int64_t>(kAtOnce) * step) {
        int32_t page[kAtOnce];
#pragma unroll
        for (int j = 0; j < kAtOnce; ++j) {
            const int64_t i = i0 + static_cast<int64_t>(j) * step;
            page[j] = 0;
            if (i < total) {
                int lo = 0, hi = p.R;  // s_back[lo] <= i < s_back[hi]
                while (hi - lo > 1) {
                    const int mid = (lo + hi) >> 1;
                    if (s_back[place(mid)] <= i) lo = mid;
                    else hi = mid;
                }
                page[j] = p.table[lo * p.table_stride + s_keep[place(lo)] + (static_cast<int>(i) - s_back[place(lo)])];
            }
        }
#pragma unroll
        for (int j = 0; j < kAtOnce; ++j) {
            const int64_t i = i0 + static_cast<int64_t>(j) * step;
            if (i >= total) break;
            const int64_t at = g0 + i;
            p.ring[at >= p.pages ? at - p.pages : at] = page[j];
        }
    }
}

template <int kThreads>
int launch_trim(const TrimParams& p, int sms, smd_stream_t stream) {
    const size_t smem = (2 * static_cast<size_t>(place(p.R)) + 2) * 4;  // at most 68 KB
    static SharedLimit limit;
    const int rc = limit.raise(trim_kernel<kThreads>, (2 * place(kMaxRequests) + 2) * 4);
    if (rc != SMD_OK) return rc;
    const int64_t rows = static_cast<int64_t>(p.R) * p.width;  // the most pages that go back
    const int64_t want = ((rows < p.pages ? rows : p.pages) + kAtOnce * kThreads - 1) / (kAtOnce * kThreads);
    const int grid = static_cast<int>(want < 1 ? 1 : want < 2 * sms ? want : 2 * sms);
    return launch_pdl(trim_kernel<kThreads>, dim3(grid), kThreads, smem, stream, p);
}

}  // namespace
}  // namespace smd

extern "C" int smd_block_trim(const int32_t* lengths, const int32_t* drop, int32_t R, const int32_t* table,
                              int64_t table_stride, int32_t width, int32_t* ring, int32_t pages,
                              const int64_t* state, int32_t page_size, int32_t* new_lengths,
                              int64_t* new_state, smd_stream_t stream) {
    using namespace smd;
    if (R < 0 || R > kMaxRequests || pages < 1 || page_size < 1 ||
        static_cast<int64_t>(pages) * page_size >= (1ll << 31) || width < 1 || table_stride < width ||
        static_cast<int64_t>(width) * page_size >= (1ll << 31))
        return SMD_ERR_SHAPE;
    if (ring == nullptr || state == nullptr || new_state == nullptr ||
        (R > 0 && (lengths == nullptr || drop == nullptr || table == nullptr || new_lengths == nullptr)))
        return SMD_ERR_NULL;
    for (const void* a : {static_cast<const void*>(lengths), static_cast<const void*>(drop),
                          static_cast<const void*>(table), static_cast<const void*>(ring),
                          static_cast<const void*>(new_lengths)})
        if (!aligned(a, 4)) return SMD_ERR_ALIGN;
    if (!aligned(state, 8) || !aligned(new_state, 8)) return SMD_ERR_ALIGN;
    const int sms = device_sms();
    if (sms <= 0) return SMD_ERR_DEVICE;
    int shift = -1;
    if ((page_size & (page_size - 1)) == 0)
        for (shift = 0; 1 << shift < page_size;) ++shift;
    const TrimParams p{lengths, drop, R, table, table_stride, width, ring, pages, state, page_size, shift,
                       new_lengths, new_state};
    return R <= kSmall ? launch_trim<kSmall>(p, sms, stream) : launch_trim<kThreadsMost>(p, sms, stream);
}

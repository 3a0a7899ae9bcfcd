// Pages and slots of a step from the requests' lengths (smd_block_tables).
//
// need_r = ceil((len_r + n_r) / P) - ceil(len_r / P); request r's new pages are
// ring[(taken + sum_{q<r} need_q + j) mod pages]. The sums are exclusive
// prefix sums over the requests: of the pages needed (which decides who is
// granted them), of the tokens of those granted, and of the pages that ended
// requests return.
//
// What bounds it: a few bytes a request and 8 bytes a token are moved, so it is
// the latency of three dependent rounds (lengths, sums, table or ring entry)
// for a step, and the 8 bytes a token for admitted prompts. One launch: every
// block computes the sums for itself (at most 8192 requests, from L2) and then
// writes its share of the tokens; no block waits for another, so the arrays
// that are read may not be the ones that are written.
#include "smd_internal.h"
#include "smd_paged.h"
#include "smd_ptx.cuh"

namespace smd {
namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxRequests = 8192;
constexpr int kTokensPerBlock = 4 * kThreads;

struct TableParams {
    const int32_t* lengths;
    const int32_t* new_tokens;
    int32_t R;
    int32_t* table;
    int64_t table_stride;
    int32_t width;
    int32_t* ring;
    int32_t pages;
    const int64_t* state;
    int32_t P, T;
    int32_t* new_lengths;
    int64_t* new_state;
    int32_t* starts;
    int32_t* slots;
    int32_t* positions;
    int32_t* status;
};

struct Request {
    int64_t len, want;  // tokens held; wanted (0 where its row is too narrow)
    int64_t have, need; // pages held; needed
    bool ended, narrow;
};

__device__ __forceinline__ Request request(const TableParams& p, int r) {
    Request q;
    q.len = max(static_cast<int64_t>(p.lengths[r]), static_cast<int64_t>(0));
    q.len = min(q.len, static_cast<int64_t>(p.width) * p.P);
    const int n = p.new_tokens[r];
    q.ended = n < 0;
    q.want = max(n, 0);
    q.have = (q.len + p.P - 1) / p.P;
    q.narrow = (q.len + q.want + p.P - 1) / p.P > p.width;
    if (q.narrow) q.want = 0;
    q.need = (q.len + q.want + p.P - 1) / p.P - q.have;
    return q;
}

// The sum of v over the threads before this one; *total over all.
__device__ __forceinline__ int64_t scan(int64_t v, int64_t* buf, int64_t* total) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    int64_t inc = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t u = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += u;
    }
    __syncthreads();
    if (lane == 31) buf[warp] = inc;
    __syncthreads();
    int64_t before = inc - v, all = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        const int64_t u = buf[w];
        if (w < warp) before += u;
        all += u;
    }
    *total = all;
    return before;
}

// s_start[r]: tokens granted before request r. s_page[r]: the page count before
// request r, of those taken, or of those returned where it has ended.
__global__ void __launch_bounds__(kThreads) block_tables_kernel(const TableParams p) {
    extern __shared__ int32_t smem[];
    int32_t* const s_start = smem;
    int32_t* const s_page = smem + p.R + 1;
    __shared__ int64_t buf[kWarps];
    const int tid = threadIdx.x;
    pdl_entry();

    const int per = (p.R + kThreads - 1) / kThreads;
    const int r0 = min(tid * per, p.R), r1 = min(r0 + per, p.R);
    const int64_t taken = p.state[0], given = p.state[1];
    int64_t need = 0, back = 0, total_need, total_back, total_tokens, total_granted;
    bool refused = false;
    for (int r = r0; r < r1; ++r) {
        const Request q = request(p, r);
        need += q.need;
        back += q.ended ? q.have : 0;
        refused = refused || q.narrow;
    }
    const int64_t need0 = scan(need, buf, &total_need);
    const int64_t back0 = scan(back, buf, &total_back);
    // Tokens of the requests whose pages fit.
    int64_t off = need0, tokens = 0;
    for (int r = r0; r < r1; ++r) {
        const Request q = request(p, r);
        off += q.need;
        if (q.need == 0 || off <= given - taken) tokens += q.want;
    }
    int64_t tok = scan(tokens, buf, &total_tokens);
    // Who is granted. Tokens past T are refused to every later request, so the
    // sum of those granted before r is the sum of those that fit.
    int64_t granted = 0, used = 0, bk = back0;
    off = need0;
    for (int r = r0; r < r1; ++r) {
        const Request q = request(p, r);
        const bool fits = q.need == 0 || off + q.need <= given - taken;
        const bool ok = fits && (q.want == 0 || tok + q.want <= p.T);
        s_start[r] = static_cast<int32_t>(min(tok, static_cast<int64_t>(p.T)));
        s_page[r] = static_cast<int32_t>(q.ended ? bk : off);
        if (fits) tok += q.want;
        off += q.need;
        bk += q.ended ? q.have : 0;
        granted += ok ? q.want : 0;
        used += ok ? q.need : 0;
        refused = refused || !ok;
        if (blockIdx.x == 0)
            p.new_lengths[r] = q.ended ? 0 : static_cast<int32_t>(q.len + (ok ? q.want : 0));
    }
    scan(granted, buf, &total_granted);
    scan(used, buf, &total_need);
    const int32_t total = static_cast<int32_t>(total_granted);
    // A request that did not fit T, and those after it, start at the total.
    for (int r = r0; r < r1; ++r) s_start[r] = min(s_start[r], total);
    if (tid == 0) s_start[p.R] = total;
    __syncthreads();

    const auto in_ring = [&](int64_t i) {
        i = i >= p.pages || i < 0 ? i % p.pages : i;
        return i < 0 ? i + p.pages : i;
    };
    const int64_t tk = in_ring(taken), gv = in_ring(given);
    // Tokens: the slot of each, and the table entry of each page that one begins.
    const int step = static_cast<int>(gridDim.x) * kThreads;
    for (int t = blockIdx.x * kThreads + tid; t < p.T; t += step) {
        if (t >= total) {
            p.slots[t] = -1;
            if (p.positions != nullptr) p.positions[t] = -1;
            continue;
        }
        int lo = 0, hi = p.R;  // s_start[lo] <= t < s_start[hi]
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (s_start[mid] <= t) lo = mid;
            else hi = mid;
        }
        const int len = min(max(p.lengths[lo], 0), p.width * p.P);
        const int pos = len + t - s_start[lo], blk = pos / p.P, in = pos - blk * p.P;
        const int have = (len + p.P - 1) / p.P;
        int32_t* const entry = p.table + lo * p.table_stride + blk;
        int page;
        if (blk < have) {
            page = *entry;
        } else {
            page = p.ring[in_ring(tk + s_page[lo] + blk - have)];
            if (in == 0) *entry = page;
        }
        p.slots[t] = page * p.P + in;
        if (p.positions != nullptr) p.positions[t] = pos;
    }
    // Pages that go back.
    for (int r = blockIdx.x * kWarps + (tid >> 5); r < p.R; r += gridDim.x * kWarps) {
        if (p.new_tokens[r] >= 0) continue;
        const int len = min(max(p.lengths[r], 0), p.width * p.P);
        const int have = (len + p.P - 1) / p.P;
        for (int j = tid & 31; j < have; j += 32)
            p.ring[in_ring(gv + s_page[r] + j)] = p.table[r * p.table_stride + j];
    }
    for (int r = blockIdx.x * kThreads + tid; r <= p.R; r += step) p.starts[r] = s_start[r];
    if (blockIdx.x == 0) {
        if (__syncthreads_or(refused) && tid == 0 && p.status != nullptr)
            atomicCAS(p.status, 0, SMD_ERR_PAGES);
        if (tid == 0) {
            p.new_state[0] = taken + total_need;
            p.new_state[1] = given + total_back;
        }
    }
}

}  // namespace
}  // namespace smd

extern "C" int smd_block_tables(const int32_t* lengths, const int32_t* new_tokens, int32_t R,
                                int32_t* table, int64_t table_stride, int32_t width, int32_t* ring,
                                int32_t pages, const int64_t* state, int32_t page_size, int32_t T,
                                int32_t* new_lengths, int64_t* new_state, int32_t* starts,
                                int32_t* slots, int32_t* positions, int32_t* status,
                                smd_stream_t stream) {
    using namespace smd;
    if (R < 0 || R > kMaxRequests || T < 0 || pages < 1 || page_size < 1 ||
        static_cast<int64_t>(pages) * page_size >= (1ll << 31) || width < 1 ||
        table_stride < width || static_cast<int64_t>(width) * page_size >= (1ll << 31))
        return SMD_ERR_SHAPE;
    if (ring == nullptr || state == nullptr || new_state == nullptr || starts == nullptr ||
        (T > 0 && slots == nullptr) ||
        (R > 0 && (lengths == nullptr || new_tokens == nullptr || table == nullptr ||
                   new_lengths == nullptr)))
        return SMD_ERR_NULL;
    for (const void* a : {static_cast<const void*>(lengths), static_cast<const void*>(new_tokens),
                          static_cast<const void*>(table), static_cast<const void*>(ring),
                          static_cast<const void*>(new_lengths), static_cast<const void*>(starts),
                          static_cast<const void*>(slots), static_cast<const void*>(positions),
                          static_cast<const void*>(status)})
        if (!aligned(a, 4)) return SMD_ERR_ALIGN;
    if (!aligned(state, 8) || !aligned(new_state, 8)) return SMD_ERR_ALIGN;
    const int sms = device_sms();
    if (sms <= 0) return SMD_ERR_DEVICE;
    const TableParams p{lengths, new_tokens, R, table, table_stride, width, ring, pages, state,
                        page_size, T, new_lengths, new_state, starts, slots, positions, status};
    const size_t smem = (2 * static_cast<size_t>(R) + 1) * 4;  // at most 64 KB
    static_assert((2 * kMaxRequests + 1) * 4 <= 80 * 1024, "shared memory of the sums");
    if (smem > 48 * 1024 &&
        cudaFuncSetAttribute(block_tables_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             (2 * kMaxRequests + 1) * 4) != cudaSuccess) {
        (void)cudaGetLastError();
        return SMD_ERR_DEVICE;
    }
    const int64_t want = (static_cast<int64_t>(T) + kTokensPerBlock - 1) / kTokensPerBlock;
    const int grid = static_cast<int>(want < 1 ? 1 : want < 2 * sms ? want : 2 * sms);
    return launch_pdl(block_tables_kernel, dim3(grid), kThreads, smem, stream, p);
}

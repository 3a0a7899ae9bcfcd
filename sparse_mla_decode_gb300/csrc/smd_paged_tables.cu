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
//
// Measured (GB300, back to back in a CUDA graph): 96 requests with a token each 5.1
// us, 700 requests with 280 thousand tokens 9.9 us.
#include "smd_internal.h"
#include "smd_paged.h"
#include "smd_ptx.cuh"

namespace smd {
namespace {

constexpr int kMaxRequests = 8192;
constexpr int kSmall = 128, kThreadsMost = 512;  // threads of a block

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
    bool wide;  // slots and positions take 16-byte stores
};

struct Request {
    int len, want;   // tokens held; wanted (0 where its row is too narrow)
    int have, need;  // pages held; needed
    bool ended, narrow;
};

__device__ __forceinline__ Request request(const TableParams& p, int r) {
    Request q;
    const int room = p.width * p.P;
    q.len = min(max(p.lengths[r], 0), room);
    const int n = p.new_tokens[r];
    q.ended = n < 0;
    q.narrow = n > room - q.len;
    q.want = q.narrow ? 0 : max(n, 0);
    q.have = pages_of(q.len, p.P);
    q.need = pages_of(q.len + q.want, p.P) - q.have;
    return q;
}

// The sums of a and b over the threads before this one, in place; the totals.
template <int kWarps>
__device__ __forceinline__ void scan2(int64_t& a, int64_t& b, int64_t (*buf)[2], int64_t& all_a,
                                      int64_t& all_b) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    int64_t ia = a, ib = b;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t ua = __shfl_up_sync(0xffffffffu, ia, o), ub = __shfl_up_sync(0xffffffffu, ib, o);
        if (lane >= o) ia += ua, ib += ub;
    }
    if (lane == 31) buf[warp][0] = ia, buf[warp][1] = ib;
    __syncthreads();
    int64_t ba = ia - a, bb = ib - b;
    all_a = all_b = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        if (w < warp) ba += buf[w][0], bb += buf[w][1];
        all_a += buf[w][0], all_b += buf[w][1];
    }
    a = ba;
    b = bb;
}

// s_start[r]: tokens granted before request r. s_page[r]: the page count before
// request r, of those taken, or of those returned where it has ended.
template <int kThreads>
__global__ void __launch_bounds__(kThreads) block_tables_kernel(const TableParams p) {
    constexpr int kWarps = kThreads / 32;
    extern __shared__ int32_t smem[];
    int32_t* const s_start = smem;
    int32_t* const s_page = smem + p.R + 1;
    __shared__ int64_t buf[2][kWarps][2];
    __shared__ int s_most[2][kWarps];
    const int tid = threadIdx.x;
    pdl_entry();

    const int per = (p.R + kThreads - 1) / kThreads;
    const int r0 = min(tid * per, p.R), r1 = min(r0 + per, p.R);
    const int64_t taken = p.state[0], given = p.state[1];
    int64_t need = 0, back = 0, all_need, all_back;
    bool refused = false;
    Request one{};  // the thread's request where it has one only
    for (int r = r0; r < r1; ++r) {
        one = request(p, r);
        need += one.need;
        back += one.ended ? one.have : 0;
        refused = refused || one.narrow;
    }
    scan2<kWarps>(need, back, buf[0], all_need, all_back);
    // Tokens of the requests whose pages fit.
    int64_t off = need, tokens = 0, none = 0, all_tokens, all_none;
    for (int r = r0; r < r1; ++r) {
        if (per > 1) one = request(p, r);
        off += one.need;
        if (one.need == 0 || off <= given - taken) tokens += one.want;
    }
    scan2<kWarps>(tokens, none, buf[1], all_tokens, all_none);
    // Who is granted. Pages or tokens that run out are refused to every later request that
    // wants any, so what is granted before r is what fits before r.
    int64_t tok = tokens;
    int granted = 0, used = 0;  // sums up to the last request that is granted any
    off = need;
    for (int r = r0; r < r1; ++r) {
        if (per > 1) one = request(p, r);
        const bool fits = one.need == 0 || off + one.need <= given - taken;
        const bool ok = fits && (one.want == 0 || tok + one.want <= p.T);
        s_start[r] = static_cast<int32_t>(min(tok, static_cast<int64_t>(p.T)));
        s_page[r] = static_cast<int32_t>(one.ended ? back : off);
        if (ok && one.want > 0) granted = static_cast<int>(tok + one.want);
        if (ok && one.need > 0) used = static_cast<int>(off + one.need);
        if (fits) tok += one.want;
        off += one.need;
        back += one.ended ? one.have : 0;
        refused = refused || !ok;
        if (blockIdx.x == 0)
            p.new_lengths[r] = one.ended ? 0 : one.len + (ok ? one.want : 0);
    }
    granted = __reduce_max_sync(0xffffffffu, granted);
    used = __reduce_max_sync(0xffffffffu, used);
    if ((tid & 31) == 0) s_most[0][tid >> 5] = granted, s_most[1][tid >> 5] = used;
    __syncthreads();
    int total = 0, total_used = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        total = max(total, s_most[0][w]);
        total_used = max(total_used, s_most[1][w]);
    }
    if (tid == 0) s_start[p.R] = total;
    __syncthreads();
    // A request that did not fit T, and those after it, start at the total.
    const auto start = [&](int r) { return min(s_start[r], total); };

    const auto in_ring = [&](int64_t i) {
        i = i >= p.pages || i < 0 ? i % p.pages : i;
        return i < 0 ? i + p.pages : i;
    };
    const int64_t tk = in_ring(taken), gv = in_ring(given);
    const int room = p.width * p.P;
    // Tokens, four a thread: the slot of each, and the table entry of each page that one begins.
    const int64_t step = static_cast<int64_t>(gridDim.x) * kThreads * 4;
    for (int64_t t4 = (static_cast<int64_t>(blockIdx.x) * kThreads + tid) * 4; t4 < p.T; t4 += step) {
        int slot[4], pos[4];
        int r = 0;
        if (t4 < total) {
            int hi = p.R;  // start(r) <= t4 < start(hi)
            while (hi - r > 1) {
                const int mid = (r + hi) >> 1;
                if (s_start[mid] <= t4) r = mid;
                else hi = mid;
            }
        }
        int len = 0, from = 0, until = -1, have = 0, last_blk = -1, page = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int64_t t = t4 + i;
            slot[i] = pos[i] = -1;
            if (t >= total) continue;
            if (i == 0 || t >= until) {
                while (start(r + 1) <= t) ++r;
                len = min(max(p.lengths[r], 0), room);
                from = start(r);
                until = start(r + 1);
                have = pages_of(len, p.P);
                last_blk = -1;
            }
            pos[i] = len + static_cast<int>(t) - from;
            const int blk = static_cast<int>(static_cast<uint32_t>(pos[i]) / static_cast<uint32_t>(p.P));
            const int in = pos[i] - blk * p.P;
            if (blk != last_blk) {
                int32_t* const entry = p.table + r * p.table_stride + blk;
                if (blk < have) {
                    page = *entry;
                } else {
                    page = p.ring[in_ring(tk + s_page[r] + blk - have)];
                    if (in == 0) *entry = page;
                }
                last_blk = blk;
            }
            slot[i] = page * p.P + in;
        }
        if (p.wide && t4 + 4 <= p.T) {
            *reinterpret_cast<int4*>(p.slots + t4) = make_int4(slot[0], slot[1], slot[2], slot[3]);
            if (p.positions != nullptr)
                *reinterpret_cast<int4*>(p.positions + t4) = make_int4(pos[0], pos[1], pos[2], pos[3]);
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (t4 + i < p.T) {
                    p.slots[t4 + i] = slot[i];
                    if (p.positions != nullptr) p.positions[t4 + i] = pos[i];
                }
        }
    }
    // Pages that go back, kBack loads of a lane in flight.
    constexpr int kBack = 8;
    const int warps = gridDim.x * kWarps, lane = tid & 31;
    for (int q0 = blockIdx.x * kWarps + (tid >> 5); q0 < p.R; q0 += 32 * warps) {
        const int own = q0 + lane * warps;  // a warp's requests, one a lane
        const bool ended = own < p.R && p.new_tokens[own] < 0;
        const int held = ended ? pages_of(min(max(p.lengths[own], 0), room), p.P) : 0;
        for (uint32_t left = __ballot_sync(0xffffffffu, ended); left != 0; left &= left - 1) {
            const int l = __ffs(left) - 1, r = q0 + l * warps;
            const int have = __shfl_sync(0xffffffffu, held, l);
            for (int j = lane; j < have; j += 32 * kBack) {
                int32_t page[kBack];
#pragma unroll
                for (int i = 0; i < kBack; ++i)
                    page[i] = j + 32 * i < have ? p.table[r * p.table_stride + j + 32 * i] : 0;
#pragma unroll
                for (int i = 0; i < kBack; ++i)
                    if (j + 32 * i < have) p.ring[in_ring(gv + s_page[r] + j + 32 * i)] = page[i];
            }
        }
    }
    for (int r = blockIdx.x * kThreads + tid; r <= p.R; r += gridDim.x * kThreads) p.starts[r] = start(r);
    if (blockIdx.x == 0) {
        if (__syncthreads_or(refused) && tid == 0 && p.status != nullptr)
            atomicCAS(p.status, 0, SMD_ERR_PAGES);
        if (tid == 0) {
            p.new_state[0] = taken + total_used;
            p.new_state[1] = given + all_back;
        }
    }
}

template <int kThreads>
int launch_tables(const TableParams& p, int sms, smd_stream_t stream) {
    constexpr int kTokensPerBlock = 4 * kThreads;  // of one turn
    const size_t smem = (2 * static_cast<size_t>(p.R) + 1) * 4;  // at most 64 KB
    static_assert((2 * kMaxRequests + 1) * 4 <= 80 * 1024, "shared memory of the sums");
    static SharedLimit limit;
    const int rc = limit.raise(block_tables_kernel<kThreads>, (2 * kMaxRequests + 1) * 4);
    if (rc != SMD_OK) return rc;
    const int64_t want = (static_cast<int64_t>(p.T) + kTokensPerBlock - 1) / kTokensPerBlock;
    const int grid = static_cast<int>(want < 1 ? 1 : want < 2 * sms ? want : 2 * sms);
    return launch_pdl(block_tables_kernel<kThreads>, dim3(grid), kThreads, smem, stream, p);
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
                        page_size, T, new_lengths, new_state, starts, slots, positions, status,
                        aligned(slots, 16) && aligned(positions, 16)};
    // Few requests take small blocks, whose sums are over fewer warps. 128 / 512 threads: 96
    // requests with a token each 5.1 / 5.9 us, 100 with 16 tokens 5.1 / 6.2, with 400 4.4 / 5.5.
    return R <= kSmall ? launch_tables<kSmall>(p, sms, stream)
                       : launch_tables<kThreadsMost>(p, sms, stream);
}

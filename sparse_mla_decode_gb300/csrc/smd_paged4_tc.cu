// Attention over a paged E2M1 cache on the tcgen05 tensor cores, 128 columns
// (smd_paged4_decode; other sizes: smd_paged_decode.cuh).
//
// The definition, the cuts of the batch and the joins are smd_paged_decode.cuh's; a worker is
// four warps here, and a tile 128 tokens. For a tile of a unit with N query rows (16 or 32):
//   S^T [128 tokens x N] = K Q^T,  P = 2^(S f - m),  O^T [128 columns x N] += V^T P
// Tokens (then columns) are the MMA's 128 rows, so that every lane of the tensor cores
// has work whatever the number of query rows, and the rows are its N.
//
// What bounds it: 144 bytes of a (token, kv head) are few for what has to be done to them: 256
// codes converted to f16 and multiplied by their scales. Both operands that come
// from codes are therefore formed in registers and stored into tensor memory,
// from where tcgen05.mma takes its A operand: shared memory holds codes only (K and V in
// f16 through shared memory would be written and read again at 128 bytes a cycle). K: thread t of
// the worker converts token t, its lane of tensor memory. V: transposing ldmatrix gives a thread
// four columns of two tokens, whose nibbles are put side by side (the f16 pairs of
// an A operand run along the tokens); the store's 16x128b shape takes them as an MMA fragment,
// so that lane 32 w + 16 m + 8 y + g holds column 32 w + 4 g + 2 m + y.
//
// Two warps beside the workers keep the engines busy: one fills the workers' rings by tensor copies
// (8 lanes a worker; list and table entries are loaded one and two tiles ahead), one issues
// all MMAs as operands become ready. A worker's tile: K converted and handed over; half of V
// (its own 32 columns of tensor memory) while S^T is made; the weights; the other half of V, over
// K's columns, while the first half's products run. An MMA of 128 x N x 16 takes some 50 cycles
// whatever N is up to 64, 800 a tile, and a tile's 18 KB take HBM as long: the workers on an SM (four
// at 16 rows, three at 32: 128 and 160 columns of tensor memory each) are there to hide
// one another's conversions. A thread has one token's N logits: no reduction over tokens is
// needed but for the sums, once a unit, and the maximum, which is moved only when a logit exceeds
// it by more than 2^8 (the worker's vote; accumulators in tensor memory then come down by
// 2^(old - new)).
#include "smd_paged4_tc.h"

namespace smd {
namespace {

constexpr int kTile = 128;              // tokens
constexpr int kCols = 128;              // columns of a head
constexpr int kSideBytes = kTile * kCols / 2, kScaleBytes = kTile * kCols / 16;
constexpr int kSlotBytes = 2 * (kSideBytes + kScaleBytes);
constexpr int kFar = 0x7ffffff0;        // the position of tokens that no row sees (15 more fit an int)
constexpr int kTcUnitCost = 1;          // what a unit's begin and end cost, in tiles

// N query rows of a unit, W workers, ST slots of a worker's ring.
template <int N_, int W_, int ST_>
struct TcShape {
    static constexpr int N = N_, W = W_, ST = ST_;
    static constexpr int threads = 128 * W + 32;       // the workers' and the copies' warp
    static constexpr int joiners = 128 * W;            // threads of the joins
    // Tensor memory of a worker: K's operand (later V's second half), V's first half, S^T, O^T.
    static constexpr int t_v = 64, t_s = 96, t_o = 96 + N, t_cols = 96 + 2 * N;
    static_assert(W * t_cols <= 512 && W <= 4, "tensor memory");
    static constexpr int off_q = ST * kSlotBytes;
    static constexpr int off_p = off_q + N * kCols * 2;
    static constexpr int worker_bytes = off_p + N * kTile * 2;
    static_assert(worker_bytes % 1024 == 0, "swizzle atoms");
    static_assert(N * kCols * 4 == worker_bytes - off_q, "a worker's accumulators fit its queries' and weights' places");
    // Of a worker, beside that: logit factors and maxima of row pairs, limits, NaN
    // blocks, sums of the warps, positions of 16 tokens each, the last of a tile.
    static constexpr int off_lim = 8 * N, off_nan = off_lim + 4 * N,
                         off_red = off_nan + 4 * N, off_pos = off_red + 16 * N, off_last = off_pos + ST * 32,
                         row_bytes = off_last + 16;
    static constexpr int off_rows = W * worker_bytes;
    static constexpr int bars = 2 * ST + 5;  // of a worker: full, empty, K, S, P, V, O
    static constexpr int off_bar = off_rows + W * row_bytes;
    static constexpr int off_scan = off_bar + W * bars * 8;
    static constexpr int off_tmem = off_scan + 4 * ((threads / 32 + 3) / 4 * 4);
    static constexpr int off_ml = off_tmem + 16;
    static constexpr int off_left = off_ml + W * N * 8;
    static constexpr int off_range = off_left + W * 64;  // [W] tiles of a worker, whether it has stopped
    static constexpr int off_prefix = off_range + 32;
    static constexpr int smem(int entries) { return off_prefix + 4 * (2 * entries + 1) + 1024; }
    static_assert(sizeof(Left) <= 64 && off_ml % 8 == 0 && off_bar % 8 == 0 && row_bytes % 16 == 0, "places");
    static_assert(smem(kMaxEntries) + 64 <= 227 * 1024, "one CTA of an SM");
};

__device__ __forceinline__ void worker_sync(int id) {
    asm volatile("barrier.cta.sync %0, 128;" ::"r"(id) : "memory");
}

__device__ __forceinline__ bool worker_and(int id, bool v) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbarrier.cta.red.and.pred q, %2, 128, p;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"(static_cast<uint32_t>(v)), "r"(id)
        : "memory");
    return r != 0;
}

__device__ __forceinline__ bool worker_or(int id, bool v) { return !worker_and(id, !v); }

// Whether phase `parity` of a barrier is complete; does not wait.
__device__ __forceinline__ bool mbar_poll(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\tmbarrier.test_wait.parity.acquire.cta.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok != 0;
}

__device__ __forceinline__ uint32_t lds_volatile(uint32_t addr) {
    uint32_t v;
    asm volatile("ld.volatile.shared.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
    return v;
}

// One lane of the warp, by its value's truth.
__device__ __forceinline__ uint32_t elected() {
    uint32_t r;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
    return r;
}

// D (+)= A B of kind f16: A (128 rows) in tensor memory, B in shared memory. Called by a whole warp
// in step, issued by the lane where `one` holds: in uniform control flow the operands stay in
// uniform registers, and an MMA of 128 x 16 x 16 goes out every 13 cycles instead of 50 out of a
// branch that one lane takes.
__device__ __forceinline__ void umma_f16_ta(uint32_t d, uint32_t a, uint64_t b_desc, uint32_t idesc,
                                            uint32_t accumulate, uint32_t one) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(b_desc), "r"(idesc), "r"(accumulate), "r"(one)
        : "memory");
}

__device__ __forceinline__ void umma_commit_one(uint32_t bar, uint32_t one) {
    asm volatile(
        "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %1, 0;\n\t"
        "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(bar),
        "r"(one)
        : "memory");
}

// Instruction descriptor of kind::f16: f16 A (K-major) and B, FP32 D, M = 128.
__host__ __device__ constexpr uint32_t idesc_f16(int N, int mn_major_b) {
    return (1u << 4) | (static_cast<uint32_t>(mn_major_b) << 16) | (static_cast<uint32_t>(N >> 3) << 17) |
           (8u << 24);
}

// 32 words of this thread's lane.
__device__ __forceinline__ void tmem_st32(uint32_t at, const uint32_t (&v)[32]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, "
        "%13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, "
        "%32};" ::"r"(at),
        "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]),
        "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15]), "r"(v[16]),
        "r"(v[17]), "r"(v[18]), "r"(v[19]), "r"(v[20]), "r"(v[21]), "r"(v[22]), "r"(v[23]), "r"(v[24]),
        "r"(v[25]), "r"(v[26]), "r"(v[27]), "r"(v[28]), "r"(v[29]), "r"(v[30]), "r"(v[31])
        : "memory");
}

__device__ __forceinline__ void tmem_st16(uint32_t at, const uint32_t (&v)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, "
        "%13, %14, %15, %16};" ::"r"(at),
        "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]),
        "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
        : "memory");
}

// MMA A fragments of 16 lanes by 32 tokens (16 words).
__device__ __forceinline__ void tmem_st_frag(uint32_t at, const uint32_t (&v)[8]) {
    asm volatile("tcgen05.st.sync.aligned.16x128b.x4.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(at),
                 "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                 : "memory");
}

__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ void tmem_ldn(uint32_t at, float (&v)[16]) { tmem_ld16(at, v); }
__device__ __forceinline__ void tmem_ldn(uint32_t at, float (&v)[32]) { tmem_ld32(at, v); }

__device__ __forceinline__ void tmem_stn(uint32_t at, const float (&v)[16]) {
    uint32_t w[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) w[i] = __float_as_uint(v[i]);
    tmem_st16(at, w);
}
__device__ __forceinline__ void tmem_stn(uint32_t at, const float (&v)[32]) {
    uint32_t w[32];
#pragma unroll
    for (int i = 0; i < 32; ++i) w[i] = __float_as_uint(v[i]);
    tmem_st32(at, w);
}

__device__ __forceinline__ float max3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

// v[n] of the warp's lanes joined by op: lane l gets row l % N.
template <int N, typename Op>
__device__ __forceinline__ float reduce_rows(float (&v)[N], int lane, const Op& op) {
#pragma unroll
    for (int s = N / 2; s > 0; s >>= 1) {
        const bool up = (lane & s) != 0;
#pragma unroll
        for (int j = 0; j < s; ++j) {
            const float other = __shfl_xor_sync(0xffffffffu, up ? v[j] : v[j + s], s);
            v[j] = op(up ? v[j + s] : v[j], other);
        }
    }
    if (N == 16) v[0] = op(v[0], __shfl_xor_sync(0xffffffffu, v[0], 16));
    return v[0];
}

__device__ __forceinline__ uint4 lds_v4(uint32_t addr) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "r"(addr)
                 : "memory");
    return v;
}

__device__ __forceinline__ void sts_u4(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d)
                 : "memory");
}


template <typename S>
__global__ void __launch_bounds__(S::threads, 1)
    paged4_tc_kernel(const PagedParams p, const int box, const __grid_constant__ Maps<4> maps) {
    constexpr int N = S::N, W = S::W, ST = S::ST, D = kCols, KT = kTile;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t base = (smem_addr(smem_raw) + 1023u) & ~1023u;
    uint8_t* const gbase = smem_raw + (base - smem_addr(smem_raw));
    const int tid = threadIdx.x, lane = tid & 31, qr = lane >> 2, qi = lane & 3, wt = tid & 127;
    // Worker and warp of it, the same in a warp's registers; the warps past the workers': copies, MMAs.
    const int wk = __shfl_sync(0xffffffffu, tid >> 7, 0), ww = __shfl_sync(0xffffffffu, wt >> 5, 0);
    int32_t* const prefix = reinterpret_cast<int32_t*>(gbase + S::off_prefix);
    int32_t* const lens = prefix + p.entries + 1;
    Left* const s_left = reinterpret_cast<Left*>(gbase + S::off_left);
    float2* const s_ml = reinterpret_cast<float2*>(gbase + S::off_ml);
    const uint32_t range_at = base + S::off_range;
    const bool lists = p.lists != nullptr;
    const auto bar_of = [&](int w, int i) { return base + S::off_bar + (w * S::bars + i) * 8; };
    constexpr int kFull = 0, kEmpty = ST, kKReady = 2 * ST, kSDone = kKReady + 1, kPReady = kSDone + 1,
                  kVReady = kPReady + 1, kODone = kVReady + 1;

    if (tid == 0) {
        prefetch_map(&maps.k);
        prefetch_map(&maps.v);
        prefetch_map(&maps.k_scales);
        prefetch_map(&maps.v_scales);
    }
    if (wt == 0 && wk < W) {
        for (int i = 0; i < S::bars; ++i)
            mbar_init(bar_of(wk, i), i < ST || i == kSDone || i == kODone ? 1 : 128);
        fence_mbar_init();
        fence_proxy_async();
        s_left[wk].ended = s_left[wk].open = -1;
    }
    pdl_entry();
    fence_proxy_async_global();  // the cache may have been written by the kernel before
    if (tid < 32) tmem_alloc(base + S::off_tmem, 512);
    tc_fence_before();
    const int total = scan_entries<KT, 256>(p, prefix, lens, reinterpret_cast<int32_t*>(gbase + S::off_scan));
    tc_fence_after();
    const uint32_t tmem = lds_u32(base + S::off_tmem);

    const auto find = [&](int t, int unit_cost) {  // the entry at t (below the last one's end)
        int lo = 0, hi = p.entries;
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (prefix[mid] + unit_cost * p.x_units * mid <= t) lo = mid;
            else hi = mid;
        }
        return lo;
    };
    const int cost = total + kTcUnitCost * p.x_units * p.entries;
    const int per = max((cost + p.workers - 1) / p.workers, 1);
    const auto tiles_before = [&](int64_t at) {  // tiles that lie before a cost position
        if (at >= cost) return total;
        const int c = static_cast<int>(at), e = find(c, kTcUnitCost);
        const int nt = (prefix[e + 1] - prefix[e]) / p.x_units;
        const int rem = c - prefix[e] - kTcUnitCost * p.x_units * e, x = rem / (nt + kTcUnitCost);
        return prefix[e] + x * nt + max(rem - x * (nt + kTcUnitCost) - kTcUnitCost, 0);
    };
    // The workers' ranges: where one ends the next begins. Lane w has worker w's.
    const int cut = tiles_before((static_cast<int64_t>(blockIdx.x) * W + min(lane, W)) * per);
    if (tid < W) sts64(range_at + 8 * tid, 0, 0);
    __syncthreads();

    if (wk == W) {
        // ---- copies: lanes 8 w .. 8 w + 7 are worker w's, one for each box of a tile
        const int w = min(lane >> 3, W - 1), j = lane & 7;
        const unsigned group = 0xffu << (lane & 24);
        const int t0 = __shfl_sync(0xffffffffu, cut, w), t1 = __shfl_sync(0xffffffffu, cut, w + 1);
        const int n = lane >> 3 < W ? t1 - t0 : 0;
        const int boxes = KT / box, step_blk = KT / p.page_size, step_off = KT % p.page_size;
        const bool has_box = j < boxes;
        const uint32_t ring = base + w * S::worker_bytes;
        int* const s_pos = reinterpret_cast<int*>(gbase + S::off_rows + w * S::row_bytes + S::off_pos);
        int* const s_last = reinterpret_cast<int*>(gbase + S::off_rows + w * S::row_bytes + S::off_last);
        // The tile that is looked up: its entry, unit, tiles of the unit from it on, the lane's page of the
        // request or list and token in it, request, kv head, listed pages.
        int e = 0, x = 0, left = 0, blk = 0, off = 0, r = 0, head = 0, count = 0;
        const auto enter = [&](int tile) {
            const int b = lists ? e / p.heads : e;
            r = lists ? b / p.G : e;
            head = lists ? e - b * p.heads : x / p.row_tiles;
            count = !lists ? 0 : p.counts != nullptr ? max(min(p.counts[e], p.K), 0) : p.K;
            const int first = tile * KT + j * box;
            blk = first / p.page_size;
            off = first - blk * p.page_size;
        };
        const auto advance = [&]() {
            if (--left > 0) {
                blk += step_blk;
                off += step_off;
                if (off >= p.page_size) {
                    off -= p.page_size;
                    ++blk;
                }
                return;
            }
            if (++x == p.x_units) {
                ++e;
                x = 0;
            }
            left = (prefix[e + 1] - prefix[e]) / p.x_units;
            enter(0);
        };
        // Tile kk + 2's page of the request is loaded (lists), tile kk + 1's table entry, tile kk is copied.
        int l_page = -1, l_off = 0, l_head = 0, l_len = 0, l_r = 0;
        int c_page = -1, c_off = 0, c_head = 0, c_pos = kFar;
        const auto look = [&]() {
            l_page = !has_box ? -1 : !lists ? blk : blk < count ? p.lists[static_cast<int64_t>(e) * p.K + blk] : -1;
            l_off = off, l_head = head, l_len = lens[e], l_r = r;
        };
        const auto resolve = [&]() {
            c_page = -1, c_off = l_off, c_head = l_head, c_pos = kFar;
            const int64_t pos = static_cast<int64_t>(l_page) * p.page_size + l_off;
            if (l_page < 0 || pos >= l_len) return;
            c_pos = static_cast<int>(pos);
            c_page = p.table[static_cast<int64_t>(l_r) * p.table_stride + l_page];
        };
        int looked = 0;
        if (n > 0) {
            e = find(t0, 0);
            const int nt = (prefix[e + 1] - prefix[e]) / p.x_units;
            x = (t0 - prefix[e]) / nt;
            const int tile = t0 - prefix[e] - x * nt;
            left = nt - tile;
            enter(tile);
            look();
            resolve();
            if (++looked < n) {
                advance();
                look();
            }
        }
        int kk = 0;
        while (true) {
            const bool active = kk < n && lds_volatile(range_at + 8 * w + 4) == 0;
            if (!__any_sync(0xffffffffu, active)) break;
            const int s = kk % ST;
            bool ready = active && (kk < ST || mbar_poll(bar_of(w, kEmpty + s), (kk / ST - 1) & 1));
            ready = __shfl_sync(0xffffffffu, ready, lane & 24);
            if (!ready) continue;
            const uint32_t bar = bar_of(w, kFull + s), dst = ring + s * kSlotBytes;
            if (has_box)
                for (int i = 0; i < box / 16; ++i)
                    s_pos[8 * s + j * (box / 16) + i] = c_pos == kFar ? kFar : c_pos + 16 * i;
            int last = has_box ? c_pos + (c_pos == kFar ? 15 : box - 1) : 0;
#pragma unroll
            for (int o = 1; o < 8; o <<= 1) last = max(last, __shfl_xor_sync(group, last, o));
            if (j == 0) s_last[s] = last;
            __syncwarp(group);
            if (j == 0) mbar_arrive_expect_tx(bar, kSlotBytes + (kk + 1 == p.stall ? 16 : 0));
            __syncwarp(group);
            if (has_box) {
                const int page = c_page >= 0 && c_page < p.pages ? c_page : -1;
                const uint32_t codes = dst + j * box * (D / 2), scales = dst + 2 * kSideBytes + j * box * (D / 16);
                tma_load_4d(codes, &maps.k, 0, c_off, c_head, page, bar);
                tma_load_3d(scales, &maps.k_scales, c_off, c_head, page, bar);
                tma_load_4d(codes + kSideBytes, &maps.v, 0, c_off, c_head, page, bar);
                tma_load_3d(scales + kScaleBytes, &maps.v_scales, c_off, c_head, page, bar);
            }
            ++kk;
            if (kk < n) resolve();
            if (++looked < n) {
                advance();
                look();
            }
        }
        // No copy may outlive the worker's memory.
        for (int i = max(kk - ST, 0); i < kk; ++i) {
            bool done = true;
            mbar_wait(bar_of(w, kFull + i % ST), (i / ST) & 1, done, p.status, p.budget_ns, true);
        }
    } else {
        // ---- a worker
        const int worker = static_cast<int>(blockIdx.x) * W + wk, bar_id = 1 + wk;
        const int t0 = __shfl_sync(0xffffffffu, cut, wk), t1 = __shfl_sync(0xffffffffu, cut, wk + 1);
        const uint32_t ring = base + wk * S::worker_bytes, q_at = ring + S::off_q, p_at = ring + S::off_p;
        uint8_t* const rows = gbase + S::off_rows + wk * S::row_bytes;
        float* const s_fm = reinterpret_cast<float*>(rows);  // [N / 2] f, f, -m, -m
        int* const s_lim = reinterpret_cast<int*>(rows + S::off_lim);
        uint32_t* const s_nan = reinterpret_cast<uint32_t*>(rows + S::off_nan);
        float* const s_red = reinterpret_cast<float*>(rows + S::off_red);
        const int* const s_pos = reinterpret_cast<const int*>(rows + S::off_pos);
        const int* const s_last = reinterpret_cast<const int*>(rows + S::off_last);
        const uint32_t fm_at = base + S::off_rows + wk * S::row_bytes;
        const uint32_t my_lanes = static_cast<uint32_t>(32 * ww) << 16, t_a = tmem + S::t_cols * wk + my_lanes;
        bool ok = true;  // until a wait runs out; the same in a worker's threads outside the tile loop
        int k = 0, t = t0, e = t0 < t1 ? find(t0, 0) : 0;
        // The unit of tile t: entry e, unit x of its x_units, each of nt tiles.
        int nt = 1, x = 0;
        if (t0 < t1) {
            nt = (prefix[e + 1] - prefix[e]) / p.x_units;
            x = (t0 - prefix[e]) / nt;
        }
        // Half h of K's columns (this thread's token), and of V's tokens (the warp's 32 columns).
        const auto convert_k = [&](uint32_t kc, uint32_t ks, int h) {
            uint32_t sc, a[32];
            sc = lds_u32(ks + 8 * wt + 4 * h);
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                const uint4 v = lds_v4(kc + piece<64, KT>(wt, 2 * h + c));
                const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const uint32_t by = scale_pair(sc, 0, 0x4400u + 0x11u * (2 * c + (j >> 1)));
                    uint32_t f[4];
                    e2m1_to_f16(w[j], f);
#pragma unroll
                    for (int z = 0; z < 4; ++z) a[16 * c + 4 * j + z] = mul_f16x2(f[z], by);
                }
            }
            tmem_st32(t_a + 32 * h, a);
        };
        // Products of half h of the tokens, onto those before.
        const uint32_t one = elected(), t_w = __shfl_sync(0xffffffffu, tmem, 0) + S::t_cols * wk;
        const auto products = [&](int h, bool more) {
#pragma unroll
            for (int z = 0; z < KT / 32; ++z)
                umma_f16_ta(t_w + S::t_o, t_w + (h == 0 ? S::t_v : 0) + 8 * z,
                            umma_desc(p_at + (4 * h + z) * 32 * N, 16, 16 * N, N == 32 ? 4 : 6), idesc_f16(N, 1),
                            more || z > 0, one);
        };
        // A warp issues MMAs once all of the worker's operands are there (in step: one lane's branch
        // would take their operands out of uniform registers).
        const auto multiply = [&](int ready, const auto& issue) {
            mbar_wait(bar_of(wk, ready), k & 1, ok, p.status, p.budget_ns, true);
            __syncwarp();
            tc_fence_after();
            issue();
        };
        const uint32_t v_sel = 0x40u + 0x11u * (2 * (ww & 1) + (qr >> 2));
        const auto convert_v = [&](uint32_t vc, uint32_t vs, int h) {
            const uint32_t sc = vs + 4 * (ww >> 1) + 16 * qi, to = t_a + (h == 0 ? S::t_v : 0);
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                uint32_t vr[4], fr[2][8];
                ldsm4_t(vc + piece<64, KT>(64 * h + 32 * q + lane, ww), vr);
#pragma unroll
                for (int j = 0; j < 4; ++j) {  // tokens 64 h + 32 q + 8 j ..
                    const uint32_t at = sc + 8 * (64 * h + 32 * q + 8 * j);
                    const uint32_t by = scale_pair(lds_u32(at), lds_u32(at + 8), v_sel);
                    uint32_t f[4];
                    pairs_to_f16(vr[j], f);
#pragma unroll
                    for (int z = 0; z < 4; ++z)  // column 2 m + y of the four
                        fr[z >> 1][2 * j + (z & 1)] = mul_f16x2(f[z], by);
                }
                tmem_st_frag(to + 16 * q, fr[0]);
                tmem_st_frag(to + (16u << 16) + 16 * q, fr[1]);
            }
        };

#pragma unroll 1
        while (t < t1) {
            Unit u;
            {
                const int rt = p.row_tiles == 1 ? 0 : x % p.row_tiles;
                u.b0 = lists ? e / p.heads : e * p.G;
                u.head = lists ? e - u.b0 * p.heads : p.row_tiles == 1 ? x : x / p.row_tiles;
                u.m0 = rt * N;
                u.m_real = min(p.rows - u.m0, N);
            }
            const int u0 = prefix[e] + x * nt, u1 = u0 + nt, tend = min(u1, t1);
            const int len = lens[e], m_real = u.m_real;
            const auto row_limit = [&](int m) {  // the tokens that row m of the tile sees
                return lists ? len : max(len - p.G + 1 + u.verify_row(p, m), 0);
            };
            const int min_lim = row_limit(0), max_lim = row_limit(m_real - 1);

            // The queries as f16, scaled to [2^14, 2^15) by a power of two of each row: the second operand.
            {
                constexpr int kPer = 128 / N, kPieces = 16 / kPer;  // threads of a row; their 16-byte pieces
                const int n = wt / kPer, c0 = wt % kPer * kPieces;
                uint4 w[kPieces];
#pragma unroll
                for (int c = 0; c < kPieces; ++c) w[c] = make_uint4(0, 0, 0, 0);
                if (n < m_real) {
                    const int64_t b = u.b(p, n);
                    const int a = u.a(p, n);
                    const uint4* const row =
                        reinterpret_cast<const uint4*>(p.q + b * p.q_stride + static_cast<int64_t>(a) * D);
#pragma unroll
                    for (int c = 0; c < kPieces; ++c) w[c] = __ldg(row + c0 + c);
                }
                float a = 0.0f;
#pragma unroll
                for (int c = 0; c < kPieces; ++c) {
                    a = fmaxf(a, fmaxf(fabsf(bf_lo(w[c].x)), fabsf(bf_hi(w[c].x))));
                    a = fmaxf(a, fmaxf(fabsf(bf_lo(w[c].y)), fabsf(bf_hi(w[c].y))));
                    a = fmaxf(a, fmaxf(fabsf(bf_lo(w[c].z)), fabsf(bf_hi(w[c].z))));
                    a = fmaxf(a, fmaxf(fabsf(bf_lo(w[c].w)), fabsf(bf_hi(w[c].w))));
                }
#pragma unroll
                for (int s = 1; s < kPer; s <<= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, s));
                const int ex = static_cast<int>(__float_as_uint(a) >> 23);
                const int ue = min(14 + 127 - ex + 127, 253);
                float up = a > 0.0f && ex < 255 ? __uint_as_float(static_cast<uint32_t>(ue) << 23) : 1.0f;
                if (wt % kPer == 0) {
                    const float f = fmaxf(fabsf(p.scale_log2) / up * head_power(p.k_exp, u.head), 1.17549435e-38f);
                    s_fm[4 * (n >> 1) + (n & 1)] = f;
                    s_fm[4 * (n >> 1) + 2 + (n & 1)] = n < m_real ? -kNone : 0.0f;  // a row of zeros: weights of 1
                    s_lim[n] = n < m_real ? row_limit(n) : max_lim;
                    s_nan[n] = 0;
                }
                if (p.scale_log2 < 0.0f) up = -up;
#pragma unroll
                for (int c = 0; c < kPieces; ++c) {
                    const uint32_t v[4] = {w[c].x, w[c].y, w[c].z, w[c].w};
                    uint32_t f[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) f[j] = f16x2(bf_lo(v[j]) * up, bf_hi(v[j]) * up);
                    const int cc = c0 + c;
                    sts_u4(q_at + (cc >> 3) * (N * 128) + n * 128 + (((cc & 7) ^ (n & 7)) << 4), f[0], f[1], f[2], f[3]);
                }
            }
            fence_proxy_async();
            worker_sync(bar_id);
            float l[N];
#pragma unroll
            for (int n = 0; n < N; ++n) l[n] = 0.0f;
            bool started = false;

#pragma unroll 1
            for (; t < tend && ok; ++t, ++k) {
                const int slot = k % ST;
                const uint32_t kc = ring + slot * kSlotBytes, vc = kc + kSideBytes, ks = vc + kSideBytes, vs = ks + kScaleBytes;
                mbar_wait(bar_of(wk, kFull + slot), (k / ST) & 1, ok, p.status, p.budget_ns);
                const int pos = s_pos[8 * slot + (wt >> 4)] + (wt & 15);
                const bool masked = s_last[slot] >= min_lim;  // some row does not see some token
                if (masked) {
                    // A NaN among the scales of this token's V: rows that see it get it in the block's
                    // columns at the end, and 0 stands in its place for the products.
                    uint32_t w0, w1;
                    lds64(vs + 8 * wt, w0, w1);
                    if (pos >= max_lim) {
                        sts64(vs + 8 * wt, 0, 0);
                    } else if (pos >= min_lim) {
                        const uint32_t n0 = nan_bytes(w0), n1 = nan_bytes(w1);
                        if ((n0 | n1) != 0) {
                            uint32_t blocks = 0;
                            for (int j = 0; j < 4; ++j) {
                                blocks |= (n0 >> (8 * j + 7) & 1u) << j;
                                blocks |= (n1 >> (8 * j + 7) & 1u) << (4 + j);
                            }
                            for (int n = 0; n < m_real; ++n)
                                if (pos < s_lim[n]) atomicOr(&s_nan[n], blocks);
                            sts64(vs + 8 * wt, w0 & ~((n0 >> 7) * 0xffu), w1 & ~((n1 >> 7) * 0xffu));
                        }
                    }
                    fence_proxy_async();  // before the slot is copied into again
                    worker_sync(bar_id);
                }
                // K, the half first that V's second half of the tile before did not take.
                convert_k(kc, ks, 1);
                if (k > 0) mbar_wait(bar_of(wk, kODone), (k - 1) & 1, ok, p.status, p.budget_ns, true);
                tc_fence_after();
                convert_k(kc, ks, 0);
                tmem_wait_st();
                tc_fence_before();
                mbar_arrive_local(bar_of(wk, kKReady));
                if (ww == 3) multiply(kKReady, [&]() {
#pragma unroll
                    for (int s = 0; s < D / 16; ++s)
                        umma_f16_ta(t_w + S::t_s, t_w + 8 * s,
                                    umma_desc(q_at + (s >> 2) * (N * 128) + (s & 3) * 32, 16, 1024, 2),
                                    idesc_f16(N, 0), s > 0, one);
                    umma_commit_one(bar_of(wk, kSDone), one);
                });
                convert_v(vc, vs, 0);
                mbar_wait(bar_of(wk, kSDone), k & 1, ok, p.status, p.budget_ns, true);
                tc_fence_after();

                float xs[N], over = kNone;
                const auto logits = [&]() {  // the token's, -infinity where a row does not see it
                    tmem_ldn(t_a + S::t_s, xs);
                    if (masked && pos >= min_lim) {
#pragma unroll
                        for (int n = 0; n < N; ++n)
                            if (pos >= s_lim[n]) xs[n] = -INFINITY;
                    }
                };
                const auto exponents = [&]() {
#pragma unroll
                    for (int n = 0; n < N; n += 2) {
                        const float4 fm = lds_f4(fm_at + 8 * n);
                        unpack2(fma2(pack2(xs[n], xs[n + 1]), pack2(fm.x, fm.y), pack2(fm.z, fm.w)), xs[n], xs[n + 1]);
                    }
                };
                logits();
                exponents();
#pragma unroll
                for (int n = 0; n < N; n += 2) over = max3(over, xs[n], xs[n + 1]);
                if (worker_or(bar_id, over > kSlack + kPShift || !ok)) {
                    ok = worker_and(bar_id, ok);
                    if (!ok) break;
                    logits();
#pragma unroll
                    for (int n = 0; n < N; ++n) xs[n] = fmaf(xs[n], s_fm[4 * (n >> 1) + (n & 1)], -kPShift);
                    const float most = reduce_rows<N>(xs, lane, [](float a, float b) { return fmaxf(a, b); });
                    if (lane < N) s_red[ww * N + lane] = most;
                    worker_sync(bar_id);
                    if (wt < N) {
                        float* const minus = &s_fm[4 * (wt >> 1) + 2 + (wt & 1)];
                        const float was = -*minus;
                        const float now = fmaxf(fmaxf(was, fmaxf(s_red[wt], s_red[N + wt])),
                                                fmaxf(s_red[2 * N + wt], s_red[3 * N + wt]));
                        *minus = -now;
                        s_red[wt] = now > was ? ex2_approx(was - now) : 1.0f;
                    }
                    worker_sync(bar_id);
#pragma unroll
                    for (int n = 0; n < N; ++n) l[n] *= s_red[n];
                    if (started) {
                        tmem_ldn(t_a + S::t_o, xs);
#pragma unroll
                        for (int n = 0; n < N; ++n) xs[n] *= s_red[n];
                        tmem_stn(t_a + S::t_o, xs);
                    }
                    logits();
                    exponents();
                }
                // Weights: a token's N values in a row of shared memory.
                {
                    uint32_t w[N / 2];
#pragma unroll
                    for (int n = 0; n < N; n += 2) {
                        const float a = ex2_approx(xs[n]), b = ex2_approx(xs[n + 1]);
                        unpack2(add2(pack2(l[n], l[n + 1]), pack2(a, b)), l[n], l[n + 1]);
                        w[n >> 1] = f16x2(a, b);
                    }
#pragma unroll
                    for (int c = 0; c < N / 8; ++c)
                        sts_u4(p_at + piece<2 * N, KT>(wt, c), w[4 * c], w[4 * c + 1], w[4 * c + 2], w[4 * c + 3]);
                }
                tmem_wait_st();
                fence_proxy_async();
                tc_fence_before();
                mbar_arrive_local(bar_of(wk, kPReady));
                if (ww == 2) multiply(kPReady, [&]() { products(0, started); });
                convert_v(vc, vs, 1);
                mbar_arrive_local(bar_of(wk, kEmpty + slot));
                tmem_wait_st();
                tc_fence_before();
                mbar_arrive_local(bar_of(wk, kVReady));
                if (ww == 2) multiply(kVReady, [&]() {
                    products(1, true);
                    umma_commit_one(bar_of(wk, kODone), one);
                });
                started = true;
            }

            if (k > 0 && started) mbar_wait(bar_of(wk, kODone), (k - 1) & 1, ok, p.status, p.budget_ns, true);
            ok = worker_and(bar_id, ok);
            if (!ok) {
                // A wait ran out: this unit and the worker's later ones are NaN (a NaN sum stays one
                // through every join), and nothing more is copied or multiplied.
                t = tend;
#pragma unroll
                for (int n = 0; n < N; ++n) l[n] = NAN;
                if (wt == 0) asm volatile("st.volatile.shared.u32 [%0], %1;" ::"r"(range_at + 8 * wk + 4), "r"(1) : "memory");
            }
            tc_fence_after();

            // The unit's rows, or this worker's part of them.
            {
                const float sum = reduce_rows<N>(l, lane, [](float a, float b) { return a + b; });
                if (lane < N) s_red[ww * N + lane] = sum;
            }
            worker_sync(bar_id);
            const bool whole = u0 >= t0 && u1 <= t1, open = u1 > t1;
            if (!whole) {
                const int unit = e * p.x_units + x, at = u0 + kTcUnitCost * (unit + 1);  // its first tile
                u.first_cta = at / per / W;
                u.last_cta = (at + nt - 1) / per / W;
                Left* const left = s_left + wk;
                if (wt == 0 && open) {
                    left->open = unit;
                    left->open_begins = u0 >= t0;
                    left->open_unit = u;
                } else if (wt == 0) {
                    left->ended = unit;
                    left->ended_unit = u;
                }
            }
            // The accumulators go where the queries and weights were, a row's columns together (as the joins
            // want it), and from there on: this runs once a unit, out of instructions that are not
            // cached, so it is kept short.
            {
                float o[N];
                const float vref = started ? head_power(p.v_exp, u.head) : 0.0f;
                if (started) tmem_ldn(t_a + S::t_o, o);
                const int col = 32 * ww + 4 * (lane & 7) + 2 * (lane >> 4) + (lane >> 3 & 1);
#pragma unroll
                for (int n = 0; n < N; ++n)
                    asm volatile("st.shared.f32 [%0], %1;" ::"r"(q_at + n * D * 4 +
                                                                (((col >> 2) ^ ((n >> 1 & 3) << 1)) << 4) + 4 * (col & 3)),
                                 "f"(started ? o[n] * vref : 0.0f)
                                 : "memory");
            }
            worker_sync(bar_id);
#pragma unroll 1
            for (int i = wt; i < m_real * (D / 4); i += 128) {
                const int n = i / (D / 4), c = i % (D / 4);
                const uint32_t at = q_at + n * D * 4 + ((c ^ ((n >> 1 & 3) << 1)) << 4);
                float4 v = lds_f4(at);
                const float sum = (s_red[n] + s_red[N + n]) + (s_red[2 * N + n] + s_red[3 * N + n]);
                const float top = -s_fm[4 * (n >> 1) + 2 + (n & 1)];
                const bool nan = (s_nan[n] >> (c >> 2) & 1u) != 0;
                if (nan) v = make_float4(NAN, NAN, NAN, NAN);
                if (whole) {
                    write_row(p, u, D, n, 4 * c, v, top, sum);
                    continue;
                }
                const float2 ml = make_float2(top == kNone ? -INFINITY : top, sum);
                if (open) {
                    if (nan) sts_v4(at, v);
                    if (c == 0) s_ml[wk * N + n] = ml;
                } else {
                    const int64_t to = static_cast<int64_t>(worker) * N + n;
                    reinterpret_cast<float4*>(p.head + to * D)[c] = v;
                    if (c == 0) p.head_ml[to] = ml;
                }
            }
            tc_fence_before();
            worker_sync(bar_id);  // the rows' words and the accumulators are free again
            if (tend < t1 && ++x == p.x_units) {
                ++e;  // every entry has a tile
                x = 0;
                nt = (prefix[e + 1] - prefix[e]) / p.x_units;
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (tid < 32) {
        tc_fence_after();
        tmem_free(tmem, 512);
    }
    join_units<D, N, S::joiners, W, true>(p, base + S::off_q, S::worker_bytes, s_left, s_ml);
}

template <typename S>
int launch_tc(PagedParams p, const Maps<4>& maps, int box, int sms, int64_t tiles, smd_stream_t stream) {
    static SharedLimit limit;
    auto kernel = paged4_tc_kernel<S>;
    const int rc = limit.raise(kernel, S::smem(kMaxEntries));
    if (rc != SMD_OK) return rc;
    const int64_t want = (tiles + S::W - 1) / S::W;
    const int64_t grid = want < sms ? want : sms;
    p.workers = static_cast<int>(grid) * S::W;
    set_workspace(p, sms, S::N, kCols);
    return launch_pdl(kernel, dim3(static_cast<unsigned>(grid)), S::threads, S::smem(p.entries), stream, p, box,
                      maps);
}

}  // namespace

int paged4_tc(const PagedParams& p, const Maps<4>& maps, int box, int rows, int sms, int64_t tiles,
              smd_stream_t stream) {
    return rows == 16 ? launch_tc<TcShape<16, 4, 2>>(p, maps, box, sms, tiles, stream)
                      : launch_tc<TcShape<32, 3, 3>>(p, maps, box, sms, tiles, stream);
}

}  // namespace smd

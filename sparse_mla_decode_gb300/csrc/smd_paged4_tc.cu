// Attention over a paged E2M1 cache on the tcgen05 tensor cores, 128 columns
// (smd_paged4_decode; other sizes: smd_paged_decode.cuh).
//
// The definition, the cuts of the batch and the joins are smd_paged_decode.cuh's; a worker is
// four warps here, and a tile 128 tokens. For a tile of a unit with R query rows (8, 16 or 32):
//   S^T [128 tokens x R] = K Q^T,  P = 2^(S f - m),  O^T [128 columns x R] += V^T P
// Tokens (then columns) are the MMA's 128 rows, so that every lane of the tensor cores
// has work whatever the number of query rows, and the rows are its N.
//
// What bounds it: 144 bytes of a (token, kv head) are few for what has to be done to them. 256 codes
// converted to f16 and multiplied by their scales took half of the instructions of this kernel's
// first form. So K is not converted: the tensor cores multiply E2M1 codes with E4M3 scales of 16
// along the columns as the cache holds them, out of shared memory where the copies put them. The
// queries, the other operand, are E2M1 too then, six digits in base 8 of a value: two MMAs of 128 x 48 x 64
// at 8 rows, and 20 additions a token for the digits, instead of 64 conversions, 64 multiplications and 16
// more for the scales. (The scales go into tensor memory; a negative one, which the MMA takes for a positive,
// turns its codes' signs.) V's scales are of 16 columns, which the second product does not add over: V is
// formed in registers and stored into tensor memory, from where tcgen05.mma takes its f16 operand.
// Transposing ldmatrix gives a thread four columns of two tokens, whose nibbles are put side
// by side (the f16 pairs of an A operand run along the tokens); the store's 16x128b shape takes them as
// an MMA fragment, so that lane 32 w + 16 m + 8 y + g holds column 32 w + 4 g + 2 m + y.
//
// A worker's tile is a chain: scales, S^T, the weights, V, the product. The four workers of an SM (three
// at 32 rows: 96, 104 and 152 columns of tensor memory each; V lies over the logits that were read) hide
// one another's waits; two tiles' logits in flight for three workers were slower (98 us for 91, when one warp copied
// for all workers; not measured since), and so were warps of one job each (K, V, weights) in turn on a pipeline's tiles
// (211 for 92 at 16 rows, then, too). Each worker has
// a warp for its copies, which looks up 4 to 32 tiles at once, a lane for each box: with one such warp for
// all workers the round trips for table entries bound the kernel (91 us; 147 with pages of 16 tokens).
// A thread has one token's logits: no reduction over tokens is needed but for the sums, once a unit,
// and the maximum, which is moved only when a logit exceeds it by more than 2^8 (the worker's vote;
// accumulators in tensor memory then come down by 2^(old - new)).
//
// Measured (GB300, device time; of the rate at which the GPU copies), pages of 64 tokens:
//   64 requests of 1024 .. 8192 tokens, 8 / 16 / 32 / 64 rows    73 us 70% / 82 us 63% / 115 us 45% / 208 us 26%
//   the same with pages of 16 tokens, 8 / 16 / 32 rows           89 us / 94 us / 123 us
//   64 listed pages in each of 64 requests, 8 / 16 / 32 rows     69 us 66% / 78 us 59% / 108 us 43%
//   16 requests up to 65536 tokens, 8 / 16 / 32 rows             110 us 83% / 121 us 76% / 170 us 54%
//   200 requests up to 300 tokens, 8 / 16 / 32 rows              29 us / 36 us / 57 us
//   one request of 777 tokens, 8 / 16 / 32 rows                  12.6 us / 14.5 us / 17.5 us
// At 8 rows instructions are issued in 59% of the cycles and the logic pipe is busy for 47% (V's
// conversions are most of it); copies alone take 68 us of the 73. Start and joins are some 12 us, as in
// smd_paged_decode.cu. At 32 rows three workers wait for one another's chains (51% of the issue slots).
#include "smd_paged4_tc.h"

namespace smd {
namespace {

constexpr int kTile = 128;              // tokens
constexpr int kCols = 128;              // columns of a head
constexpr int kSideBytes = kTile * kCols / 2, kScaleBytes = kTile * kCols / 16;
constexpr int kSlotBytes = 2 * (kSideBytes + kScaleBytes);
constexpr int kFar = 0x7ffffff0;        // the position of tokens that no row sees (15 more fit an int)
constexpr int kDigits = 6;              // of a query's value

// R query rows of a unit, W workers, ST slots of a worker's ring.
template <int R_, int W_, int ST_>
struct TcShape {
    static constexpr int R = R_, W = W_, ST = ST_;
    // What a unit's begin and end cost, in tiles: 1 / 3 / 4 / 6 / 9 at 8 rows 75.6 / 74.4 / 75.1 / 75.9 / 79.2 us
    // (the first measurement above), at 32 rows 130 / 120 / 117 / 118 / 123.
    static constexpr int unit_cost = R == 8 ? 3 : 4;
    static constexpr int threads = 160 * W;            // four warps of each worker, and one that copies for it
    static constexpr int joiners = 128 * W;            // threads of the joins
    static constexpr int N = R < 16 ? 16 : R;          // columns of P and O
    // A digit j has columns with number j / DS; the scales of set j % DS hold its 8^-(j % DS).
    static constexpr int DN = R == 8 ? 6 : 3, DS = kDigits / DN, NS = DN * R;
    // Tensor memory of a worker: the digits' logits (later V's operand), O^T, block scales of K and Q.
    static constexpr int t_o = NS < 64 ? 64 : NS, t_sa = t_o + N, t_sb = t_sa + 8, t_cols = t_sb + 8 * DS;
    static_assert(W * t_cols <= 512 && W <= 4 && t_cols % 4 == 0, "tensor memory");
    static constexpr int off_q = ST * kSlotBytes;
    static constexpr int off_p = off_q + DS * NS * kCols / 2;
    static constexpr int worker_bytes = off_p + N * kTile * 2;
    static_assert(worker_bytes % 1024 == 0, "swizzle atoms");
    static_assert(R * kCols * 4 <= worker_bytes - off_q, "a worker's accumulators fit its queries' and weights' places");
    // Of a worker, beside that: logit factors and maxima of row pairs, limits, NaN
    // blocks, sums of the warps, block scales, positions of 16 tokens each, the last of a tile.
    static constexpr int off_lim = 8 * R, off_nan = off_lim + 4 * R,
                         off_red = off_nan + 4 * R, off_sb = off_red + 16 * R, off_pos = off_sb + 8 * DS * R,
                         off_last = off_pos + ST * 32, row_bytes = off_last + 16;
    static constexpr int off_rows = W * worker_bytes;
    static constexpr int bars = 2 * ST + 4;  // of a worker: full, empty, K, S, V, O
    static constexpr int off_bar = off_rows + W * row_bytes;
    static constexpr int off_scan = off_bar + W * bars * 8;
    static constexpr int off_tmem = off_scan + 4 * ((threads / 32 + 3) / 4 * 4);
    static constexpr int off_ml = off_tmem + 16;
    static constexpr int off_left = off_ml + W * R * 8;
    static constexpr int off_range = off_left + W * 64;  // [W] whether a worker has stopped
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

// The same of E2M1 codes with E4M3 scales (their signs do not count) of 16 along K = 64 in tensor memory,
// A in shared memory too.
__device__ __forceinline__ void umma_e2m1(uint32_t d, uint64_t a_desc, uint64_t b_desc, uint32_t idesc, uint32_t a_scales,
                                          uint32_t b_scales, uint32_t accumulate, uint32_t one) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %6, 0;\n\tsetp.ne.b32 q, %7, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::mxf4nvf4.block_scale.scale_vec::4X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(a_scales), "r"(b_scales), "r"(accumulate), "r"(one)
        : "memory");
}

// Its instruction descriptor: FP32 D, M = 128.
__host__ __device__ constexpr uint32_t idesc_e2m1(int N) {
    return (1u << 7) | (1u << 10) | (static_cast<uint32_t>(N >> 3) << 17) | (8u << 24);
}

// Instruction descriptor of kind::f16: f16 A (K-major) and B, FP32 D, M = 128.
__host__ __device__ constexpr uint32_t idesc_f16(int N, int mn_major_b) {
    return (1u << 4) | (static_cast<uint32_t>(mn_major_b) << 16) | (static_cast<uint32_t>(N >> 3) << 17) |
           (8u << 24);
}

// 16 words of this thread's lane, and 8.
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

__device__ __forceinline__ void tmem_st8(uint32_t at, const uint32_t (&v)[8]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(at),
                 "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                 : "memory");
}

__device__ __forceinline__ void tmem_ldn(uint32_t at, float (&v)[8]) { tmem_ld8(at, v); }
__device__ __forceinline__ void tmem_ldn(uint32_t at, float (&v)[16]) { tmem_ld16(at, v); }
__device__ __forceinline__ void tmem_ldn(uint32_t at, float (&v)[32]) { tmem_ld32(at, v); }

__device__ __forceinline__ void tmem_stn(uint32_t at, const float (&v)[8]) {
    uint32_t w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = __float_as_uint(v[i]);
    tmem_st8(at, w);
}
template <int N>
__device__ __forceinline__ void tmem_stn(uint32_t at, const float (&v)[N]) {
#pragma unroll
    for (int c = 0; c < N; c += 16) {
        uint32_t w[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) w[i] = __float_as_uint(v[c + i]);
        tmem_st16(at + c, w);
    }
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
#pragma unroll
    for (int s = N; s < 32; s <<= 1) v[0] = op(v[0], __shfl_xor_sync(0xffffffffu, v[0], s));
    return v[0];
}

__device__ __forceinline__ void sts_u4(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d)
                 : "memory");
}


template <typename S>
__global__ void __launch_bounds__(S::threads, 1)
    paged4_tc_kernel(const PagedParams p, const int box, const __grid_constant__ Maps<4> maps) {
    constexpr int R = S::R, N = S::N, W = S::W, ST = S::ST, NS = S::NS, DS = S::DS, RS = R < 16 ? R : 16, D = kCols, KT = kTile;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t base = (smem_addr(smem_raw) + 1023u) & ~1023u;
    uint8_t* const gbase = smem_raw + (base - smem_addr(smem_raw));
    const int tid = threadIdx.x, lane = tid & 31, qr = lane >> 2, qi = lane & 3, wt = tid & 127;
    // Worker and warp of it, the same in a warp's registers; the warps past the workers' copy for them.
    const int ww = __shfl_sync(0xffffffffu, wt >> 5, 0), warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
    const bool copies = warp >= 4 * W;
    const int wk = copies ? warp - 4 * W : warp >> 2;
    int32_t* const prefix = reinterpret_cast<int32_t*>(gbase + S::off_prefix);
    int32_t* const lens = prefix + p.entries + 1;
    Left* const s_left = reinterpret_cast<Left*>(gbase + S::off_left);
    float2* const s_ml = reinterpret_cast<float2*>(gbase + S::off_ml);
    const uint32_t range_at = base + S::off_range;
    const bool lists = p.lists != nullptr;
    const auto bar_of = [&](int w, int i) { return base + S::off_bar + (w * S::bars + i) * 8; };
    constexpr int kFull = 0, kEmpty = ST, kKReady = 2 * ST, kSDone = kKReady + 1, kVReady = kSDone + 1,
                  kODone = kVReady + 1;

    if (tid == 0) {
        prefetch_map(&maps.k);
        prefetch_map(&maps.v);
        prefetch_map(&maps.k_scales);
        prefetch_map(&maps.v_scales);
    }
    if (wt == 0 && !copies) {
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
    const int cost = total + S::unit_cost * p.x_units * p.entries;
    const int per = max((cost + p.workers - 1) / p.workers, 1);
    const auto tiles_before = [&](int64_t at) {  // tiles that lie before a cost position
        if (at >= cost) return total;
        const int c = static_cast<int>(at), e = find(c, S::unit_cost);
        const int nt = (prefix[e + 1] - prefix[e]) / p.x_units;
        const int rem = c - prefix[e] - S::unit_cost * p.x_units * e, x = rem / (nt + S::unit_cost);
        if (uncut(nt, per)) return prefix[e] + x * nt;
        return prefix[e] + x * nt + max(rem - x * (nt + S::unit_cost) - S::unit_cost, 0);
    };
    // The workers' ranges: where one ends the next begins. Lane w has worker w's.
    const int cut = tiles_before((static_cast<int64_t>(blockIdx.x) * W + min(lane, W)) * per);
    const int t0 = __shfl_sync(0xffffffffu, cut, wk), t1 = __shfl_sync(0xffffffffu, cut, wk + 1);
    if (tid < W) sts32(range_at + 4 * tid, 0);
    __syncthreads();

    if (copies) {
        // ---- lane j + boxes i copies box j of tile i of those that are looked up together
        const int boxes = KT / box, at_once = 32 / boxes, mine = lane / boxes, j = lane % boxes;
        const int n = t1 - t0;
        const uint32_t ring = base + wk * S::worker_bytes;
        int* const s_pos = reinterpret_cast<int*>(gbase + S::off_rows + wk * S::row_bytes + S::off_pos);
        int* const s_last = reinterpret_cast<int*>(gbase + S::off_rows + wk * S::row_bytes + S::off_last);
        int page = -1, off = 0, head = 0, pos = kFar, last = 0;
        const auto look = [&](int kk) {
            page = -1, off = 0, head = 0, pos = kFar;
            if (kk < n) {
                const int t = t0 + kk, e = find(t, 0), nt = (prefix[e + 1] - prefix[e]) / p.x_units;
                const int x = (t - prefix[e]) / nt, first = (t - prefix[e] - x * nt) * KT + j * box;
                const int b = lists ? e / p.heads : e, r = lists ? b / p.G : e;
                head = lists ? e - b * p.heads : x / p.row_tiles;
                int blk = first / p.page_size;
                off = first - blk * p.page_size;
                if (lists) {
                    const int count = p.counts != nullptr ? max(min(p.counts[e], p.K), 0) : p.K;
                    blk = blk < count ? p.lists[static_cast<int64_t>(e) * p.K + blk] : -1;
                }
                const int64_t to = static_cast<int64_t>(blk) * p.page_size + off;
                if (blk >= 0 && to < lens[e]) {
                    pos = static_cast<int>(to);
                    page = p.table[static_cast<int64_t>(r) * p.table_stride + blk];
                    if (page >= p.pages) page = -1;
                }
            }
            page = max(page, -1);
            last = pos + (pos == kFar ? 15 : box - 1);
            for (int o = 1; o < boxes; o <<= 1) last = max(last, __shfl_xor_sync(0xffffffffu, last, o));
        };
        int kk = 0;
        bool run = true;
#pragma unroll 1
        for (; kk < n; ++kk) {
            const int i = kk & (at_once - 1), s = kk % ST;
            if (i == 0) look(kk + mine);
            // The worker's waits are bounded, and the last that runs out stops this.
            while (run && kk >= ST && !mbar_test(bar_of(wk, kEmpty + s), (kk / ST - 1) & 1))
                run = lds_volatile(range_at + 4 * wk) == 0;
            run = __all_sync(0xffffffffu, run);
            if (!run) break;
            const uint32_t bar = bar_of(wk, kFull + s), dst = ring + s * kSlotBytes;
            if (mine == i) {
                for (int z = 0; z < box / 16; ++z) s_pos[8 * s + j * (box / 16) + z] = pos == kFar ? kFar : pos + 16 * z;
                if (j == 0) s_last[s] = last;
            }
            __syncwarp();
            if (lane == 0) mbar_arrive_expect_tx(bar, kSlotBytes + (kk + 1 == p.stall ? 16 : 0));
            __syncwarp();
            if (mine == i) {
                const uint32_t codes = dst + j * box * (D / 2), scales = dst + 2 * kSideBytes + j * box * (D / 16);
                tma_load_4d(codes, &maps.k, 0, off, head, page, bar);
                tma_load_3d(scales, &maps.k_scales, off, head, page, bar);
                tma_load_4d(codes + kSideBytes, &maps.v, 0, off, head, page, bar);
                tma_load_3d(scales + kScaleBytes, &maps.v_scales, off, head, page, bar);
            }
        }
        // No copy may outlive the worker's memory.
        for (int i = max(kk - ST, 0); i < kk; ++i) {
            bool done = true;
            mbar_wait(bar_of(wk, kFull + i % ST), (i / ST) & 1, done, p.status, p.budget_ns, true);
        }
    } else {
        // ---- a worker
        const int worker = static_cast<int>(blockIdx.x) * W + wk, bar_id = 1 + wk;
        const uint32_t ring = base + wk * S::worker_bytes, q_at = ring + S::off_q, p_at = ring + S::off_p;
        uint8_t* const rows = gbase + S::off_rows + wk * S::row_bytes;
        float* const s_fm = reinterpret_cast<float*>(rows);  // [R / 2] f, f, -m, -m
        int* const s_lim = reinterpret_cast<int*>(rows + S::off_lim);
        uint32_t* const s_nan = reinterpret_cast<uint32_t*>(rows + S::off_nan);
        float* const s_red = reinterpret_cast<float*>(rows + S::off_red);
        const int* const s_pos = reinterpret_cast<const int*>(rows + S::off_pos);
        const int* const s_last = reinterpret_cast<const int*>(rows + S::off_last);
        const uint32_t fm_at = base + S::off_rows + wk * S::row_bytes, sb_at = fm_at + S::off_sb;
        const uint32_t my_lanes = static_cast<uint32_t>(32 * ww) << 16, t_a = tmem + S::t_cols * wk + my_lanes;
        bool ok = true;  // until a wait runs out; the same in a worker's threads outside the tile loop
        int k = 0, t = t0, e = t0 < t1 ? find(t0, 0) : 0;
        // The unit of tile t: entry e, unit x of its x_units, each of nt tiles.
        int nt = 1, x = 0;
        if (t0 < t1) {
            nt = (prefix[e + 1] - prefix[e]) / p.x_units;
            x = (t0 - prefix[e]) / nt;
        }
        // Logits, some digits apart; products of all tokens, onto those before.
        const uint32_t one = elected(), t_w = __shfl_sync(0xffffffffu, tmem, 0) + S::t_cols * wk;
        const auto make_logits = [&](uint32_t kc) {
#pragma unroll
            for (int i = 0; i < DS * (D / 64); ++i) {
                const int set = i / (D / 64), half = i % (D / 64);
                umma_e2m1(t_w, umma_desc(kc + 32 * half, 16, 512, 4),
                          umma_desc(q_at + set * (NS * 64) + 32 * half, 16, 512, 4), idesc_e2m1(NS),
                          t_w + S::t_sa + 4 * half, t_w + S::t_sb + 8 * set + 4 * half, i > 0, one);
            }
            umma_commit_one(bar_of(wk, kSDone), one);
        };
        const auto products = [&](bool more) {
#pragma unroll
            for (int z = 0; z < KT / 16; ++z)
                umma_f16_ta(t_w + S::t_o, t_w + 8 * z, umma_desc(p_at + z * 32 * N, 16, 16 * N, N == 32 ? 4 : 6),
                            idesc_f16(N, 1), more || z > 0, one);
            umma_commit_one(bar_of(wk, kODone), one);
        };
        // A warp issues MMAs once all of the worker's operands are there (in step: one lane's branch
        // would take their operands out of uniform registers).
        const auto multiply = [&](int ready, int parity, const auto& issue) {
            mbar_wait(bar_of(wk, ready), parity, ok, p.status, p.budget_ns, true);
            __syncwarp();
            tc_fence_after();
            issue();
        };
        const uint32_t v_sel = 0x40u + 0x11u * (2 * (ww & 1) + (qr >> 2));
        const auto convert_v = [&](uint32_t vc, uint32_t vs) {
            const uint32_t sc = vs + 4 * (ww >> 1) + 16 * qi;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                uint32_t vr[4], fr[2][8];
                ldsm4_t(vc + piece<64, KT>(32 * q + lane, ww), vr);
#pragma unroll
                for (int j = 0; j < 4; ++j) {  // tokens 32 q + 8 j ..
                    const uint32_t at = sc + 8 * (32 * q + 8 * j);
                    const uint32_t by = scale_pair(lds_u32(at), lds_u32(at + 8), v_sel);
                    uint32_t f[4];
                    pairs_to_f16(vr[j], f);
#pragma unroll
                    for (int z = 0; z < 4; ++z)  // column 2 m + y of the four
                        fr[z >> 1][2 * j + (z & 1)] = mul_f16x2(f[z], by);
                }
                tmem_st_frag(t_a + 16 * q, fr[0]);
                tmem_st_frag(t_a + (16u << 16) + 16 * q, fr[1]);
            }
        };

#pragma unroll 1
        while (t < t1) {
            Unit u;
            {
                const int rt = p.row_tiles == 1 ? 0 : x % p.row_tiles;
                u.b0 = lists ? e / p.heads : e * p.G;
                u.head = lists ? e - u.b0 * p.heads : p.row_tiles == 1 ? x : x / p.row_tiles;
                u.m0 = rt * R;
                u.m_real = min(p.rows - u.m0, R);
            }
            const int u0 = prefix[e] + x * nt, u1 = u0 + nt, tend = min(u1, t1);
            const int len = lens[e], m_real = u.m_real;
            const auto row_limit = [&](int m) {  // the tokens that row m of the tile sees
                return lists ? len : max(len - p.G + 1 + u.verify_row(p, m), 0);
            };
            const int min_lim = row_limit(0), max_lim = row_limit(m_real - 1);

            // The queries as digits: in a block of 16 columns a value is 2^e (the block's scale; 2^-14 of the row's
            // largest or more) times a sum of 8^-j d_j, d_j in -4 .. 3, whose codes are E2M1's of d_j / 2. That is
            // exact for values of 2^-8 of the block's largest and more; smaller ones are off by at most 2^-16 of it.
            {
                constexpr int kPer = 128 / R, kPieces = 16 / kPer;  // threads of a row; their 8 columns each
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
                // Exponents of the blocks and of the row.
                constexpr int kBlocks = kPieces < 2 ? 1 : kPieces / 2;
                int eb[kBlocks], top = 1;
#pragma unroll
                for (int c = 0; c < kBlocks; ++c) {
                    uint32_t a = 0;
#pragma unroll
                    for (int z = 2 * c; z < min(2 * c + 2, kPieces); ++z) {
                        const uint32_t v[4] = {w[z].x, w[z].y, w[z].z, w[z].w};
#pragma unroll
                        for (int j = 0; j < 4; ++j) a = max(a, max(v[j] & 0x7f80u, (v[j] >> 16) & 0x7f80u));
                    }
                    eb[c] = static_cast<int>(a >> 7);
                    if (kPieces < 2) eb[c] = max(eb[c], __shfl_xor_sync(0xffffffffu, eb[c], 1));
                    top = max(top, eb[c]);
                }
#pragma unroll
                for (int s = 1; s < kPer; s <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, s));
                const bool nan = top == 255;  // or an infinity: all of the row's logits are NaN
                if (wt % kPer == 0) {
                    // Logits are 2^(top - 127 - 7) times what the products give.
                    const float base2 = __uint_as_float(top > 7 ? static_cast<uint32_t>(top - 7) << 23 : 1u << (15 + top));
                    const float f = fmaxf(fabsf(p.scale_log2) * (base2 * head_power(p.k_exp, u.head)), 1.17549435e-38f);
                    s_fm[4 * (n >> 1) + (n & 1)] = f;
                    s_fm[4 * (n >> 1) + 2 + (n & 1)] = n < m_real ? -kNone : 0.0f;  // a row of zeros: weights of 1
                    s_lim[n] = n < m_real ? row_limit(n) : max_lim;
                    s_nan[n] = 0;
                }
#pragma unroll
                for (int c = 0; c < kPieces; ++c) {
                    const int e2 = max(eb[c >> 1], max(top - 14, 1));
                    if (kPieces >= 2 ? c % 2 == 0 : wt % 2 == 0)
#pragma unroll
                        for (int z = 0; z < DS; ++z) {
                            const int e4 = e2 - top + 8 - 3 * z;  // -9 or more: E4M3's last three are subnormal
                            asm volatile("st.shared.u8 [%0], %1;" ::"r"(sb_at + 8 * (z * R + n) + ((c0 + c) >> 1)),
                                         "r"(nan ? 0x7f : e4 >= -6 ? (e4 + 7) << 3 : 1 << (e4 + 9))
                                         : "memory");
                        }
                    // y in [1, 2) where the block is largest, with 15 binary places
                    const float up = __uint_as_float(e2 < 254 ? static_cast<uint32_t>(254 - e2) << 23 : 1u << 22);
                    const float places = p.scale_log2 < 0.0f ? -32768.0f : 32768.0f;
                    const uint32_t v[4] = {w[c].x, w[c].y, w[c].z, w[c].w};
                    uint32_t y[8];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        y[2 * j] = nan ? 0 : __float2int_rn(bf_lo(v[j]) * up * places) + 0444444;
                        y[2 * j + 1] = nan ? 0 : __float2int_rn(bf_hi(v[j]) * up * places) + 0444444;
                    }
                    const int cc = c0 + c;
#pragma unroll
                    for (int j = 0; j < kDigits; ++j) {
                        uint32_t o = 0;  // d_j + 4
#pragma unroll
                        for (int z = 0; z < 8; ++z) o |= (y[z] >> (3 * (kDigits - 1 - j)) & 7u) << (4 * z);
                        const uint32_t minus = (~(o >> 2) & 0x11111111u) * 15u;
                        const uint32_t code = ((0xccccccccu - o) & minus) | ((o ^ 0x44444444u) & ~minus);
                        sts32(q_at + piece<64, KT>((j % DS * S::DN + j / DS) * R + n, cc >> 2) + 4 * (cc & 3), code);
                    }
                }
                if (R < 16) sts_u4(p_at + piece<2 * N, KT>(wt, 1), 0, 0, 0, 0);  // columns without a row
            }
            fence_proxy_async();
            worker_sync(bar_id);
#pragma unroll
            for (int i = 0; i < DS; ++i) {  // their scales: column c of the lane l has row 32 c + l's
                uint32_t w0, w1;
                lds64(sb_at + 8 * (i * R + lane % R), w0, w1);
                const uint32_t v[8] = {w0, w0, w0, w0, w1, w1, w1, w1};
                tmem_st8(t_a + S::t_sb + 8 * i, v);
            }
            float l[R];
#pragma unroll
            for (int n = 0; n < R; ++n) l[n] = 0.0f;
            bool started = false;

            const bool alive = ok;  // the same in the worker's threads
#pragma unroll 1
            for (; alive && t < tend; ++t, ++k) {  // until a vote finds that a wait has run out
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
                // K's block scales, without signs: those turn the codes'.
                {
                    uint32_t v[8], w0, w1;
#pragma unroll
                    for (int c = 0; c < 4; ++c) lds64(ks + 8 * (32 * c + lane), v[c], v[4 + c]);
                    lds64(ks + 8 * wt, w0, w1);
                    if (((w0 | w1) & 0x80808080u) != 0) {
                        for (int c = 0; c < 8; ++c)
                            if ((c < 4 ? w0 : w1) >> (8 * (c & 3) + 7) & 1u) {
                                const uint32_t at = kc + piece<64, KT>(wt, c >> 1) + 8 * (c & 1);
                                uint32_t a, b;
                                lds64(at, a, b);
                                sts64(at, a ^ 0x88888888u, b ^ 0x88888888u);
                            }
                        fence_proxy_async();
                    }
#pragma unroll
                    for (int c = 0; c < 8; ++c) v[c] &= 0x7f7f7f7fu;
                    tmem_st8(t_a + S::t_sa, v);
                }
                tmem_wait_st();
                tc_fence_before();
                mbar_arrive_local(bar_of(wk, kKReady));
                if (ww == 3) multiply(kKReady, k & 1, [&]() {
                    if (k > 0) {  // the logits' place is free again
                        mbar_wait(bar_of(wk, kODone), (k - 1) & 1, ok, p.status, p.budget_ns, true);
                        tc_fence_after();
                    }
                    make_logits(kc);
                });
                mbar_wait(bar_of(wk, kSDone), k & 1, ok, p.status, p.budget_ns, true);
                tc_fence_after();
                bool stop = false;
#pragma unroll
                for (int r0 = 0; r0 < R; r0 += RS) {  // some rows at a time: their logits are registers
                    float xs[RS], over = kNone;
                    // The token's logits out of their digits', -infinity where a row does not see it.
                    const auto logits = [&]() {
                        uint64_t x[RS / 2];
                        const uint64_t by = DS == 1 ? pack2(0.125f, 0.125f) : pack2(0.015625f, 0.015625f);  // 8^-DS
                        const auto add = [&](const float* d, int digits, bool first) {
#pragma unroll
                            for (int z = digits - 1; z >= 0; --z)
#pragma unroll
                                for (int n = 0; n < RS; n += 2) {
                                    const uint64_t v = pack2(d[RS * z + n], d[RS * z + n + 1]);
                                    x[n >> 1] = first && z == digits - 1 ? v : fma2(x[n >> 1], by, v);
                                }
                        };
                        if (RS < R) {
#pragma unroll
                            for (int z = S::DN - 1; z >= 0; --z) {
                                float d[RS];
                                tmem_ldn(t_a + R * z + r0, d);
                                add(d, 1, z == S::DN - 1);
                            }
                        } else {
                            constexpr int kEach = 32 / RS, kFirst = (NS - 1) / 32;  // digits of a load; the last ones' load
#pragma unroll
                            for (int c = kFirst; c >= 0; --c) {
                                if (NS - 32 * c >= 32) {
                                    float d[32];
                                    tmem_ld32(t_a + 32 * c, d);
                                    add(d, kEach, c == kFirst);
                                } else {
                                    float d[16];
                                    tmem_ld16(t_a + 32 * c, d);
                                    add(d, kEach / 2, true);
                                }
                            }
                        }
#pragma unroll
                        for (int n = 0; n < RS; n += 2) unpack2(x[n >> 1], xs[n], xs[n + 1]);
                        if (masked && pos >= min_lim) {
#pragma unroll
                            for (int n = 0; n < RS; ++n)
                                if (pos >= s_lim[r0 + n]) xs[n] = -INFINITY;
                        }
                    };
                    const auto exponents = [&]() {
#pragma unroll
                        for (int n = 0; n < RS; n += 2) {
                            const float4 fm = lds_f4(fm_at + 8 * (r0 + n));
                            unpack2(fma2(pack2(xs[n], xs[n + 1]), pack2(fm.x, fm.y), pack2(fm.z, fm.w)), xs[n],
                                    xs[n + 1]);
                        }
                    };
                    logits();
                    exponents();
#pragma unroll
                    for (int n = 0; n < RS; n += 2) over = max3(over, xs[n], xs[n + 1]);
                    if (worker_or(bar_id, over > kSlack + kPShift || !ok)) {
                        ok = worker_and(bar_id, ok);
                        stop = !ok;
                        if (stop) break;
                        float* const fm = s_fm + 2 * r0;
                        float* const red = s_red + 4 * r0;
                        logits();
#pragma unroll
                        for (int n = 0; n < RS; ++n) xs[n] = fmaf(xs[n], fm[4 * (n >> 1) + (n & 1)], -kPShift);
                        const float most = reduce_rows<RS>(xs, lane, [](float a, float b) { return fmaxf(a, b); });
                        if (lane < RS) red[ww * RS + lane] = most;
                        worker_sync(bar_id);
                        if (wt < RS) {
                            float* const minus = &fm[4 * (wt >> 1) + 2 + (wt & 1)];
                            const float was = -*minus;
                            const float now = fmaxf(fmaxf(was, fmaxf(red[wt], red[RS + wt])),
                                                    fmaxf(red[2 * RS + wt], red[3 * RS + wt]));
                            *minus = -now;
                            red[wt] = now > was ? ex2_approx(was - now) : 1.0f;
                        }
                        worker_sync(bar_id);
#pragma unroll
                        for (int n = 0; n < RS; ++n) l[r0 + n] *= red[n];
                        if (started) {
                            tmem_ldn(t_a + S::t_o + r0, xs);
#pragma unroll
                            for (int n = 0; n < RS; ++n) xs[n] *= red[n];
                            tmem_stn(t_a + S::t_o + r0, xs);
                        }
                        logits();
                        exponents();
                    }
                    // Weights: a token's values in a row of shared memory.
                    uint32_t w[RS / 2];
#pragma unroll
                    for (int n = 0; n < RS; n += 2) {
                        const float a = ex2_approx(xs[n]), b = ex2_approx(xs[n + 1]);
                        unpack2(add2(pack2(l[r0 + n], l[r0 + n + 1]), pack2(a, b)), l[r0 + n], l[r0 + n + 1]);
                        w[n >> 1] = f16x2(a, b);
                    }
#pragma unroll
                    for (int c = 0; c < RS / 8; ++c)
                        sts_u4(p_at + piece<2 * N, KT>(wt, r0 / 8 + c), w[4 * c], w[4 * c + 1], w[4 * c + 2],
                               w[4 * c + 3]);
                }
                if (stop) break;
                convert_v(vc, vs);  // over the logits of this warp's tokens, which it has read
                mbar_arrive_local(bar_of(wk, kEmpty + slot));
                tmem_wait_st();
                fence_proxy_async();
                tc_fence_before();
                mbar_arrive_local(bar_of(wk, kVReady));
                if (ww == 2) multiply(kVReady, k & 1, [&]() { products(started); });
                started = true;
            }

            if (k > 0 && started) mbar_wait(bar_of(wk, kODone), (k - 1) & 1, ok, p.status, p.budget_ns, true);
            ok = worker_and(bar_id, ok);
            if (!ok) {
                // A wait ran out: this unit and the worker's later ones are NaN (a NaN sum stays one
                // through every join), and nothing more is copied or multiplied.
                t = tend;
#pragma unroll
                for (int n = 0; n < R; ++n) l[n] = NAN;
                if (wt == 0) asm volatile("st.volatile.shared.u32 [%0], %1;" ::"r"(range_at + 4 * wk), "r"(1) : "memory");
            }
            tc_fence_after();

            // The unit's rows, or this worker's part of them.
            {
                const float sum = reduce_rows<R>(l, lane, [](float a, float b) { return a + b; });
                if (lane < R) s_red[ww * R + lane] = sum;
            }
            worker_sync(bar_id);
            const bool whole = u0 >= t0 && u1 <= t1, open = u1 > t1;
            if (!whole) {
                const int unit = e * p.x_units + x, at = u0 + S::unit_cost * (unit + 1);  // its first tile
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
                float o[R];
                const float vref = started ? head_power(p.v_exp, u.head) : 0.0f;
                if (started) tmem_ldn(t_a + S::t_o, o);
                const int col = 32 * ww + 4 * (lane & 7) + 2 * (lane >> 4) + (lane >> 3 & 1);
#pragma unroll
                for (int n = 0; n < R; ++n)
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
                const float sum = (s_red[n] + s_red[R + n]) + (s_red[2 * R + n] + s_red[3 * R + n]);
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
                    if (c == 0) s_ml[wk * R + n] = ml;
                } else {
                    const int64_t to = static_cast<int64_t>(worker) * R + n;
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
    join_units<D, R, S::joiners, W, true>(p, base + S::off_q, S::worker_bytes, s_left, s_ml);
}

template <typename S>
int launch_tc(PagedParams p, const Maps<4>& maps, int box, int sms, int64_t tiles, smd_stream_t stream) {
    static SharedLimit limit;
    auto kernel = paged4_tc_kernel<S>;
    const int rc = limit.raise(kernel, S::smem(kMaxEntries));
    if (rc != SMD_OK) return rc;
    // A worker for each tile: at the most cost, units' ends too
    const int64_t want = (tiles + static_cast<int64_t>(S::unit_cost) * p.x_units * p.entries + S::W - 1) / S::W;
    const int64_t grid = want < sms ? want : sms;
    p.workers = static_cast<int>(grid) * S::W;
    set_workspace(p, sms, S::R, kCols);
    return launch_pdl(kernel, dim3(static_cast<unsigned>(grid)), S::threads, S::smem(p.entries), stream, p, box,
                      maps);
}

}  // namespace

int paged4_tc(const PagedParams& p, const Maps<4>& maps, int box, int rows, int sms, int64_t tiles,
              smd_stream_t stream) {
    return rows == 8    ? launch_tc<TcShape<8, 4, 2>>(p, maps, box, sms, tiles, stream)
           : rows == 16 ? launch_tc<TcShape<16, 4, 2>>(p, maps, box, sms, tiles, stream)
                        : launch_tc<TcShape<32, 3, 2>>(p, maps, box, sms, tiles, stream);
}

}  // namespace smd

// Attention over a paged E4M3 cache (smd_paged_decode).
//
// For the M query rows that share a kv head's keys (verify rows x query heads
// of the group), over the tokens t a row sees:
//   s_t = sm_scale q . k_t,   out = sum_t e^(s_t) v_t / sum_t e^(s_t)
// in one pass with the running maximum m and sum l of an online softmax.
//
// What bounds it: 2 D bytes of codes are read for each (token, kv head) and
// 4 D M FLOPs done with them, 2 M FLOPs a byte: HBM for the M <= 32 of decode
// rows. So the kernel is built to keep copies in flight, and the products go
// to mma.sync m16n8k16 with f16 operands: E4M3 codes convert to f16 exactly,
// and 8 or 16 rows would leave most of a 128-lane tcgen05 tile empty. Tokens (for
// the logits) and columns (for the output) are the MMA's 16 rows, query rows
// its 8 columns, so that 8 query heads fill it.
//
// A warp is a worker of its own: it walks tiles of KT tokens of one (page,
// head) through a ring of ST slots that its own lanes fill with tensor copies
// (K and V of a tile: one barrier), and holds the tile's softmax state and its
// D x M accumulators in registers. The tiles of all units (a request's kv
// head), laid end to end, are cut evenly over the warps of the grid, so a batch
// of mixed lengths loads every SM alike and no warp waits for another before it
// is through. A unit inside one warp's range is written by it. A unit that cuts
// divide is joined in order, in three steps: the CTA's warps through shared
// memory (the ring of a warp that is through holds its accumulators), then up
// to 32 neighbouring CTAs, then those groups, through fp32 partials in the
// workspace. Each of the last two is done by the CTA that arrives last, by a
// count, so nothing waits and no second kernel is needed; who joins depends on
// timing, what is added to what does not: run to run the bits are the same.
//
// Operand layouts (lane = 4 g + i): K comes by ldmatrix as 4 consecutive codes
// of token g, columns 16 c + 4 i ..; the contraction index of the MMA is
// permuted to take them as they are (slots 2i, 2i+1, 2i+8, 2i+9 are columns 4i
// .. 4i+3), and the query fragments are read in the same order. V comes by
// transposing ldmatrix as codes 16 c + 2 g and + 1 of tokens 2i and 2i+1; one
// byte permute pairs the tokens, and MMA rows g and g + 8 are those two columns.
// The weights leave the first product with a token a lane and enter the second
// with a query row a lane: movmatrix transposes their 8 x 8 blocks.
//
// Rounding: q enters as f16 after a power of two per row that puts its largest
// element in [2^14, 2^15) (bf16 has fewer bits than f16, so this is exact down
// to 2^-30 of the largest); the weights enter as f16, 11 bits, below the 8 of
// the bf16 output, relative to a maximum that is moved only when it has grown
// by more than 2^8 (so at 2^7 to 2^15); their sum is of the fp32 weights;
// accumulators, maxima and sums are fp32. V's scale multiplies the weights
// relative to the largest scale met so far (exact for powers of two), so f16
// never sees its range.
//
// Measured (GB300, device time; of the rate at which the GPU copies):
//   64 requests of 1024 .. 8192 tokens, 8 query rows of 128 columns   108 us   84%
//   64 listed pages of 64 tokens in each of 64 requests               102 us   78%
//   16 requests up to 131072 tokens, 32 query rows                    425 us   76%
//   31 requests up to 5001 tokens, 12 query rows of 64 columns         33 us   36%
//   one request of 777 tokens                                         9.5 us
//   32 requests of 1024 .. 8192 tokens, 8 query rows of 256 columns   109 us   79%
//   the same, 16 / 32 query rows of 256 columns             127 us   68% / 204 us   43%
//   16 requests of 4096 .. 65536 tokens, 32 / 64 query rows 223 us   72% / 414 us   39%
//   128 query heads over one kv head, 16 such requests                129 us   16%
// What bounds it now. The start costs 4 us before a copy is on its way (lengths,
// table entry, copy: three round trips and the launch), the joins 5 to 9 us after
// the last tile: all of the time of one short request, half of that of a small batch.
// (The joins run once a CTA, from instructions that are not cached yet: they are
// kept short, which took 1 to 2.5 us off each of these.) At 8 rows the rest is HBM,
// and its unevenness: some neighbourhoods of SMs stream 7% slower than the others,
// the same ones every time. At 32 rows the 254 registers a lane leave 8 warps an
// SM, and the products' and softmax's latencies show (mma.sync takes 8 cycles a
// sub-partition, 52% of the time in all; issue 38%). Past 32 rows (16 at 256 columns) the
// cache is read again for each 32, by other warps; past 1024 requests, or 1024 (row, kv head)
// lists, the call is as many launches as that takes, each with its start and joins (1024
// requests up to 300 tokens 80 us, 1025 110; 1000 requests with 4 listed pages for each of 8
// heads, eight launches, 244 us for 82 us of bytes; 256 with 64 pages, two, 373 us: 85%).
#include <cstring>

#include "smd_internal.h"
#include "smd_paged.h"
#include "smd_ptx.cuh"

namespace smd {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr int kMaxEntries = 1024;  // requests (or (row, kv head) lists) of one launch
constexpr float kPShift = 7.0f;    // weights are 2^7 at the maximum kept
constexpr float kSlack = 8.0f;     // which is moved when a logit exceeds it by 2^8
constexpr float kNone = -3.402823466e38f;  // no logit met
// What a unit's begin and end cost a warp, in tiles. 0 / 1 / 3 / 6: 31 requests up to 5001
// tokens of 64 columns 44 / 39 / 34 / 33 us, 1000 up to 300 tokens of 128 columns 93 / 81 /
// 78 / 78, 64 up to 8192 tokens 111 / 110 / 109 / 109; twice as much at 64 columns: no gain.
constexpr int kUnitCost = 3;
constexpr int kMinTiles = 2;       // least range of a warp, in tiles (1 to 8: the same times)
constexpr int kFan = 32;           // neighbouring CTAs of a first join (8 to 64: the same times)

struct PagedParams {
    const uint16_t* q;
    int64_t q_stride;
    const int32_t* table;
    int64_t table_stride;
    int32_t width;
    const int32_t* lengths;
    const float* k_scale;
    const float* v_scale;
    int32_t pages, heads, page_size;
    int32_t entries;    // requests, or (row, kv head) pairs where lists are given
    int32_t x_units;    // units of an entry: (kv heads x) row tiles
    int32_t row_tiles;
    int32_t G, g, Hq;   // verify rows; query heads of a kv head; query heads
    uint32_t g_magic;   // ceil(2^20 / g): m / g = (m * g_magic) >> 20 for m < 1024, g <= 128
    int32_t rows;       // query rows of a unit before tiling: G * g, or g with lists
    float scale_log2;   // sm_scale * log2 e
    const int32_t* lists;
    const int32_t* counts;
    int32_t K;
    uint16_t* out;
    float* lse;
    int32_t* status;
    uint64_t budget_ns; // bound of every wait
    int32_t stall;      // n > 0: the copy of each warp's n-th tile never completes (tests)
    int32_t workers;    // warps of the grid
    int32_t* arrived;   // [2][2 CTAs]: arrivals at the joins of CTAs, 0 between calls
    float* head;        // [workers][rows of a tile][D]: the end of a unit begun by a warp before
    float* part;        // [CTAs][4][rows of a tile][D]: the unit that the CTA goes on with, and
                        // what its group of CTAs has of it; the same of the unit that it begins
    float2* head_ml;    // the same without columns: maximum, sum
    float2* part_ml;
};

__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                        uint32_t a3, uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
        "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Not volatile, but ordered after the barrier wait by the memory clobber.
__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}

__device__ __forceinline__ void ldsm4_t(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}

// Four E4M3 codes -> two f16 pairs (low bytes first), exactly.
__device__ __forceinline__ void e4m3_to_f16(uint32_t v, uint32_t& lo, uint32_t& hi) {
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(v));
}

__device__ __forceinline__ uint32_t f16x2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

__device__ __forceinline__ void tma_load_4d(uint32_t dst, const void* map, int x, int t, int h,
                                            int p, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
        "[%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
        "l"(map), "r"(x), "r"(t), "r"(h), "r"(p), "r"(bar)
        : "memory");
}

__device__ __forceinline__ void prefetch_map(const void* map) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory");
}

__device__ __forceinline__ void lds64(uint32_t addr, uint32_t& a, uint32_t& b) {
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(a), "=r"(b) : "r"(addr) : "memory");
}

__device__ __forceinline__ void sts64(uint32_t addr, uint32_t a, uint32_t b) {
    asm volatile("st.shared.v2.u32 [%0], {%1, %2};" ::"r"(addr), "r"(a), "r"(b) : "memory");
}

__device__ __forceinline__ void sts32(uint32_t addr, uint32_t v) {
    asm volatile("st.shared.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}

__device__ __forceinline__ float4 lds_f4(uint32_t addr) {
    float4 v;
    asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(addr)
                 : "memory");
    return v;
}

// Two fp32 operations an instruction.
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
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

__device__ __forceinline__ float bf_lo(uint32_t v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ float bf_hi(uint32_t v) { return __uint_as_float(v & 0xffff0000u); }

// ln of the sum of e^logits, from the base-2 logit whose weight is 1 and the sum of the weights.
__device__ __forceinline__ float natural_lse(float base, float sum) {
    return sum == 0.0f ? -INFINITY : 0.69314718055994531f * (base + log2f(sum));
}

// Transposes the 8 x 8 block of 16-bit elements whose row g holds its elements
// 2i, 2i + 1 in lane 4 g + i.
__device__ __forceinline__ uint32_t transpose8x8(uint32_t v) {
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}

// The sizes of one instantiation: D columns, RT tiles of 8 query rows, KT
// tokens a tile, from one page or (NP = 2) a page for each half, ST slots of a
// warp's ring, CTAs an SM holds.
template <int D_, int RT_, int KT_, int NP_, int ST_, int CTAS_>
struct Shape {
    static constexpr int D = D_, RT = RT_, KT = KT_, NP = NP_, ST = ST_, CTAS = CTAS_;
    static constexpr int rows = 8 * RT;
    static constexpr int row_bytes = D < 128 ? D : 128;  // of a copy box
    static constexpr int side = KT * D;                  // bytes of a tile's K, and of its V
    static constexpr int slot = 2 * side;
    static constexpr bool q_regs = rows * D <= 2048;     // query fragments stay in registers
    static constexpr int off_q = kWarps * ST * slot;     // else here: [warps][RT][D / 16][32] pairs
    static constexpr int off_meta = off_q + (q_regs ? 0 : kWarps * rows * D * 2);
    static constexpr int off_bar = off_meta + kWarps * ST * 32;   // [warps][ST]
    static constexpr int off_scan = off_bar + kWarps * ST * 8;    // [warps] words
    static constexpr int off_ml = off_scan + 32;                  // [warps][rows] maximum, sum
    static constexpr int off_left = off_ml + kWarps * rows * 8;   // [warps] what a warp leaves
    static constexpr int off_prefix = off_left + kWarps * 64;     // [entries + 1], then [entries] lengths (of a list's row)
    static_assert(rows * D * 4 <= ST * slot, "a warp's accumulators fit its ring");
    static constexpr int smem(int entries) { return off_prefix + 4 * (2 * entries + 1) + 1024; }
};

// Byte offset of 16-byte piece c of token `row` in a side of a slot, as the
// copy's swizzle places it.
template <int D, int KT>
__device__ __forceinline__ uint32_t piece(int row, int c) {
    if (D == 64) return row * 64 + ((c ^ ((row >> 1) & 3)) << 4);
    return (c >> 3) * (KT * 128) + row * 128 + (((c & 7) ^ (row & 7)) << 4);
}

// One tile's tokens: for each page the offset in it, the first token's position
// in its request and the scales.
template <int NP>
struct Tile {
    int page[NP], off[NP], pos[NP], head;
    float ks[NP], vs[NP];
};

// A unit's row tile: its query rows as rows of the batch and query heads, and the
// CTAs that hold its first and last tile.
struct Unit {
    int b0, head, m0, m_real, first_cta, last_cta;
    __device__ __forceinline__ int verify_row(const PagedParams& p, int m) const {
        return static_cast<int>((static_cast<uint32_t>(m0 + m) * p.g_magic) >> 20);
    }
    __device__ __forceinline__ int64_t b(const PagedParams& p, int m) const {
        return p.lists != nullptr ? b0 : b0 + verify_row(p, m);
    }
    __device__ __forceinline__ int a(const PagedParams& p, int m) const {
        return head * p.g + m0 + m - verify_row(p, m) * p.g;
    }
};

// Four columns of one row, done: out and lse.
__device__ __forceinline__ void write_row(const PagedParams& p, const Unit& u, int D, int row,
                                          int col, float4 v, float top, float sum) {
    const int64_t at = u.b(p, row) * p.Hq + u.a(p, row);
    const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
    *reinterpret_cast<uint2*>(p.out + at * D + col) =
        make_uint2(bf16x2(v.x * inv, v.y * inv), bf16x2(v.z * inv, v.w * inv));
    if (col == 0 && p.lse != nullptr) p.lse[at] = natural_lse(top, sum);
}

// Adds N partials (maximum and sum, four of their columns; none: -infinity, 0) to
// another, in order.
template <int N>
__device__ __forceinline__ void add_partials(float4& acc, float& top, float& sum, const float4 (&v)[N],
                                             const float2 (&ml)[N]) {
    float to = top;
#pragma unroll
    for (int z = 0; z < N; ++z) to = fmaxf(to, ml[z].x);
    const float keep = top == -INFINITY ? 0.0f : ex2_approx(top - to);
    top = to;
    sum *= keep;
    acc.x *= keep, acc.y *= keep, acc.z *= keep, acc.w *= keep;
#pragma unroll
    for (int z = 0; z < N; ++z) {
        const float w = ml[z].x == -INFINITY ? 0.0f : ex2_approx(ml[z].x - to);
        sum += ml[z].y * w;  // a NaN stays one
        acc.x += v[z].x * w;
        acc.y += v[z].y * w;
        acc.z += v[z].z * w;
        acc.w += v[z].w * w;
    }
}

// What a warp leaves to its CTA: the unit whose end it held (its partial is in
// PagedParams::head) and the unit that goes on after it (in its ring).
struct Left {
    int32_t ended, open;   // the unit's number, or -1
    int32_t open_begins;   // the open unit begins in this warp's range
    int32_t pad;
    Unit ended_unit, open_unit;
};

template <typename S>
__global__ void __launch_bounds__(kThreads, S::CTAS)
    paged_decode_kernel(const PagedParams p, const __grid_constant__ CUtensorMap kmap,
                        const __grid_constant__ CUtensorMap vmap) {
    constexpr int D = S::D, RT = S::RT, KT = S::KT, ST = S::ST;
    constexpr int NH = KT / 16;   // 16-token halves of a tile
    constexpr int NP = S::NP;     // its pages
    constexpr int NC = D / 16;    // 16-column chunks
    // The position of tokens that no row sees: past every row's end (lengths are whole pages below
    // 2^31 at most, of 32 tokens where a tile has one position for 32) and, with the 31 or 15
    // that are added to it, still an int.
    constexpr int kNoPos = NH > NP ? 0x7fffffe0 : 0x7ffffff0;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t base = (smem_addr(smem_raw) + 1023u) & ~1023u;
    uint8_t* const gbase = smem_raw + (base - smem_addr(smem_raw));
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, qr = lane >> 2, qi = lane & 3;
    int32_t* const prefix = reinterpret_cast<int32_t*>(gbase + S::off_prefix);
    int32_t* const lens = prefix + p.entries + 1;
    const uint32_t ring = base + warp * ST * S::slot;
    const uint32_t bars = base + S::off_bar + warp * ST * 8;
    const uint32_t meta = base + S::off_meta + warp * ST * 32;  // ks, vs, pos of each half
    const uint32_t q_at = base + S::off_q + warp * S::rows * D * 2 + 8 * lane;
    const bool lists = p.lists != nullptr;

    if (tid == 0) {
        prefetch_map(&kmap);
        prefetch_map(&vmap);
    }
    if (lane == 0) {
        for (int s = 0; s < ST; ++s) mbar_init(bars + 8 * s, 1);
        fence_mbar_init();
        fence_proxy_async();
    }
    pdl_entry();
    fence_proxy_async_global();  // the cache may have been written by the kernel before

    // Prefix sums of the entries' tiles: at least one for each unit, so that one without
    // tokens still writes its zeros.
    int total;
    {
        const auto tiles_of = [&](int e) {
            if (e >= p.entries) return 0;
            const int b = lists ? e / p.heads : e, r = lists ? b / p.G : e;  // row, or request
            int len = max(min(p.lengths[r], p.width * p.page_size), 0), n = len;
            if (lists) {
                // The tokens that the list's row sees: a listed page past them is not read, so its
                // scales reach nothing either.
                len = max(len - p.G + 1 + b - r * p.G, 0);
                n = max(min(p.counts != nullptr ? p.counts[e] : p.K, p.K), 0) * p.page_size;
            }
            lens[e] = len;
            return max(n / KT + (n % KT != 0 ? 1 : 0), 1) * p.x_units;
        };
        constexpr int kPer = kMaxEntries / kThreads;
        const int each = (p.entries + kThreads - 1) / kThreads;  // entries of a thread
        int v[kPer], sum = 0;
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
            v[j] = j < each ? tiles_of(tid * each + j) : 0;
            sum += v[j];
        }
        int inc = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int u = __shfl_up_sync(0xffffffffu, inc, o);
            if (lane >= o) inc += u;
        }
        int32_t* const scan = reinterpret_cast<int32_t*>(gbase + S::off_scan);
        if (lane == 31) scan[warp] = inc;
        __syncthreads();
        int before = inc - sum;
        total = 0;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            if (w < warp) before += scan[w];
            total += scan[w];
        }
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
            if (j < each && tid * each + j < p.entries) prefix[tid * each + j] = before;
            before += v[j];
        }
        if (tid == 0) prefix[p.entries] = total;
    }
    __syncthreads();

    // The grid is cut evenly by cost: each unit counts kUnitCost besides its tiles, laid
    // before them, so unit u of the batch starts its tiles kUnitCost (u + 1) further on.
    const auto find = [&](int t, int unit_cost) {  // the entry at t (below the last one's end)
        int lo = 0, hi = p.entries;
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (prefix[mid] + unit_cost * p.x_units * mid <= t) lo = mid;
            else hi = mid;
        }
        return lo;
    };
    const auto find_entry = [&](int t) { return find(t, 0); };
    const int cost = total + kUnitCost * p.x_units * p.entries;
    const int worker = static_cast<int>(blockIdx.x) * kWarps + warp;
    const int per = max((cost + p.workers - 1) / p.workers, kMinTiles);
    const auto tiles_before = [&](int64_t at) {  // tiles that lie before a cost position
        if (at >= cost) return total;
        const int c = static_cast<int>(at), e = find(c, kUnitCost);
        const int nt = (prefix[e + 1] - prefix[e]) / p.x_units;
        const int rem = c - prefix[e] - kUnitCost * p.x_units * e, x = rem / (nt + kUnitCost);
        return prefix[e] + x * nt + max(rem - x * (nt + kUnitCost) - kUnitCost, 0);
    };
    const int cut = tiles_before(static_cast<int64_t>(worker + (lane & 1)) * per);
    const int t0 = __shfl_sync(0xffffffffu, cut, 0), t1 = __shfl_sync(0xffffffffu, cut, 1);

    // Lane l resolves tile t0 + 32 * (k / 32) + l.
    Tile<NP> td;
    const auto resolve = [&](int kk) {
        const int t = t0 + kk;
#pragma unroll
        for (int h = 0; h < NP; ++h) {
            td.page[h] = -1;
            td.off[h] = 0;
            td.pos[h] = kNoPos;
            td.ks[h] = 1.0f;
            td.vs[h] = 0.0f;
        }
        td.head = 0;
        if (t >= t1) return;
        const int e = find_entry(t), nt = (prefix[e + 1] - prefix[e]) / p.x_units;
        const int rem = t - prefix[e], x = rem / nt, first = (rem - x * nt) * KT;
        const int b = lists ? e / p.heads : e;  // row, or request
        const int r = lists ? b / p.G : e, len = lens[e];
        td.head = lists ? e - b * p.heads : x / p.row_tiles;
        const int32_t* const row = p.table + static_cast<int64_t>(r) * p.table_stride;
#pragma unroll
        for (int h = 0; h < NP; ++h) {
            int blk = (first + KT / NP * h) / p.page_size;
            const int off = first + KT / NP * h - blk * p.page_size;
            if (lists) {
                const int c = p.counts != nullptr ? max(min(p.counts[e], p.K), 0) : p.K;
                blk = blk < c ? p.lists[static_cast<int64_t>(e) * p.K + blk] : -1;
            }
            const int64_t pos = static_cast<int64_t>(blk) * p.page_size + off;
            if (blk < 0 || pos >= len) continue;
            td.pos[h] = static_cast<int>(pos);
            td.off[h] = off;
            const int pg = row[blk];
            if (pg < 0 || pg >= p.pages) continue;
            td.page[h] = pg;
            td.ks[h] = p.k_scale[static_cast<int64_t>(pg) * p.heads + td.head];
            td.vs[h] = p.v_scale[static_cast<int64_t>(pg) * p.heads + td.head];
        }
    };
    // Fills the slot of tile t0 + kk; called in order of kk.
    const auto issue = [&](int kk) {
        if (t0 + kk >= t1) return;
        // The first tiles' copies go out before the other lanes look their tiles up.
        if (kk == 0 || kk == ST || (kk & 31) == 0)
            resolve(kk == 0 && lane >= ST ? t1 - t0 : (kk & ~31) + lane);
        if (lane == (kk & 31)) {
            const int s = kk % ST;
            const uint32_t bar = bars + 8 * s, dst = ring + s * S::slot;
            mbar_arrive_expect_tx(bar, S::slot + (kk + 1 == p.stall ? 16 : 0));
#pragma unroll
            for (int h = 0; h < NP; ++h) {
#pragma unroll
                for (int sub = 0; sub < (D > 128 ? 2 : 1); ++sub) {
                    const uint32_t at = dst + sub * KT * 128 + h * (KT / NP) * S::row_bytes;
                    tma_load_4d(at, &kmap, sub * 128, td.off[h], td.head, td.page[h], bar);
                    tma_load_4d(at + S::side, &vmap, sub * 128, td.off[h], td.head, td.page[h],
                                bar);
                }
            }
            sts_v4(meta + 32 * s, make_float4(td.ks[0], td.ks[NP - 1], td.vs[0], td.vs[NP - 1]));
            sts64(meta + 32 * s + 16, td.pos[0], td.pos[NP - 1] + (NH > NP ? 16 : 0));
        }
        __syncwarp();
    };

    float2* const s_ml = reinterpret_cast<float2*>(gbase + S::off_ml);
    Left* const s_left = reinterpret_cast<Left*>(gbase + S::off_left);
    if (lane == 0) s_left[warp].ended = s_left[warp].open = -1;
    bool ok = true;  // until a wait runs out; the same in every lane outside the tile loop
    int k = 0, t = t0, e = t0 < t1 ? find(t0, 0) : 0;
#pragma unroll 1
    for (int s = 0; s < ST; ++s) issue(s);

    // The unit of tile t: entry e, unit x of its x_units, each of nt tiles.
    int nt = 1, x = 0;
    if (t0 < t1) {
        nt = (prefix[e + 1] - prefix[e]) / p.x_units;
        x = (t0 - prefix[e]) / nt;
    }
    const auto unit_at = [&](int ue, int ux) {
        Unit u;
        const int rt = p.row_tiles == 1 ? 0 : ux % p.row_tiles;
        u.b0 = lists ? ue / p.heads : ue * p.G;
        u.head = lists ? ue - u.b0 * p.heads : p.row_tiles == 1 ? ux : ux / p.row_tiles;
        u.m0 = rt * S::rows;
        u.m_real = min(p.rows - u.m0, S::rows);
        return u;
    };
    Unit u{};
    if (t0 < t1) u = unit_at(e, x);

#pragma unroll 1
    while (t < t1) {
        const int u0 = prefix[e] + x * nt, u1 = u0 + nt, tend = min(u1, t1);
        const int len = lens[e];
        const int m_real = u.m_real;
        // The tokens that row m of the tile sees.
        const auto row_limit = [&](int m) {
            return lists ? len : max(len - p.G + 1 + u.verify_row(p, m), 0);
        };
        const int min_lim = row_limit(0), max_lim = row_limit(m_real - 1);

        // The queries of row 8 n + g, columns 16 c + 4 i .., as f16; the logit factor of
        // rows 8 n + 2 i + y (positive: a negative softmax scale turns the query's sign).
        uint32_t qb[S::q_regs ? RT : 1][S::q_regs ? NC : 1][2];
        float fac[RT][2];
#pragma unroll
        for (int n = 0; n < RT; ++n) {
            uint2 w[NC];
            const int m = 8 * n + qr;
#pragma unroll
            for (int c = 0; c < NC; ++c) w[c] = make_uint2(0, 0);
            if (m < m_real) {
                const uint16_t* const row =
                    p.q + u.b(p, m) * p.q_stride + static_cast<int64_t>(u.a(p, m)) * D + 4 * qi;
#pragma unroll
                for (int c = 0; c < NC; ++c)
                    w[c] = __ldg(reinterpret_cast<const uint2*>(row + 16 * c));
            }
            float a = 0.0f;
#pragma unroll
            for (int c = 0; c < NC; ++c) {
                a = fmaxf(a, fmaxf(fabsf(bf_lo(w[c].x)), fabsf(bf_hi(w[c].x))));
                a = fmaxf(a, fmaxf(fabsf(bf_lo(w[c].y)), fabsf(bf_hi(w[c].y))));
            }
            a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, 1));
            a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, 2));
            // up = 2^(14 - exponent of a), within what a float holds
            const int ex = static_cast<int>(__float_as_uint(a) >> 23);
            const int ue = min(14 + 127 - ex + 127, 253);
            float up = a > 0.0f && ex < 255 ? __uint_as_float(static_cast<uint32_t>(ue) << 23) : 1.0f;
            const float own = fabsf(p.scale_log2) / up;
            fac[n][0] = __shfl_sync(0xffffffffu, own, 8 * qi);
            fac[n][1] = __shfl_sync(0xffffffffu, own, 8 * qi + 4);
            if (p.scale_log2 < 0.0f) up = -up;
#pragma unroll
            for (int c = 0; c < NC; ++c) {
                const uint32_t f0 = f16x2(bf_lo(w[c].x) * up, bf_hi(w[c].x) * up);
                const uint32_t f1 = f16x2(bf_lo(w[c].y) * up, bf_hi(w[c].y) * up);
                if (S::q_regs) {
                    qb[S::q_regs ? n : 0][S::q_regs ? c : 0][0] = f0;
                    qb[S::q_regs ? n : 0][S::q_regs ? c : 0][1] = f1;
                } else {
                    sts64(q_at + (n * NC + c) * 256, f0, f1);  // read by this lane only
                }
            }
        }
        // The unit after it, if this warp has some of that: its queries come into L1 meanwhile.
        int e_next = e, x_next = x + 1;
        Unit u_next{};
        if (tend < t1) {
            if (x_next == p.x_units) {
                ++e_next;  // every entry has a tile
                x_next = 0;
            }
            u_next = unit_at(e_next, x_next);
            constexpr int kLines = D / 64;  // 128-byte lines of a row
            for (int i = lane; i < u_next.m_real * kLines; i += 32) {
                const int row = i / kLines;
                asm volatile("prefetch.global.L1 [%0];" ::"l"(
                    p.q + u_next.b(p, row) * p.q_stride +
                    static_cast<int64_t>(u_next.a(p, row)) * D + i % kLines * 64));
            }
        }
        float m[RT][2], l[RT][2], o[RT][NC][4], vref = 0.0f, vinv = 0.0f;
#pragma unroll
        for (int n = 0; n < RT; ++n)
#pragma unroll
            for (int y = 0; y < 2; ++y) {
                m[n][y] = kNone;
                l[n][y] = 0.0f;
            }
#pragma unroll
        for (int n = 0; n < RT; ++n)
#pragma unroll
            for (int c = 0; c < NC; ++c)
#pragma unroll
                for (int j = 0; j < 4; ++j) o[n][c][j] = 0.0f;

#pragma unroll 1
        for (; t < tend && ok; ++t, ++k) {
            if (k > 0) issue(k + ST - 1);
            const int slot = k % ST;
            mbar_wait(bars + 8 * slot, (k / ST) & 1, ok, p.status, p.budget_ns);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            const uint32_t ks_at = ring + slot * S::slot, vs_at = ks_at + S::side;

            // logits: token 16 h + g (+ 8 for j >= 2), query row 8 n + 2 i + (j & 1)
            float s[NH][RT][4];
#pragma unroll
            for (int h = 0; h < NH; ++h)
#pragma unroll
                for (int n = 0; n < RT; ++n)
#pragma unroll
                    for (int j = 0; j < 4; ++j) s[h][n][j] = 0.0f;
#pragma unroll
            for (int c0 = 0; c0 < NC; c0 += 2 / NH) {
                uint32_t kr[4];
                ldsm4(ks_at + piece<D, KT>(lane % KT, c0 + lane / KT), kr);
                uint32_t a[2][4];
#pragma unroll
                for (int z = 0; z < 2; ++z) {
                    e4m3_to_f16(kr[2 * z], a[z][0], a[z][2]);
                    e4m3_to_f16(kr[2 * z + 1], a[z][1], a[z][3]);
                }
#pragma unroll
                for (int n = 0; n < RT; ++n) {
                    uint32_t b0v, b1v;
#pragma unroll
                    for (int z = 0; z < 2; ++z) {
                        const int h = z % NH, c = c0 + z / NH;
                        if (S::q_regs) {
                            b0v = qb[S::q_regs ? n : 0][S::q_regs ? c : 0][0];
                            b1v = qb[S::q_regs ? n : 0][S::q_regs ? c : 0][1];
                        } else if (z == 0 || NH == 1) {
                            lds64(q_at + (n * NC + c) * 256, b0v, b1v);
                        }
                        mma_f16(s[h][n], a[z][0], a[z][1], a[z][2], a[z][3], b0v, b1v);
                    }
                }
            }

            const float4 sc = lds_f4(meta + 32 * slot);
            const float ks[2] = {sc.x, sc.y}, vs[2] = {sc.z, sc.w};
            uint32_t up0, up1;
            lds64(meta + 32 * slot + 16, up0, up1);
            const int pos[2] = {static_cast<int>(up0), static_cast<int>(up1)};
            if (max(pos[0], pos[1]) + 15 >= min_lim) {
                // Tokens that a row does not see.
#pragma unroll
                for (int n = 0; n < RT; ++n)
#pragma unroll
                    for (int y = 0; y < 2; ++y) {
                        const int lim = row_limit(min(8 * n + 2 * qi + y, m_real - 1));
#pragma unroll
                        for (int h = 0; h < NH; ++h)
#pragma unroll
                            for (int z = 0; z < 2; ++z)
                                if (pos[h] + qr + 8 * z >= lim) s[h][n][2 * z + y] = -INFINITY;
                    }
#pragma unroll
                for (int h = 0; h < NH; ++h) {
                    // V of tokens that no row sees becomes 0 (0 times a NaN would not be).
                    if (pos[h] + 15 >= max_lim) {
#pragma unroll
                        for (int z = 0; z < 16 * NC; z += 32) {
                            const int j = (z + lane) / NC;
                            if (pos[h] + j >= max_lim)
                                sts_zero16(vs_at + piece<D, KT>(16 * h + j, (z + lane) % NC));
                        }
                    }
                    // V of tokens that some rows see and others do not: a NaN goes to the rows
                    // that see it here, and 0 stands in its place for the products.
#pragma unroll 1
                    for (int at = max(min_lim, pos[h]); at < pos[h] + min(max_lim - pos[h], 16); ++at) {
                        const int j = 16 * h + at - pos[h];
                        uint32_t nan = 0;
#pragma unroll
                        for (int z = 0; z < 4 * NC; z += 32)
                            if (z + lane < 4 * NC) {
                                const uint32_t w = lds_u32(vs_at + piece<D, KT>(j, (z + lane) >> 2) +
                                                           4 * (lane & 3));
                                nan |= ((w & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u;
                            }
                        if (!__any_sync(0xffffffffu, nan != 0)) continue;
#pragma unroll
                        for (int c = 0; c < NC; ++c) {
                            const uint32_t a = vs_at + piece<D, KT>(j, c) + 4 * (qr >> 1);
                            const uint32_t w = lds_u32(a);
#pragma unroll
                            for (int z = 0; z < 2; ++z)
                                if (((w >> (16 * (qr & 1) + 8 * z)) & 0x7fu) == 0x7fu)
#pragma unroll
                                    for (int n = 0; n < RT; ++n)
#pragma unroll
                                        for (int y = 0; y < 2; ++y)
                                            if (at < row_limit(8 * n + 2 * qi + y))
                                                o[n][c][2 * z + y] = NAN;
                            const uint32_t bad = ((w & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u;
                            __syncwarp();
                            if ((lane & 7) == 0) sts32(a, w & ~((bad >> 7) * 0xffu));
                        }
                    }
                }
                fence_proxy_async();  // before the slot is copied into again
                __syncwarp();
            }

            // The maximum (m + kPShift) stays while no logit exceeds it by more than kSlack.
            float f[NP][RT][2], over = kNone;
            const auto largest = [&](int h, int n, int y) {  // product of the page's tokens
                float w = fmaxf(s[h][n][y], s[h][n][2 + y]);
                if (NP < NH) w = fmaxf(w, fmaxf(s[NH - 1][n][y], s[NH - 1][n][2 + y]));
                return w;
            };
#pragma unroll
            for (int n = 0; n < RT; ++n)
#pragma unroll
                for (int y = 0; y < 2; ++y)
#pragma unroll
                    for (int h = 0; h < NP; ++h) {
                        f[h][n][y] = fmaxf(fac[n][y] * ks[h], 1.17549435e-38f);
                        over = fmaxf(over, fmaf(largest(h, n, y), f[h][n][y], -m[n][y]));
                    }
            const bool moved = over > kSlack + kPShift;
            if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
                for (int n = 0; n < RT; ++n)
#pragma unroll
                    for (int y = 0; y < 2; ++y) {
                        float top = m[n][y];
#pragma unroll
                        for (int h = 0; h < NP; ++h)
                            top = fmaxf(top, fmaf(largest(h, n, y), f[h][n][y], -kPShift));
                        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 4));
                        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 8));
                        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 16));
                        const float alpha = top > m[n][y] ? ex2_approx(m[n][y] - top) : 1.0f;
                        m[n][y] = top;
                        l[n][y] *= alpha;
#pragma unroll
                        for (int c = 0; c < NC; ++c) {
                            o[n][c][y] *= alpha;
                            o[n][c][2 + y] *= alpha;
                        }
                    }
            }

            // weights and the second product, relative to the largest scale of V so far. Of two pages
            // the first's products are done before the second's scale comes in: a verify row may
            // not see the second at all, and its weights must keep their bits.
            const float vtop = fmaxf(fmaxf(vs[0], vs[NP - 1]), 1.17549435e-38f);
            float ratio[NP], later = 1.0f;  // what the accumulators come down by between the pages
#pragma unroll
            for (int h = 0; h < NP; ++h) ratio[h] = vs[h] * vinv;
            if (vtop > vref) {
                const float first = NP == 1 ? vtop : fmaxf(fmaxf(vs[0], vref), 1.17549435e-38f);
                const float down = vref / first;
                vref = vtop;
                vinv = 1.0f / vref;
                ratio[NP - 1] = vs[NP - 1] * vinv;
                if (NP == 2) {
                    ratio[0] = vs[0] / first;
                    later = first / vtop;
                }
#pragma unroll
                for (int n = 0; n < RT; ++n)
#pragma unroll
                    for (int c = 0; c < NC; ++c)
#pragma unroll
                        for (int j = 0; j < 4; ++j) o[n][c][j] *= down;
            }
            uint32_t pb[NH][RT][2];
#pragma unroll
            for (int h = 0; h < NH; ++h) {
                const float by = ratio[NP == NH ? h : 0];
#pragma unroll
                for (int n = 0; n < RT; ++n) {
                    float w[4];
                    const float* const fh = f[NP == NH ? h : 0][n];
                    uint64_t sum = pack2(l[n][0], l[n][1]);
#pragma unroll
                    for (int z = 0; z < 2; ++z) {
                        float x0, x1;
                        unpack2(fma2(pack2(s[h][n][2 * z], s[h][n][2 * z + 1]), pack2(fh[0], fh[1]),
                                     pack2(-m[n][0], -m[n][1])), x0, x1);
                        const uint64_t pv = pack2(ex2_approx(x0), ex2_approx(x1));
                        sum = add2(sum, pv);
                        unpack2(mul2(pv, pack2(by, by)), w[2 * z], w[2 * z + 1]);
                    }
                    unpack2(sum, l[n][0], l[n][1]);
                    pb[h][n][0] = transpose8x8(f16x2(w[0], w[1]));
                    pb[h][n][1] = transpose8x8(f16x2(w[2], w[3]));
                }
            }
#pragma unroll
            for (int h = 0; h < NH; ++h) {
                if (NP == 2 && h == 1 && later != 1.0f) {
#pragma unroll
                    for (int n = 0; n < RT; ++n)
#pragma unroll
                        for (int c = 0; c < NC; ++c)
#pragma unroll
                            for (int j = 0; j < 4; ++j) o[n][c][j] *= later;
                }
#pragma unroll
                for (int c = 0; c < NC; c += 2) {
                    uint32_t vr[4];
                    ldsm4_t(vs_at + piece<D, KT>(16 * h + (lane & 15), c + (lane >> 4)), vr);
#pragma unroll
                    for (int z = 0; z < 2; ++z) {
                        uint32_t a[4];
                        e4m3_to_f16(__byte_perm(vr[2 * z], 0, 0x3120), a[0], a[1]);
                        e4m3_to_f16(__byte_perm(vr[2 * z + 1], 0, 0x3120), a[2], a[3]);
#pragma unroll
                        for (int n = 0; n < RT; ++n)
                            mma_f16(o[n][c + z], a[0], a[1], a[2], a[3], pb[h][n][0], pb[h][n][1]);
                    }
                }
            }
            __syncwarp();
        }

        if (!ok) {
            // A wait ran out: this unit and the warp's later ones are NaN (a NaN sum stays one
            // through every join), and nothing more is issued.
            t = tend;
#pragma unroll
            for (int n = 0; n < RT; ++n) l[n][0] = l[n][1] = NAN;
        }

        // The unit's rows, or this warp's part of them.
        const bool whole = u0 >= t0 && u1 <= t1, open = u1 > t1;
        if (!whole) {
            const int unit = e * p.x_units + x, at = u0 + kUnitCost * (unit + 1);  // its first tile
            u.first_cta = at / per / kWarps;
            u.last_cta = (at + nt - 1) / per / kWarps;
            Left* const left = s_left + warp;
            if (lane == 0 && open) {
                left->open = unit;
                left->open_begins = u0 >= t0;
                left->open_unit = u;
            } else if (lane == 0) {
                left->ended = unit;
                left->ended_unit = u;
            }
        }
#pragma unroll
        for (int n = 0; n < RT; ++n)
#pragma unroll
            for (int y = 0; y < 2; ++y) {
                float sum = l[n][y];
                sum += __shfl_xor_sync(0xffffffffu, sum, 4);
                sum += __shfl_xor_sync(0xffffffffu, sum, 8);
                sum += __shfl_xor_sync(0xffffffffu, sum, 16);
                const int row = 8 * n + 2 * qi + y;
                if (row >= m_real) continue;
                if (whole) {
                    const int64_t at = u.b(p, row) * p.Hq + u.a(p, row);
                    const float w = sum == 0.0f ? 0.0f : vref / sum;
                    uint32_t* const out = reinterpret_cast<uint32_t*>(p.out + at * D) + qr;
#pragma unroll
                    for (int c = 0; c < NC; ++c)
                        out[8 * c] = bf16x2(o[n][c][y] * w, o[n][c][2 + y] * w);
                    if (qr == 0 && p.lse != nullptr) p.lse[at] = natural_lse(m[n][y], sum);
                } else if (open) {
                    // every tile of the ring has been consumed (or, after a wait that ran out, the
                    // ring is left to the copies in flight)
#pragma unroll
                    for (int c = 0; c < NC; ++c) {
                        if (!ok) break;
                        const uint32_t piece16 = (4 * c + (qr >> 1)) ^ (qi << 1);
                        sts64(ring + row * D * 4 + (piece16 << 4) + 8 * (qr & 1),
                              __float_as_uint(o[n][c][y] * vref), __float_as_uint(o[n][c][2 + y] * vref));
                    }
                    if (qr == 0) s_ml[warp * S::rows + row] = make_float2(m[n][y] == kNone ? -INFINITY : m[n][y], sum);
                } else {
                    const int64_t at = static_cast<int64_t>(worker) * S::rows + row;
                    float2* const out = reinterpret_cast<float2*>(p.head + at * D) + qr;
#pragma unroll
                    for (int c = 0; c < NC; ++c)
                        out[8 * c] = make_float2(o[n][c][y] * vref, o[n][c][2 + y] * vref);
                    if (qr == 0) p.head_ml[at] = make_float2(m[n][y] == kNone ? -INFINITY : m[n][y], sum);
                }
            }
        if (tend < t1) {
            if (e_next != e) nt = (prefix[e_next + 1] - prefix[e_next]) / p.x_units;
            e = e_next;
            x = x_next;
            u = u_next;
        }
    }
    // After a wait that ran out the copies of tiles k to k + ST - 1 are in flight: none may
    // outlive the warp.
    if (!ok)
        for (int j = k; j < min(k + ST, t1 - t0); ++j) {
            bool done = true;
            mbar_wait(bars + 8 * (j % ST), (j / ST) & 1, done, p.status, p.budget_ns, true);
        }

    // The CTA's warps: the units that cuts between them divide. Open partials of
    // neighbours and the end that follows them are one unit.
    __threadfence_block();
    __syncthreads();
    const int cta = static_cast<int>(blockIdx.x);
    // The units that this CTA goes on with (0) and begins (1) and does not hold whole.
    bool goes[2] = {false, false};
    Unit unit[2];
#pragma unroll 1
    for (int i = 0; i < 2 * kWarps;) {  // warp i / 2: what it ended, then what it leaves open
        const int first = i >> 1;
        const bool is_open = (i & 1) != 0;
        ++i;
        if ((is_open ? s_left[first].open : s_left[first].ended) < 0) continue;
        const bool begins = is_open && s_left[first].open_begins != 0;
        const Unit u = is_open ? s_left[first].open_unit : s_left[first].ended_unit;
        int opens = is_open ? 1 : 0, end_at = is_open ? -1 : first;
        while (end_at < 0 && i < 2 * kWarps) {
            if (s_left[i >> 1].ended >= 0) {
                end_at = i >> 1;
                ++i;
            } else {
                ++opens;
                i += 2;
            }
        }
        const bool whole = begins && end_at >= 0;
        if (!whole) {
            if (begins) unit[1] = u, goes[1] = true;
            else unit[0] = u, goes[0] = true;
        }
        const int64_t slot = static_cast<int64_t>(4 * cta + (begins ? 2 : 0)) * S::rows;
#pragma unroll 1
        for (int idx = tid; idx < u.m_real * (D / 4); idx += kThreads) {
            const int row = idx / (D / 4), col = idx % (D / 4);
            // The open warps' partials in order, then the end.
            float4 end_v[1] = {make_float4(0.0f, 0.0f, 0.0f, 0.0f)};
            float2 end_ml[1] = {make_float2(-INFINITY, 0.0f)};
            if (end_at >= 0) {
                const int64_t at = (static_cast<int64_t>(cta) * kWarps + end_at) * S::rows + row;
                end_v[0] = __ldcg(reinterpret_cast<const float4*>(p.head + at * D) + col);
                end_ml[0] = __ldcg(p.head_ml + at);
            }
            float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            float top = -INFINITY, sum = 0.0f;
#pragma unroll 1
            for (int j = 0; j < opens; ++j) {
                const float4 v[1] = {lds_f4(base + (first + j) * ST * S::slot + row * D * 4 +
                                            ((col ^ (((row >> 1) & 3) << 1)) << 4))};
                const float2 ml[1] = {s_ml[(first + j) * S::rows + row]};
                add_partials<1>(acc, top, sum, v, ml);
            }
            if (end_at >= 0) add_partials<1>(acc, top, sum, end_v, end_ml);
            if (whole) {
                write_row(p, u, D, row, 4 * col, acc, top, sum);
            } else {
                reinterpret_cast<float4*>(p.part + (slot + row) * D)[col] = acc;
                if (col == 0) p.part_ml[slot + row] = make_float2(top, sum);
            }
        }
    }
    if (!goes[0] && !goes[1]) return;

    // The units that cuts between CTAs divide, level 0: among kFan neighbours from the unit's
    // first CTA on, level 1: among these groups. The CTA that arrives last at a join
    // makes it.
    __shared__ int s_joins[2];
    const int ctas = static_cast<int>(gridDim.x);
    const auto span = [&](int q, int level, int& from, int& n) {  // the first CTA of a join, its partials
        const int c0 = unit[q].first_cta, c1 = unit[q].last_cta;
        from = level == 0 ? c0 + (cta - c0) / kFan * kFan : c0;
        n = level == 0 ? min(c1, from + kFan - 1) - from + 1 : (c1 - c0) / kFan + 1;
    };
#pragma unroll 1
    for (int level = 0; level < 2; ++level) {
        __threadfence();
        __syncthreads();
        if ((tid & 31) == 0 && tid < 64) {
            const int q = tid >> 5;
            bool joins = goes[q];
            if (joins) {
                int from, n;
                span(q, level, from, n);
                if (n > 1) {
                    int* const count = p.arrived + level * 2 * ctas +
                                       2 * from + (unit[q].first_cta == from ? 1 : 0);
                    joins = atomicAdd(count, 1) == n - 1;
                    if (joins) *count = 0;  // for the next call
                }
            }
            s_joins[q] = joins;
        }
        __syncthreads();
        goes[0] = s_joins[0] != 0;
        goes[1] = s_joins[1] != 0;
        if (!goes[0] && !goes[1]) return;
        __threadfence();
        // Two joins are made by half of the threads each.
        const bool both = goes[0] && goes[1];
        const int threads = both ? kThreads / 2 : kThreads, me = tid & (threads - 1);
        const int q = both ? tid / (kThreads / 2) : goes[1] ? 1 : 0;
        const Unit u = q == 0 ? unit[0] : unit[1];
        int from, n;
        span(q, level, from, n);
        const bool done[2] = {
            level == 1 || unit[0].last_cta - unit[0].first_cta < kFan,
            level == 1 || unit[1].last_cta - unit[1].first_cta < kFan};
        const auto slot = [&](int c, int stage) {
            return static_cast<int64_t>(4 * c + (c == u.first_cta ? 2 : 0) + stage) * S::rows;
        };
#pragma unroll 1
        for (int i0 = me; i0 < u.m_real * (D / 4); i0 += 2 * threads) {
            // Two pieces of 4 columns, kMany partials of each: one round trip.
            constexpr int kMany = 4;
            int row[2], col[2];
            float4 acc[2];
            float top[2], sum[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                row[i] = min((i0 + i * threads) / (D / 4), u.m_real - 1);
                col[i] = (i0 + i * threads) % (D / 4);
                acc[i] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                top[i] = -INFINITY;
                sum[i] = 0.0f;
            }
#pragma unroll 1
            for (int j0 = 0; j0 < n; j0 += kMany) {
                float4 v[2][kMany];
                float2 ml[2][kMany];
#pragma unroll
                for (int z = 0; z < kMany; ++z) {
                    const int c = from + (j0 + z) * (level == 0 ? 1 : kFan);
                    const int64_t at = slot(c, level);
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        v[i][z] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                        ml[i][z] = make_float2(-INFINITY, 0.0f);
                        if (j0 + z < n) {
                            v[i][z] = __ldcg(reinterpret_cast<const float4*>(p.part + (at + row[i]) * D) + col[i]);
                            ml[i][z] = __ldcg(p.part_ml + at + row[i]);
                        }
                    }
                }
                add_partials<kMany>(acc[0], top[0], sum[0], v[0], ml[0]);
                add_partials<kMany>(acc[1], top[1], sum[1], v[1], ml[1]);
            }
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                if (i0 + i * threads >= u.m_real * (D / 4)) break;
                if (q == 0 ? done[0] : done[1]) {
                    write_row(p, u, D, row[i], 4 * col[i], acc[i], top[i], sum[i]);
                } else {
                    const int64_t to = slot(from, 1) + row[i];
                    reinterpret_cast<float4*>(p.part + to * D)[col[i]] = acc[i];
                    if (col[i] == 0) p.part_ml[to] = make_float2(top[i], sum[i]);
                }
            }
        }
        goes[0] = goes[0] && !done[0];
        goes[1] = goes[1] && !done[1];
        if (!goes[0] && !goes[1]) return;
    }
}

constexpr int kWorkersPerSm = 12;  // most warps on an SM (the workspace has room for them)

template <typename S>
int launch_decode(PagedParams p, const CUtensorMap& kmap, const CUtensorMap& vmap, int sms,
                  int64_t tiles, smd_stream_t stream) {
    static_assert(S::CTAS * kWarps <= kWorkersPerSm, "the workspace's workers");
    static_assert(S::CTAS * (S::smem(kMaxEntries) + 64 + 1024) <= 228 * 1024, "CTAs of an SM");
    static SharedLimit limit;
    auto kernel = paged_decode_kernel<S>;
    const int rc = limit.raise(kernel, S::smem(kMaxEntries));
    if (rc != SMD_OK) return rc;
    const int64_t most = static_cast<int64_t>(sms) * kWorkersPerSm;
    const int64_t want = (tiles + kWarps - 1) / kWarps;  // a tile for each warp
    int64_t grid = static_cast<int64_t>(sms) * S::CTAS;
    if (grid > want) grid = want;
    p.workers = static_cast<int>(grid) * kWarps;
    // The workspace: counts, then the partials of warps and CTAs.
    float* at = reinterpret_cast<float*>(p.arrived) + 4 * most;
    const int64_t part_rows = most * S::rows;
    p.head = at;
    p.part = p.head + part_rows * S::D;
    p.head_ml = reinterpret_cast<float2*>(p.part + part_rows * S::D);
    p.part_ml = p.head_ml + part_rows;
    return launch_pdl(kernel, dim3(static_cast<unsigned>(grid)), kThreads, S::smem(p.entries), stream,
                      p, kmap, vmap);
}

// Counts, and for each warp a partial of its own and a quarter of its CTA's four,
// of up to 32 rows (16 at 256 columns).
int64_t workspace_bytes(int sms, int D) {
    const int64_t most = static_cast<int64_t>(sms) * kWorkersPerSm;
    return 4 * most * (4 + 2 * (D == 256 ? 16 : 32) * (D + 2));
}

}  // namespace
}  // namespace smd

extern "C" int64_t smd_paged_workspace_bytes(const smd_paged_cache_t* cache) {
    if (cache == nullptr) return SMD_ERR_NULL;
    if (!smd::paged_ready(cache)) return SMD_ERR_PLAN;
    const int sms = smd::device_sms();
    if (sms <= 0) return SMD_ERR_DEVICE;
    return smd::workspace_bytes(sms, cache->head_dim);
}

extern "C" int smd_paged_decode(const uint16_t* q, int64_t q_stride, const smd_paged_cache_t* cache,
                                const int32_t* table, int64_t table_stride, int32_t width,
                                const int32_t* lengths, int32_t R, int32_t row_group, int32_t Hq,
                                float sm_scale, const int32_t* block_lists,
                                const int32_t* block_counts, int32_t K, uint16_t* out, float* lse,
                                int32_t* status, void* workspace, int64_t workspace_bytes,
                                smd_stream_t stream) {
    return smd_paged_decode_ex(q, q_stride, cache, table, table_stride, width, lengths, R, row_group, Hq,
                               sm_scale, block_lists, block_counts, K, out, lse, status, workspace,
                               workspace_bytes, stream, nullptr);
}

extern "C" int smd_paged_decode_ex(const uint16_t* q, int64_t q_stride,
                                   const smd_paged_cache_t* cache, const int32_t* table,
                                   int64_t table_stride, int32_t width, const int32_t* lengths,
                                   int32_t R, int32_t row_group, int32_t Hq, float sm_scale,
                                   const int32_t* block_lists, const int32_t* block_counts, int32_t K,
                                   uint16_t* out, float* lse, int32_t* status, void* workspace,
                                   int64_t workspace_bytes, smd_stream_t stream,
                                   const smd_plan_t* force) {
    using namespace smd;
    bool skip;
    int rc = check_paged_rows(q, q_stride, cache, table, table_stride, width, lengths, R, row_group,
                              Hq, &skip);
    if (rc != SMD_OK) return rc;
    const int D = cache->head_dim, P = cache->page_size;
    if (cache->k == nullptr) return SMD_ERR_NULL;
    if (block_lists != nullptr &&
        (K < 0 || static_cast<int64_t>(K) * P >= (1ll << 31) || row_group * cache->heads > kMaxEntries ||
         static_cast<int64_t>(R) * row_group * cache->heads >= (1ll << 31)))
        return SMD_ERR_SHAPE;
    if (skip) return SMD_OK;
    if (out == nullptr || workspace == nullptr) return SMD_ERR_NULL;
    if (!aligned(out, 16) || !aligned(lse, 4) || !aligned(status, 4) || !aligned(block_lists, 4) ||
        !aligned(block_counts, 4))
        return SMD_ERR_ALIGN;
    const int sms = device_sms();
    if (sms <= 0) return SMD_ERR_DEVICE;
    if (!aligned(workspace, 16) || workspace_bytes < smd::workspace_bytes(sms, D))
        return SMD_ERR_WORKSPACE;

    const bool lists = block_lists != nullptr;
    const int g = Hq / cache->heads, rows = lists ? g : row_group * g;
    // Tiles of 8 query rows that a warp holds: as many as there are rows for, up to what its
    // registers take. 16 requests up to 65536 tokens, 4 / 2 at 32 rows 226 / 340 us, at 16
    // rows 213 / 189; 2 / 1 at 8 rows 113 / 109 (64 requests up to 8192 tokens).
    const int most_tiles = D == 256 ? 2 : 4;
    const int RT = rows <= 8 ? 1 : rows <= 16 ? 2 : most_tiles, KT = D == 256 ? 16 : 32;
    PagedParams p{};
    p.q_stride = q_stride;
    p.table_stride = table_stride;
    p.width = width;
    p.k_scale = cache->k_scale;
    p.v_scale = cache->v_scale;
    p.pages = cache->pages;
    p.heads = cache->heads;
    p.page_size = P;
    p.row_tiles = (rows + 8 * RT - 1) / (8 * RT);
    p.x_units = lists ? p.row_tiles : cache->heads * p.row_tiles;
    p.G = row_group;
    p.g = g;
    p.g_magic = ((1u << 20) + static_cast<uint32_t>(g) - 1) / static_cast<uint32_t>(g);
    p.Hq = Hq;
    p.rows = rows;
    p.scale_log2 = sm_scale * 1.4426950408889634f;
    p.K = K;
    p.status = status;
    p.budget_ns = force != nullptr && force->wait_budget_us > 0
                      ? static_cast<uint64_t>(force->wait_budget_us) * 1000ull
                      : kWaitBudgetNs;
    p.stall = force != nullptr ? force->inject_stall : 0;
    p.arrived = static_cast<int32_t*>(workspace);
    const bool halves = page_box_tokens(*cache) < KT;  // a tile spans two pages
    CUtensorMap maps[2];
    std::memcpy(maps, &cache->map[1], sizeof maps);

    // Requests of one launch: their entries fit the prefix table, their tiles an int.
    const int64_t per_entry = (static_cast<int64_t>(lists ? K : width) * P + KT - 1) / KT + 1 + kUnitCost;
    const int64_t per_request =
        static_cast<int64_t>(lists ? row_group * cache->heads : 1) * p.x_units * per_entry;
    const int entries_of = lists ? row_group * cache->heads : 1;
    if (per_request >= (1ll << 30)) return SMD_ERR_SHAPE;
    int64_t step = kMaxEntries / entries_of;
    if (step > (1ll << 30) / per_request) step = (1ll << 30) / per_request;
    for (int64_t r = 0; r < R; r += step) {
        const int n = static_cast<int>(R - r < step ? R - r : step);
        const int64_t row = r * row_group;
        p.q = q + row * q_stride;
        p.table = table + r * table_stride;
        p.lengths = lengths + r;
        p.entries = n * entries_of;
        p.lists = lists ? block_lists + row * cache->heads * K : nullptr;
        p.counts = lists && block_counts != nullptr ? block_counts + row * cache->heads : nullptr;
        p.out = out + row * Hq * D;
        p.lse = lse != nullptr ? lse + row * Hq : nullptr;
        const int64_t tiles = n * per_request;
        const auto launch = [&](auto shape) {
            return launch_decode<decltype(shape)>(p, maps[0], maps[1], sms, tiles, stream);
        };
        if (D == 64)
            rc = halves    ? (RT == 1   ? launch(Shape<64, 1, 32, 2, 4, 3>{})
                              : RT == 2 ? launch(Shape<64, 2, 32, 2, 4, 3>{})
                                        : launch(Shape<64, 4, 32, 2, 4, 2>{}))
                 : RT == 1 ? launch(Shape<64, 1, 32, 1, 4, 3>{})
                 : RT == 2 ? launch(Shape<64, 2, 32, 1, 4, 3>{})
                           : launch(Shape<64, 4, 32, 1, 4, 2>{});
        else if (D == 128)
            rc = halves    ? (RT == 1   ? launch(Shape<128, 1, 32, 2, 2, 3>{})
                              : RT == 2 ? launch(Shape<128, 2, 32, 2, 2, 3>{})
                                        : launch(Shape<128, 4, 32, 2, 2, 2>{}))
                 : RT == 1 ? launch(Shape<128, 1, 32, 1, 2, 3>{})
                 : RT == 2 ? launch(Shape<128, 2, 32, 1, 2, 3>{})
                           : launch(Shape<128, 4, 32, 1, 2, 2>{});
        else
            rc = RT == 1 ? launch(Shape<256, 1, 16, 1, 2, 3>{}) : launch(Shape<256, 2, 16, 1, 2, 2>{});
        if (rc != SMD_OK) return rc;
    }
    return SMD_OK;
}

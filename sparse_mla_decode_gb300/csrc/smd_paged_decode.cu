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
// D x M accumulators in registers. No CTA barrier is passed until the tokens
// of a unit (a request's kv head) end, where the CTA's warps join their
// states through shared memory (the slots they have just consumed).
//
// The tiles of all units, laid end to end, are cut evenly over the grid, so a
// batch of mixed lengths loads every SM alike; a unit cut by a CTA boundary
// leaves fp32 partials in the workspace, joined in CTA order by a second
// kernel (run-to-run the same bits; no atomics, no flags).
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
#include <atomic>
#include <cstring>
#include <cstdlib>
#include <cstdlib>

#include "smd_internal.h"
#include "smd_paged.h"
#include "smd_ptx.cuh"

namespace smd {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr int kMaxEntries = 1024;  // requests (or (row, kv head) lists) of one launch
constexpr int kNoPos = 0x3fffffff; // the position of tokens that no row sees
constexpr float kPShift = 7.0f;    // weights are formed at 2^7 of the maximum kept
constexpr float kSlack = 8.0f;     // which is moved when a logit exceeds it by 2^8
constexpr int kJoinRows = 4;       // rows of a unit that a CTA of the join takes
constexpr int kUnitCost = 8;       // what ending a unit costs a CTA, in tiles

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
    int32_t rows;       // query rows of a unit before tiling: G * g, or g with lists
    float scale_log2;   // sm_scale * log2 e
    const int32_t* lists;
    const int32_t* counts;
    int32_t K;
    uint16_t* out;
    float* lse;
    int32_t* status;
    int32_t* desc;      // [grid][2]: the unit a CTA starts and does not end, its last CTA
    float* part;        // [grid][2][rows of a tile][D]
    float* part_ml;     // [grid][2][rows of a tile][2]: maximum, sum
    int32_t box;        // tokens of a copy box
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

// Transposes the 8 x 8 block of 16-bit elements whose row g holds its elements
// 2i, 2i + 1 in lane 4 g + i.
__device__ __forceinline__ uint32_t transpose8x8(uint32_t v) {
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}

// The sizes of one instantiation: D columns, RT tiles of 8 query rows, KT
// tokens a tile, ST slots of a warp's ring, CTAs an SM holds.
template <int D_, int RT_, int KT_, int ST_, int CTAS_>
struct Shape {
    static constexpr int D = D_, RT = RT_, KT = KT_, ST = ST_, CTAS = CTAS_;
    static constexpr int rows = 8 * RT;
    static constexpr int row_bytes = D < 128 ? D : 128;  // of a copy box
    static constexpr int side = KT * D;                  // bytes of a tile's K, and of its V
    static constexpr int slot = 2 * side;
    static constexpr int q_pitch = 2 * D + 32;           // 8-byte reads of 4 rows hit 4 bank groups
    static constexpr int off_q = kWarps * ST * slot;
    static constexpr int off_qf = off_q + rows * q_pitch;         // [rows] logit factors
    static constexpr int off_lim = off_qf + rows * 4;             // [rows] tokens that a row sees
    static constexpr int off_ml = off_lim + rows * 4;             // [warps][rows] maximum, sum
    static constexpr int off_meta = off_ml + kWarps * rows * 8;   // [warps][ST][8] words
    static constexpr int off_bar = off_meta + kWarps * ST * 32;
    static constexpr int off_scan = off_bar + kWarps * ST * 8;    // [warps + 1] words
    static constexpr int off_prefix = off_scan + 32;              // [entries + 1]
    static constexpr int smem(int entries) { return off_prefix + 4 * (entries + 1) + 1024; }
};

// Byte offset of 16-byte piece c of token `row` in a side of a slot, as the
// copy's swizzle places it.
template <int D, int KT>
__device__ __forceinline__ uint32_t piece(int row, int c) {
    if (D == 64) return row * 64 + ((c ^ ((row >> 1) & 3)) << 4);
    return (c >> 3) * (KT * 128) + row * 128 + (((c & 7) ^ (row & 7)) << 4);
}

// The tokens an entry's units walk, in tiles of KT; at least one tile, so that
// a unit without tokens still writes its zeros.
template <int KT>
__device__ __forceinline__ int entry_tiles(const PagedParams& p, int e) {
    int n;
    if (p.lists != nullptr) {
        int c = p.counts != nullptr ? p.counts[e] : p.K;
        n = max(min(c, p.K), 0) * p.page_size;
    } else {
        n = max(min(p.lengths[e], p.width * p.page_size), 0);
    }
    return max((n + KT - 1) / KT, 1);
}

// One tile's tokens: for each 16 of them the page, the offset in it, the first
// token's position in its request and the scales.
template <int NH>
struct Tile {
    int page[NH], off[NH], pos[NH], head;
    float ks[NH], vs[NH];
};

template <typename S>
__global__ void __launch_bounds__(kThreads, S::CTAS)
    paged_decode_kernel(const PagedParams p, const __grid_constant__ CUtensorMap kmap,
                        const __grid_constant__ CUtensorMap vmap) {
    constexpr int D = S::D, RT = S::RT, KT = S::KT, ST = S::ST;
    constexpr int NH = KT / 16;   // 16-token halves of a tile
    constexpr int NC = D / 16;    // 16-column chunks
    constexpr bool kQRegs = RT * D <= 256;  // query fragments stay in registers
    extern __shared__ uint8_t smem_raw[];
    const uint32_t base = (smem_addr(smem_raw) + 1023u) & ~1023u;
    uint8_t* const gbase = smem_raw + (base - smem_addr(smem_raw));
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, qr = lane >> 2, qi = lane & 3;
    int32_t* const prefix = reinterpret_cast<int32_t*>(gbase + S::off_prefix);
    float2* const ml = reinterpret_cast<float2*>(gbase + S::off_ml);
    float* const qf = reinterpret_cast<float*>(gbase + S::off_qf);
    int32_t* const lims = reinterpret_cast<int32_t*>(gbase + S::off_lim);
    const uint32_t ring = base + warp * ST * S::slot;
    const uint32_t bars = base + S::off_bar + warp * ST * 8;
    const uint32_t meta = base + S::off_meta + warp * ST * 32;  // ks, vs, pos of each half

    if (lane == 0) {
        for (int s = 0; s < ST; ++s) mbar_init(bars + 8 * s, 1);
        fence_mbar_init();
        fence_proxy_async();
    }
    pdl_entry();
    fence_proxy_async_global();  // the cache may have been written by the kernel before

    // Prefix sums of the entries' tiles.
    constexpr int kPer = kMaxEntries / kThreads;
    int total;
    {
        int v[kPer], sum = 0;
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
            const int e = tid * kPer + j;
            v[j] = e < p.entries ? entry_tiles<KT>(p, e) * p.x_units : 0;
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
        for (int w = 0; w < kWarps; ++w) {
            if (w < warp) before += scan[w];
            total += scan[w];
        }
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
            const int e = tid * kPer + j;
            if (e <= p.entries) prefix[e] = before;
            before += v[j];
        }
        if (tid == kThreads - 1 && p.entries == kMaxEntries) prefix[kMaxEntries] = before;
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
    const int grid = static_cast<int>(gridDim.x);
    const int per = max((cost + grid - 1) / grid, kWarps + kUnitCost);
    const auto tiles_before = [&](int64_t at) {  // tiles that lie before a cost position
        if (at >= cost) return total;
        const int c = static_cast<int>(at), e = find(c, kUnitCost);
        const int nt = (prefix[e + 1] - prefix[e]) / p.x_units;
        const int rem = c - prefix[e] - kUnitCost * p.x_units * e, x = rem / (nt + kUnitCost);
        return prefix[e] + x * nt + max(rem - x * (nt + kUnitCost) - kUnitCost, 0);
    };
    const int64_t at0 = static_cast<int64_t>(blockIdx.x) * per;
    const int t0 = tiles_before(at0), t1 = tiles_before(at0 + per);
    if (tid == 0) {
        p.desc[2 * blockIdx.x] = -1;
    }
    if (t0 >= t1) return;

    // Lane l resolves tile 32 * (k / 32) + l of this warp's tiles.
    Tile<NH> td;
    const int my_tiles = (t1 - t0 - warp + kWarps - 1) / kWarps;
    const auto resolve = [&](int kk) {
        const int t = t0 + warp + kWarps * kk;
#pragma unroll
        for (int h = 0; h < NH; ++h) {
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
        const int b = p.lists != nullptr ? e / p.heads : e;      // row, or request
        const int r = p.lists != nullptr ? b / p.G : e;
        td.head = p.lists != nullptr ? e - b * p.heads : x / p.row_tiles;
        const int len = max(min(p.lengths[r], p.width * p.page_size), 0);
        const int32_t* const row = p.table + static_cast<int64_t>(r) * p.table_stride;
#pragma unroll
        for (int h = 0; h < NH; ++h) {
            int blk = (first + 16 * h) / p.page_size;
            const int off = first + 16 * h - blk * p.page_size;
            if (p.lists != nullptr) {
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
    // Fills the slot of this warp's tile kk; all lanes call it in order of kk.
    const auto issue = [&](int kk) {
        if (kk >= my_tiles) return;
        if ((kk & 31) == 0) resolve(kk + lane);
        if (lane == (kk & 31)) {
            const int s = kk % ST;
            const uint32_t bar = bars + 8 * s, dst = ring + s * S::slot;
            mbar_arrive_expect_tx(bar, S::slot);
#pragma unroll
            for (int h = 0; h < NH; ++h) {
                if (h > 0 && p.box != 16) break;
#pragma unroll
                for (int sub = 0; sub < (D > 128 ? 2 : 1); ++sub) {
                    const uint32_t at = dst + sub * KT * 128 + h * 16 * S::row_bytes;
                    tma_load_4d(at, &kmap, sub * 128, td.off[h], td.head, td.page[h], bar);
                    tma_load_4d(at + S::side, &vmap, sub * 128, td.off[h], td.head, td.page[h],
                                bar);
                }
            }
            sts_v4(meta + 32 * s, make_float4(td.ks[0], td.ks[NH - 1], td.vs[0], td.vs[NH - 1]));
            sts64(meta + 32 * s + 16, td.pos[0], td.pos[NH - 1]);
        }
        __syncwarp();
    };

    // Row m (of the unit, before tiling): verify row and query head.
    const auto row_limit = [&](int m, int b, int len) {
        const int i = p.lists != nullptr ? b % p.G : m / p.g;
        return max(len - p.G + 1 + i, 0);
    };
    // The unit's queries as f16 in shared memory, with each row's logit factor
    // (positive: a negative softmax scale turns the query's sign) and limit.
    const auto load_q = [&](int e, int x) {
        const int rt = x % p.row_tiles, u_b = p.lists != nullptr ? e / p.heads : e * p.G;
        const int u_len =
            max(min(p.lengths[p.lists != nullptr ? u_b / p.G : e], p.width * p.page_size), 0);
        const int head = p.lists != nullptr ? e % p.heads : x / p.row_tiles;
        constexpr int kPieces = D / 8;
        for (int idx = tid; idx < S::rows * kPieces; idx += kThreads) {
            const int m = idx / kPieces, c = idx % kPieces, mm = rt * S::rows + m;
            uint4 v = make_uint4(0, 0, 0, 0);
            if (mm < p.rows) {
                const int64_t b = p.lists != nullptr ? e / p.heads
                                                     : static_cast<int64_t>(e) * p.G + mm / p.g;
                v = *reinterpret_cast<const uint4*>(p.q + b * p.q_stride +
                                                    static_cast<int64_t>(head * p.g + mm % p.g) * D +
                                                    8 * c);
            }
            const uint32_t w[4] = {v.x, v.y, v.z, v.w};
            float f[8], a = 0.0f;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                f[2 * j] = __uint_as_float(w[j] << 16);
                f[2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
                a = fmaxf(a, fmaxf(fabsf(f[2 * j]), fabsf(f[2 * j + 1])));
            }
#pragma unroll
            for (int o = 1; o < kPieces; o <<= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, o));
            // up = 2^(14 - exponent of a), within what a float holds
            const int ex = static_cast<int>(__float_as_uint(a) >> 23);
            const int ue = min(14 + 127 - ex + 127, 253);
            float up = a > 0.0f && ex < 255 ? __uint_as_float(static_cast<uint32_t>(ue) << 23) : 1.0f;
            if (c == 0) {
                qf[m] = fabsf(p.scale_log2) / up;
                lims[m] = mm < p.rows ? row_limit(mm, u_b, u_len) : 0;
            }
            if (p.scale_log2 < 0.0f) up = -up;
            const uint32_t at = base + S::off_q + m * S::q_pitch + 16 * c;
            asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(at),
                         "r"(f16x2(f[0] * up, f[1] * up)), "r"(f16x2(f[2] * up, f[3] * up)),
                         "r"(f16x2(f[4] * up, f[5] * up)), "r"(f16x2(f[6] * up, f[7] * up))
                         : "memory");
        }
    };

    bool ok = true;
    int k = 0, t = t0, e = find_entry(t0);
#pragma unroll 1
    for (int s = 0; s < ST - 1; ++s) issue(s);
    {
        const int nt = (prefix[e + 1] - prefix[e]) / p.x_units;
        load_q(e, (t0 - prefix[e]) / nt);
    }
    __syncthreads();

#pragma unroll 1
    while (t < t1) {
        while (prefix[e + 1] <= t) ++e;
        const int nt = (prefix[e + 1] - prefix[e]) / p.x_units, x = (t - prefix[e]) / nt;
        const int u0 = prefix[e] + x * nt, u1 = u0 + nt, tend = min(u1, t1);
        const int rt = x % p.row_tiles, b0 = p.lists != nullptr ? e / p.heads : e * p.G;
        const int m_real = min(p.rows - rt * S::rows, S::rows);
        const int min_lim = lims[0], max_lim = lims[m_real - 1];
        float m[RT][2], l[RT][2], o[RT][NC][4], vref = 0.0f;
        uint32_t qb[kQRegs ? RT : 1][kQRegs ? NC : 1][2];
#pragma unroll
        for (int n = 0; n < RT; ++n)
#pragma unroll
            for (int y = 0; y < 2; ++y) {
                m[n][y] = -INFINITY;
                l[n][y] = 0.0f;
            }
#pragma unroll
        for (int n = 0; n < RT; ++n)
#pragma unroll
            for (int c = 0; c < NC; ++c)
#pragma unroll
                for (int j = 0; j < 4; ++j) o[n][c][j] = 0.0f;
        const uint32_t q_at = base + S::off_q + qr * S::q_pitch + 8 * qi;
        if (kQRegs) {
#pragma unroll
            for (int n = 0; n < (kQRegs ? RT : 0); ++n)
#pragma unroll
                for (int c = 0; c < NC; ++c)
                    lds64(q_at + n * 8 * S::q_pitch + 32 * c, qb[n][c][0], qb[n][c][1]);
        }

#pragma unroll 1
        for (; t0 + warp + kWarps * k < tend; ++k) {
            issue(k + ST - 1);
            const int slot = k % ST;
            mbar_wait(bars + 8 * slot, (k / ST) & 1, ok, p.status, kWaitBudgetNs);
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
                        if (kQRegs) {
                            b0v = qb[kQRegs ? n : 0][kQRegs ? c : 0][0];
                            b1v = qb[kQRegs ? n : 0][kQRegs ? c : 0][1];
                        } else if (z == 0 || NH == 1) {
                            lds64(q_at + n * 8 * S::q_pitch + 32 * c, b0v, b1v);
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
                        const int lim = lims[8 * n + 2 * qi + y];
#pragma unroll
                        for (int h = 0; h < NH; ++h)
#pragma unroll
                            for (int z = 0; z < 2; ++z)
                                if (pos[h] + qr + 8 * z >= lim) s[h][n][2 * z + y] = -INFINITY;
                    }
                // V of tokens that no row sees becomes 0 (0 times a NaN would not be).
#pragma unroll 1
                for (int z = lane; z < KT * NC; z += 32) {
                    const int j = z / NC;
                    if ((j < 16 ? pos[0] : pos[1]) + (j & 15) >= max_lim)
                        sts_zero16(vs_at + piece<D, KT>(j, z % NC));
                }
                // V of tokens that some rows see and others do not: a NaN goes to the rows
                // that see it here, and 0 stands in its place for the products.
                if (min_lim < max_lim) {
#pragma unroll 1
                    for (int j = 0; j < KT; ++j) {
                        const int at = (j < 16 ? pos[0] : pos[1]) + (j & 15);
                        if (at < min_lim || at >= max_lim) continue;
                        bool nan = false;
#pragma unroll 1
                        for (int z = lane; z < 4 * NC; z += 32) {
                            const uint32_t w = lds_u32(vs_at + piece<D, KT>(j, z >> 2) + 4 * (z & 3));
                            nan = nan || (((w & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u) != 0;
                        }
                        if (!__any_sync(0xffffffffu, nan)) continue;
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
                                            if (at < lims[8 * n + 2 * qi + y])
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

            // The maximum stays while no logit exceeds it by more than kSlack.
            float f[NH][RT][2], v[RT][2];
            bool moved = false;
#pragma unroll
            for (int n = 0; n < RT; ++n)
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                    const float fac = qf[8 * n + 2 * qi + y];
                    v[n][y] = -INFINITY;
#pragma unroll
                    for (int h = 0; h < NH; ++h) {
                        f[h][n][y] = fmaxf(fac * ks[h], 1.17549435e-38f);
                        v[n][y] = fmaxf(v[n][y], fmaxf(s[h][n][y], s[h][n][2 + y]) * f[h][n][y]);
                    }
                    moved = moved || v[n][y] > m[n][y] + kSlack;
                }
            if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
                for (int n = 0; n < RT; ++n)
#pragma unroll
                    for (int y = 0; y < 2; ++y) {
                        float top = fmaxf(m[n][y], v[n][y]);
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

            // weights and the second product
#pragma unroll
            for (int h = 0; h < NH; ++h) {
                if (vs[h] > vref) {
                    const float down = vref / vs[h];
                    vref = vs[h];
#pragma unroll
                    for (int n = 0; n < RT; ++n)
#pragma unroll
                        for (int c = 0; c < NC; ++c)
#pragma unroll
                            for (int j = 0; j < 4; ++j) o[n][c][j] *= down;
                }
                const float ratio = vref > 0.0f ? vs[h] / vref : 0.0f;
                uint32_t pb[RT][2];
#pragma unroll
                for (int n = 0; n < RT; ++n) {
                    float w[4];
#pragma unroll
                    for (int y = 0; y < 2; ++y) {
                        const float top = m[n][y] == -INFINITY ? 0.0f : m[n][y] - kPShift;
#pragma unroll
                        for (int z = 0; z < 2; ++z) {
                            const float pv = ex2_approx(fmaf(s[h][n][2 * z + y], f[h][n][y], -top));
                            l[n][y] += pv;
                            w[2 * z + y] = pv * ratio;
                        }
                    }
                    pb[n][0] = transpose8x8(f16x2(w[0], w[1]));
                    pb[n][1] = transpose8x8(f16x2(w[2], w[3]));
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
                            mma_f16(o[n][c + z], a[0], a[1], a[2], a[3], pb[n][0], pb[n][1]);
                    }
                }
            }
            __syncwarp();
        }

        // The warps' states become the CTA's. Warp w holds tiles of this unit if one of
        // its turns fell into [t, tend); the slot it consumed last takes its accumulators.
#pragma unroll
        for (int n = 0; n < RT; ++n)
#pragma unroll
            for (int y = 0; y < 2; ++y) {
                float v = l[n][y];
                v += __shfl_xor_sync(0xffffffffu, v, 4);
                v += __shfl_xor_sync(0xffffffffu, v, 8);
                v += __shfl_xor_sync(0xffffffffu, v, 16);
                if (qr == 0) ml[warp * S::rows + 8 * n + 2 * qi + y] = make_float2(m[n][y], v);
            }
        __syncthreads();
        const bool mine = k > 0 && t0 + warp + kWarps * (k - 1) >= t;
        float wgt[RT][2];
#pragma unroll
        for (int n = 0; n < RT; ++n)
#pragma unroll
            for (int y = 0; y < 2; ++y) {
                float top = -INFINITY;
#pragma unroll
                for (int w = 0; w < kWarps; ++w)
                    top = fmaxf(top, ml[w * S::rows + 8 * n + 2 * qi + y].x);
                wgt[n][y] = m[n][y] == -INFINITY ? 0.0f : vref * ex2_approx(m[n][y] - top);
            }
        const bool whole = u0 >= t0 && u1 <= t1;
        const int part_at = (2 * static_cast<int>(blockIdx.x) + (u0 >= t0 ? 1 : 0)) * S::rows;
        if (!whole && u0 >= t0 && tid == 0) {
            p.desc[2 * blockIdx.x] = e * p.x_units + x;
            // the CTA that holds the unit's last tile
            p.desc[2 * blockIdx.x + 1] = (u1 - 1 + kUnitCost * (e * p.x_units + x + 1)) / per;
        }
        constexpr int kRound = RT < KT / 16 ? RT : KT / 16;  // row tiles that a slot holds in fp32
#pragma unroll
        for (int n0 = 0; n0 < RT; n0 += kRound) {
                if (mine) {
                    const uint32_t buf = ring + ((k - 1) % ST) * S::slot;
#pragma unroll
                    for (int n = 0; n < kRound; ++n)
#pragma unroll
                        for (int c = 0; c < NC; ++c) {
                            const float(&v)[4] = o[n0 + n][c];
#pragma unroll
                            for (int y = 0; y < 2; ++y) {
                                const uint32_t unit = (4 * c + (qr >> 1)) ^ (qi << 1);
                                const float w = wgt[n0 + n][y];
                                sts64(buf + (8 * n + 2 * qi + y) * D * 4 + (unit << 4) + 8 * (qr & 1),
                                      __float_as_uint(v[y] * w), __float_as_uint(v[2 + y] * w));
                            }
                        }
                    fence_proxy_async();
                }
                __syncthreads();
                if (n0 == 0 && tend < t1) {
                    // The next unit's queries: every warp is past its tiles of this one.
                    int en = e;
                    while (prefix[en + 1] <= tend) ++en;
                    const int ntn = (prefix[en + 1] - prefix[en]) / p.x_units;
                    load_q(en, (tend - prefix[en]) / ntn);
                }
                for (int idx = tid; idx < 8 * kRound * (D / 4); idx += kThreads) {
                    const int row = idx / (D / 4), unit = idx % (D / 4), mm = 8 * n0 + row;
                    if (mm >= m_real) continue;
                    float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                    float top = -INFINITY, sum = 0.0f;
                    for (int w = 0; w < kWarps; ++w) top = fmaxf(top, ml[w * S::rows + mm].x);
                    for (int w = 0; w < kWarps; ++w) {
                        // the last of warp w's tiles before tend
                        const int last = (tend - t0 - 1 - w) >= 0 ? (tend - t0 - 1 - w) / kWarps : -1;
                        if (last < 0 || t0 + w + kWarps * last < t) continue;
                        const float2 s = ml[w * S::rows + mm];
                        sum += s.y * (s.x == -INFINITY ? 0.0f : ex2_approx(s.x - top));  // a NaN stays one
                        const float4 f =
                            lds_f4(base + (w * ST + last % ST) * S::slot + row * D * 4 +
                                   ((unit ^ (((row >> 1) & 3) << 1)) << 4));
                        acc.x += f.x;
                        acc.y += f.y;
                        acc.z += f.z;
                        acc.w += f.w;
                    }
                    const int col = 4 * unit;
                    if (whole) {
                        const int ma = rt * S::rows + mm;
                        const int b = p.lists != nullptr ? b0 : b0 + ma / p.g;
                        const int head = p.lists != nullptr ? e % p.heads : x / p.row_tiles;
                        const int64_t at = static_cast<int64_t>(b) * p.Hq + head * p.g + ma % p.g;
                        const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
                        uint2 v = make_uint2(bf16x2(acc.x * inv, acc.y * inv),
                                             bf16x2(acc.z * inv, acc.w * inv));
                        *reinterpret_cast<uint2*>(p.out + at * D + col) = v;
                        if (col == 0 && p.lse != nullptr)
                            p.lse[at] = sum == 0.0f ? -INFINITY
                                                    : 0.69314718055994531f * (top - kPShift + log2f(sum));
                    } else {
                        *reinterpret_cast<float4*>(p.part + static_cast<int64_t>(part_at + mm) * D + col) = acc;
                        if (col == 0)
                            *reinterpret_cast<float2*>(p.part_ml + 2 * static_cast<int64_t>(part_at + mm)) =
                                make_float2(top, sum);
                    }
                }
                __syncthreads();
            }
        t = tend;
    }
    // A wait that ran out left its copy in flight: none may outlive the CTA.
    if (!ok)
        for (int j = max(k - ST, 0); j < k; ++j) {
            bool done = true;
            mbar_wait(bars + 8 * (j % ST), (j / ST) & 1, done, p.status, kWaitBudgetNs, true);
        }
}

// Joins the partials of the units that a CTA boundary cut. Block (c, y): the
// unit that CTA c starts, rows 4 y ..; two warps a row take its CTAs in turn,
// their sums are added in that order.
template <int D>
__global__ void __launch_bounds__(2 * kJoinRows * 32) paged_join_kernel(const PagedParams p, int rows) {
    pdl_entry();
    const int unit = p.desc[2 * blockIdx.x];
    if (unit < 0) return;
    const int c0 = static_cast<int>(blockIdx.x), c1 = p.desc[2 * blockIdx.x + 1];
    const int e = unit / p.x_units, x = unit % p.x_units, rt = x % p.row_tiles;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, half = warp & 1;
    const int mm = blockIdx.y * kJoinRows + (warp >> 1), ma = rt * rows + mm;
    const bool real = mm < rows && ma < p.rows;
    constexpr int kV = D / 128 > 0 ? D / 128 : 1;  // float4 of a lane
    __shared__ float4 other[kJoinRows][kV][32];
    const auto at = [&](int c) { return static_cast<int64_t>(2 * c + (c == c0 ? 1 : 0)) * rows + mm; };
    float top = -INFINITY, sum = 0.0f;
    float4 acc[kV];
#pragma unroll
    for (int v = 0; v < kV; ++v) acc[v] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (real) {
        for (int c = c0 + lane; c <= c1; c += 32) top = fmaxf(top, p.part_ml[2 * at(c)]);
        top = warp_max(top);
        for (int c = c0 + lane; c <= c1; c += 32) {
            const float m = p.part_ml[2 * at(c)];
            sum += p.part_ml[2 * at(c) + 1] * (m == -INFINITY ? 0.0f : ex2_approx(m - top));
        }
        sum = warp_sum(sum);
#pragma unroll 4
        for (int c = c0 + half; c <= c1; c += 2) {
            const float m = p.part_ml[2 * at(c)];
            const float w = m == -INFINITY ? 0.0f : ex2_approx(m - top);
#pragma unroll
            for (int v = 0; v < kV; ++v)
                if (D >= 128 || lane < D / 4) {
                    const float4 f = reinterpret_cast<const float4*>(p.part + at(c) * D)[32 * v + lane];
                    acc[v].x += f.x * w;
                    acc[v].y += f.y * w;
                    acc[v].z += f.z * w;
                    acc[v].w += f.w * w;
                }
        }
        if (half == 1)
#pragma unroll
            for (int v = 0; v < kV; ++v) other[warp >> 1][v][lane] = acc[v];
    }
    __syncthreads();
    if (!real || half == 1) return;
    const int b = p.lists != nullptr ? e / p.heads : e * p.G + ma / p.g;
    const int head = p.lists != nullptr ? e % p.heads : x / p.row_tiles;
    const int64_t row = static_cast<int64_t>(b) * p.Hq + head * p.g + ma % p.g;
    const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
#pragma unroll
    for (int v = 0; v < kV; ++v)
        if (D >= 128 || lane < D / 4) {
            const float4 f = other[warp >> 1][v][lane];
            const uint2 u = make_uint2(bf16x2((acc[v].x + f.x) * inv, (acc[v].y + f.y) * inv),
                                       bf16x2((acc[v].z + f.z) * inv, (acc[v].w + f.w) * inv));
            reinterpret_cast<uint2*>(p.out + row * D)[32 * v + lane] = u;
        }
    if (lane == 0 && p.lse != nullptr)
        p.lse[row] = sum == 0.0f ? -INFINITY : 0.69314718055994531f * (top - kPShift + log2f(sum));
}

constexpr int kMaxDevices = 64;
constexpr int kWaves = 1;       // CTAs launched for each that an SM holds
constexpr int kGridPerSm = 6;   // most CTAs for each SM (the workspace has room for them)

template <typename S>
int launch_decode(PagedParams p, const CUtensorMap& kmap, const CUtensorMap& vmap, int sms,
                  int64_t tiles, smd_stream_t stream) {
    static_assert(S::CTAS * (S::smem(kMaxEntries) + 1024) <= 228 * 1024, "CTAs of an SM");
    static std::atomic<bool> ready[kMaxDevices];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return SMD_ERR_DEVICE;
    auto kernel = paged_decode_kernel<S>;
    if (!ready[dev]) {
        if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 S::smem(kMaxEntries)) != cudaSuccess) {
            (void)cudaGetLastError();
            return SMD_ERR_DEVICE;
        }
        ready[dev] = true;
    }
    // At least kWarps tiles a CTA, so that each warp has one.
    const int64_t most = static_cast<int64_t>(sms) * kGridPerSm;
    const int64_t want = (tiles + kWarps - 1) / kWarps;
    const char* ev = getenv("SMD_W"); int64_t grid = static_cast<int64_t>(sms) * S::CTAS * (ev ? atoi(ev) : kWaves);
    if (grid > most) grid = most;
    if (grid > want) grid = want;
    p.part = reinterpret_cast<float*>(p.desc) + 4 * most;  // 16-byte aligned
    p.part_ml = p.part + most * 2 * S::rows * S::D;
    int rc = launch_pdl(kernel, dim3(static_cast<unsigned>(grid)), kThreads, S::smem(p.entries),
                        stream, p, kmap, vmap);
    if (rc != SMD_OK) return rc;
    const int join_rows = p.rows < S::rows ? p.rows : S::rows;
    return launch_pdl(paged_join_kernel<S::D>,
                      dim3(static_cast<unsigned>(grid), (join_rows + kJoinRows - 1) / kJoinRows),
                      2 * kJoinRows * 32, 0, stream, p, static_cast<int>(S::rows));
}

// A CTA's descriptor and two partials of up to 32 rows (16 at 256 columns).
int64_t workspace_bytes(int sms, int D) {
    const int64_t most = static_cast<int64_t>(sms) * kGridPerSm;
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
    using namespace smd;
    bool skip;
    int rc = check_paged_rows(q, q_stride, cache, table, table_stride, width, lengths, R, row_group,
                              Hq, &skip);
    if (rc != SMD_OK) return rc;
    const int D = cache->head_dim, P = cache->page_size;
    if (cache->k == nullptr) return SMD_ERR_NULL;
    if (block_lists != nullptr &&
        (K < 0 || static_cast<int64_t>(K) * P >= (1ll << 31) ||
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
    const int most_tiles = D == 256 ? 2 : 4;  // of 8 rows: what the registers hold
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
    p.Hq = Hq;
    p.rows = rows;
    p.scale_log2 = sm_scale * 1.4426950408889634f;
    p.K = K;
    p.status = status;
    p.desc = static_cast<int32_t*>(workspace);
    p.box = page_box_tokens(*cache);
    CUtensorMap maps[2];
    std::memcpy(maps, &cache->map[1], sizeof maps);

    // Requests of one launch: their entries fit the prefix table, their tiles an int.
    const int64_t per_entry = (static_cast<int64_t>(lists ? K : width) * P + KT - 1) / KT + 1;
    const int64_t per_request =
        static_cast<int64_t>(lists ? row_group * cache->heads : 1) * p.x_units * per_entry;
    const int entries_of = lists ? row_group * cache->heads : 1;
    if (entries_of > kMaxEntries || per_request >= (1ll << 30)) return SMD_ERR_SHAPE;
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
            rc = RT == 1   ? launch(Shape<64, 1, 32, 4, 3>{})
                 : RT == 2 ? launch(Shape<64, 2, 32, 4, 3>{})
                           : launch(Shape<64, 4, 32, 4, 2>{});
        else if (D == 128)
            rc = RT == 1   ? launch(Shape<128, 1, 32, 2, 3>{})
                 : RT == 2 ? launch(Shape<128, 2, 32, 2, 3>{})
                           : launch(Shape<128, 4, 32, 3, 2>{});
        else
            rc = RT == 1 ? launch(Shape<256, 1, 16, 2, 3>{}) : launch(Shape<256, 2, 16, 3, 2>{});
        if (rc != SMD_OK) return rc;
    }
    return SMD_OK;
}

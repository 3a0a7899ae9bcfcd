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
// and M = 8 or 16 rows would leave most of a 128-lane tcgen05 tile empty.
//
// A warp is a worker of its own: it walks tiles of KT tokens of one (page,
// head) through a ring of ST slots that its own lanes fill with tensor copies
// (K and V of a tile: one barrier), and holds the tile's softmax state and its
// M x D accumulators in registers. No CTA barrier is passed until the tokens
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
// transposing ldmatrix as two codes each of tokens 2i and 2i+1; one byte
// permute pairs the tokens, and the even and odd columns of a 16-column chunk
// go to two MMAs, whose results leave a lane 4 consecutive columns.
//
// Rounding: q enters as f16 after a power of two per row that puts its largest
// element in [2^14, 2^15) (bf16 has fewer bits than f16, so this is exact down
// to 2^-30 of the largest); the weights enter as f16 at 2^14 of the running
// maximum, 11 bits, below the 8 of the bf16 output; their sum is of the fp32
// weights; accumulators, maxima and sums are fp32. V's scale multiplies the
// weights relative to the largest scale met so far (exact for powers of two),
// so f16 never sees its range.
#include <atomic>
#include <cstring>

#include "smd_internal.h"
#include "smd_paged.h"
#include "smd_ptx.cuh"

namespace smd {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr int kMaxEntries = 1024;  // requests (or (row, kv head) lists) of one launch
constexpr int kNoPos = 0x3fffffff; // the position of tokens that no row sees
constexpr float kPShift = 14.0f;   // weights are formed at 2^14 of the maximum
constexpr int kJoinRows = 4;       // rows of a unit that a CTA of the join takes

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

// The sizes of one instantiation: D columns, MT tiles of 16 query rows, KT
// tokens a tile, ST slots of a warp's ring.
template <int D, int MT, int KT, int ST>
struct Shape {
    static constexpr int rows = 16 * MT;
    static constexpr int row_bytes = D < 128 ? D : 128;  // of a copy box
    static constexpr int side = KT * D;                  // bytes of a tile's K, and of its V
    static constexpr int slot = 2 * side;
    static constexpr int q_pitch = 2 * D + 32;           // 8-byte reads of 4 rows hit 4 bank groups
    static constexpr int off_q = kWarps * ST * slot;
    static constexpr int off_qf = off_q + rows * q_pitch;         // [rows] logit factors
    static constexpr int off_ml = off_qf + rows * 4;              // [warps][rows] maximum, sum
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

template <int D, int MT, int KT, int ST>
__global__ void __launch_bounds__(kThreads, (D == 256 || (D == 128 && MT == 2)) ? 2 : 3)
    paged_decode_kernel(const PagedParams p, const __grid_constant__ CUtensorMap kmap,
                        const __grid_constant__ CUtensorMap vmap) {
    using S = Shape<D, MT, KT, ST>;
    constexpr int NT = KT / 8;    // key tiles of an MMA
    constexpr int NH = KT / 16;   // k-steps of the second product
    constexpr int NC = D / 16;    // 16-column chunks
    constexpr bool kQRegs = MT == 1 && D <= 128;  // query fragments stay in registers
    extern __shared__ uint8_t smem_raw[];
    const uint32_t base = (smem_addr(smem_raw) + 1023u) & ~1023u;
    uint8_t* const gbase = smem_raw + (base - smem_addr(smem_raw));
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, qr = lane >> 2, qi = lane & 3;
    int32_t* const prefix = reinterpret_cast<int32_t*>(gbase + S::off_prefix);
    float2* const ml = reinterpret_cast<float2*>(gbase + S::off_ml);
    float* const qf = reinterpret_cast<float*>(gbase + S::off_qf);
    const uint32_t ring = base + warp * ST * S::slot;
    const uint32_t bars = base + S::off_bar + warp * ST * 8;
    volatile uint32_t* const meta =
        reinterpret_cast<uint32_t*>(gbase + S::off_meta) + warp * ST * 8;

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

    const int grid = static_cast<int>(gridDim.x);
    const int per = max((total + grid - 1) / grid, kWarps);
    const int t0 = min(static_cast<int>(blockIdx.x) * per, total), t1 = min(t0 + per, total);
    if (tid == 0) {
        p.desc[2 * blockIdx.x] = -1;
    }
    if (t0 >= t1) return;

    const auto find_entry = [&](int t) {  // the entry of tile t (< total)
        int lo = 0, hi = p.entries;       // prefix[lo] <= t < prefix[hi]
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (prefix[mid] <= t) lo = mid;
            else hi = mid;
        }
        return lo;
    };

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
            td.ks[h] = td.vs[h] = 0.0f;
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
        fence_proxy_async();
        __syncwarp();
        if (lane == (kk & 31)) {
            const int s = kk % ST;
            const uint32_t bar = bars + 8 * s, dst = ring + s * S::slot;
            mbar_arrive_expect_tx(bar, S::slot);
            const int step = p.box == 16 ? 1 : NH;
            for (int h = 0; h < NH; h += step) {
#pragma unroll
                for (int sub = 0; sub < (D > 128 ? 2 : 1); ++sub) {
                    const uint32_t at = dst + sub * KT * 128 + h * 16 * S::row_bytes;
                    tma_load_4d(at, &kmap, sub * 128, td.off[h], td.head, td.page[h], bar);
                    tma_load_4d(at + S::side, &vmap, sub * 128, td.off[h], td.head, td.page[h],
                                bar);
                }
            }
#pragma unroll
            for (int h = 0; h < NH; ++h) {
                meta[8 * s + 3 * h] = __float_as_uint(td.ks[h]);
                meta[8 * s + 3 * h + 1] = __float_as_uint(td.vs[h]);
                meta[8 * s + 3 * h + 2] = static_cast<uint32_t>(td.pos[h]);
            }
        }
        __syncwarp();
    };

    // Row m (of the unit, before tiling): verify row and query head.
    const auto row_limit = [&](int m, int b, int len) {
        const int i = p.lists != nullptr ? b % p.G : m / p.g;
        return max(len - p.G + 1 + i, 0);
    };
    // The unit's queries as f16 in shared memory, with each row's logit factor.
    const auto load_q = [&](int e, int x) {
        const int rt = x % p.row_tiles;
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
            const float up = a > 0.0f && ex < 255 ? __uint_as_float(static_cast<uint32_t>(ue) << 23) : 1.0f;
            const uint32_t at = base + S::off_q + m * S::q_pitch + 16 * c;
            asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(at),
                         "r"(f16x2(f[0] * up, f[1] * up)), "r"(f16x2(f[2] * up, f[3] * up)),
                         "r"(f16x2(f[4] * up, f[5] * up)), "r"(f16x2(f[6] * up, f[7] * up))
                         : "memory");
            if (c == 0) qf[m] = p.scale_log2 / up;
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
        const int r = p.lists != nullptr ? b0 / p.G : e;
        const int len = max(min(p.lengths[r], p.width * p.page_size), 0);
        const int m_real = min(p.rows - rt * S::rows, S::rows);
        const int min_lim = row_limit(rt * S::rows, b0, len);
        const int max_lim = row_limit(rt * S::rows + m_real - 1, b0, len);
        int lim[MT][2];
        float fac[MT][2], m[MT][2], l[MT][2], o[MT][NC][2][4], vref = 0.0f;
        uint32_t qa[kQRegs ? NC : 1][4];
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int row = 16 * i + 8 * j + qr;
                lim[i][j] = row_limit(rt * S::rows + min(row, m_real - 1), b0, len);
                fac[i][j] = qf[row];
                m[i][j] = -INFINITY;
                l[i][j] = 0.0f;
            }
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int c = 0; c < NC; ++c)
#pragma unroll
                for (int j = 0; j < 8; ++j) o[i][c][j >> 2][j & 3] = 0.0f;
        const uint32_t q_at = base + S::off_q + qr * S::q_pitch + 8 * qi;
        if (kQRegs) {
#pragma unroll
            for (int c = 0; c < (kQRegs ? NC : 0); ++c) {
                lds64(q_at + 32 * c, qa[c][0], qa[c][2]);
                lds64(q_at + 8 * S::q_pitch + 32 * c, qa[c][1], qa[c][3]);
            }
        }

#pragma unroll 1
        for (; t0 + warp + kWarps * k < tend; ++k) {
            issue(k + ST - 1);
            const int slot = k % ST;
            mbar_wait(bars + 8 * slot, (k / ST) & 1, ok, p.status, kWaitBudgetNs);
            const uint32_t ks_at = ring + slot * S::slot, vs_at = ks_at + S::side;

            // logits
            float s[MT][NT][4];
#pragma unroll
            for (int i = 0; i < MT; ++i)
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int j = 0; j < 4; ++j) s[i][n][j] = 0.0f;
#pragma unroll
            for (int c0 = 0; c0 < NC; c0 += 4 / NT) {
                uint32_t kr[4];
                const int row = lane % KT, cc = c0 + lane / KT;
                ldsm4(ks_at + piece<D, KT>(row, cc), kr);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int c = c0 + j / NT, n = j % NT;
                    uint32_t b0v, b1v;
                    e4m3_to_f16(kr[j], b0v, b1v);
#pragma unroll
                    for (int i = 0; i < MT; ++i) {
                        uint32_t a[4];
                        if (kQRegs) {
#pragma unroll
                            for (int z = 0; z < 4; ++z) a[z] = qa[kQRegs ? c : 0][z];
                        } else {
                            lds64(q_at + i * 16 * S::q_pitch + 32 * c, a[0], a[2]);
                            lds64(q_at + (i * 16 + 8) * S::q_pitch + 32 * c, a[1], a[3]);
                        }
                        mma_f16(s[i][n], a[0], a[1], a[2], a[3], b0v, b1v);
                    }
                }
            }

            // scale, mask
            float ks[NH], vs[NH];
            int pos[NH];
#pragma unroll
            for (int h = 0; h < NH; ++h) {
                ks[h] = __uint_as_float(meta[8 * slot + 3 * h]);
                vs[h] = __uint_as_float(meta[8 * slot + 3 * h + 1]);
                pos[h] = static_cast<int>(meta[8 * slot + 3 * h + 2]);
            }
#pragma unroll
            for (int i = 0; i < MT; ++i)
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int j = 0; j < 4; ++j) s[i][n][j] *= fac[i][j >> 1] * ks[n >> 1];
            bool tail = false;
#pragma unroll
            for (int h = 0; h < NH; ++h) tail = tail || pos[h] + 15 >= min_lim;
            if (tail) {
#pragma unroll
                for (int i = 0; i < MT; ++i)
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            if (pos[n >> 1] + 8 * (n & 1) + 2 * qi + (j & 1) >= lim[i][j >> 1])
                                s[i][n][j] = -INFINITY;
                // V of tokens that no row sees becomes 0 (0 times a NaN would not be).
#pragma unroll
                for (int z = lane; z < KT * NC; z += 32) {
                    const int j = z / NC;
                    if (pos[NH == 1 ? 0 : j >> 4] + (j & 15) >= max_lim)
                        sts_zero16(vs_at + piece<D, KT>(j, z % NC));
                }
                // V of tokens that some rows see and others do not: a NaN goes to the rows
                // that see it here, and 0 stands in its place for the products.
                if (min_lim < max_lim) {
#pragma unroll 1
                    for (int j = 0; j < KT; ++j) {
                        const int at = pos[NH == 1 ? 0 : j >> 4] + (j & 15);
                        if (at < min_lim || at >= max_lim) continue;
#pragma unroll
                        for (int c = 0; c < NC; ++c) {
                            const uint32_t a = vs_at + piece<D, KT>(j, c) + 4 * qi;
                            const uint32_t w = lds_u32(a);
                            uint32_t nan = 0;
#pragma unroll
                            for (int z = 0; z < 4; ++z)
                                if (((w >> (8 * z)) & 0x7fu) == 0x7fu) {
                                    nan |= 0xffu << (8 * z);
#pragma unroll
                                    for (int i = 0; i < MT; ++i)
#pragma unroll
                                        for (int y = 0; y < 2; ++y)
                                            if (at < lim[i][y])
                                                o[i][c][z & 1][2 * y + (z >> 1)] = NAN;
                                }
                            __syncwarp();
                            if (nan != 0 && qr == 0) sts32(a, w & ~nan);
                        }
                    }
                }
                __syncwarp();
            }

            // the running maximum
#pragma unroll
            for (int i = 0; i < MT; ++i) {
                float alpha[2];
                bool moved = false;
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                    float v = m[i][y];
#pragma unroll
                    for (int n = 0; n < NT; ++n)
                        v = fmaxf(v, fmaxf(s[i][n][2 * y], s[i][n][2 * y + 1]));
                    v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 1));
                    v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 2));
                    alpha[y] = v > m[i][y] ? ex2_approx(m[i][y] - v) : 1.0f;
                    moved = moved || v > m[i][y];
                    m[i][y] = v;
                }
                if (__any_sync(0xffffffffu, moved)) {
                    l[i][0] *= alpha[0];
                    l[i][1] *= alpha[1];
#pragma unroll
                    for (int c = 0; c < NC; ++c)
#pragma unroll
                        for (int j = 0; j < 8; ++j) o[i][c][j >> 2][j & 3] *= alpha[(j >> 1) & 1];
                }
            }

            // weights and the second product
#pragma unroll
            for (int h = 0; h < NH; ++h) {
                if (vs[h] > vref) {
                    const float down = vref / vs[h];
                    vref = vs[h];
#pragma unroll
                    for (int i = 0; i < MT; ++i)
#pragma unroll
                        for (int c = 0; c < NC; ++c)
#pragma unroll
                            for (int j = 0; j < 8; ++j) o[i][c][j >> 2][j & 3] *= down;
                }
                const float ratio = vref > 0.0f ? vs[h] / vref : 0.0f;
                uint32_t pa[MT][4];
#pragma unroll
                for (int i = 0; i < MT; ++i) {
                    float w[2][4];
#pragma unroll
                    for (int y = 0; y < 2; ++y) {
                        const float top = m[i][y] == -INFINITY ? 0.0f : m[i][y] - kPShift;
#pragma unroll
                        for (int n = 0; n < 2; ++n)
#pragma unroll
                            for (int j = 0; j < 2; ++j) {
                                const float pv = ex2_approx(s[i][2 * h + n][2 * y + j] - top);
                                l[i][y] += pv;
                                w[n][2 * y + j] = pv * ratio;
                            }
                    }
                    pa[i][0] = f16x2(w[0][0], w[0][1]);
                    pa[i][1] = f16x2(w[0][2], w[0][3]);
                    pa[i][2] = f16x2(w[1][0], w[1][1]);
                    pa[i][3] = f16x2(w[1][2], w[1][3]);
                }
#pragma unroll
                for (int c = 0; c < NC; c += 2) {
                    uint32_t vr[4];
                    ldsm4_t(vs_at + piece<D, KT>(16 * h + (lane & 15), c + (lane >> 4)), vr);
#pragma unroll
                    for (int z = 0; z < 2; ++z) {
                        uint32_t e0, e1, o0, o1;
                        e4m3_to_f16(__byte_perm(vr[2 * z], 0, 0x3120), e0, o0);
                        e4m3_to_f16(__byte_perm(vr[2 * z + 1], 0, 0x3120), e1, o1);
#pragma unroll
                        for (int i = 0; i < MT; ++i) {
                            mma_f16(o[i][c + z][0], pa[i][0], pa[i][1], pa[i][2], pa[i][3], e0, e1);
                            mma_f16(o[i][c + z][1], pa[i][0], pa[i][1], pa[i][2], pa[i][3], o0, o1);
                        }
                    }
                }
            }
            __syncwarp();
        }

        // The warps' states become the CTA's. Warp w holds tiles of this unit if one of
        // its turns fell into [t, tend); the slot it consumed last takes its accumulators.
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int y = 0; y < 2; ++y) {
                float v = l[i][y];
                v += __shfl_xor_sync(0xffffffffu, v, 1);
                v += __shfl_xor_sync(0xffffffffu, v, 2);
                if (qi == 0) ml[warp * S::rows + 16 * i + 8 * y + qr] = make_float2(m[i][y], v);
            }
        __syncthreads();
        const bool mine = k > 0 && t0 + warp + kWarps * (k - 1) >= t;
        float wgt[MT][2];
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int y = 0; y < 2; ++y) {
                float top = -INFINITY;
                for (int w = 0; w < kWarps; ++w)
                    top = fmaxf(top, ml[w * S::rows + 16 * i + 8 * y + qr].x);
                wgt[i][y] = m[i][y] == -INFINITY ? 0.0f : vref * ex2_approx(m[i][y] - top);
            }
        const bool whole = u0 >= t0 && u1 <= t1;
        const int part_at = (2 * static_cast<int>(blockIdx.x) + (u0 >= t0 ? 1 : 0)) * S::rows;
        if (!whole && u0 >= t0 && tid == 0) {
            p.desc[2 * blockIdx.x] = e * p.x_units + x;
            p.desc[2 * blockIdx.x + 1] = (u1 - 1) / per;
        }
        constexpr int kCols = S::slot / 64;  // columns of 16 rows that a slot holds in fp32
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int c0 = 0; c0 < D; c0 += kCols) {
                if (mine) {
                    const uint32_t buf = ring + ((k - 1) % ST) * S::slot;
#pragma unroll
                    for (int c = 0; c < kCols / 16; ++c) {
                        const float(&v)[2][4] = o[i][c0 / 16 + c];
#pragma unroll
                        for (int y = 0; y < 2; ++y) {
                            const uint32_t unit = 4 * c + qi;
                            const float w = wgt[i][y];
                            float4 f = make_float4(v[0][2 * y] * w, v[1][2 * y] * w,
                                                   v[0][2 * y + 1] * w, v[1][2 * y + 1] * w);
                            sts_v4(buf + (8 * y + qr) * kCols * 4 + ((unit ^ ((qr & 1) << 2)) << 4), f);
                        }
                    }
                    fence_proxy_async();
                }
                __syncthreads();
                if (i == 0 && c0 == 0 && tend < t1) {
                    // The next unit's queries: every warp is past its tiles of this one.
                    int en = e;
                    while (prefix[en + 1] <= tend) ++en;
                    const int ntn = (prefix[en + 1] - prefix[en]) / p.x_units;
                    load_q(en, (tend - prefix[en]) / ntn);
                }
                for (int idx = tid; idx < 16 * (kCols / 4); idx += kThreads) {
                    const int row = idx / (kCols / 4), unit = idx % (kCols / 4), mm = 16 * i + row;
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
                            lds_f4(base + (w * ST + last % ST) * S::slot + row * kCols * 4 +
                                   ((unit ^ ((row & 1) << 2)) << 4));
                        acc.x += f.x;
                        acc.y += f.y;
                        acc.z += f.z;
                        acc.w += f.w;
                    }
                    const int col = c0 + 4 * unit;
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

template <int D, int MT, int KT, int ST>
int launch_decode(PagedParams p, const CUtensorMap& kmap, const CUtensorMap& vmap, int sms,
                  int64_t tiles, smd_stream_t stream) {
    using S = Shape<D, MT, KT, ST>;
    constexpr int kResident = (D == 256 || (D == 128 && MT == 2)) ? 2 : 3;
    static_assert(kResident * (S::smem(kMaxEntries) + 1024) <= 228 * 1024, "CTAs of an SM");
    static std::atomic<bool> ready[kMaxDevices];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return SMD_ERR_DEVICE;
    auto kernel = paged_decode_kernel<D, MT, KT, ST>;
    if (!ready[dev]) {
        if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 S::smem(kMaxEntries)) != cudaSuccess) {
            (void)cudaGetLastError();
            return SMD_ERR_DEVICE;
        }
        ready[dev] = true;
    }
    // At least kWarps tiles a CTA, so that each warp has one.
    const int64_t most = static_cast<int64_t>(sms) * kResident, want = (tiles + kWarps - 1) / kWarps;
    const int grid = static_cast<int>(want < most ? want : most);
    p.part = reinterpret_cast<float*>(p.desc) + 4 * most;  // 16-byte aligned
    p.part_ml = p.part + most * 2 * S::rows * D;
    int rc = launch_pdl(kernel, dim3(grid), kThreads, S::smem(p.entries), stream, p, kmap, vmap);
    if (rc != SMD_OK) return rc;
    const int join_rows = p.rows < S::rows ? p.rows : S::rows;
    return launch_pdl(paged_join_kernel<D>, dim3(grid, (join_rows + kJoinRows - 1) / kJoinRows),
                      2 * kJoinRows * 32, 0, stream, p, static_cast<int>(S::rows));
}

// Workspace of the widest instantiation at D columns: a CTA's descriptor and two
// partials of its rows.
int64_t workspace_bytes(int sms, int D) {
    const int64_t three = 3 * 16, two = 2 * 32;
    const int64_t rows = sms * (D == 64 ? 3 * 32 : D == 128 ? (three > two ? three : two) : 2 * 16);
    return 4 * (4 * 3 * static_cast<int64_t>(sms) + 2 * rows * (D + 2));
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
    const int MT = D == 256 || rows <= 16 ? 1 : 2, KT = D == 256 ? 16 : 32;
    PagedParams p{};
    p.q_stride = q_stride;
    p.table_stride = table_stride;
    p.width = width;
    p.k_scale = cache->k_scale;
    p.v_scale = cache->v_scale;
    p.pages = cache->pages;
    p.heads = cache->heads;
    p.page_size = P;
    p.row_tiles = (rows + 16 * MT - 1) / (16 * MT);
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
        if (D == 64)
            rc = MT == 1 ? launch_decode<64, 1, 32, 4>(p, maps[0], maps[1], sms, tiles, stream)
                         : launch_decode<64, 2, 32, 3>(p, maps[0], maps[1], sms, tiles, stream);
        else if (D == 128)
            rc = MT == 1 ? launch_decode<128, 1, 32, 2>(p, maps[0], maps[1], sms, tiles, stream)
                         : launch_decode<128, 2, 32, 3>(p, maps[0], maps[1], sms, tiles, stream);
        else
            rc = launch_decode<256, 1, 16, 3>(p, maps[0], maps[1], sms, tiles, stream);
        if (rc != SMD_OK) return rc;
    }
    return SMD_OK;
}

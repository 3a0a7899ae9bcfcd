// The score of each page of a paged cache for a query (smd_block_scores).
//
// With hi, lo the channelwise bounds of a page's keys, every key k of it has
//   q . k <= sum_c max(q_c hi_c, q_c lo_c) = q+ . hi + q- . lo,
// q+ = max(q, 0), q- = min(q, 0): a product of 2 D columns, for which
// mma.sync m16n8k16 takes bf16 operands as they are (exact products, fp32
// sums). The page's score is the largest over the query heads of the kv head,
// so a page stays if any of them may need it; one bf16 rounding at the end.
//
// What bounds it: 4 D bytes of bounds for each (page, head), read once, 4 D M
// FLOPs with them: HBM. So nothing is staged: a warp takes 16 pages (the rows of
// the MMA), a lane reads 16-byte pieces of two pages' bounds straight into the
// operand registers. The contraction index is permuted to allow it: lane
// 4 g + i holds columns 32 j + 8 i .. + 7 of pages g and g + 8, and the query
// fragments q+ and q-, in shared memory in the order of the lanes, are made to
// match. The query rows pass over these registers 8 at a time.
//
// Measured (GB300): 48 requests of 8192 .. 131072 tokens in pages of 64, 8 heads of
// 128 columns: 33 us for 8 query rows a head (89% of the copy rate for the 201
// MB), 37 us for 16 rows, 76 us for 64 rows, where each 8 more rows cost 6 us: 3 of
// MMAs, 3 of reads of the query fragments from shared memory.
#include "smd_internal.h"
#include "smd_paged.h"
#include "smd_ptx.cuh"

namespace smd {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr int kGroup = 16 * kWarps;  // pages that a block's warps take at once
// Such turns of a block: the waits for length, page and query are paid once a block. The
// 201 MB above take 34.3 us at two turns, 33.4 at four, 35.4 at eight (too few blocks).
constexpr int kMostSteps = 4;

struct ScoreParams {
    const uint16_t* q;
    int64_t q_stride;
    const uint16_t* bounds;
    const int32_t* table;
    int64_t table_stride;
    int32_t width;
    const int32_t* lengths;
    int32_t pages, heads, P, G, g, r0;
    int32_t i0, i_end;  // verify rows of this launch
    int32_t keep_first, keep_last;
    uint16_t* scores;
    int64_t score_stride;
    int32_t cols, cols_log2;  // columns of the MMA that one verify row takes: a power of two up to 8
    int32_t parts;      // MMAs that one verify row takes (more than 8 query heads)
    int32_t tiles;      // MMAs over all rows
    int32_t steps;      // turns of a block
};

__device__ __forceinline__ void mma_bf16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 "
        "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t pos2(uint32_t v) {
    uint32_t r;
    asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(v), "r"(0u));
    return r;
}

__device__ __forceinline__ uint32_t neg2(uint32_t v) {
    uint32_t r;
    asm("min.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(v), "r"(0u));
    return r;
}

template <int D>
__global__ void __launch_bounds__(kThreads) block_scores_kernel(const ScoreParams p) {
    constexpr int kJ = D / 32;  // 16-byte pieces of a lane, per bound and page
    extern __shared__ __align__(16) uint8_t smem[];
    // [tiles][kJ][sign][32 lanes]: the second operand's registers of two MMAs
    uint4* const qs = reinterpret_cast<uint4*>(smem);
    __shared__ int s_sees[kPagedMaxGroup];  // pages that a verify row sees
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, gr = lane >> 2, gi = lane & 3;
    const int head = blockIdx.y, r = blockIdx.z + p.r0;
    const int block0 = blockIdx.x * kGroup * p.steps, block1 = block0 + kGroup * p.steps;
    pdl_entry();
    const int len = max(min(p.lengths[r], p.width * p.P), 0);
    const int have = pages_of(len, p.P);  // pages that the last verify row sees
    const int64_t b0 = static_cast<int64_t>(r) * p.G;

    // Pages that no row sees: NaN.
    for (int i = p.i0; i < p.i_end; ++i) {
        uint16_t* const row = p.scores + ((b0 + i) * p.heads + head) * p.score_stride;
        for (int c = max(have, block0) + tid; c < min(block1, p.width); c += kThreads)
            row[c] = 0x7fffu;
    }
    if (block0 >= have) return;
    uint16_t* const scores = p.scores + (b0 * p.heads + head) * p.score_stride;
    const int64_t row_step = p.heads * p.score_stride;

    // The pages of a turn, one turn ahead of the bounds; those are on their way while the
    // products of the turn before (at first, while the queries) are dealt with.
    int page[2];
    const auto look_up = [&](int c0) {
#pragma unroll
        for (int z = 0; z < 2; ++z) {
            const int c = c0 + 8 * z + gr;
            page[z] = c < min(have, block1) ? p.table[r * p.table_stride + c] : -1;
        }
    };
    uint4 hi[2][kJ], lo[2][kJ];
    const auto load = [&]() {
#pragma unroll
        for (int z = 0; z < 2; ++z) {
            const int pg = page[z];
#pragma unroll
            for (int j = 0; j < kJ; ++j) hi[z][j] = lo[z][j] = make_uint4(0, 0, 0, 0);
            if (pg >= 0 && pg < p.pages) {
                const uint4* const b = reinterpret_cast<const uint4*>(
                    p.bounds + (static_cast<int64_t>(pg) * p.heads + head) * 2 * D + 8 * gi);
#pragma unroll
                for (int j = 0; j < kJ; ++j) {
                    hi[z][j] = __ldcs(b + 4 * j);
                    lo[z][j] = __ldcs(b + D / 8 + 4 * j);
                }
            }
        }
    };
    look_up(block0 + 16 * warp);
    load();
    look_up(block0 + 16 * warp + kGroup);
    if (tid < p.i_end - p.i0)
        s_sees[tid] = pages_of(max(len - p.G + 1 + p.i0 + tid, 0), p.P);
    for (int idx = tid; idx < p.tiles * kJ * 32; idx += kThreads) {
        // Column l / 4 of a tile, the pieces of lane l. Columns beyond the heads repeat the
        // last one, which leaves the maximum as it is.
        const int l = idx & 31, j = (idx >> 5) % kJ, tile = (idx >> 5) / kJ;
        int i, a;
        if (p.parts > 1) {
            i = tile / p.parts;
            a = (tile % p.parts) * 8 + (l >> 2);
        } else {
            i = (tile * 8 + (l >> 2)) >> p.cols_log2;
            a = (l >> 2) & (p.cols - 1);
        }
        i = min(p.i0 + i, p.i_end - 1);
        a = min(a, p.g - 1);
        const uint4 v = *reinterpret_cast<const uint4*>(
            p.q + (b0 + i) * p.q_stride + static_cast<int64_t>(head * p.g + a) * D + 32 * j + 8 * (l & 3));
        uint4* const to = qs + static_cast<int64_t>(tile * kJ + j) * 64 + l;
        to[0] = make_uint4(pos2(v.x), pos2(v.y), pos2(v.z), pos2(v.w));
        to[32] = make_uint4(neg2(v.x), neg2(v.y), neg2(v.z), neg2(v.w));
    }
    __syncthreads();

#pragma unroll 1
    for (int c0 = block0 + 16 * warp; c0 < min(have, block1); c0 += kGroup) {
        float run[2] = {0.0f, 0.0f};
#pragma unroll 1
        for (int tile = 0; tile < p.tiles; ++tile) {
            __syncwarp();  // some lanes wrote the scores of the tile before; the MMAs are the warp's
            // page g: columns 2 i, 2 i + 1; page g + 8. Four sums, so that the MMAs do not wait
            // for one another.
            float d[4] = {}, d1[4] = {}, d2[4] = {}, d3[4] = {};
            const uint4* const q = qs + static_cast<int64_t>(tile) * kJ * 64 + lane;
#pragma unroll
            for (int j = 0; j < kJ; ++j) {
                const uint4 a = q[j * 64], b = q[j * 64 + 32];
                mma_bf16(d, hi[0][j].x, hi[1][j].x, hi[0][j].y, hi[1][j].y, a.x, a.y);
                mma_bf16(d1, hi[0][j].z, hi[1][j].z, hi[0][j].w, hi[1][j].w, a.z, a.w);
                mma_bf16(d2, lo[0][j].x, lo[1][j].x, lo[0][j].y, lo[1][j].y, b.x, b.y);
                mma_bf16(d3, lo[0][j].z, lo[1][j].z, lo[0][j].w, lo[1][j].w, b.z, b.w);
            }
#pragma unroll
            for (int z = 0; z < 4; ++z) d[z] = (d[z] + d1[z]) + (d2[z] + d3[z]);
            // The largest over a verify row's columns.
            if (p.cols >= 2) {
                d[0] = fmaxf(d[0], d[1]);
                d[2] = fmaxf(d[2], d[3]);
            }
            if (p.cols >= 4) {
                d[0] = fmaxf(d[0], __shfl_xor_sync(0xffffffffu, d[0], 1));
                d[2] = fmaxf(d[2], __shfl_xor_sync(0xffffffffu, d[2], 1));
            }
            if (p.cols >= 8) {
                d[0] = fmaxf(d[0], __shfl_xor_sync(0xffffffffu, d[0], 2));
                d[2] = fmaxf(d[2], __shfl_xor_sync(0xffffffffu, d[2], 2));
            }
            int i = (tile * 8 + 2 * gi) >> p.cols_log2;
            if (p.parts > 1) {
                i = tile / p.parts;
                const int part = tile - i * p.parts;
                run[0] = part == 0 ? d[0] : fmaxf(run[0], d[0]);
                run[1] = part == 0 ? d[2] : fmaxf(run[1], d[2]);
                if (part + 1 < p.parts) continue;
                d[0] = run[0];
                d[2] = run[1];
            }
            if ((2 * gi & (p.cols - 1)) != 0) continue;
            for (int y = 0; y < (p.cols == 1 ? 2 : 1); ++y, ++i) {
                if (p.i0 + i >= p.i_end) break;
                const int sees = s_sees[i];
                uint16_t* const out = scores + (p.i0 + i) * row_step;
#pragma unroll
                for (int z = 0; z < 2; ++z) {
                    const int c = c0 + 8 * z + gr;
                    uint16_t v = static_cast<uint16_t>(bf16x2(y == 0 ? d[2 * z] : d[2 * z + 1], 0.0f));
                    if (c < p.keep_first || c >= sees - p.keep_last) v = 0x7f80u;
                    if (c >= sees) v = 0x7fffu;
                    if (c < have) out[c] = v;
                }
            }
        }
        load();
        look_up(c0 + 2 * kGroup);
    }
}

template <int D>
int launch_scores(ScoreParams p, int R, int sms, smd_stream_t stream) {
    constexpr int kTile = 32 * D, kMost = 176 * 1024;  // shared bytes of an MMA's columns
    static_assert(kMost / kTile >= kPagedMaxHeads / 8, "a verify row's query heads fit");
    static SharedLimit limit;
    int rc = limit.raise(block_scores_kernel<D>, kMost);
    if (rc != SMD_OK) return rc;
    // Turns of a block: few where there are few pages, so that the blocks still fill the device.
    const int64_t groups = (static_cast<int64_t>(p.width) + kGroup - 1) / kGroup;
    p.steps = kMostSteps;
    while (p.steps > 1 && groups / p.steps * p.heads * R < 8ll * sms) p.steps /= 2;
    const unsigned gx = static_cast<unsigned>((groups + p.steps - 1) / p.steps);
    // Verify rows of one launch: all of them, unless many query heads fill the shared memory.
    const int rows = p.tiles * kTile <= kMost ? p.G : kMost / kTile / p.parts;
    for (p.i0 = 0; p.i0 < p.G; p.i0 += rows) {
        p.i_end = p.i0 + rows < p.G ? p.i0 + rows : p.G;
        const int n = p.i_end - p.i0;
        p.tiles = p.parts > 1 ? n * p.parts : (n * p.cols + 7) / 8;
        for (p.r0 = 0; p.r0 < R; p.r0 += 65535) {
            const int z = R - p.r0 < 65535 ? R - p.r0 : 65535;
            rc = launch_pdl(
                block_scores_kernel<D>, dim3(gx, static_cast<unsigned>(p.heads), static_cast<unsigned>(z)),
                kThreads, static_cast<size_t>(p.tiles) * kTile, stream, p);
            if (rc != SMD_OK) return rc;
        }
    }
    return SMD_OK;
}

}  // namespace
}  // namespace smd

extern "C" int smd_block_scores(const uint16_t* q, int64_t q_stride, const smd_paged_cache_t* cache,
                                const int32_t* table, int64_t table_stride, int32_t width,
                                const int32_t* lengths, int32_t R, int32_t row_group, int32_t Hq,
                                int32_t keep_first, int32_t keep_last, uint16_t* scores,
                                int64_t score_stride, smd_stream_t stream) {
    using namespace smd;
    if (cache == nullptr) return SMD_ERR_NULL;
    bool skip;
    int rc = check_paged_rows(q, q_stride, shape_of(cache), table, table_stride, width, lengths, R, row_group,
                              Hq, &skip);
    if (rc != SMD_OK) return rc;
    if (cache->bounds == nullptr) return SMD_ERR_NULL;
    if (keep_first < 0 || keep_last < 0 || score_stride < width) return SMD_ERR_SHAPE;
    if (skip) return SMD_OK;
    if (scores == nullptr) return SMD_ERR_NULL;
    if (!aligned(scores, 2)) return SMD_ERR_ALIGN;
    const int sms = device_sms();
    if (sms <= 0) return SMD_ERR_DEVICE;
    ScoreParams p{};
    p.q = q;
    p.q_stride = q_stride;
    p.bounds = cache->bounds;
    p.table = table;
    p.table_stride = table_stride;
    p.width = width;
    p.lengths = lengths;
    p.pages = cache->pages;
    p.heads = cache->heads;
    p.P = cache->page_size;
    p.G = row_group;
    p.g = Hq / cache->heads;
    p.keep_first = keep_first;
    p.keep_last = keep_last;
    p.scores = scores;
    p.score_stride = score_stride;
    p.cols = 1;
    while (p.cols < p.g && p.cols < 8) p.cols *= 2, ++p.cols_log2;
    p.parts = (p.g + 7) / 8;
    p.tiles = p.parts > 1 ? p.G * p.parts : (p.G * p.cols + 7) / 8;
    return cache->head_dim == 64    ? launch_scores<64>(p, R, sms, stream)
           : cache->head_dim == 128 ? launch_scores<128>(p, R, sms, stream)
                                    : launch_scores<256>(p, R, sms, stream);
}

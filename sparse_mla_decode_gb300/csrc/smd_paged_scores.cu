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
// FLOPs with them: HBM. So nothing is staged: a warp takes 8 pages (the columns
// of the MMA), a lane reads 16-byte pieces of one page's bounds straight into
// the operand registers. The contraction index is permuted to allow it: lane
// 4 g + i holds columns 32 j + 8 i .. + 7 of page g, and the query fragments,
// in shared memory, are read in the same order. The M query rows pass over
// these registers 16 at a time.
#include "smd_internal.h"
#include "smd_paged.h"
#include "smd_ptx.cuh"

namespace smd {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr int kSteps = 4;                          // groups of 8 pages of a warp
constexpr int kPagesPerBlock = 8 * kWarps * kSteps;

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
    int32_t lanes;      // rows of the MMA that one verify row takes: a power of two up to 16
    int32_t parts;      // MMAs that one verify row takes (more than 16 query heads)
    int32_t m_tiles;    // MMAs over all rows
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

// Query row of MMA row `s` of tile mt: verify row i and head j of the group.
// Rows beyond the heads repeat the last one, which leaves the maximum as it is.
__device__ __forceinline__ void row_of(const ScoreParams& p, int mt, int s, int& i, int& j) {
    if (p.parts > 1) {
        i = p.i0 + mt / p.parts;
        j = (mt % p.parts) * 16 + s;
    } else {
        i = p.i0 + mt * (16 / p.lanes) + s / p.lanes;
        j = s % p.lanes;
    }
    i = min(i, p.i_end - 1);
    j = min(j, p.g - 1);
}

template <int D>
__global__ void __launch_bounds__(kThreads) block_scores_kernel(const ScoreParams p) {
    constexpr int kPitch = 2 * D + 64;  // 16-byte reads of two rows hit different banks
    constexpr int kJ = D / 32;          // 16-byte pieces of a lane, per bound
    extern __shared__ __align__(16) uint8_t smem[];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, gr = lane >> 2, gi = lane & 3;
    const int head = blockIdx.y, r = blockIdx.z + p.r0;
    const int first = blockIdx.x * kPagesPerBlock + warp * 8 * kSteps;
    pdl_entry();
    const int len = max(min(p.lengths[r], p.width * p.P), 0);
    const int have = (len + p.P - 1) / p.P;  // pages that the last verify row sees
    const int64_t b0 = static_cast<int64_t>(r) * p.G;

    // Pages that no row sees: NaN.
    for (int i = p.i0; i < p.i_end; ++i) {
        uint16_t* const row = p.scores + ((b0 + i) * p.heads + head) * p.score_stride;
        for (int c = max(have, static_cast<int>(blockIdx.x) * kPagesPerBlock) + tid;
             c < min(static_cast<int>(blockIdx.x + 1) * kPagesPerBlock, p.width); c += kThreads)
            row[c] = 0x7fffu;
    }
    if (static_cast<int>(blockIdx.x) * kPagesPerBlock >= have) return;

    int page[kSteps];
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
        const int c = first + 8 * s + gr;
        page[s] = c < have ? p.table[r * p.table_stride + c] : -1;
    }
    for (int idx = tid; idx < p.m_tiles * 16 * (D / 8); idx += kThreads) {
        const int row = idx / (D / 8), c = idx % (D / 8);
        int i, j;
        row_of(p, row >> 4, row & 15, i, j);
        *reinterpret_cast<uint4*>(smem + row * kPitch + 16 * c) = *reinterpret_cast<const uint4*>(
            p.q + (b0 + i) * p.q_stride + static_cast<int64_t>(head * p.g + j) * D + 8 * c);
    }
    __syncthreads();

#pragma unroll 1
    for (int s = 0; s < kSteps; ++s) {
        const int c0 = first + 8 * s;
        if (c0 >= have) break;
        uint4 hi[kJ], lo[kJ];
        const int pg = page[s];
        if (pg >= 0 && pg < p.pages) {
            const uint4* const b = reinterpret_cast<const uint4*>(
                p.bounds + (static_cast<int64_t>(pg) * p.heads + head) * 2 * D + 8 * gi);
#pragma unroll
            for (int j = 0; j < kJ; ++j) {
                hi[j] = __ldcs(b + 4 * j);
                lo[j] = __ldcs(b + D / 8 + 4 * j);
            }
        } else {
#pragma unroll
            for (int j = 0; j < kJ; ++j) hi[j] = lo[j] = make_uint4(0, 0, 0, 0);
        }
        float run[4];
#pragma unroll 1
        for (int mt = 0; mt < p.m_tiles; ++mt) {
            float d[4] = {0.0f, 0.0f, 0.0f, 0.0f};
            const uint8_t* const q0 = smem + (mt * 16 + gr) * kPitch + 16 * gi;
#pragma unroll
            for (int j = 0; j < kJ; ++j) {
                const uint4 x = *reinterpret_cast<const uint4*>(q0 + 64 * j);
                const uint4 y = *reinterpret_cast<const uint4*>(q0 + 8 * kPitch + 64 * j);
                mma_bf16(d, pos2(x.x), pos2(y.x), pos2(x.y), pos2(y.y), hi[j].x, hi[j].y);
                mma_bf16(d, neg2(x.x), neg2(y.x), neg2(x.y), neg2(y.y), lo[j].x, lo[j].y);
                mma_bf16(d, pos2(x.z), pos2(y.z), pos2(x.w), pos2(y.w), hi[j].z, hi[j].w);
                mma_bf16(d, neg2(x.z), neg2(y.z), neg2(x.w), neg2(y.w), lo[j].z, lo[j].w);
            }
            // The largest over a verify row's MMA rows: lanes of equal gi, and for
            // 16 of them both halves.
#pragma unroll
            for (int o = 4; o < 32; o <<= 1) {
                if (o >= 4 * p.lanes) break;
#pragma unroll
                for (int z = 0; z < 4; ++z) d[z] = fmaxf(d[z], __shfl_xor_sync(0xffffffffu, d[z], o));
            }
            if (p.lanes == 16) {
                d[0] = d[2] = fmaxf(d[0], d[2]);
                d[1] = d[3] = fmaxf(d[1], d[3]);
            }
            if (p.parts > 1) {
                const int part = mt % p.parts;
#pragma unroll
                for (int z = 0; z < 4; ++z) run[z] = part == 0 ? d[z] : fmaxf(run[z], d[z]);
                if (part + 1 < p.parts) continue;
#pragma unroll
                for (int z = 0; z < 4; ++z) d[z] = run[z];
            }
#pragma unroll
            for (int y = 0; y < 2; ++y) {
                if (y == 1 && p.lanes == 16) break;
                const int row = 8 * y + gr;
                const int i =
                    p.i0 + (p.parts > 1 ? mt / p.parts : mt * (16 / p.lanes) + row / p.lanes);
                if (row % p.lanes != 0 || i >= p.i_end) continue;
                const int sees = (max(len - p.G + 1 + i, 0) + p.P - 1) / p.P;
                uint16_t* const out =
                    p.scores + ((b0 + i) * p.heads + head) * p.score_stride + c0 + 2 * gi;
#pragma unroll
                for (int z = 0; z < 2; ++z) {
                    const int c = c0 + 2 * gi + z;
                    if (c >= have) continue;
                    uint16_t v = static_cast<uint16_t>(bf16x2(d[2 * y + z], 0.0f) & 0xffffu);
                    if (c < p.keep_first || c >= sees - p.keep_last) v = 0x7f80u;
                    if (c >= sees) v = 0x7fffu;
                    out[z] = v;
                }
            }
        }
    }
}

template <int D>
int launch_scores(ScoreParams p, int R, smd_stream_t stream) {
    constexpr int kTile = 16 * (2 * D + 64), kMost = 176 * 1024;  // shared bytes of an MMA's rows
    static_assert(kMost / kTile >= kPagedMaxHeads / 16, "a verify row's query heads fit");
    if (p.m_tiles * kTile > 48 * 1024 &&
        cudaFuncSetAttribute(block_scores_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             kMost) != cudaSuccess) {
        (void)cudaGetLastError();
        return SMD_ERR_DEVICE;
    }
    const unsigned gx = static_cast<unsigned>((p.width + kPagesPerBlock - 1) / kPagesPerBlock);
    // Verify rows of one launch: all of them, unless many query heads fill the shared memory.
    const int rows = p.m_tiles * kTile <= kMost ? p.G : kMost / kTile / p.parts;
    for (p.i0 = 0; p.i0 < p.G; p.i0 += rows) {
        p.i_end = p.i0 + rows < p.G ? p.i0 + rows : p.G;
        const int n = p.i_end - p.i0;
        p.m_tiles = p.parts > 1 ? n * p.parts : (n * p.lanes + 15) / 16;
        for (p.r0 = 0; p.r0 < R; p.r0 += 65535) {
            const int z = R - p.r0 < 65535 ? R - p.r0 : 65535;
            const int rc = launch_pdl(
                block_scores_kernel<D>, dim3(gx, static_cast<unsigned>(p.heads), static_cast<unsigned>(z)),
                kThreads, static_cast<size_t>(p.m_tiles) * kTile, stream, p);
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
    bool skip;
    int rc = check_paged_rows(q, q_stride, cache, table, table_stride, width, lengths, R, row_group,
                              Hq, &skip);
    if (rc != SMD_OK) return rc;
    if (cache->bounds == nullptr) return SMD_ERR_NULL;
    if (keep_first < 0 || keep_last < 0 || score_stride < width) return SMD_ERR_SHAPE;
    if (skip) return SMD_OK;
    if (scores == nullptr) return SMD_ERR_NULL;
    if (!aligned(scores, 2)) return SMD_ERR_ALIGN;
    if (device_sms() <= 0) return SMD_ERR_DEVICE;
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
    p.lanes = 1;
    while (p.lanes < p.g && p.lanes < 16) p.lanes *= 2;
    p.parts = (p.g + 15) / 16;
    p.m_tiles = p.parts > 1 ? p.G * p.parts : (p.G * p.lanes + 15) / 16;
    return cache->head_dim == 64    ? launch_scores<64>(p, R, stream)
           : cache->head_dim == 128 ? launch_scores<128>(p, R, stream)
                                    : launch_scores<256>(p, R, stream);
}

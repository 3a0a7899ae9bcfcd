// Attention over a paged E2M1 cache (smd_paged4_decode). 128 columns: smd_paged4_tc.cu; 64 and 256:
// the kernel in smd_paged_decode.cuh, with mma.sync.
//
// Measured of the latter (GB300, device time; of the rate at which the GPU copies), 64 requests of
// 1024 .. 8192 tokens, 8 / 16 / 32 query rows:
//    64 columns    55 us 47% / 70 us 37% / 104 us 25%
//   256 columns   156 us 66% / 207 us 50% / 373 us 28% (16 rows at a time: the cache is read twice)
// 5 requests up to 777 tokens, 12 rows of 64 columns, pages of 16: 12.5 us, start and joins.
// What bounds it: conversions. A tile of 32 tokens takes 720 instructions at 8 rows of 128 columns, 64
// conversions and 64 multiplications for K and as many for V among them; the logic pipe, which converts,
// is busy two thirds of the time that is not start or joins. More warps change nothing.
#include <cstring>

#include "smd_paged4_tc.h"
#include "smd_paged_decode.cuh"

extern "C" int64_t smd_paged4_workspace_bytes(const smd_paged4_cache_t* cache) {
    if (cache == nullptr) return SMD_ERR_NULL;
    if (!smd::paged_ready(cache)) return SMD_ERR_PLAN;
    const int sms = smd::device_sms();
    if (sms <= 0) return SMD_ERR_DEVICE;
    return smd::workspace_bytes(sms, cache->head_dim);
}

extern "C" int smd_paged4_decode(const uint16_t* q, int64_t q_stride, const smd_paged4_cache_t* cache,
                                 const int32_t* table, int64_t table_stride, int32_t width,
                                 const int32_t* lengths, int32_t R, int32_t row_group, int32_t Hq,
                                 float sm_scale, const int32_t* block_lists,
                                 const int32_t* block_counts, int32_t K, uint16_t* out, float* lse,
                                 int32_t* status, void* workspace, int64_t workspace_bytes,
                                 smd_stream_t stream) {
    return smd_paged4_decode_ex(q, q_stride, cache, table, table_stride, width, lengths, R, row_group, Hq,
                                sm_scale, block_lists, block_counts, K, out, lse, status, workspace,
                                workspace_bytes, stream, nullptr);
}

extern "C" int smd_paged4_decode_ex(const uint16_t* q, int64_t q_stride,
                                    const smd_paged4_cache_t* cache, const int32_t* table,
                                    int64_t table_stride, int32_t width, const int32_t* lengths,
                                    int32_t R, int32_t row_group, int32_t Hq, float sm_scale,
                                    const int32_t* block_lists, const int32_t* block_counts,
                                    int32_t K, uint16_t* out, float* lse, int32_t* status,
                                    void* workspace, int64_t workspace_bytes, smd_stream_t stream,
                                    const smd_plan_t* force) {
    using namespace smd;
    if (cache == nullptr) return SMD_ERR_NULL;
    PagedParams p{};
    p.k_exp = cache->k_exp;
    p.v_exp = cache->v_exp;
    Maps<4> maps;
    std::memcpy(&maps, &cache->map[1], sizeof maps);
    const int D = cache->head_dim;
    const DecodeCall call{q, q_stride, table, table_stride, width, lengths, R, row_group, Hq, sm_scale,
                          block_lists, block_counts, K, out, lse, status, workspace, workspace_bytes,
                          stream, force};
    return run_decode(call, shape_of(cache), p, [&](const PagedParams& p, int64_t tiles, int RT, int sms) {
        // 128 columns: tcgen05. mma.sync (smd_paged_decode.cuh), measured in its place with 64 requests of
        // 1024 .. 8192 tokens, tcgen05 / mma.sync in us: pages of 64 tokens, 8 / 16 / 32 query rows 73 / 84,
        // 82 / 111, 115 / 167; pages of 16 89 / 92, 94 / 119, 123 / 179; one request of 777 tokens 12.6 / 11.3.
        if (D == 128)
            return paged4_tc(p, maps, tc_box_tokens(cache->page_size), 8 * RT, sms, (tiles + 3) / 4, stream);
        const bool halves = page_box_tokens(cache->page_size, D) < (D == 256 ? 16 : 32);  // a tile spans two pages
        const auto launch = [&](auto shape) {
            return launch_decode<decltype(shape)>(p, maps, sms, tiles, stream);
        };
        if (D == 64)
            return halves    ? (RT == 1   ? launch(Shape<64, 1, 32, 2, 3, 3, 4>{})
                              : RT == 2 ? launch(Shape<64, 2, 32, 2, 3, 3, 4>{})
                                        : launch(Shape<64, 4, 32, 2, 4, 2, 4>{}))
                 : RT == 1 ? launch(Shape<64, 1, 32, 1, 3, 3, 4>{})
                 : RT == 2 ? launch(Shape<64, 2, 32, 1, 3, 3, 4>{})
                           : launch(Shape<64, 4, 32, 1, 4, 2, 4>{});
        return RT == 1 ? launch(Shape<256, 1, 16, 1, 3, 3, 4>{}) : launch(Shape<256, 2, 16, 1, 3, 2, 4>{});
    });
}

// Attention over a paged E4M3 cache (smd_paged_decode); the kernel is in
// smd_paged_decode.cuh.
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

#include "smd_paged_decode.cuh"

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
    if (cache == nullptr) return SMD_ERR_NULL;
    PagedParams p{};
    p.k_scale = cache->k_scale;
    p.v_scale = cache->v_scale;
    Maps<8> maps;
    std::memcpy(&maps, &cache->map[1], sizeof maps);
    const int D = cache->head_dim;
    const DecodeCall call{q, q_stride, table, table_stride, width, lengths, R, row_group, Hq, sm_scale,
                          block_lists, block_counts, K, out, lse, status, workspace, workspace_bytes,
                          stream, force};
    return run_decode(call, shape_of(cache), p, [&](const PagedParams& p, int64_t tiles, int RT, int sms) {
        const bool halves = page_box_tokens(cache->page_size, D) < (D == 256 ? 16 : 32);  // a tile spans two pages
        const auto launch = [&](auto shape) {
            return launch_decode<decltype(shape)>(p, maps, sms, tiles, stream);
        };
        if (D == 64)
            return halves    ? (RT == 1   ? launch(Shape<64, 1, 32, 2, 4, 3>{})
                              : RT == 2 ? launch(Shape<64, 2, 32, 2, 4, 3>{})
                                        : launch(Shape<64, 4, 32, 2, 4, 2>{}))
                 : RT == 1 ? launch(Shape<64, 1, 32, 1, 4, 3>{})
                 : RT == 2 ? launch(Shape<64, 2, 32, 1, 4, 3>{})
                           : launch(Shape<64, 4, 32, 1, 4, 2>{});
        if (D == 128)
            return halves    ? (RT == 1   ? launch(Shape<128, 1, 32, 2, 2, 3>{})
                              : RT == 2 ? launch(Shape<128, 2, 32, 2, 2, 3>{})
                                        : launch(Shape<128, 4, 32, 2, 2, 2>{}))
                 : RT == 1 ? launch(Shape<128, 1, 32, 1, 2, 3>{})
                 : RT == 2 ? launch(Shape<128, 2, 32, 1, 2, 3>{})
                           : launch(Shape<128, 4, 32, 1, 2, 2>{});
        return RT == 1 ? launch(Shape<256, 1, 16, 1, 2, 3>{}) : launch(Shape<256, 2, 16, 1, 2, 2>{});
    });
}

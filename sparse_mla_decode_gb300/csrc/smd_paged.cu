// The descriptions of paged caches (smd_paged_cache_init, smd_paged4_cache_init) and the
// checks that the calls on them share. Host code only.
#include <cstring>

#include "smd_internal.h"
#include "smd_paged.h"

namespace smd {

namespace {

bool strides_ok(const int64_t (&s)[3], int row_bytes) {
    for (int i = 0; i < 3; ++i)
        if (s[i] <= 0 || s[i] >= (1ll << 40)) return false;
    return s[2] >= row_bytes;
}

bool shape_ok(int pages, int heads, int page_size, int head_dim) {
    return pages >= 1 && heads >= 1 && heads <= 65535 && page_size >= 16 && page_size <= 256 &&
           page_size % 16 == 0 && (head_dim == 64 || head_dim == 128 || head_dim == 256) &&
           static_cast<int64_t>(pages) * page_size < (1ll << 31);
}

bool steps_of_16(const int64_t (&s)[3]) { return s[0] % 16 == 0 && s[1] % 16 == 0 && s[2] % 16 == 0; }

// cuTensorMapEncodeTiled, looked up through the runtime (the library does not
// link the driver library, so it loads on machines without one).
using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                   const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                   const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                   CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn() {
    static EncodeTiledFn fn = [] {
        void* f = nullptr;
        cudaDriverEntryPointQueryResult q{};
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault,
                                             &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess) {
            (void)cudaGetLastError();
            f = nullptr;
        }
        return reinterpret_cast<EncodeTiledFn>(f);
    }();
    return fn;
}

// The tensor map of codes over (byte of a token, token, head, page), with a box of up to 128
// bytes by `tokens`, swizzled over its row. False if encoding failed.
bool encode_codes(CUtensorMap* out, const void* ptr, const int64_t (&stride)[3], int row_bytes, int tokens,
                  const CacheShape& c) {
    EncodeTiledFn encode = encode_fn();
    if (encode == nullptr) return false;
    const cuuint64_t dims[4] = {
        static_cast<cuuint64_t>(row_bytes), static_cast<cuuint64_t>(c.page_size),
        static_cast<cuuint64_t>(c.heads), static_cast<cuuint64_t>(c.pages)};
    const cuuint64_t strides[3] = {static_cast<cuuint64_t>(stride[2]),
                                   static_cast<cuuint64_t>(stride[1]),
                                   static_cast<cuuint64_t>(stride[0])};
    const cuuint32_t box[4] = {static_cast<cuuint32_t>(row_bytes < 128 ? row_bytes : 128),
                               static_cast<cuuint32_t>(tokens), 1, 1};
    const cuuint32_t estr[4] = {1, 1, 1, 1};
    // L2 fetches no more than a row where rows of 64 bytes lie apart (E4M3, 310 requests of up to
    // 5001 tokens, 12 query rows, token-major pages of 16: 185 us against 273 at 128 bytes, whose
    // other half is another head's; 31 requests 32.9 against 34.1).
    const bool apart = row_bytes < 128 && stride[2] != row_bytes;
    const CUtensorMapL2promotion fetch = !apart            ? CU_TENSOR_MAP_L2_PROMOTION_L2_128B
                                         : row_bytes == 64 ? CU_TENSOR_MAP_L2_PROMOTION_L2_64B
                                                           : CU_TENSOR_MAP_L2_PROMOTION_NONE;
    return encode(out, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, const_cast<void*>(ptr), dims, strides, box,
                  estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                  row_bytes == 32   ? CU_TENSOR_MAP_SWIZZLE_32B
                  : row_bytes == 64 ? CU_TENSOR_MAP_SWIZZLE_64B
                                    : CU_TENSOR_MAP_SWIZZLE_128B,
                  fetch, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The tensor map of block scales [pages, heads, tokens * head_dim / 16] in elements of `element`
// bytes (1 or 8), with a box of `tokens` tokens' scales (at most 256 elements): a page outside the
// pool reads as zeros.
bool encode_scales(CUtensorMap* out, const void* ptr, int element, int tokens, const CacheShape& c) {
    EncodeTiledFn encode = encode_fn();
    if (encode == nullptr) return false;
    const int token = c.head_dim / 16;  // bytes
    const cuuint64_t row = static_cast<cuuint64_t>(c.page_size) * token;
    const cuuint64_t dims[3] = {row / element, static_cast<cuuint64_t>(c.heads), static_cast<cuuint64_t>(c.pages)};
    const cuuint64_t strides[2] = {row, row * c.heads};
    const cuuint32_t box[3] = {static_cast<cuuint32_t>(tokens * token / element), 1, 1};
    const cuuint32_t estr[3] = {1, 1, 1};
    return encode(out, element == 8 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT64 : CU_TENSOR_MAP_DATA_TYPE_UINT8, 3,
                  const_cast<void*>(ptr), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                  CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

int device_sms() {
    int dev = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
        (void)cudaGetLastError();
        return 0;
    }
    return sms;
}

int check_paged_rows(const uint16_t* q, int64_t q_stride, const CacheShape& cache,
                     const int32_t* table, int64_t table_stride, int32_t width,
                     const int32_t* lengths, int32_t R, int32_t row_group, int32_t Hq, bool* skip) {
    *skip = false;
    if (!cache.ready) return SMD_ERR_PLAN;
    const int64_t row = static_cast<int64_t>(Hq) * cache.head_dim;
    if (R < 0 || row_group < 1 || row_group > kPagedMaxGroup || Hq < 1 || Hq % cache.heads != 0 ||
        Hq / cache.heads > kPagedMaxHeads || Hq > 65535 || width < 1 || table_stride < width ||
        static_cast<int64_t>(width) * cache.page_size >= (1ll << 31) ||
        static_cast<int64_t>(R) * row_group * Hq >= (1ll << 31) || q_stride < row ||
        q_stride % 8 != 0)
        return SMD_ERR_SHAPE;
    if (R == 0) {
        *skip = true;
        return SMD_OK;
    }
    if (q == nullptr || table == nullptr || lengths == nullptr) return SMD_ERR_NULL;
    if (!aligned(q, 16) || !aligned(table, 4) || !aligned(lengths, 4)) return SMD_ERR_ALIGN;
    return SMD_OK;
}

}  // namespace smd

extern "C" int smd_paged_cache_init(smd_paged_cache_t* c) {
    using namespace smd;
    if (c == nullptr) return SMD_ERR_NULL;
    std::memset(c->map, 0, sizeof c->map);
    const bool kv = c->k != nullptr;
    if (kv != (c->v != nullptr) || (!kv && c->bounds == nullptr) ||
        (kv && (c->k_scale == nullptr || c->v_scale == nullptr)))
        return SMD_ERR_NULL;
    if (!shape_ok(c->pages, c->heads, c->page_size, c->head_dim))
        return SMD_ERR_SHAPE;
    if (!aligned(c->bounds, 16) || !aligned(c->k_scale, 4) || !aligned(c->v_scale, 4))
        return SMD_ERR_ALIGN;
    if (kv) {
        if (!strides_ok(c->k_stride, c->head_dim) || !strides_ok(c->v_stride, c->head_dim))
            return SMD_ERR_SHAPE;
        if (!steps_of_16(c->k_stride) || !steps_of_16(c->v_stride)) return SMD_ERR_ALIGN;
        if (!aligned(c->k, 16) || !aligned(c->v, 16)) return SMD_ERR_ALIGN;
        CUtensorMap maps[2];
        const CacheShape shape = shape_of(c);
        const int box = page_box_tokens(c->page_size, c->head_dim);
        if (!encode_codes(&maps[0], c->k, c->k_stride, c->head_dim, box, shape) ||
            !encode_codes(&maps[1], c->v, c->v_stride, c->head_dim, box, shape))
            return SMD_ERR_DEVICE;
        std::memcpy(&c->map[1], maps, sizeof maps);
    }
    c->map[0] = kPagedMark;
    return SMD_OK;
}

extern "C" int smd_paged4_cache_init(smd_paged4_cache_t* c) {
    using namespace smd;
    if (c == nullptr) return SMD_ERR_NULL;
    std::memset(c->map, 0, sizeof c->map);
    if (c->k == nullptr || c->v == nullptr || c->k_scales == nullptr || c->v_scales == nullptr)
        return SMD_ERR_NULL;
    if (!shape_ok(c->pages, c->heads, c->page_size, c->head_dim) ||
        !strides_ok(c->k_stride, c->head_dim / 2) || !strides_ok(c->v_stride, c->head_dim / 2))
        return SMD_ERR_SHAPE;
    if (!steps_of_16(c->k_stride) || !steps_of_16(c->v_stride) || !aligned(c->k, 16) ||
        !aligned(c->v, 16) || !aligned(c->k_scales, 16) || !aligned(c->v_scales, 16) ||
        !aligned(c->k_exp, 4) || !aligned(c->v_exp, 4) || !aligned(c->bounds, 16))
        return SMD_ERR_ALIGN;
    CUtensorMap maps[4];
    const CacheShape shape = shape_of(c);
    const bool tc = c->head_dim == 128;
    const int box = tc ? tc_box_tokens(c->page_size) : page_box_tokens(c->page_size, c->head_dim);
    if (!encode_codes(&maps[0], c->k, c->k_stride, c->head_dim / 2, box, shape) ||
        !encode_codes(&maps[1], c->v, c->v_stride, c->head_dim / 2, box, shape) ||
        !encode_scales(&maps[2], c->k_scales, tc ? 8 : 1, box, shape) ||
        !encode_scales(&maps[3], c->v_scales, tc ? 8 : 1, box, shape))
        return SMD_ERR_DEVICE;
    std::memcpy(&c->map[1], maps, sizeof maps);
    c->map[0] = kPaged4Mark;
    return SMD_OK;
}

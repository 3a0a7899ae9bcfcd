// The description of a paged cache (smd_paged_cache_init) and the checks that
// the calls on it share. Host code only.
#include <cstring>

#include "smd_internal.h"
#include "smd_paged.h"

namespace smd {

namespace {

bool strides_ok(const int64_t (&s)[3], int head_dim) {
    for (int i = 0; i < 3; ++i)
        if (s[i] <= 0 || s[i] >= (1ll << 40)) return false;
    return s[2] >= head_dim;
}

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

bool encode_page_map(CUtensorMap* out, const void* ptr, const int64_t (&stride)[3],
                     const smd_paged_cache_t& c) {
    EncodeTiledFn encode = encode_fn();
    if (encode == nullptr) return false;
    const cuuint64_t dims[4] = {
        static_cast<cuuint64_t>(c.head_dim), static_cast<cuuint64_t>(c.page_size),
        static_cast<cuuint64_t>(c.heads), static_cast<cuuint64_t>(c.pages)};
    const cuuint64_t strides[3] = {static_cast<cuuint64_t>(stride[2]),
                                   static_cast<cuuint64_t>(stride[1]),
                                   static_cast<cuuint64_t>(stride[0])};
    const cuuint32_t box[4] = {static_cast<cuuint32_t>(c.head_dim < 128 ? c.head_dim : 128),
                               static_cast<cuuint32_t>(page_box_tokens(c)), 1, 1};
    const cuuint32_t estr[4] = {1, 1, 1, 1};
    // L2 fetches no more than a row where rows of 64 bytes lie apart (310 requests of up to
    // 5001 tokens, 12 query rows, token-major pages of 16: 185 us against 273 at 128 bytes, whose
    // other half is another head's; 31 requests 32.9 against 34.1).
    const CUtensorMapL2promotion fetch = c.head_dim < 128 && stride[2] != c.head_dim
                                             ? CU_TENSOR_MAP_L2_PROMOTION_L2_64B
                                             : CU_TENSOR_MAP_L2_PROMOTION_L2_128B;
    return encode(out, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, const_cast<void*>(ptr), dims, strides, box,
                  estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                  c.head_dim < 128 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B, fetch,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

int check_paged_rows(const uint16_t* q, int64_t q_stride, const smd_paged_cache_t* cache,
                     const int32_t* table, int64_t table_stride, int32_t width,
                     const int32_t* lengths, int32_t R, int32_t row_group, int32_t Hq, bool* skip) {
    *skip = false;
    if (cache == nullptr) return SMD_ERR_NULL;
    if (!paged_ready(cache)) return SMD_ERR_PLAN;
    const int64_t row = static_cast<int64_t>(Hq) * cache->head_dim;
    if (R < 0 || row_group < 1 || row_group > kPagedMaxGroup || Hq < 1 || Hq % cache->heads != 0 ||
        Hq / cache->heads > kPagedMaxHeads || Hq > 65535 || width < 1 || table_stride < width ||
        static_cast<int64_t>(width) * cache->page_size >= (1ll << 31) ||
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
    if (c->pages < 1 || c->heads < 1 || c->heads > 65535 || c->page_size < 16 ||
        c->page_size > 256 || c->page_size % 16 != 0 ||
        (c->head_dim != 64 && c->head_dim != 128 && c->head_dim != 256) ||
        static_cast<int64_t>(c->pages) * c->page_size >= (1ll << 31))
        return SMD_ERR_SHAPE;
    if (!aligned(c->bounds, 16) || !aligned(c->k_scale, 4) || !aligned(c->v_scale, 4))
        return SMD_ERR_ALIGN;
    if (kv) {
        if (!strides_ok(c->k_stride, c->head_dim) || !strides_ok(c->v_stride, c->head_dim))
            return SMD_ERR_SHAPE;
        for (int i = 0; i < 3; ++i)
            if (c->k_stride[i] % 16 != 0 || c->v_stride[i] % 16 != 0) return SMD_ERR_ALIGN;
        if (!aligned(c->k, 16) || !aligned(c->v, 16)) return SMD_ERR_ALIGN;
        CUtensorMap maps[2];
        if (!encode_page_map(&maps[0], c->k, c->k_stride, *c) ||
            !encode_page_map(&maps[1], c->v, c->v_stride, *c))
            return SMD_ERR_DEVICE;
        std::memcpy(&c->map[1], maps, sizeof maps);
    }
    c->map[0] = kPagedMark;
    return SMD_OK;
}

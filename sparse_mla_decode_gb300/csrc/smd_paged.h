// Declarations shared by the paged-cache calls (smd_block_tables,
// smd_paged_append, smd_block_scores, smd_paged_decode).
#pragma once

#include <atomic>
#include <cstdint>

#include <cuda.h>
#include <cuda_runtime.h>

#include "smd.h"

namespace smd {

constexpr int kPagedMaxGroup = 8;    // verify rows of a request
constexpr int kPagedMaxHeads = 128;  // query heads of a kv head

// What smd_paged_cache_init leaves in smd_paged_cache_t::map: a mark, then the
// tensor maps of k and v (absent in a cache of bounds only).
constexpr uint64_t kPagedMark = 0x736d645061676564ull;
static_assert(sizeof(CUtensorMap) == 128, "two maps and the mark fit smd_paged_cache_t::map");

inline bool paged_ready(const smd_paged_cache_t* c) { return c->map[0] == kPagedMark; }

inline bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// Pages that hold a number of tokens (0 to 2^31 - 1).
__device__ __forceinline__ int pages_of(int tokens, int P) {
    return static_cast<int>((static_cast<uint32_t>(tokens) + static_cast<uint32_t>(P) - 1) /
                            static_cast<uint32_t>(P));
}

// Tokens of one copy box: the largest of 32 and 16 that divides a page (16 at
// 256 columns, where the decode's tile holds 16 tokens).
inline int page_box_tokens(const smd_paged_cache_t& c) {
    return c.page_size % 32 == 0 && c.head_dim < 256 ? 32 : 16;
}

// The tensor map of one side of a cache over (column, token, head, page), with
// a box of up to 128 columns by page_box_tokens() tokens (128-byte swizzle; 64
// at 64 columns). False if encoding failed.
bool encode_page_map(CUtensorMap* out, const void* ptr, const int64_t (&stride)[3],
                     const smd_paged_cache_t& c);

// Rows of queries as smd_block_scores and smd_paged_decode take them, checked;
// *skip is set where there is nothing to do.
int check_paged_rows(const uint16_t* q, int64_t q_stride, const smd_paged_cache_t* cache,
                     const int32_t* table, int64_t table_stride, int32_t width,
                     const int32_t* lengths, int32_t R, int32_t row_group, int32_t Hq, bool* skip);

// SMs of the current device; 0 on failure.
int device_sms();

constexpr int kMaxDevices = 64;

// A kernel's limit of dynamic shared memory, raised once on each device, whatever the
// first call asks for: below the raised limit the static bytes count with the dynamic
// ones, so whether one call fits must not rest on its own dynamic bytes alone.
struct SharedLimit {
    std::atomic<bool> ready[kMaxDevices];

    template <typename... Params>
    int raise(void (*kernel)(Params...), int bytes) {
        int dev = 0;
        if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) {
            (void)cudaGetLastError();
            return SMD_ERR_DEVICE;
        }
        if (ready[dev]) return SMD_OK;
        if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) !=
            cudaSuccess) {
            (void)cudaGetLastError();
            return SMD_ERR_DEVICE;
        }
        ready[dev] = true;
        return SMD_OK;
    }
};

// Launches `kernel` with programmatic stream serialization, as every kernel of
// the library; an smd_status.
template <typename... Params, typename... Args>
int launch_pdl(void (*kernel)(Params...), dim3 grid, int threads, size_t smem, smd_stream_t stream,
               const Args&... args) {
    cudaLaunchConfig_t lc{};
    lc.gridDim = grid;
    lc.blockDim = dim3(static_cast<unsigned>(threads), 1, 1);
    lc.dynamicSmemBytes = smem;
    lc.stream = reinterpret_cast<cudaStream_t>(stream);
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    lc.attrs = attr;
    lc.numAttrs = 1;
    if (cudaLaunchKernelEx(&lc, kernel, static_cast<Params>(args)...) != cudaSuccess) {
        (void)cudaGetLastError();
        return SMD_ERR_LAUNCH;
    }
    return SMD_OK;
}

}  // namespace smd

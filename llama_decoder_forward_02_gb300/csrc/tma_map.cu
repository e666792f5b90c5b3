// Host-side creation of the TMA descriptors (CUtensorMap) that the tcgen05
// kernels load their fp16 operand tiles with: a row-major [rows][cols] matrix
// read in boxes of box_rows x 64 elements with 128-byte swizzle, the layout
// the kernels' shared-memory matrix descriptors expect.  The driver entry
// point is looked up once through the runtime, so the library links no
// driver library directly.
#include <cuda.h>
#include <mutex>

#include "gemm_tc_common.cuh"
#include "kernels.h"

namespace llm {

namespace {

typedef CUresult (*EncodeTiledFn)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                  const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn() {
    static std::once_flag once;
    static EncodeTiledFn fn = nullptr;
    std::call_once(once, [] {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) ==
                cudaSuccess && q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<EncodeTiledFn>(p);
    });
    return fn;
}

// A row-major [rows][cols] matrix of elements of `size` bytes, in boxes of box_rows x box_cols.
bool encode(TmaMap *m, CUtensorMapDataType type, int size, const void *ptr, long long rows, int cols, int box_rows, int box_cols,
            CUtensorMapSwizzle swizzle) {
    static_assert(sizeof(TmaMap) == sizeof(CUtensorMap), "TmaMap must hold a CUtensorMap");
    EncodeTiledFn fn = encode_fn();
    if (!fn || !ptr || rows < 1 || (reinterpret_cast<uintptr_t>(ptr) & 15)) return false;
    const cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
    const cuuint64_t strides[1] = {(cuuint64_t)cols * size};
    const cuuint32_t box[2] = {(cuuint32_t)box_cols, (cuuint32_t)box_rows};
    const cuuint32_t estr[2] = {1, 1};
    auto call = [&] {
        return fn(reinterpret_cast<CUtensorMap *>(m), type, 2, const_cast<void *>(ptr), dims, strides, box, estr,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    };
    CUresult r = call();
    // the driver wants a context that is current, which a host thread has only after a call of the runtime's that
    // needs one: such a thread's first call may be ours
    int dev = 0;
    if (r == CUDA_ERROR_INVALID_CONTEXT && cudaGetDevice(&dev) == cudaSuccess && cudaSetDevice(dev) == cudaSuccess) r = call();
    return r == CUDA_SUCCESS;
}

}  // namespace

bool make_operand_map(TmaMap *m, const f16 *ptr, int rows, int cols, int box_rows) {
    return cols % 64 == 0 &&
           encode(m, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2, ptr, rows, cols, box_rows, tcg::BK, CU_TENSOR_MAP_SWIZZLE_128B);
}

bool make_cache_map(TmaMap *m, const f16 *ptr, long long rows, int head_dim) {
    return (head_dim == 32 || head_dim % 64 == 0) && rows < (1ll << 31) &&
           encode(m, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2, ptr, rows, head_dim, 128, 64, CU_TENSOR_MAP_SWIZZLE_128B);
}

bool make_cache8_map(TmaMap *m, const uint8_t *ptr, long long rows, int head_dim) {
    return head_dim <= 128 && head_dim % 32 == 0 && rows < (1ll << 31) &&
           encode(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, ptr, rows, head_dim, 128, head_dim,
                  head_dim == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE);
}

bool make_f32_tile_map(TmaMap *m, const float *ptr, int rows, int cols) {
    return cols % 32 == 0 && encode(m, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 4, ptr, rows, cols, 128, 32, CU_TENSOR_MAP_SWIZZLE_128B);
}

}  // namespace llm

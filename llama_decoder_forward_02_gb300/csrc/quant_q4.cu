// Q4_0 weight blocks for the decode GEMVs (q4.cuh has the encoding and the
// layout of the codes).  A Q4_0 matrix [N][K], K a multiple of 256, is N rows
// of K / 256 chunks of 144 bytes: the codes of two 128-element groups, then
// the chunk's 8 fp16 scales, so that any run of chunks of a row is one
// 16-byte aligned copy that brings codes and scales together.
#include "common.cuh"
#include "kernels.h"
#include "q4.cuh"

namespace llm {

namespace {

// One thread per block: thread b of the grid takes block b % (K/32) of row
// b / (K/32).  q4 == nullptr skips the encoded copy; write_back replaces the
// fp16 elements by the weights the block stands for (one rounding).  Set-up
// work, bound by the fp16 reads and writes.
__global__ void quantize_q4_0_kernel(f16 *w, int N, int K, uint8_t *q4, int write_back) {
    const int nb = K / q4::BLOCK;
    const long long b = (long long)blockIdx.x * blockDim.x + threadIdx.x;
    if (b >= (long long)N * nb) return;
    const int row = (int)(b / nb), blk = (int)(b - (long long)row * nb);
    f16 *src = w + (size_t)row * K + (size_t)blk * q4::BLOCK;
    uint4 raw[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) raw[i] = reinterpret_cast<const uint4 *>(src)[i];
    const __half *h = reinterpret_cast<const __half *>(raw);
    float m = 0.f;
#pragma unroll
    for (int i = 0; i < q4::BLOCK; ++i) {
        const float v = __half2float(h[i]);
        if (fabsf(v) > fabsf(m)) m = v;
    }
    const float d = m * -0.125f;                     // exact: fp16 values are normal fp32 numbers
    int c[q4::BLOCK];
#pragma unroll
    for (int i = 0; i < q4::BLOCK; ++i) c[i] = q4::code_of(__half2float(h[i]), d);
    const __half dh = __float2half_rn(d);
    if (q4) {
        const int in_chunk = blk & 7;
        uint8_t *chunk = q4 + (size_t)row * ((size_t)K / q4::CHUNK * q4::CHUNK_BYTES) +
                         (size_t)(blk >> 3) * q4::CHUNK_BYTES;
        uint32_t *words = reinterpret_cast<uint32_t *>(chunk) + (in_chunk >> 2) * 16 + (in_chunk & 3);
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            uint32_t word = 0;
#pragma unroll
            for (int e = 0; e < 8; ++e) word |= (uint32_t)c[8 * t + e] << q4::shift_of(e);
            words[4 * t] = word;
        }
        reinterpret_cast<__half *>(chunk + 128)[in_chunk] = dh;
    }
    if (write_back) {
        const float ds = __half2float(dh);
        uint4 out[4];
        uint32_t *o = reinterpret_cast<uint32_t *>(out);
#pragma unroll
        for (int i = 0; i < q4::BLOCK / 2; ++i)
            o[i] = pack_h2((float)(c[2 * i] - 8) * ds, (float)(c[2 * i + 1] - 8) * ds);
#pragma unroll
        for (int i = 0; i < 4; ++i) reinterpret_cast<uint4 *>(src)[i] = out[i];
    }
}

}  // namespace

size_t q4_0_row_bytes(int K) { return (size_t)K / q4::CHUNK * q4::CHUNK_BYTES; }

cudaError_t launch_quantize_q4_0(f16 *w, int N, int K, uint8_t *q4, bool write_back, cudaStream_t st) {
    if (N < 1 || K < q4::BLOCK || K % q4::BLOCK || (q4 && K % q4::CHUNK)) return cudaErrorInvalidValue;
    const long long nblk = (long long)N * (K / q4::BLOCK);
    quantize_q4_0_kernel<<<(unsigned)((nblk + 255) / 256), 256, 0, st>>>(w, N, K, q4, write_back ? 1 : 0);
    return cudaGetLastError();
}

}  // namespace llm

// Q4_0: four-bit codes with one scale for 32 elements, as the weights of the
// decode GEMVs and the KV cache hold them.  "LLama.cpp — how it works" names
// four-bit types among the quantised tensor element types ("The GGUF format
// (reference)") and the quantised cache ("KV-cache") without a layout.  The
// one taken: a row is cut into blocks of 32 consecutive elements; with m the
// block's element of largest magnitude (the first of equals), a block keeps
// the scale m / -8 (float32, stored as fp16) and codes
//   c = clamp(nearest integer to w / (m / -8), ties to even, + 8, 0, 15),
// and stands for d * (c - 8) with the stored d: m itself takes code 0 and the
// fifteen levels 0..15 reach 7/8 of it on the other side.  A block of zeros
// has d = 0 and codes 8.
//
// Codes lie eight to a 32-bit word.  In a group of NB blocks (a cache row of
// 32 NB elements; 128 consecutive elements, NB = 4, of a weight row) word
// t * NB + b, t = 0..3, holds elements 32 b + 8 t + {0..7}: element 8 t + 2 i
// in bits 4 i.., element 8 t + 2 i + 1 in bits 16 + 4 i...  So one AND with
// 0x000F000F leaves two neighbouring elements in the halves of a register,
// which is how an mma.sync fragment wants them, and the 4 NB bytes that lane t
// of a fragment row needs are contiguous.  The ANDed halves are used as they
// are: as fp16 bit patterns they are the subnormals c * 2^-24 (or, for the
// nibbles at bits 4 and 20, c * 2^-20), which the tensor cores multiply
// exactly.
#pragma once
#include "common.cuh"
#include "kernels.h"

namespace llm {
namespace q4 {

constexpr int BLOCK = 32;                // elements of a block
constexpr int CHUNK = 256;               // elements of a weight chunk
constexpr int CHUNK_BYTES = 144;         // ... its codes (2 x 64 bytes), then 8 fp16 scales

// bits of element e of an eight-element word
__host__ __device__ constexpr int shift_of(int e) { return 4 * (e >> 1) + 16 * (e & 1); }

// The code of v in a block of scale d (unrounded).  |v / d| <= 8; R is float
// where v is exact, double where a caller resolves a value next to a border.
template <class R>
__device__ __forceinline__ int code_of(R v, R d) {
    if (d == R(0)) return 8;
    const R q = v / d;
    int c = (int)rint(q) + 8;
    return c < 0 ? 0 : c > 15 ? 15 : c;
}

// Whether q = v / d in float32, next to the integer k, lies so near a code
// border that its last bits could decide: |q| <= 8 with a relative error below
// 24 * 2^-24 (a norm, a rotation and the quotient) is 1.2e-5 off at most.
__device__ __forceinline__ bool near_border(float q, float k) {
    constexpr float NEAR = 2e-5f;
    return fabsf(fabsf(q - k) - 0.5f) < NEAR || q > 8.f - NEAR;
}

// The code of a lane's element u of the block that its warp holds, and the
// block's scale.  Returns whether R does not settle the code.
template <class R>
__device__ __forceinline__ bool encode_lane(R u, R &d, int &code) {
    R top = fabs(u);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        const R other = __shfl_xor_sync(0xffffffffu, top, o);
        top = other > top ? other : top;
    }
    const unsigned has = __ballot_sync(0xffffffffu, fabs(u) == top);     // the first of that magnitude gives the sign
    d = __shfl_sync(0xffffffffu, u, has ? __ffs(has) - 1 : 0) * R(-0.125);
    if constexpr (sizeof(R) == 4) {
        const float q = d != 0.f ? u * __frcp_rn(d) : 0.f, k = rintf(q);
        code = min(max((int)k + 8, 0), 15);
        return d != 0.f && (!(fabsf(d) > 1e-30f) || near_border(q, k));
    } else {
        code = code_of(u, d);
        return false;
    }
}

}  // namespace q4
}  // namespace llm

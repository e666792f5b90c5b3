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
// of a fragment row needs are contiguous.  Decode attention uses K's ANDed
// halves as they are: as fp16 bit patterns they are the subnormals c * 2^-24 (or,
// for the nibbles at bits 4 and 20, c * 2^-20), which the tensor cores multiply
// exactly.  Everything else reads c - 8 (Widen).
#pragma once
#include "common.cuh"
#include "kernels.h"

namespace llm {
namespace q4 {

constexpr int BLOCK = 32;                // elements of a block
constexpr int CHUNK = 256;               // elements of a weight chunk
constexpr int CHUNK_BYTES = 144;         // ... its codes (2 x 64 bytes), then 8 fp16 scales

// scales at and below which a product's remainder leaves float32's range, and a
// factor that brings such a block back
constexpr float TINY = 1e-30f, RAISE = 0x1p96f;

// bits of element e of an eight-element word
__host__ __device__ constexpr int shift_of(int e) { return 4 * (e >> 1) + 16 * (e & 1); }

// c - 8 of the codes at bits 0 and 16 / at bits 4 and 20 of a word, as an fp16
// pair: (w & 0x000F000F) | 0x64006400 reads 1024 + c in both halves, (w &
// 0x00F000F0) | 0x54005400 reads 64 + c, and less 1032 and 72 that is c - 8.  One
// LOP3 takes at most one constant as an immediate, so the masks and biases are
// kept in registers the compiler cannot see through (with immediates it emits
// two: 20% more instructions in all).
struct Widen {
    uint32_t m0, e0, m1, e1;
    __device__ __forceinline__ Widen() {
        asm volatile("mov.b32 %0, 0x000F000F;\n\tmov.b32 %1, 0x64006400;\n\tmov.b32 %2, 0x00F000F0;\n\tmov.b32 %3, 0x54005400;"
                     : "=r"(m0), "=r"(e0), "=r"(m1), "=r"(e1));
    }
    __device__ __forceinline__ static uint32_t pick(uint32_t w, uint32_t m, uint32_t e, uint32_t bias) {
        uint32_t v;
        asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(v) : "r"(w), "r"(m), "r"(e));       // (w & m) | e
        const __half2 r = __hsub2(*reinterpret_cast<const __half2 *>(&v), *reinterpret_cast<const __half2 *>(&bias));
        return *reinterpret_cast<const uint32_t *>(&r);
    }
    __device__ __forceinline__ uint32_t low(uint32_t w) const { return pick(w, m0, e0, 0x64086408u); }
    __device__ __forceinline__ uint32_t high(uint32_t w) const { return pick(w, m1, e1, 0x54805480u); }
};

// The code of v in a block of scale d (unrounded), v exact.  |v / d| <= 8.
__device__ __forceinline__ int code_of(float v, float d) {
    if (d == 0.f) return 8;
    const int c = (int)rintf(v / d) + 8;
    return c < 0 ? 0 : c > 15 ? 15 : c;
}

// Values next to a code border are settled in pairs of floats, h + l with l at
// most half an ulp of h: sums and products of floats are exact as pairs (Knuth's
// two-sum, a product and its FMA remainder), those of pairs good to 2^-44, and
// this GPU's float64 units are a sixtieth of its float32 ones (a warp that
// resolved its borders in float64 took 6.5 us).
struct Pair { float h, l; };
__device__ __forceinline__ Pair two_sum(float a, float b) {
    const float s = __fadd_rn(a, b), t = __fsub_rn(s, a);
    return Pair{s, __fadd_rn(__fsub_rn(a, __fsub_rn(s, t)), __fsub_rn(b, t))};
}
__device__ __forceinline__ Pair two_prod(float a, float b) {
    const float p = __fmul_rn(a, b);
    return Pair{p, __fmaf_rn(a, b, -p)};
}
__device__ __forceinline__ Pair settle(float h, float l) {          // |l| well below |h|
    const float s = __fadd_rn(h, l);
    return Pair{s, __fsub_rn(l, __fsub_rn(s, h))};
}
__device__ __forceinline__ Pair operator+(Pair a, Pair b) {
    const Pair s = two_sum(a.h, b.h);
    return settle(s.h, __fadd_rn(s.l, __fadd_rn(a.l, b.l)));
}
__device__ __forceinline__ Pair operator*(Pair a, float b) {
    const Pair p = two_prod(a.h, b);
    return settle(p.h, __fmaf_rn(a.l, b, p.l));
}
__device__ __forceinline__ Pair operator*(Pair a, Pair b) {
    const Pair p = two_prod(a.h, b.h);
    return settle(p.h, __fmaf_rn(a.h, b.l, __fmaf_rn(a.l, b.h, p.l)));
}
__device__ __forceinline__ Pair magnitude(Pair a) { return a.h < 0.f ? Pair{-a.h, -a.l} : a; }
// of two magnitudes
__device__ __forceinline__ bool larger(Pair a, Pair b) { return a.h > b.h || (a.h == b.h && a.l > b.l); }
__device__ __forceinline__ Pair shfl_xor(Pair a, int o) {
    return Pair{__shfl_xor_sync(0xffffffffu, a.h, o), __shfl_xor_sync(0xffffffffu, a.l, o)};
}
__device__ __forceinline__ Pair shfl(Pair a, int from) {
    return Pair{__shfl_sync(0xffffffffu, a.h, from), __shfl_sync(0xffffffffu, a.l, from)};
}

// The code of v: which side of the border b nearest to v / d it lies on is the
// sign of v - b d.  On the border the even integer.
__device__ __forceinline__ int code_of(Pair v, Pair d) {
    if (d.h == 0.f) return 8;
    const float q = v.h * __frcp_rn(d.h), k = rintf(q), b = q >= k ? k + 0.5f : k - 0.5f;
    const Pair p = two_prod(b, d.h);
    const float t = __fadd_rn(__fsub_rn(__fsub_rn(v.h, p.h), p.l), __fmaf_rn(-b, d.l, v.l));
    const int lo = (int)floorf(b);
    const int c = 8 + (t == 0.f ? lo + (lo & 1) : lo + ((t > 0.f) == (d.h > 0.f)));
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
// block's scale.  Returns whether float32 does not settle the code.
__device__ __forceinline__ bool encode_lane(float u, float &d, int &code) {
    float top = fabsf(u);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        const float other = __shfl_xor_sync(0xffffffffu, top, o);
        top = other > top ? other : top;
    }
    const unsigned has = __ballot_sync(0xffffffffu, fabsf(u) == top);     // the first of that magnitude gives the sign
    d = __shfl_sync(0xffffffffu, u, has ? __ffs(has) - 1 : 0) * -0.125f;
    const float q = d != 0.f ? u * __frcp_rn(d) : 0.f, k = rintf(q);
    code = min(max((int)k + 8, 0), 15);
    return d != 0.f && (!(fabsf(d) > TINY) || near_border(q, k));
}
// ... of the pair u, whose remainder is lost below TINY: the caller scales.
__device__ __forceinline__ void encode_lane(Pair u, float &d, int &code) {
    Pair top = magnitude(u);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        const Pair other = shfl_xor(top, o);
        if (larger(other, top)) top = other;
    }
    const Pair mine = magnitude(u);
    const unsigned has = __ballot_sync(0xffffffffu, mine.h == top.h && mine.l == top.l);
    const Pair m = shfl(u, has ? __ffs(has) - 1 : 0), d2{m.h * -0.125f, m.l * -0.125f};
    code = code_of(u, d2);
    d = d2.h;
}

}  // namespace q4
}  // namespace llm

// Microscaled 4-bit format: constants, the scale buffer's layout and the
// quantisation of a run of values held in registers, shared by the row
// quantiser, the norm step and the decode weight layout.
#pragma once

#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "common.cuh"

namespace as {

__host__ __device__ constexpr int fp4_block(int fmt) { return fmt == AS_FP4_MX ? 32 : 16; }
// 512-byte scale tiles (128 rows x 4 blocks) along K
__host__ __device__ constexpr int fp4_sf_ktiles(int K, int fmt)
{
    return (K + 4 * fp4_block(fmt) - 1) / (4 * fp4_block(fmt));
}
// Byte of row r, block b in the scale buffer with kt tiles along K.
__host__ __device__ __forceinline__ size_t fp4_sf_byte(int r, int b, int kt)
{
    return ((size_t)(r >> 7) * kt + (b >> 2)) * 512 + (size_t)(r & 31) * 16 + ((r >> 5) & 3) * 4 + (b & 3);
}

constexpr uint32_t F32_INF_BITS = 0x7F800000u;

// Row scale S = 2^e of the NV format from the bits of the row's largest
// finite |v|: the smallest e >= -126 with amax <= 2688 * 2^e.  2688 =
// 1.3125 * 2^11, so e = k - 11 for a mantissa up to 1.3125 and k - 10 above
// (amax = 1.m * 2^k).  Returns e (0 for a zero row).
__device__ __forceinline__ int nv_row_exponent(uint32_t amax_bits)
{
    if (amax_bits == 0u) return 0;
    const int k = (int)(amax_bits >> 23) - 127;
    const int e = k - 11 + ((amax_bits & 0x7FFFFFu) > 0x280000u ? 1 : 0);
    return e < -126 ? -126 : e;
}

__device__ __forceinline__ float pow2f(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }  // -126..127

// Two E2M1 codes, lo in the low four bits: round to nearest even, saturating.
__device__ __forceinline__ uint32_t e2m1x2(float lo, float hi)
{
    uint32_t r;
    asm("{\n\t.reg .b8 t;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 t, %2, %1;\n\t"
        "cvt.u32.u8 %0, t;\n\t}"
        : "=r"(r)
        : "f"(lo), "f"(hi));
    return r;
}

// Two values of a byte of codes, as float32.
__device__ __forceinline__ float2 e2m1x2_value(uint32_t byte)
{
    uint32_t h;
    asm("{\n\t.reg .b8 t;\n\t"
        "cvt.u8.u32 t, %1;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, t;\n\t}"
        : "=r"(h)
        : "r"(byte));
    return __half22float2(*reinterpret_cast<const __half2 *>(&h));
}

__device__ __forceinline__ float e4m3_value(uint32_t byte)
{
    return __half2float(__half(__nv_cvt_fp8_to_halfraw((__nv_fp8_storage_t)byte, __NV_E4M3)));
}

// Scale byte -> value (E8M0 0 is 2^-127, 0xFF is NaN).
template <int FMT>
__device__ __forceinline__ float fp4_scale_value(uint32_t byte)
{
    if constexpr (FMT == AS_FP4_NV) return e4m3_value(byte);
    return byte == 0u ? __uint_as_float(0x00400000u)
                      : (byte == 255u ? __uint_as_float(0x7FFFFFFFu) : __uint_as_float(byte << 23));
}

// What a block's largest |v| (float32 bits) decides: the scale byte, the
// factor `pre` that divides the row scale (or, MX, the whole scale) out
// exactly, and the E4M3 scale `s` left to divide by (NV).  s = 0: codes 0.
//
// The codes are those of the exact quotient: a border between two codes is
// t * s with t of at most three and s of four significant bits.
//   NV: the scale is E4M3(fl32(amax * 2^-e / 6)); fl32 of that quotient never
//   lands on a border between two E4M3 values unless the quotient is one,
//   since one float32 step of amax moves amax / 6 by more than half a step.
//   MX: s is a power of two, multiplying by its inverse is exact.
struct Fp4Block {
    uint32_t byte;
    float pre, s;
};
template <int FMT>
__device__ __forceinline__ Fp4Block fp4_block_scale(uint32_t amax_bits, float inv_row)
{
    Fp4Block b;
    const bool bad = amax_bits >= F32_INF_BITS;
    if constexpr (FMT == AS_FP4_MX) {
        const int f = (int)(amax_bits >> 23);  // biased exponent, 0 for subnormals
        const int e = amax_bits == 0u ? 127 : (f > 2 ? f - 2 : 0);
        b.byte = bad ? 255u : (uint32_t)e;
        b.pre = bad ? 0.0f : __uint_as_float((uint32_t)(254 - e) << 23);
        b.s = bad ? 0.0f : 1.0f;
    } else {
        const float q = __fdiv_rn(__fmul_rn(__uint_as_float(amax_bits), inv_row), 6.0f);
        b.byte = bad ? 127u : (uint32_t)__nv_cvt_float_to_fp8(q, __NV_SATFINITE, __NV_E4M3);
        b.pre = inv_row;
        b.s = bad ? 0.0f : e4m3_value(b.byte);
    }
    return b;
}

// Codes of 8 values of one block (channel order, low four bits first).
// EXACT8: every value has at most 8 significant bits (bf16).  Then one
// truncating multiply by r = fl32(1/s) decides every code as the exact
// quotient does: off a border the quotient is at least 2^-16 away from it,
// and on a border the truncated product is the border itself (checked for all
// 8 mantissas of s against all 128 of v).  Otherwise the quotient is rounded
// correctly; fl32(v / s) lies on a border only when v / s does (one float32
// step of v moves it by more than half a step of the border).
template <int FMT, bool EXACT8>
__device__ __forceinline__ uint32_t fp4_codes8(const float *v, const Fp4Block &b, float r)
{
    const bool none = !(b.s > 0.0f);
    uint32_t w = 0u;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float q[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const float x = __fmul_rn(v[2 * i + k], b.pre);
            if constexpr (FMT == AS_FP4_MX) q[k] = x;
            else if constexpr (EXACT8) q[k] = __fmul_rz(x, r);
            else q[k] = __fdiv_rn(x, none ? 1.0f : b.s);
        }
        w |= e2m1x2(q[0], q[1]) << (8 * i);
    }
    return none ? 0u : w;
}
template <int FMT, bool EXACT8>
__device__ __forceinline__ uint2 fp4_codes16(const float (&v)[16], const Fp4Block &b)
{
    const float r = (FMT == AS_FP4_NV && EXACT8) ? __frcp_rn(b.s > 0.0f ? b.s : 1.0f) : 1.0f;
    const uint32_t lo = fp4_codes8<FMT, EXACT8>(v, b, r), hi = fp4_codes8<FMT, EXACT8>(v + 8, b, r);
    return make_uint2(lo, hi);
}

// Largest |v| bits of the block that 16 values belong to; MX blocks span two
// neighbouring lanes (all 32 lanes take part).
template <int FMT>
__device__ __forceinline__ uint32_t fp4_block_amax(uint32_t m)
{
    if constexpr (FMT == AS_FP4_MX) m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
    return m;
}

}  // namespace as

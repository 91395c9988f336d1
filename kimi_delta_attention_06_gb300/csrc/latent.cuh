// latent.cuh -- the latent cache's row formats and small device helpers of the latent
// attention kernels.
#pragma once
#include <cstdint>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include "common.cuh"

namespace kda {

constexpr int kLatDim = 512;                     // latent values a token
constexpr int kLatRope = 64;                     // shared position key values a token
constexpr int kLatQ = kLatDim + kLatRope;        // absorbed query length
constexpr int kLatRowBf16 = kLatQ * 2;           // 1152 bytes: latent, position key
// 656 bytes: 512 codes, the position key (64 bf16), the fp32 scale, 12 bytes of zero
constexpr int kLatRowE4m3 = kLatDim + 2 * kLatRope + 16;
constexpr int kLatScaleAt = kLatDim + 2 * kLatRope;
constexpr int kStatusIndex = -1;                 // KDA_ERR_INVALID_ARG, recorded on the device

__host__ __device__ constexpr int lat_row_bytes(bool e4m3) { return e4m3 ? kLatRowE4m3 : kLatRowBf16; }

__device__ __forceinline__ float lat_ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Smallest e with x <= 448 * 2^e = 1.75 * 2^(8 + e), in [-117, most]; 0 for x = 0 (x >= 0 by its bits).  A cache
// row's scale ends at 2^119; the largest finite x needs 120.
__device__ __forceinline__ int lat_scale_exponent(uint32_t bits, int most = 119) {
    const int e = static_cast<int>(bits >> 23) - 127 - 8 + ((bits & 0x7fffffu) > 0x600000u ? 1 : 0);
    return bits == 0 ? 0 : max(-117, min(most, e));
}

// Two e4m3 codes (low byte first) -> two floats.
__device__ __forceinline__ float2 e4m3x2_to_f32(uint32_t w) {
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(w & 0xFFFFu), __NV_E4M3);
    return __half22float2(__half2(h));
}
// Two floats -> two e4m3 codes (low byte first), nearest even, magnitudes above 448 -> 448, NaN stays NaN.
__device__ __forceinline__ uint32_t f32x2_to_e4m3x2(float lo, float hi) {
    return __nv_cvt_float2_to_fp8x2(make_float2(lo, hi), __NV_SATFINITE, __NV_E4M3);
}

// Splitting fp16 pairs (packed bits) into 8-bit terms, by the formats' definitions and in integer
// arithmetic: the conversion instructions to 8-bit types take 16 clocks a warp here, these 3.
// e5m2 is fp16 with 2 of its 10 fraction bits, so rounding the magnitude's low byte away rounds to
// e5m2; the code is the upper byte.  (Halves round up; a NaN is not kept.)
__device__ __forceinline__ uint32_t f16x2_round_e5m2(uint32_t h) { return (h + 0x00800080u) & 0xff00ff00u; }
// e4m3 codes of x are the bits 13..7 of fp16 values x / 2^8 and the sign (both formats' subnormals line
// up: 2^-6 / 2^8 = 2^-14), for |x| <= 448.  Here h holds x / 2^8 (at most 1.75: no carry leaves its
// half) and the result is the rounded x / 2^8.
__device__ __forceinline__ uint32_t f16x2_round_e4m3(uint32_t h) { return (h + 0x00400040u) & 0xff80ff80u; }
// The two e4m3 codes of such a rounded pair, in bytes 0 and 2 (bytes 1 and 3: anything).
__device__ __forceinline__ uint32_t e4m3_codes(uint32_t r) { return ((r >> 7) & 0x007f007fu) | ((r >> 8) & ~0x007f007fu); }
__device__ __forceinline__ uint32_t f16x2_sub(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}
__device__ __forceinline__ uint32_t f32x2_to_f16x2(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}

}  // namespace kda

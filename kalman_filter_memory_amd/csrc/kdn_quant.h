// kdn_quant.h -- the 8-bit format the norm, the quantiser and the 8-bit product
// share (gfx950 only, internal): e4m3 without infinities (largest value 448),
// one float32 scale per 128 columns (x 1 or 128 rows), value = element * scale.
#pragma once

#include "kdn_device.h"

namespace kdn {

constexpr int kQuantBlock = 128;           // columns (and weight rows) per scale
constexpr float kQuantInvMax = 1.f / 448.f;  // of the largest e4m3 value
constexpr float kQuantScaleMin = 0x1p-126f;  // smallest normal float

// |x| as its bits: ordered like the value, with infinity above every number and
// NaN above infinity, so that an integer maximum keeps a NaN (fmaxf drops it)
__device__ __forceinline__ uint32_t abs_bits(float x) { return __float_as_uint(x) & 0x7fffffffu; }

template <int CTRL> __device__ __forceinline__ uint32_t dpp_u(uint32_t x) {
    return __builtin_amdgcn_update_dpp(0, x, CTRL, 0xF, 0xF, false);
}
__device__ __forceinline__ uint32_t umax(uint32_t a, uint32_t b) { return a > b ? a : b; }

// maximum over the 16 aligned lanes of a DPP row, returned to each of them
__device__ __forceinline__ uint32_t row_umax(uint32_t x) {
    x = umax(x, dpp_u<0xB1>(x));   // quad_perm xor 1
    x = umax(x, dpp_u<0x4E>(x));   // quad_perm xor 2
    x = umax(x, dpp_u<0x141>(x));  // row_half_mirror
    return umax(x, dpp_u<0x140>(x));  // row_mirror
}

// scale of a block whose largest |x| has these bits: max times the float32 1 / 448, at
// least 2^-126 (an all-zero block gets 2^-126); a NaN or an infinity is kept.  The
// product and not a division, because that is what torch's max / 448 is on the GPU: half
// of the two's scales differ by a unit, which moves up to 0.1 % of the elements of a
// bfloat16 tensor (many quotients lie next to a border), and the operand would not be
// the same.
__device__ __forceinline__ float quant_scale(uint32_t amax_bits) {
    const float s = __uint_as_float(amax_bits) * kQuantInvMax;
    return s < kQuantScaleMin ? kQuantScaleMin : s;
}

// eight values over their scale as eight e4m3 bytes, round to nearest even; inv is
// 1 / scale in 64 bits.  The quotient is float32's, correctly rounded: x inv is within
// 2^-52 of it, relative, and a quotient of two floats lies at least 2^-49 from any
// point halfway between floats (x is not halfway (25 bits) times scale (24 bits), and
// both are multiples of one unit of that product's 49 bits).  A product with the float32
// 1 / scale is up to two units off and puts an element in 10^7 on the other side of a
// border.  (us, bfloat16, with that product, with this and with a float32 division: norm
// to 8 bits 32768 x 2048 81.3, 82.4, 85.4; quantiser 6192 x 2048 7.1, 8.0, 10.7, 32768 x
// 2048 rows 32.2, 33.8, 37.1.)
// |x| / scale <= 448 (1 + 2^-22) and e4m3 rounds everything below 464 to 448, so no clamp
// is needed; NaN stays NaN.
__device__ __forceinline__ u32x2 quant8(const float* x, double inv) {
    float y[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = float(double(x[i]) * inv);
    int lo = 0, hi = 0;
    lo = __builtin_amdgcn_cvt_pk_fp8_f32(y[0], y[1], lo, false);
    lo = __builtin_amdgcn_cvt_pk_fp8_f32(y[2], y[3], lo, true);
    hi = __builtin_amdgcn_cvt_pk_fp8_f32(y[4], y[5], hi, false);
    hi = __builtin_amdgcn_cvt_pk_fp8_f32(y[6], y[7], hi, true);
    return u32x2{static_cast<uint32_t>(lo), static_cast<uint32_t>(hi)};
}

// eight floats at p (16-byte aligned) in E
template <typename E> __device__ __forceinline__ void store8(E* p, const float* f) {
    u32x4* o = reinterpret_cast<u32x4*>(p);
    if constexpr (sizeof(E) == 2) {
        *o = u32x4{pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]), pack_bf16(f[4], f[5]),
                   pack_bf16(f[6], f[7])};
    } else {
        o[0] = u32x4{__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]),
                     __float_as_uint(f[3])};
        o[1] = u32x4{__float_as_uint(f[4]), __float_as_uint(f[5]), __float_as_uint(f[6]),
                     __float_as_uint(f[7])};
    }
}

}  // namespace kdn

// 4-bit weights to BF16, in registers.
//
// code x scale is a BF16 number exactly (2 significant bits times at most 4),
// but for its range: values carry a factor, and the product is multiplied by
// its inverse (unscale).
// The three magnitude bits of a code, moved to bits 6..8 of a 16-bit half, are
// a BF16 of 2^-126 times the code's value (subnormal for the code 0.5), so one
// BF16 multiplication makes the value, its scaling and the factor.
//   NVFP4: values carry 2^-16 (2^126 x 448 is past BF16's range): by 2^110 x scale.
//   MXFP4: they carry 2^-2 (6 x 2^127 is past it): by 2^124 x scale, which fits up
//          to a scale of 2^3; blocks with larger scales (WIDE) take two
//          multiplications.
#pragma once

#include "mx4_internal.h"

namespace tgemm {
namespace mx4_decode {

template <int FMT> __device__ constexpr float unscale() { return FMT == TGEMM_NVFP4 ? 65536.0f : 4.0f; }

// The factor of a scale byte, as two BF16 halves.
template <int FMT>
__device__ __forceinline__ uint32_t factor(uint32_t byte) {
    uint32_t h;
    if (FMT == TGEMM_MXFP4) h = byte == 255 ? 0x7FC0u : byte <= 130 ? (byte + 124) << 7 : byte << 7;
    else h = __float_as_uint(e4m3_value(byte & 0x7F) * 1.298074214633707e33f) >> 16;     // 2^110
    return h | h << 16;
}
// MXFP4 blocks with such a scale need 2^124 as a factor of its own.
__device__ __forceinline__ bool wide(uint32_t byte) { return byte > 130; }

__device__ __forceinline__ uint32_t mul2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// Eight codes (a word) to four pairs, each a BF16 of 2^-126 times its value:
// pair i holds codes i (low half) and i + 4.
__device__ __forceinline__ void pairs(uint32_t w, uint32_t (&v)[4]) {
    constexpr uint32_t MAG = 0x01C001C0u, SIGN = 0x80008000u;
    v[0] = (w << 6 & MAG) | (w << 12 & SIGN);
    v[1] = (w << 2 & MAG) | (w << 8 & SIGN);
    v[2] = (w >> 2 & MAG) | (w << 4 & SIGN);
    v[3] = (w >> 6 & MAG) | (w & SIGN);
}

constexpr uint32_t TWO_124 = 0x7D807D80u;

// The pairs' values, scaled.
template <bool WIDE>
__device__ __forceinline__ void values(uint32_t w, uint32_t f, uint32_t (&v)[4]) {
    pairs(w, v);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (WIDE) v[i] = mul2(v[i], TWO_124);
        v[i] = mul2(v[i], f);
    }
}

// 32 codes of a row (16 bytes) to BF16, in order.
template <bool WIDE>
__device__ __forceinline__ void decode_run(uint4 (&out)[4], const uint4& codes, uint32_t f0, uint32_t f1) {
    const uint32_t w[4] = {codes.x, codes.y, codes.z, codes.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        uint32_t v[4];
        pairs(w[j], v);
        const uint32_t f = j < 2 ? f0 : f1;
        uint32_t r[4] = {__byte_perm(v[0], v[1], 0x5410), __byte_perm(v[2], v[3], 0x5410),
                         __byte_perm(v[0], v[1], 0x7632), __byte_perm(v[2], v[3], 0x7632)};
        if (WIDE)
#pragma unroll
            for (int i = 0; i < 4; ++i) r[i] = mul2(r[i], TWO_124);
#pragma unroll
        for (int i = 0; i < 4; ++i) r[i] = mul2(r[i], f);
        out[j] = make_uint4(r[0], r[1], r[2], r[3]);
    }
}

}  // namespace mx4_decode
}  // namespace tgemm

// Packed codes in registers: a lane's field of 32 consecutive channels of one
// row (BITS words of the little-endian stream) and its codes as fp32 values.
#pragma once

#include "common.hpp"

namespace ttq {

template <int BITS>
struct CodeWords {
    uint32_t w[BITS];
};

template <int BITS>
__device__ __forceinline__ void load_codes(CodeWords<BITS>& c, const uint32_t* __restrict__ p) {
    if constexpr (BITS == 4) {
        const u32x4 v = ld_nc((const u32x4*)p);
#pragma unroll
        for (int i = 0; i < 4; ++i) c.w[i] = v[i];
    } else if constexpr (BITS == 2) {
        const u32x2 v = ld_nc((const u32x2*)p);
        c.w[0] = v[0];
        c.w[1] = v[1];
    } else {
#pragma unroll
        for (int i = 0; i < BITS; ++i) c.w[i] = ld_nc(p + i);
    }
}

// Code i (0..31) of a lane's 32-code field.
template <int BITS>
__device__ __forceinline__ uint32_t code_at(const CodeWords<BITS>& c, int i) {
    const int bit = BITS * i;
    const int wi = bit >> 5, off = bit & 31;
    uint32_t v = c.w[wi] >> off;
    if (off + BITS > 32) v |= c.w[wi + 1] << (32 - off);
    return v & ((1u << BITS) - 1);
}

constexpr int kTChan = 32;                        // channels per lane field

template <int N>
__device__ __forceinline__ float cvt_ubyte(uint32_t v) {
    float f;
    if constexpr (N == 0) asm("v_cvt_f32_ubyte0 %0, %1" : "=v"(f) : "v"(v));
    else if constexpr (N == 1) asm("v_cvt_f32_ubyte1 %0, %1" : "=v"(f) : "v"(v));
    else if constexpr (N == 2) asm("v_cvt_f32_ubyte2 %0, %1" : "=v"(f) : "v"(v));
    else asm("v_cvt_f32_ubyte3 %0, %1" : "=v"(f) : "v"(v));
    return f;
}

// The 32 codes of a lane's field as fp32 values, code i at bits BITS*i of the
// little-endian bit stream.
template <int BITS>
__device__ __forceinline__ void field_codes(const CodeWords<BITS>& c, float (&q)[kTChan]) {
    if constexpr (BITS == 4) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t lo = c.w[i] & 0x0F0F0F0Fu, hi = (c.w[i] >> 4) & 0x0F0F0F0Fu;
            q[8 * i + 0] = cvt_ubyte<0>(lo);
            q[8 * i + 1] = cvt_ubyte<0>(hi);
            q[8 * i + 2] = cvt_ubyte<1>(lo);
            q[8 * i + 3] = cvt_ubyte<1>(hi);
            q[8 * i + 4] = cvt_ubyte<2>(lo);
            q[8 * i + 5] = cvt_ubyte<2>(hi);
            q[8 * i + 6] = cvt_ubyte<3>(lo);
            q[8 * i + 7] = cvt_ubyte<3>(hi);
        }
    } else if constexpr (BITS == 2) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const uint32_t m = (c.w[i] >> (2 * j)) & 0x03030303u;   // codes 4 b + j of this word
                q[16 * i + j] = cvt_ubyte<0>(m);
                q[16 * i + 4 + j] = cvt_ubyte<1>(m);
                q[16 * i + 8 + j] = cvt_ubyte<2>(m);
                q[16 * i + 12 + j] = cvt_ubyte<3>(m);
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < kTChan; ++i) q[i] = (float)code_at<BITS>(c, i);
    }
}

// 4x4 exchange between the lane quarters (16-lane rows) and the four words of
// a lane: word j of quarter q becomes word q of quarter j.
__device__ __forceinline__ void swap_quarters(u32x4& w) {
    const auto a = __builtin_amdgcn_permlane32_swap(w[0], w[2], false, false);
    const auto b = __builtin_amdgcn_permlane32_swap(w[1], w[3], false, false);
    const auto c = __builtin_amdgcn_permlane16_swap(a[0], b[0], false, false);
    const auto d = __builtin_amdgcn_permlane16_swap(a[1], b[1], false, false);
    w = u32x4{c[0], c[1], d[0], d[1]};
}

}  // namespace ttq

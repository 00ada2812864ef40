// Microscaled (MX) rows, shared by the kernels that write or read them.
//
// A row of K values is cut into blocks of 32; a block holds 32 small floats
// (e4m3: 4 exponent and 3 mantissa bits, largest 448; e2m1: 2 and 1, largest
// 6) and one scale byte b that stands for 2^(b - 127) (255: not a number).
// value = element * 2^(b - 127).  Internal to libmoe_dispatch.
#pragma once

#include "common.cuh"

namespace moe {

constexpr int kMxBlock = 32;        // values that share a scale
constexpr int kMxPad = 128;         // rows are zero-padded to this many values
constexpr int kMxMaxK = 1 << 18;    // widest row

inline bool mx_format_ok(int32_t f) { return f == MOE_MX_E4M3 || f == MOE_MX_E2M1; }
inline int32_t mx_padded(int32_t K) { return (K + kMxPad - 1) / kMxPad * kMxPad; }
inline int64_t mx_row_bytes(int32_t K, int32_t format) {
    return format == MOE_MX_E4M3 ? mx_padded(K) : mx_padded(K) / 2;
}
// 16-byte multiples: a row's scales can be moved by the row movers and by TMA.
inline int64_t mx_scale_bytes(int32_t K) { return (mx_padded(K) / kMxBlock + 15) / 16 * 16; }
inline bool mx_aligned(const void *q, const void *scales) {
    // 32 bytes: what the copy that widens packed 4-bit values asks of a matrix
    return (reinterpret_cast<uintptr_t>(q) & 31u) == 0 && aligned16(scales);
}

// Scale byte of a block from the bits of its largest magnitude (the unsigned
// maximum of the values' bits without their sign, so infinities and NaN win):
// the smallest power of two with which nothing saturates.  With the largest
// magnitude 1.m * 2^(E-127) and the format's largest value 1.75 * 2^8 or
// 1.5 * 2^2, that is 2^(E-127-8) (or -2), doubled if 1.m exceeds 1.75 (1.5).
// Rounding the power up, where the MX paper's rule rounds it down, keeps the
// block's largest value (up to a quarter of it would be cut off with e2m1).
template <int FMT>
__device__ __forceinline__ uint32_t mx_scale_byte(uint32_t amax_bits) {
    constexpr int emax = FMT == MOE_MX_E4M3 ? 8 : 2;
    constexpr uint32_t top = FMT == MOE_MX_E4M3 ? 0x600000u : 0x400000u;
    const int e = (int)(amax_bits >> 23);
    if (e == 255) return 255u;
    const int b = e - emax + ((amax_bits & 0x7fffffu) > top ? 1 : 0);
    return (uint32_t)(b > 0 ? b : 0);
}

// 2^(127 - b): the exact factor from a value to its element (b <= 253 here).
__device__ __forceinline__ float mx_inverse(uint32_t b) {
    return __uint_as_float((254u - b) << 23);
}

// 2^(b - 127): 2^-127 is the one subnormal, 255 is NaN.
__device__ __forceinline__ float mx_scale(uint32_t b) {
    return __uint_as_float(b == 0 ? 0x00400000u : b == 255u ? 0x7fc00000u : b << 23);
}

__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7fffffffu; }

// Two fp32 values in one register pair: sm_100 adds and multiplies them in one instruction.
typedef unsigned long long f32x2;
__device__ __forceinline__ f32x2 pair_of(float a, float b) {
    f32x2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float2 halves(f32x2 p) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(p));
    return r;
}
__device__ __forceinline__ f32x2 add2(f32x2 a, f32x2 b) {
    f32x2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ f32x2 mul2(f32x2 a, f32x2 b) {
    f32x2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ f32x2 fma2(f32x2 a, f32x2 b, f32x2 c) {
    f32x2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}

// Eight scaled values to elements, nearest with ties to even: 8 bytes (e4m3)
// or 4 bytes in .x (e2m1, even columns in the low halves).
template <int FMT>
__device__ __forceinline__ uint2 mx_pack8(const float (&v)[8]) {
    if (FMT == MOE_MX_E4M3) {
        uint32_t r[2];
#pragma unroll
        for (int i = 0; i < 2; ++i)
            asm("{\n\t.reg .b16 lo, hi;\n\t"
                "cvt.rn.satfinite.e4m3x2.f32 lo, %2, %1;\n\t"
                "cvt.rn.satfinite.e4m3x2.f32 hi, %4, %3;\n\t"
                "mov.b32 %0, {lo, hi};\n\t}"
                : "=r"(r[i])
                : "f"(v[4 * i]), "f"(v[4 * i + 1]), "f"(v[4 * i + 2]), "f"(v[4 * i + 3]));
        return make_uint2(r[0], r[1]);
    }
    uint32_t r;
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
        "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
        : "=r"(r)
        : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
    return make_uint2(r, 0u);
}

// The larger magnitude; NaN if one is.
__device__ __forceinline__ float max_abs(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(fabsf(a)), "f"(fabsf(b)));
    return r;
}

// A quarter block (8 values) of a lane whose neighbours in its group of four
// hold the rest of the block: the block's scale byte and this lane's elements.
// A lane that is not `real` has zeros, whatever v holds.  A block that holds an
// infinity or NaN gets scale 255 and zero elements: it reads back as NaN, so
// nothing that is not a number passes for one.
template <int FMT>
__device__ __forceinline__ uint2 mx_quarter(const f32x2 (&v)[4], bool real, uint32_t &byte) {
    float m[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) m[i] = max_abs(halves(v[i]).x, halves(v[i]).y);
    float top = max_abs(max_abs(m[0], m[1]), max_abs(m[2], m[3]));
    if (!real) top = 0.0f;
    top = max_abs(top, __shfl_xor_sync(MOE_FULL_MASK, top, 1));
    top = max_abs(top, __shfl_xor_sync(MOE_FULL_MASK, top, 2));
    byte = mx_scale_byte<FMT>(abs_bits(top));
    const float inv = mx_inverse(byte);
    const f32x2 inv2 = pair_of(inv, inv);
    float s[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 p = halves(mul2(v[i], inv2));
        s[2 * i] = p.x;
        s[2 * i + 1] = p.y;
    }
    const uint2 q = mx_pack8<FMT>(s);
    return byte == 255u || !real ? make_uint2(0u, 0u) : q;
}

// The same of 8 bf16 values.  Magnitudes are compared as 16-bit integers, two at a time, and
// the power of two is multiplied in bf16, which is exact down to products so small that
// they round to zero elements anyhow.
template <int FMT>
__device__ __forceinline__ uint2 mx_quarter_bf16(const uint4 &in, uint32_t &byte) {
    const uint32_t u[4] = {in.x, in.y, in.z, in.w};
    uint32_t m2 = u[0] & 0x7fff7fffu;
#pragma unroll
    for (int i = 1; i < 4; ++i)
        asm("max.u16x2 %0, %0, %1;" : "+r"(m2) : "r"(u[i] & 0x7fff7fffu));
    asm("max.u16x2 %0, %0, %1;" : "+r"(m2) : "r"(__shfl_xor_sync(MOE_FULL_MASK, m2, 1)));
    asm("max.u16x2 %0, %0, %1;" : "+r"(m2) : "r"(__shfl_xor_sync(MOE_FULL_MASK, m2, 2)));
    byte = mx_scale_byte<FMT>(max(m2 << 16, m2 & 0xffff0000u));
    const uint32_t inv = ((254u - byte) & 0xffu) * 0x00800080u;
    float s[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint32_t p;
        asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(p) : "r"(u[i]), "r"(inv));
        s[2 * i] = __uint_as_float(p << 16);
        s[2 * i + 1] = __uint_as_float(p & 0xffff0000u);
    }
    const uint2 q = mx_pack8<FMT>(s);
    return byte == 255u ? make_uint2(0u, 0u) : q;
}

// The lane's elements at vector `vec` (8 values) of a row.
template <int FMT>
__device__ __forceinline__ void mx_store_elements(uint8_t *row, int vec, uint2 q) {
    if (FMT == MOE_MX_E4M3)
        *reinterpret_cast<uint2 *>(row + 8 * (int64_t)vec) = q;
    else
        *reinterpret_cast<uint32_t *>(row + 4 * (int64_t)vec) = q.x;
}

// ... and by the first lane of each four the block's scale.
template <int FMT>
__device__ __forceinline__ void mx_store(uint8_t *row, uint8_t *scales, int vec, uint2 q,
                                         uint32_t byte) {
    mx_store_elements<FMT>(row, vec, q);
    if ((vec & 3) == 0) scales[vec >> 2] = (uint8_t)byte;
}

// Zeros behind the scales of a row's blocks (both counts are multiples of four).
__device__ __forceinline__ void mx_clear_scales(uint8_t *scales, int64_t blocks, int64_t bytes) {
    for (int64_t b = blocks; b < bytes; b += 4) *reinterpret_cast<uint32_t *>(scales + b) = 0u;
}

__device__ __forceinline__ void unpack_bf16x8(const uint4 &v, float (&f)[8]) {
    const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = __uint_as_float(u[i] << 16);
        f[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
    }
}

}  // namespace moe

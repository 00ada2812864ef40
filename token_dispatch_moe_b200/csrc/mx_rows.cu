// moe_mx_quantize and moe_mx_dequantize: bf16 rows to microscaled rows and back.
//
// Both are one pass over the data, bound by memory: a value costs 2 bytes on
// the bf16 side and 1 + 1/32 (e4m3) or 1/2 + 1/32 (e2m1) on the other.  A
// lane takes 8 values (16 bytes of bf16); four lanes hold a block and find its
// largest magnitude with two shuffles.  A block of threads takes a run of
// kRowVecs vectors of the rows laid end to end (padding included), kRowUnroll
// of them a thread, all loads issued before the first use.
#include <cuda_fp16.h>

#include "mx.cuh"
#include "rows.cuh"

namespace moe {
namespace {

constexpr int kRowThreads = 256;
constexpr int kRowUnroll = 4;
constexpr int kRowVecs = kRowThreads * kRowUnroll;

struct MxRowsArgs {
    int64_t vecs;      // rows * vpr
    uint32_t vpr;      // 8-value vectors of a padded row
    uint32_t magic;    // floor(2^32 / vpr) + 1: x / vpr = umulhi(x, magic) while x * vpr < 2^32,
                       // and x < vpr + kRowVecs with vpr <= 2^15; not used with vpr 1
    uint32_t data;     // vectors of a row that hold data
    int64_t row_bytes, scale_bytes;
};

// Row and vector of element `off` of the run that starts at (row0, vec0).
__device__ __forceinline__ int64_t place(const MxRowsArgs &a, int64_t row0, uint32_t vec0,
                                         uint32_t off, uint32_t &vec) {
    const uint32_t x = vec0 + off;
    const uint32_t r = a.vpr == 1 ? x : __umulhi(x, a.magic);
    vec = x - r * a.vpr;
    return row0 + r;
}

template <int FMT>
__global__ void __launch_bounds__(kRowThreads)
    mx_quantize_kernel(const moe_bf16_t *__restrict__ x, uint8_t *__restrict__ q,
                       uint8_t *__restrict__ scales, const MxRowsArgs a) {
    griddep_wait();
    const int64_t base = (int64_t)blockIdx.x * kRowVecs;
    const int64_t row0 = base / a.vpr;
    const uint32_t vec0 = (uint32_t)(base - row0 * a.vpr);
    uint4 in[kRowUnroll];
    int64_t row[kRowUnroll];
    uint32_t vec[kRowUnroll];
#pragma unroll
    for (int u = 0; u < kRowUnroll; ++u) {
        const uint32_t off = u * kRowThreads + threadIdx.x;
        row[u] = place(a, row0, vec0, off, vec[u]);
        in[u] = make_uint4(0u, 0u, 0u, 0u);
        if (base + off < a.vecs && vec[u] < a.data)
            in[u] = ld_stream(reinterpret_cast<const uint4 *>(x) + row[u] * a.data + vec[u]);
    }
    griddep_launch_dependents();
#pragma unroll
    for (int u = 0; u < kRowUnroll; ++u) {
        const uint32_t off = u * kRowThreads + threadIdx.x;
        float f[8];
        unpack_bf16x8(in[u], f);
        uint32_t byte;
        const uint2 e = mx_quarter<FMT>(f, byte);  // four lanes of a block share its fate
        if (base + off >= a.vecs) continue;
        uint8_t *srow = scales + row[u] * a.scale_bytes;
        mx_store<FMT>(q + row[u] * a.row_bytes, srow, (int)vec[u], e, byte);
        // the bytes behind the last block's scale
        if (vec[u] + 1 == a.vpr)
            for (int64_t b = a.vpr / 4; b < a.scale_bytes; ++b) srow[b] = 0;
    }
}

template <int FMT>
__global__ void __launch_bounds__(kRowThreads)
    mx_dequantize_kernel(const uint8_t *__restrict__ q, const uint8_t *__restrict__ scales,
                         moe_bf16_t *__restrict__ out, const MxRowsArgs a) {
    // Here vpr counts the vectors that hold data: padding is not read.
    griddep_wait();
    const int64_t base = (int64_t)blockIdx.x * kRowVecs;
    const int64_t row0 = base / a.vpr;
    const uint32_t vec0 = (uint32_t)(base - row0 * a.vpr);
    uint2 in[kRowUnroll];
    uint32_t byte[kRowUnroll];
#pragma unroll
    for (int u = 0; u < kRowUnroll; ++u) {
        const uint32_t off = u * kRowThreads + threadIdx.x;
        uint32_t vec;
        const int64_t row = place(a, row0, vec0, off, vec);
        in[u] = make_uint2(0u, 0u);
        byte[u] = 0;
        if (base + off < a.vecs) {
            const uint8_t *src = q + row * a.row_bytes;
            if (FMT == MOE_MX_E4M3)
                in[u] = __ldcs(reinterpret_cast<const uint2 *>(src) + vec);
            else
                in[u].x = __ldcs(reinterpret_cast<const uint32_t *>(src) + vec);
            byte[u] = __ldg(scales + row * a.scale_bytes + (vec >> 2));
        }
    }
    griddep_launch_dependents();
#pragma unroll
    for (int u = 0; u < kRowUnroll; ++u) {
        const int64_t i = base + u * kRowThreads + threadIdx.x;
        if (i >= a.vecs) continue;
        const float s = mx_scale(byte[u]);
        float f[8];
#pragma unroll
        for (int p = 0; p < 4; ++p) {  // two elements: exact in fp16, then exact in fp32
            uint32_t h2;
            if (FMT == MOE_MX_E4M3) {
                const uint16_t two = (uint16_t)((p < 2 ? in[u].x : in[u].y) >> (16 * (p & 1)));
                asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h2) : "h"(two));
            } else {
                const uint16_t two = (uint16_t)((in[u].x >> (8 * p)) & 0xffu);
                asm("{\n\t.reg .b8 lo, hi;\n\tmov.b16 {lo, hi}, %1;\n\t"
                    "cvt.rn.f16x2.e2m1x2 %0, lo;\n\t}"
                    : "=r"(h2)
                    : "h"(two));
            }
            const float2 v = __half22float2(*reinterpret_cast<const __half2 *>(&h2));
            f[2 * p] = v.x * s;
            f[2 * p + 1] = v.y * s;
        }
        reinterpret_cast<uint4 *>(out)[i] = pack_bf16x8(f);  // rows of out have no padding
    }
}

moe_status check_rows(const void *bf16, int64_t rows, int32_t K, int32_t format, const void *q,
                      const void *scales) {
    if (rows < 0 || K < 8 || K % 8 != 0 || !mx_format_ok(format)) return MOE_ERR_INVALID_ARG;
    if (rows == 0) return MOE_OK;
    if (!bf16 || !q || !scales || !aligned16(bf16) || !mx_aligned(q, scales))
        return MOE_ERR_INVALID_ARG;
    if (K > kMxMaxK || rows >= (int64_t)INT32_MAX) return MOE_ERR_UNSUPPORTED;
    const int64_t blocks = (rows * (mx_padded(K) / 8) + kRowVecs - 1) / kRowVecs;
    return blocks < (int64_t)INT32_MAX ? MOE_OK : MOE_ERR_UNSUPPORTED;
}

MxRowsArgs rows_args(int64_t rows, int32_t K, int32_t format, int32_t width) {
    MxRowsArgs a;
    a.vpr = (uint32_t)width / 8;
    a.data = (uint32_t)K / 8;
    a.vecs = rows * a.vpr;
    a.magic = a.vpr == 1 ? 0u : (uint32_t)((1ull << 32) / a.vpr + 1);
    a.row_bytes = mx_row_bytes(K, format);
    a.scale_bytes = mx_scale_bytes(K);
    return a;
}

}  // namespace
}  // namespace moe

extern "C" moe_status moe_mx_row_bytes(int32_t K, int32_t format, int64_t *row_bytes,
                                       int64_t *scale_bytes) {
    using namespace moe;
    if (K < 8 || K % 8 != 0 || !mx_format_ok(format) || !row_bytes || !scale_bytes)
        return MOE_ERR_INVALID_ARG;
    if (K > kMxMaxK) return MOE_ERR_UNSUPPORTED;
    *row_bytes = mx_row_bytes(K, format);
    *scale_bytes = mx_scale_bytes(K);
    return MOE_OK;
}

extern "C" moe_status moe_mx_quantize(const moe_bf16_t *x, int64_t rows, int32_t K, int32_t format,
                                      uint8_t *q, uint8_t *scales, moe_stream_t stream) {
    using namespace moe;
    const moe_status st = check_rows(x, rows, K, format, q, scales);
    if (st != MOE_OK || rows == 0) return st;
    const MxRowsArgs a = rows_args(rows, K, format, mx_padded(K));
    const dim3 grid((unsigned)((a.vecs + kRowVecs - 1) / kRowVecs));
    const cudaError_t e =
        format == MOE_MX_E4M3
            ? launch_pdl(mx_quantize_kernel<MOE_MX_E4M3>, grid, dim3(kRowThreads), 0,
                         as_cuda(stream), x, q, scales, a)
            : launch_pdl(mx_quantize_kernel<MOE_MX_E2M1>, grid, dim3(kRowThreads), 0,
                         as_cuda(stream), x, q, scales, a);
    if (e != cudaSuccess) {
        cudaGetLastError();
        return MOE_ERR_CUDA;
    }
    return launch_status();
}

extern "C" moe_status moe_mx_dequantize(const uint8_t *q, const uint8_t *scales, int64_t rows,
                                        int32_t K, int32_t format, moe_bf16_t *out,
                                        moe_stream_t stream) {
    using namespace moe;
    const moe_status st = check_rows(out, rows, K, format, q, scales);
    if (st != MOE_OK || rows == 0) return st;
    const MxRowsArgs a = rows_args(rows, K, format, K);
    const dim3 grid((unsigned)((a.vecs + kRowVecs - 1) / kRowVecs));
    const cudaError_t e =
        format == MOE_MX_E4M3
            ? launch_pdl(mx_dequantize_kernel<MOE_MX_E4M3>, grid, dim3(kRowThreads), 0,
                         as_cuda(stream), q, scales, out, a)
            : launch_pdl(mx_dequantize_kernel<MOE_MX_E2M1>, grid, dim3(kRowThreads), 0,
                         as_cuda(stream), q, scales, out, a);
    if (e != cudaSuccess) {
        cudaGetLastError();
        return MOE_ERR_CUDA;
    }
    return launch_status();
}

// moe_mx_quantize and moe_mx_dequantize: bf16 rows to microscaled rows and back.
//
// Both are one pass over the data, bound by memory: a value costs 2 bytes on
// the bf16 side and 1 + 1/32 (e4m3) or 1/2 + 1/32 (e2m1) on the other.  A
// lane takes 8 values (16 bytes of bf16); four lanes hold a block and find its
// largest magnitude with two shuffles.  A warp takes kRowUnroll * 32
// consecutive vectors of the rows laid end to end (quantize: padding
// included), all its loads issued before the first use, so its scales are 32
// consecutive bytes and go out in one store.  What bounded quantize was the
// number of instructions (110 a vector, 80 % of the issue slots busy at 4.1
// TB/s): element rows follow one another without gaps, so stores need no row
// arithmetic, nor do loads where K is a multiple of 128; magnitudes are
// compared and scaled two to a register.  Measured, e2m1: 65,536 x 2048 58 us
// (5.8 TB/s; 78 before), 368,640 x 2880 493 us (5.4; 551 before) and back
// 400 us (6.7 TB/s); e4m3 6.1 to 6.4 TB/s.
#include <cuda_fp16.h>

#include "mx.cuh"
#include "rows.cuh"

namespace moe {
namespace {

constexpr int kRowThreads = 256;
constexpr int kRowUnroll = 4;  // 32 blocks a warp: one lane for each scale
constexpr int kRowVecs = kRowThreads * kRowUnroll;

struct MxRowsArgs {
    int64_t vecs;      // rows * vpr
    uint32_t vpr;      // 8-value vectors of a row: with its padding (quantize) or without
    uint32_t magic;    // floor(2^32 / vpr) + 1: v / vpr = umulhi(v, magic) for v * vpr < 2^32, so
                       // for v < vpr + kRowVecs (vpr <= 2^15); not used with vpr 1
    uint32_t data;     // vectors of a row that hold data
    int64_t row_bytes, scale_bytes;
};

// Row and vector of the warp's vector `off` places on from its first.
struct Place {
    int64_t row;
    uint32_t vec;
    __device__ __forceinline__ Place(const MxRowsArgs &a, uint32_t off) {
        const int64_t i = (int64_t)blockIdx.x * kRowVecs;
        row = i / a.vpr;  // the same for the block
        vec = (uint32_t)(i - row * a.vpr) + (threadIdx.x >> 5) * (32 * kRowUnroll) + off;
        const uint32_t r = rows_on(a, vec);
        row += r;
        vec -= r * a.vpr;
    }
    static __device__ __forceinline__ uint32_t rows_on(const MxRowsArgs &a, uint32_t v) {
        return a.vpr == 1 ? v : __umulhi(v, a.magic);
    }
};

template <int FMT>
__global__ void __launch_bounds__(kRowThreads)
    mx_quantize_kernel(const moe_bf16_t *__restrict__ x, uint8_t *__restrict__ q,
                       uint8_t *__restrict__ scales, const MxRowsArgs a) {
    griddep_wait();
    const uint32_t lane = threadIdx.x & 31;
    const int64_t base =
        (int64_t)blockIdx.x * kRowVecs + (threadIdx.x >> 5) * (32 * kRowUnroll) + lane;
    const int left = (int)min(a.vecs - base, (int64_t)kRowVecs);  // this lane's u runs while 32 u < left
    uint4 in[kRowUnroll];
    if (a.data == a.vpr) {  // no padding: x is as flat as the elements
        const uint4 *src = reinterpret_cast<const uint4 *>(x) + base;
#pragma unroll
        for (int u = 0; u < kRowUnroll; ++u)
            in[u] = 32 * u < left ? ld_stream(src + 32 * u) : make_uint4(0u, 0u, 0u, 0u);
    } else {
        const Place at(a, lane);
        const int gap = (int)(a.vpr - a.data);
        const uint4 *src = reinterpret_cast<const uint4 *>(x) + base - at.row * gap;
#pragma unroll
        for (int u = 0; u < kRowUnroll; ++u) {
            const uint32_t v = at.vec + 32 * u, r = Place::rows_on(a, v);
            in[u] = make_uint4(0u, 0u, 0u, 0u);
            if (32 * u < left && v - r * a.vpr < a.data) in[u] = ld_stream(src + (32 * u - (int)r * gap));
        }
    }
    griddep_launch_dependents();
    uint32_t mine = 0;  // scale of the warp's block number `lane`
    uint8_t *dst = q + base * (FMT == MOE_MX_E4M3 ? 8 : 4);  // element rows follow without gaps
#pragma unroll
    for (int u = 0; u < kRowUnroll; ++u) {
        uint32_t byte;
        const uint2 e = mx_quarter_bf16<FMT>(in[u], byte);
        const uint32_t from = __shfl_sync(MOE_FULL_MASK, byte, 4 * (lane & 7));
        if ((lane >> 3) == u) mine = from;
        if (32 * u < left) mx_store_elements<FMT>(dst, 32 * u, e);
    }
    if (3 * (int)lane >= left) return;  // vector 4 * lane of the warp lies behind the last
    const Place block(a, 4 * lane);
    uint8_t *srow = scales + block.row * a.scale_bytes;
    srow[block.vec >> 2] = (uint8_t)mine;
    if (block.vec + 4 == a.vpr) mx_clear_scales(srow, a.vpr / 4, a.scale_bytes);
}

template <int FMT>
__global__ void __launch_bounds__(kRowThreads)
    mx_dequantize_kernel(const uint8_t *__restrict__ q, const uint8_t *__restrict__ scales,
                         moe_bf16_t *__restrict__ out, const MxRowsArgs a) {
    griddep_wait();
    const uint32_t lane = threadIdx.x & 31;
    const int64_t base =
        (int64_t)blockIdx.x * kRowVecs + (threadIdx.x >> 5) * (32 * kRowUnroll) + lane;
    const int left = (int)min(a.vecs - base, (int64_t)kRowVecs);  // this lane's u runs while 32 u < left
    const Place at(a, lane);
    const uint8_t *qrow = q + at.row * a.row_bytes, *srow = scales + at.row * a.scale_bytes;
    uint2 in[kRowUnroll];
    uint32_t byte[kRowUnroll];
#pragma unroll
    for (int u = 0; u < kRowUnroll; ++u) {
        const uint32_t x = at.vec + 32 * u, r = Place::rows_on(a, x), vec = x - r * a.vpr;
        in[u] = make_uint2(0u, 0u);
        byte[u] = 0;
        if (32 * u < left) {
            const uint8_t *src = qrow + r * a.row_bytes;
            if (FMT == MOE_MX_E4M3)
                in[u] = __ldcs(reinterpret_cast<const uint2 *>(src) + vec);
            else
                in[u].x = __ldcs(reinterpret_cast<const uint32_t *>(src) + vec);
            byte[u] = __ldg(srow + r * a.scale_bytes + (vec >> 2));
        }
    }
    griddep_launch_dependents();
#pragma unroll
    for (int u = 0; u < kRowUnroll; ++u) {
        if (32 * u >= left) continue;
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
        reinterpret_cast<uint4 *>(out)[base + 32 * u] = pack_bf16x8(f);  // rows of out have no padding
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

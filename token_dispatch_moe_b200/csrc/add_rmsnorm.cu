// moe_add_rmsnorm: the residual's addition and the root-mean-square norm in
// front of the router, with the experts' MX rows as a further output.
//
//   h = bf16(x + residual)                         (h = x without a residual)
//   y = bf16(h * (mean(h^2) + eps)^(-1/2) * gain)
//   mx = MX rows of y
//
// h is rounded before the norm: it is what the next layer reads, so the norm
// is the norm of the stored stream and does not depend on whether the addition
// was fused.  The MX rows are made of the rounded y: the gate and the experts
// see one and the same row, and the bits are moe_mx_quantize's on y.
//
// One pass, bound by memory (9.03 bytes a value with every output, e4m3: 65,536
// x 7168 625 to 640 us, 6.7 TB/s; 16,384 x 2048 48 us, 6.3 TB/s): a row's
// threads keep it in registers between the sum of squares and the outputs.
// Rows of more than 1024 values have a block of threads each; narrower ones
// a warp, or half a warp up to 128 values, 8 or 16 rows a block (65,536 x 128:
// 74 us with a block a row).  The sum is fp32: sums of 8, at most 8 of them in
// a thread, then a tree over the threads.
#include "mx.cuh"
#include "rows.cuh"

namespace moe {
namespace {

constexpr int kNormMaxD = 16384;

struct NormArgs {
    const moe_bf16_t *x, *residual, *gain;
    moe_bf16_t *residual_out, *y;
    uint8_t *q, *scales;
    int64_t row_bytes, scale_bytes;
    int32_t data, padded;  // 8-value vectors of a row, without and with its padding
    int64_t T;
    float eps, d, inv_d;
};

// (sum / d + eps)^(-1/2) within one unit of fp32: the quotient by one step on the remainder, the
// root by one Newton step on the hardware's estimate with the residual 1 - v y^2 kept whole.
// Every thread takes it, so the divide and square root sequences would cost (65,536 x 2880, every
// output, e2m1: 288 against 267 us); and an error of the row's factor moves a whole row's
// roundings.
__device__ __forceinline__ float inverse_root(float sum, float d, float inv_d, float eps) {
    float v = sum * inv_d;
    if (v < __int_as_float(0x7f800000)) v = fmaf(fmaf(-v, d, sum), inv_d, v);  // not of inf or NaN
    v += eps;
    const float y = rsqrtf(v);
    const float t = v * y, t_low = fmaf(v, y, -t);
    const float rest = fmaf(-t_low, y, fmaf(-t, y, 1.0f));
    const float z = fmaf(0.5f * y, rest, y);
    return z == z ? z : y;  // v = 0 or infinite: the estimate is the answer
}

// FMT -1: no MX output.  LANES threads of a warp a row (16 or 32; 0: the whole block),
// VPT vectors a thread: thread i of the row has vectors i, i + threads, ...
template <int VPT, int FMT, int LANES>
__global__ void __launch_bounds__(256) add_rmsnorm_kernel(const NormArgs a) {
    __shared__ float part[8];
    griddep_wait();
    const int threads = LANES ? LANES : blockDim.x;
    const int first = LANES ? threadIdx.x % LANES : threadIdx.x;
    const int64_t at = LANES ? (int64_t)blockIdx.x * (256 / LANES) + threadIdx.x / LANES : blockIdx.x;
    // threads of rows behind the last go along (the warp's shuffles) and write nothing
    const bool there = LANES == 0 || at < a.T;
    const int64_t row = there ? at : 0;
    const int data = there ? a.data : 0, padded = there ? a.padded : 0;
    const uint4 *x = reinterpret_cast<const uint4 *>(a.x) + row * a.data;
    const uint4 *r = reinterpret_cast<const uint4 *>(a.residual) + row * a.data;
    uint4 h[VPT], g[VPT];
    {
        uint4 rin[VPT];
#pragma unroll
        for (int u = 0; u < VPT; ++u) {
            const int v = u * threads + first;
            h[u] = rin[u] = make_uint4(0u, 0u, 0u, 0u);
            if (v < data) {
                h[u] = ld_stream(x + v);
                if (a.residual) rin[u] = ld_stream(r + v);
            }
        }
#pragma unroll
        for (int u = 0; u < VPT; ++u) {
            const int v = u * threads + first;
            g[u] = make_uint4(0u, 0u, 0u, 0u);
            if (v < data) g[u] = *(reinterpret_cast<const uint4 *>(a.gain) + v);
        }
        if (a.residual) {
#pragma unroll
            for (int u = 0; u < VPT; ++u) {
                float f[8];
                unpack_bf16x8(h[u], f);
                add_bf16x8(f, rin[u]);
                h[u] = pack_bf16x8(f);
            }
        }
    }
    griddep_launch_dependents();
    float sum = 0.0f;
#pragma unroll
    for (int u = 0; u < VPT; ++u) {
        float f[8], s = 0.0f;
        unpack_bf16x8(h[u], f);
#pragma unroll
        for (int i = 0; i < 8; ++i) s = fmaf(f[i], f[i], s);
        sum += s;
    }
#pragma unroll
    for (int o = LANES == 16 ? 8 : 16; o > 0; o >>= 1)
        sum += __shfl_xor_sync(MOE_FULL_MASK, sum, o);
    if (LANES == 0) {
        const int warps = blockDim.x >> 5;
        if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = sum;
        __syncthreads();
        sum = 0.0f;
        for (int w = 0; w < warps; ++w) sum += part[w];
    }
    const float inv = inverse_root(sum, a.d, a.inv_d, a.eps);
#pragma unroll
    for (int u = 0; u < VPT; ++u) {
        const int v = u * threads + first;
        float f[8], gf[8];
        unpack_bf16x8(h[u], f);
        unpack_bf16x8(g[u], gf);
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = f[i] * gf[i] * inv;  // h * gain is exact in fp32
        uint4 y = pack_bf16x8(f);
        if (v >= data) y = make_uint4(0u, 0u, 0u, 0u);  // 0 * a NaN row's factor is not 0
        if (v < data) {
            if (a.residual_out) reinterpret_cast<uint4 *>(a.residual_out)[row * a.data + v] = h[u];
            if (a.y) reinterpret_cast<uint4 *>(a.y)[row * a.data + v] = y;
        }
        if (FMT >= 0) {
            constexpr int F = FMT < 0 ? 0 : FMT;
            uint32_t byte;
            const uint2 e = mx_quarter_bf16<F>(y, byte);
            uint8_t *srow = a.scales + row * a.scale_bytes;
            if (v < padded) mx_store<F>(a.q + row * a.row_bytes, srow, v, e, byte);
            if (v + 1 == padded) mx_clear_scales(srow, a.padded / 4, a.scale_bytes);
        }
    }
}

template <int FMT>
cudaError_t launch_norm(const NormArgs &a, cudaStream_t s) {
    const int vecs = FMT >= 0 ? a.padded : a.data;
    if (vecs <= 128) {  // rows of up to 1024 values: half a warp or a warp each
        const dim3 block(256), grid((unsigned)((a.T + (vecs <= 16 ? 15 : 7)) / (vecs <= 16 ? 16 : 8)));
        if (vecs <= 16) return launch_pdl(add_rmsnorm_kernel<1, FMT, 16>, grid, block, 0, s, a);
        if (vecs <= 32) return launch_pdl(add_rmsnorm_kernel<1, FMT, 32>, grid, block, 0, s, a);
        if (vecs <= 64) return launch_pdl(add_rmsnorm_kernel<2, FMT, 32>, grid, block, 0, s, a);
        return launch_pdl(add_rmsnorm_kernel<4, FMT, 32>, grid, block, 0, s, a);
    }
    // The fewest vectors a thread, two at least, with which a row fits 256 threads.  Every
    // output, e2m1: 16,384 x 2048 with one 49 us, two 46, eight 51; 65,536 x 7168 with four 627,
    // eight 719; 65,536 x 2880 with two 268, eight 345.  Without MX rows the same but at 7168
    // (four 575, eight 550).
    int vpt = 2;
    while (vpt * 256 < vecs) vpt *= 2;
    const dim3 grid((unsigned)a.T), block((unsigned)(((vecs + vpt - 1) / vpt + 31) / 32 * 32));
    switch (vpt) {
        case 2: return launch_pdl(add_rmsnorm_kernel<2, FMT, 0>, grid, block, 0, s, a);
        case 4: return launch_pdl(add_rmsnorm_kernel<4, FMT, 0>, grid, block, 0, s, a);
        default: return launch_pdl(add_rmsnorm_kernel<8, FMT, 0>, grid, block, 0, s, a);
    }
}

}  // namespace
}  // namespace moe

extern "C" moe_status moe_add_rmsnorm(const moe_bf16_t *x, const moe_bf16_t *residual,
                                      const moe_bf16_t *gain, float eps, int64_t T, int32_t d,
                                      moe_bf16_t *residual_out, moe_bf16_t *y, int32_t format,
                                      uint8_t *q, uint8_t *scales, moe_stream_t stream) {
    using namespace moe;
    if (T < 0 || d < 8 || d % 8 != 0 || !(eps >= 0.0f)) return MOE_ERR_INVALID_ARG;
    if (q && (!mx_format_ok(format) || !scales)) return MOE_ERR_INVALID_ARG;
    if (!q && scales) return MOE_ERR_INVALID_ARG;
    if (T == 0) return MOE_OK;
    if (!x || !gain || (!residual_out && !y && !q) || (y && y == residual_out)) return MOE_ERR_INVALID_ARG;
    for (const void *p : {(const void *)x, (const void *)residual, (const void *)gain,
                          (const void *)residual_out, (const void *)y})
        if (!aligned16(p)) return MOE_ERR_INVALID_ARG;
    if (!mx_aligned(q, scales)) return MOE_ERR_INVALID_ARG;
    if (d > kNormMaxD || T >= (int64_t)INT32_MAX) return MOE_ERR_UNSUPPORTED;
    NormArgs a;
    a.x = x;
    a.residual = residual;
    a.gain = gain;
    a.residual_out = residual_out;
    a.y = y;
    a.q = q;
    a.scales = scales;
    a.row_bytes = q ? mx_row_bytes(d, format) : 0;
    a.scale_bytes = q ? mx_scale_bytes(d) : 0;
    a.data = d / 8;
    a.padded = mx_padded(d) / 8;
    a.T = T;
    a.eps = eps;
    a.d = (float)d;
    a.inv_d = 1.0f / (float)d;
    const cudaStream_t s = as_cuda(stream);
    const cudaError_t e = !q                        ? launch_norm<-1>(a, s)
                          : format == MOE_MX_E4M3 ? launch_norm<MOE_MX_E4M3>(a, s)
                                                  : launch_norm<MOE_MX_E2M1>(a, s);
    if (e != cudaSuccess) {
        cudaGetLastError();
        return MOE_ERR_CUDA;
    }
    return launch_status();
}

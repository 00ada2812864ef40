// moe_expert_gate_up_mx and moe_expert_down_mx: the routed experts' SwiGLU FFN
// as two grouped products on microscaled operands, over ragged expert blocks.
//
//   gate_up: h[r] = MX(act(xs[r] . W1[e]^T + b1[e], xs[r] . W3[e]^T + b3[e]))
//   down:    y[r] = bf16(h[r] . W2[e]^T + b2[e])
// e is the expert whose block [offsets[e], offsets[e+1]) holds row r; blocks
// start anywhere.  Activations (act) as moe_expert_gate_up's.
//
// sm_100a design.  The block-scaled tcgen05 MMA (mxf8f6f4: e4m3 and e2m1
// operands mix freely, a power-of-two scale per row and 32 K values) runs with
// the operands swapped: the weights are the 128-row operand, the tokens the N
// columns.  N goes in steps of 8, so a tile fits a ragged block to 8 rows (one
// decoded token costs 8 columns, not 128 rows), and a block's tiles share its
// rows evenly.
//
// A persistent grid walks tiles (block part, feature tile), features fastest:
// CTAs that run together share their tokens, and an expert's weights stay in
// L2 over its parts.  Roles of a CTA:
//   warp 0     TMA: weight and token tiles of 128 K values into a stage ring;
//              scale rows, 16 bytes (512 K values) at a time, into a second ring
//   warps 2, 3 turn raw scale rows [row][16 bytes] into the tiles that TMEM
//              wants (32 x 16 bytes, four rows' words side by side)
//   warp 1     one thread: scale tiles to TMEM (tcgen05.cp), four MMAs a stage
//   warps 4-7  epilogue: TMEM -> shared memory, transposed to token-major; each
//              thread then takes 8 features of a token: bias, activation, MX
//              block (four lanes) or bf16, and one vector store
// Two accumulators: the epilogue of a tile overlaps the next one's products.
// A gate_up tile has ft gate rows and the ft up rows of the same features in
// its 128 rows; they meet in the epilogue's shared memory.
// Every wait is bounded, as in the bf16 kernels.
#include "mx.cuh"
#include "tc.cuh"

namespace moe {
namespace {

constexpr int kXThreads = 256;
constexpr int kXBK = 128;           // K values of a stage
constexpr int kXSuper = 4;          // stages that one load of scales covers
constexpr int kXMaxE = 4096;
constexpr int kXEpiThreads = 128;
constexpr int kXChunk = 32;         // token columns the epilogue turns at a time
constexpr int kXPitch = 132;        // floats of a staged token: 16-byte aligned, off the banks
constexpr float kXOaiAlpha = 1.702f;
constexpr float kXOaiLimit = 7.0f;

struct MxFfnArgs {
    const int32_t *offsets;  // [E+1], ascending
    const float *bias0;      // gate_up: b1 [E][N]; down: b2 [E][N]
    const float *bias1;      // gate_up: b3 [E][N]
    moe_bf16_t *y;           // down: [rows][N]
    uint8_t *hq, *hs;        // gate_up: MX rows of N values
    int64_t h_row, h_scale;  // bytes of those rows
    int32_t *status;
    int64_t rows;
    int E, N, ft, f_tiles, cap, acc_cols, box, num_kb, stages, slots, tmem_cols, act, h_fmt;
    uint32_t w_count, x_count;  // bytes a barrier counts for a row of a stage: 4-bit values packed
    uint32_t a_bytes, stage_bytes, raw_b, tiled_b, slot_bytes, idesc;
    uint32_t ring, sf, stg, bars, tables;  // offsets in shared memory
};

// As in the bf16 kernel's epilogue: fast exponential and quotient, about 1e-6
// relative, far below the rounding to 8 bits.
__device__ __forceinline__ float activate(float g, float u, int act) {
    if (act == MOE_ACT_SWIGLU_OAI) {
        const float gc = fminf(g, kXOaiLimit);
        const float uc = fminf(fmaxf(u, -kXOaiLimit), kXOaiLimit);
        return __fdividef(gc, 1.0f + __expf(-kXOaiAlpha * gc)) * (uc + 1.0f);
    }
    return __fdividef(g, 1.0f + __expf(-g)) * u;
}

struct Tile {
    int e, row0, n, f0;
};

// Tile t of the walk: its expert by bisection of the part counts before each
// expert, its share of the block's rows (a multiple of 8 but for the last).
__device__ __forceinline__ Tile tile_at(const MxFfnArgs &a, const int32_t *off,
                                        const int32_t *parts, int64_t t) {
    const int p = (int)(t / a.f_tiles);
    int lo = 0, hi = a.E - 1;
    while (lo < hi) {  // the last e with parts[e] <= p
        const int mid = (lo + hi + 1) >> 1;
        if (parts[mid] <= p) lo = mid; else hi = mid - 1;
    }
    const int m = off[lo + 1] - off[lo], of = parts[lo + 1] - parts[lo];
    const int share = ((m + of - 1) / of + 7) & ~7;  // <= cap, so no part is empty
    Tile w;
    w.e = lo;
    w.row0 = off[lo] + (p - parts[lo]) * share;
    w.n = min(share, off[lo + 1] - w.row0);
    w.f0 = (int)(t - (int64_t)p * a.f_tiles) * a.ft;
    return w;
}

__device__ __forceinline__ void epi_sync() {
    asm volatile("bar.sync 1, %0;" ::"n"(kXEpiThreads) : "memory");
}

template <bool GATE_UP>
__global__ void __launch_bounds__(kXThreads, 1)
    expert_mx_kernel(const __grid_constant__ CUtensorMap map_w0,
                     const __grid_constant__ CUtensorMap map_w1,
                     const __grid_constant__ CUtensorMap map_w0s,
                     const __grid_constant__ CUtensorMap map_w1s,
                     const __grid_constant__ CUtensorMap map_x,
                     const __grid_constant__ CUtensorMap map_xs, const MxFfnArgs a) {
    extern __shared__ __align__(16) uint8_t smem_mx[];
    __shared__ int abort_s;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t raw = smem_u32(smem_mx);
    const uint32_t base = (raw + 1023u) & ~1023u;
    uint8_t *const gbase = smem_mx + (base - raw);
    const int S = a.stages, R = a.slots;
    const uint32_t bar0 = base + a.bars;
    auto full_bar = [&](int s) { return bar0 + 8u * s; };
    auto empty_bar = [&](int s) { return bar0 + 8u * (S + s); };
    auto raw_bar = [&](int r) { return bar0 + 8u * (2 * S + r); };
    auto ready_bar = [&](int r) { return bar0 + 8u * (2 * S + R + r); };
    auto free_bar = [&](int r) { return bar0 + 8u * (2 * S + 2 * R + r); };
    auto tfull_bar = [&](int b) { return bar0 + 8u * (2 * S + 3 * R + b); };
    auto tempty_bar = [&](int b) { return bar0 + 8u * (2 * S + 3 * R + 2 + b); };
    const uint32_t drain_bar = bar0 + 8u * (2 * S + 3 * R + 4);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(gbase + a.bars + 8u * (2 * S + 3 * R + 5));
    int32_t *off = reinterpret_cast<int32_t *>(gbase + a.tables);
    int32_t *parts = off + a.E + 1;

    if (threadIdx.x == 0) {
        abort_s = 0;
        for (int s = 0; s < S; ++s) {
            mbar_init(full_bar(s), 1);
            mbar_init(empty_bar(s), 1);
        }
        for (int r = 0; r < R; ++r) {
            mbar_init(raw_bar(r), 1);
            mbar_init(ready_bar(r), 2);  // one arrival per turning warp
            mbar_init(free_bar(r), 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(tfull_bar(b), 1);
            mbar_init(tempty_bar(b), 4);  // one arrival per epilogue warp
        }
        mbar_init(drain_bar, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 2) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                         smem_u32(tmem_slot)),
                     "r"(a.tmem_cols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    griddep_wait();  // offsets and tokens come from the kernels before this one
    for (int i = threadIdx.x; i <= a.E; i += blockDim.x) off[i] = __ldg(a.offsets + i);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem_base = *tmem_slot;
    // Blocks that descend or leave the buffers: nothing runs.
    bool bad = threadIdx.x == 0 && (off[0] < 0 || (int64_t)off[a.E] > a.rows);
    for (int i = threadIdx.x; i < a.E; i += blockDim.x) bad |= off[i] > off[i + 1];
    const bool any_bad = __syncthreads_or(bad);
    if (warp == 0 && !any_bad) {  // running count of parts
        int before = 0;
        for (int e0 = 0; e0 < a.E; e0 += 32) {
            const int e = e0 + lane;
            int v = e < a.E ? (off[e + 1] - off[e] + a.cap - 1) / a.cap : 0;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int w = __shfl_up_sync(MOE_FULL_MASK, v, o);
                if (lane >= o) v += w;
            }
            if (e < a.E) parts[e + 1] = before + v;
            before += __shfl_sync(MOE_FULL_MASK, v, 31);
        }
        if (lane == 0) parts[0] = 0;
    }
    __syncthreads();
    if (any_bad && threadIdx.x == 0 && blockIdx.x == 0) report(a.status, MOE_ERR_DEVICE_INDEX);
    const int64_t num_tiles = any_bad ? 0 : (int64_t)parts[a.E] * a.f_tiles;
    volatile int *abort_v = &abort_s;
    griddep_launch_dependents();

    if (warp == 0 && lane == 0) {
        uint32_t it = 0, sit = 0;
        for (int64_t t = blockIdx.x; t < num_tiles && !*abort_v; t += gridDim.x) {
            const Tile w = tile_at(a, off, parts, t);
            const int boxes = (w.n + a.box - 1) / a.box;
            const int wrow = w.e * a.N + w.f0;
            for (int kb = 0; kb < a.num_kb; ++kb, ++it) {
                if (kb % kXSuper == 0) {
                    const int r = (int)(sit % (uint32_t)R);
                    if (!mbar_wait(free_bar(r), ((sit / (uint32_t)R) & 1u) ^ 1u, a.status)) {
                        *abort_v = 1;
                        break;
                    }
                    const uint32_t sl = base + a.sf + (uint32_t)r * a.slot_bytes;
                    const int x = kb / kXSuper * 16;
                    mbar_arrive_expect_tx(raw_bar(r),
                                          (uint32_t)((GATE_UP ? 2 : 1) * a.ft) * 16u +
                                              (uint32_t)(boxes * a.box) * 16u);
                    tma_load_2d(sl, &map_w0s, raw_bar(r), x, wrow);
                    if (GATE_UP)
                        tma_load_2d(sl + (uint32_t)a.ft * 16u, &map_w1s, raw_bar(r), x, wrow);
                    for (int i = 0; i < boxes; ++i)
                        tma_load_2d(sl + 2048u + (uint32_t)(i * a.box) * 16u, &map_xs, raw_bar(r),
                                    x, w.row0 + i * a.box);
                    ++sit;
                }
                const int s = (int)(it % (uint32_t)S);
                if (!mbar_wait(empty_bar(s), ((it / (uint32_t)S) & 1u) ^ 1u, a.status)) {
                    *abort_v = 1;
                    break;
                }
                const uint32_t st = base + a.ring + (uint32_t)s * a.stage_bytes;
                mbar_arrive_expect_tx(full_bar(s),
                                      (uint32_t)((GATE_UP ? 2 : 1) * a.ft) * a.w_count +
                                          (uint32_t)(boxes * a.box) * a.x_count);
                tma_load_2d(st, &map_w0, full_bar(s), kb * kXBK, wrow);
                if (GATE_UP)
                    tma_load_2d(st + (uint32_t)a.ft * 128u, &map_w1, full_bar(s), kb * kXBK, wrow);
                for (int i = 0; i < boxes; ++i)
                    tma_load_2d(st + a.a_bytes + (uint32_t)(i * a.box) * 128u, &map_x, full_bar(s),
                                kb * kXBK, w.row0 + i * a.box);
            }
        }
        // Drain: the last loads into every stage and slot have landed before the CTA exits.
        for (uint32_t i = it > (uint32_t)S ? it - (uint32_t)S : 0u; i < it; ++i)
            if (!mbar_wait(full_bar((int)(i % (uint32_t)S)), (i / (uint32_t)S) & 1u, a.status))
                break;
        for (uint32_t i = sit > (uint32_t)R ? sit - (uint32_t)R : 0u; i < sit; ++i)
            if (!mbar_wait(raw_bar((int)(i % (uint32_t)R)), (i / (uint32_t)R) & 1u, a.status))
                break;
    } else if (warp == 1 && lane == 0) {
        uint32_t it = 0, sit = 0, j = 0;
        const uint32_t sf_col = tmem_base + 2u * (uint32_t)a.acc_cols;
        for (int64_t t = blockIdx.x; t < num_tiles && !*abort_v; t += gridDim.x, ++j) {
            const Tile w = tile_at(a, off, parts, t);
            const uint32_t n8 = (uint32_t)(w.n + 7) & ~7u;
            const uint32_t b = j & 1u;
            if (!mbar_wait(tempty_bar((int)b), ((j >> 1) & 1u) ^ 1u, a.status)) {
                *abort_v = 1;
                break;
            }
            tc_fence_after();
            const uint32_t acc = tmem_base + b * (uint32_t)a.acc_cols;
            for (int kb = 0; kb < a.num_kb; ++kb, ++it) {
                const int r = (int)(sit % (uint32_t)R);
                if (kb % kXSuper == 0 &&
                    !mbar_wait(ready_bar(r), (sit / (uint32_t)R) & 1u, a.status)) {
                    *abort_v = 1;
                    break;
                }
                const int s = (int)(it % (uint32_t)S);
                if (!mbar_wait(full_bar(s), (it / (uint32_t)S) & 1u, a.status)) {
                    *abort_v = 1;
                    break;
                }
                tc_fence_after();
                const uint32_t q = (uint32_t)(kb % kXSuper);
                const uint32_t sl = base + a.sf + (uint32_t)r * a.slot_bytes + 2048u + a.raw_b;
                const uint32_t sfa = sf_col + 16u * (q & 1u), sfb = sfa + 4u;
                tmem_cp_scales(sfa, sl + q * 512u);
                tmem_cp_scales(sfb, sl + 2048u + q * a.tiled_b);
                if (n8 > 128u) tmem_cp_scales(sfb + 4u, sl + 2048u + q * a.tiled_b + 512u);
                const uint32_t st = base + a.ring + (uint32_t)s * a.stage_bytes;
#pragma unroll
                for (uint32_t k = 0; k < 4; ++k)
                    umma_mx(acc, sw128_desc(st + 32u * k), sw128_desc(st + a.a_bytes + 32u * k),
                            mx_idesc_at(a.idesc, n8, k), sfa, sfb, (kb > 0 || k > 0) ? 1u : 0u);
                umma_commit(empty_bar(s));
                if (q == kXSuper - 1 || kb + 1 == a.num_kb) {
                    umma_commit(free_bar(r));
                    ++sit;
                }
            }
            if (*abort_v) break;
            umma_commit(tfull_bar((int)b));
        }
        // Every MMA and copy issued above has completed before the columns are freed.
        umma_commit(drain_bar);
        mbar_wait(drain_bar, 0u, a.status);
    } else if (warp == 2 || warp == 3) {
        uint32_t sit = 0;
        const int supers = (a.num_kb + kXSuper - 1) / kXSuper;
        bool ok = true;
        for (int64_t t = blockIdx.x; t < num_tiles && ok; t += gridDim.x) {
            const Tile w = tile_at(a, off, parts, t);
            // 32-row pieces in which each quarter-warp's 8 rows lie 32 rows apart, so that
            // a warp's 32 words fill 128 contiguous bytes of a tile.
            const int pa = 4, pb = (w.n + 127) / 128 * 4;
            for (int c = 0; c < supers; ++c, ++sit) {
                const int r = (int)(sit % (uint32_t)R);
                ok = __all_sync(MOE_FULL_MASK,
                                !*abort_v &&
                                    mbar_wait(raw_bar(r), (sit / (uint32_t)R) & 1u, a.status));
                if (!ok) {
                    if (lane == 0) *abort_v = 1;
                    break;
                }
                uint8_t *sl = gbase + a.sf + (size_t)r * a.slot_bytes;
                for (int i = warp - 2; i < pa + pb; i += 2) {
                    const bool is_b = i >= pa;
                    const int p = is_b ? i - pa : i;
                    // row in its group of 128, and its place in the 512-byte tile
                    const int row = 8 * (p & 3) + (lane & 7) + 32 * (lane >> 3);
                    const int g = p >> 2;
                    if (is_b && g * 128 + row >= (int)(a.raw_b >> 4)) continue;
                    const uint4 v = *reinterpret_cast<const uint4 *>(
                        sl + (is_b ? 2048 : 0) + (g * 128 + row) * 16);
                    uint8_t *dst = sl + 2048 + a.raw_b + (is_b ? 2048 + g * 512 : 0) +
                                   (row & 31) * 16 + (row >> 5) * 4;
                    const uint32_t step = is_b ? a.tiled_b : 512u;
                    *reinterpret_cast<uint32_t *>(dst) = v.x;
                    *reinterpret_cast<uint32_t *>(dst + step) = v.y;
                    *reinterpret_cast<uint32_t *>(dst + 2 * step) = v.z;
                    *reinterpret_cast<uint32_t *>(dst + 3 * step) = v.w;
                }
                fence_async_shared();
                __syncwarp();
                if (lane == 0) mbar_arrive(ready_bar(r));
            }
        }
    } else if (warp >= 4) {
        const int q = warp & 3;
        float *stg = reinterpret_cast<float *>(gbase + a.stg);
        uint32_t j = 0;
        for (int64_t t = blockIdx.x; t < num_tiles; t += gridDim.x, ++j) {
            const Tile w = tile_at(a, off, parts, t);
            const uint32_t b = j & 1u;
            // Every epilogue thread goes by the same answer: they meet at the barriers below.
            int ok = !*abort_v && mbar_wait(tfull_bar((int)b), (j >> 1) & 1u, a.status);
            asm volatile(
                "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %0, 0;\n\t"
                "barrier.red.and.pred q, 1, %1, p;\n\tselp.b32 %0, 1, 0, q;\n\t}"
                : "+r"(ok)
                : "n"(kXEpiThreads)
                : "memory");
            if (!ok) {
                if (lane == 0) *abort_v = 1;
                break;
            }
            tc_fence_after();
            const uint32_t trow =
                tmem_base + b * (uint32_t)a.acc_cols + ((uint32_t)(q * 32) << 16);
            const int64_t brow = (int64_t)w.e * a.N;
            // 8-feature groups of a token; gate_up's last tile adds those of the row's padding.
            const int own = a.ft >> 3;
            const int padded = (a.N + kMxPad - 1) / kMxPad * kMxPad;
            const int groups = GATE_UP && w.f0 + a.ft >= a.N ? (padded - w.f0) >> 3 : own;
            for (int c0 = 0; c0 < w.n; c0 += kXChunk) {
                uint32_t v[kXChunk];
                tmem_ld32(trow + (uint32_t)c0, v);
                if (c0 + kXChunk >= w.n) {  // the accumulator is free for the tile after next
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(tempty_bar((int)b));
                }
                epi_sync();  // the last chunk's readers are done
#pragma unroll
                for (int i = 0; i < kXChunk; ++i)
                    stg[i * kXPitch + 32 * q + lane] = __uint_as_float(v[i]);
                epi_sync();
                const int items = min(kXChunk, w.n - c0) * groups;
                for (int i0 = 32 * q; i0 < items; i0 += kXEpiThreads) {
                    const int i = i0 + lane;
                    const int tok = i / groups, grp = i - tok * groups;
                    const int f = w.f0 + 8 * grp;
                    const bool there = i < items, real = there && grp < own && f < a.N;
                    const int64_t row = (int64_t)w.row0 + c0 + tok;
                    float o[8];
#pragma unroll
                    for (int k = 0; k < 8; ++k) o[k] = 0.0f;
                    if (real) {
                        const float *src = stg + tok * kXPitch + 8 * grp;
#pragma unroll
                        for (int k = 0; k < 8; k += 4) {
                            const float4 g = *reinterpret_cast<const float4 *>(src + k);
                            float4 b0 = make_float4(0.f, 0.f, 0.f, 0.f), b1 = b0;
                            if (a.bias0)
                                b0 = __ldg(reinterpret_cast<const float4 *>(a.bias0 + brow + f + k));
                            o[k] = g.x + b0.x;
                            o[k + 1] = g.y + b0.y;
                            o[k + 2] = g.z + b0.z;
                            o[k + 3] = g.w + b0.w;
                            if (GATE_UP) {
                                const float4 u =
                                    *reinterpret_cast<const float4 *>(src + a.ft + k);
                                if (a.bias1)
                                    b1 = __ldg(
                                        reinterpret_cast<const float4 *>(a.bias1 + brow + f + k));
                                o[k] = activate(o[k], u.x + b1.x, a.act);
                                o[k + 1] = activate(o[k + 1], u.y + b1.y, a.act);
                                o[k + 2] = activate(o[k + 2], u.z + b1.z, a.act);
                                o[k + 3] = activate(o[k + 3], u.w + b1.w, a.act);
                            }
                        }
                    }
                    if (GATE_UP) {
                        uint32_t byte;
                        uint8_t *srow = a.hs + row * a.h_scale;
                        if (a.h_fmt == MOE_MX_E4M3) {
                            const uint2 e = mx_quarter<MOE_MX_E4M3>(o, byte);
                            if (there)
                                mx_store<MOE_MX_E4M3>(a.hq + row * a.h_row, srow, f >> 3, e, byte);
                        } else {
                            const uint2 e = mx_quarter<MOE_MX_E2M1>(o, byte);
                            if (there)
                                mx_store<MOE_MX_E2M1>(a.hq + row * a.h_row, srow, f >> 3, e, byte);
                        }
                        if (there && f + 8 == padded)
                            for (int64_t k = padded / kMxBlock; k < a.h_scale; ++k) srow[k] = 0;
                    } else if (real) {
                        uint32_t p[4];
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const __nv_bfloat162 two = __floats2bfloat162_rn(o[2 * k], o[2 * k + 1]);
                            p[k] = *reinterpret_cast<const uint32_t *>(&two);
                        }
                        *reinterpret_cast<uint4 *>(a.y + row * a.N + f) =
                            make_uint4(p[0], p[1], p[2], p[3]);
                    }
                }
            }
        }
    }

    tc_fence_before();
    __syncthreads();
    if (warp == 2) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem_base),
                     "r"(a.tmem_cols)
                     : "memory");
    }
}

bool operand_map(CUtensorMap *m, const void *q, int64_t rows, int32_t K, int32_t format, int box) {
    return format == MOE_MX_E4M3 ? make_byte_map(m, q, rows, mx_padded(K), box, 128)
                                 : make_nibble_map(m, q, rows, mx_padded(K), box);
}

template <bool GATE_UP>
moe_status launch_expert_mx(const uint8_t *xq, const uint8_t *xs, int32_t x_fmt, const uint8_t *w0,
                            const uint8_t *w0s, const uint8_t *w1, const uint8_t *w1s,
                            int32_t w_fmt, int32_t K, MxFfnArgs a, moe_stream_t stream) {
    // Token columns of a tile: enough for four times an expert's share of the rows, so that few
    // experts need a second part (which reads the weights again); a narrow tile leaves shared
    // memory to more weight stages.
    const int64_t share = 4 * ((a.rows + a.E - 1) / a.E);
    a.cap = share <= 32 ? 32 : share <= 64 ? 64 : share <= 128 ? 128 : 224;
    a.box = a.cap <= 64 ? 8 : 32;
    a.acc_cols = a.cap;
    a.ft = GATE_UP ? 64 : 128;
    a.f_tiles = (a.N + a.ft - 1) / a.ft;
    a.num_kb = mx_padded(K) / kXBK;
    const int a_rows = (GATE_UP ? 2 : 1) * a.ft;
    a.a_bytes = (uint32_t)a_rows * 128u;
    a.stage_bytes = a.a_bytes + (uint32_t)a.cap * 128u;
    a.raw_b = (uint32_t)a.cap * 16u;
    a.tiled_b = a.cap > 128 ? 1024u : 512u;
    a.slot_bytes = 2048u + a.raw_b + 2048u + 4u * a.tiled_b;
    a.slots = 2;
    a.w_count = w_fmt == MOE_MX_E4M3 ? 128u : 64u;
    a.x_count = x_fmt == MOE_MX_E4M3 ? 128u : 64u;
    a.idesc = mx_idesc(w_fmt == MOE_MX_E4M3 ? 0u : 5u, x_fmt == MOE_MX_E4M3 ? 0u : 5u, 128u);
    int cols = 32;
    while (cols < 2 * a.acc_cols + 32) cols *= 2;
    a.tmem_cols = cols;
    int dev = 0, max_smem = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&max_smem, cudaDevAttrMaxSharedMemoryPerBlockOptin, dev) !=
            cudaSuccess) {
        cudaGetLastError();
        return MOE_ERR_CUDA;
    }
    const uint32_t stg = kXChunk * kXPitch * 4, bars = 512;
    const uint32_t tables = ((uint32_t)(2 * (a.E + 1)) * 4u + 15u) / 16u * 16u;
    // alignment slack, static shared memory
    const int64_t rest = (int64_t)max_smem - 1024 - 64 - stg - bars - tables -
                         (int64_t)a.slots * a.slot_bytes;
    int64_t stages = rest / a.stage_bytes;
    if (stages > 12) stages = 12;
    if (stages < 2) return MOE_ERR_UNSUPPORTED;
    a.stages = (int)stages;
    a.ring = 0;
    a.sf = (uint32_t)a.stages * a.stage_bytes;
    a.stg = a.sf + (uint32_t)a.slots * a.slot_bytes;
    a.bars = a.stg + stg;
    a.tables = a.bars + bars;
    const size_t smem = 1024 + (size_t)a.tables + tables;
    CUtensorMap mw0, mw1, mw0s, mw1s, mx, mxs;
    const int64_t wrows = (int64_t)a.E * a.N;
    const int64_t sp = mx_scale_bytes(K);
    if (!operand_map(&mw0, w0, wrows, K, w_fmt, a.ft) ||
        !operand_map(&mw1, GATE_UP ? w1 : w0, wrows, K, w_fmt, a.ft) ||
        !make_byte_map(&mw0s, w0s, wrows, sp, a.ft, 16) ||
        !make_byte_map(&mw1s, GATE_UP ? w1s : w0s, wrows, sp, a.ft, 16) ||
        !operand_map(&mx, xq, a.rows, K, x_fmt, a.box) ||
        !make_byte_map(&mxs, xs, a.rows, sp, a.box, 16))
        return MOE_ERR_CUDA;
    if (cudaFuncSetAttribute(expert_mx_kernel<GATE_UP>,
                             cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) !=
        cudaSuccess) {
        cudaGetLastError();
        return MOE_ERR_CUDA;
    }
    // Never more CTAs than the most tiles these rows can make.
    const int64_t parts = a.rows / a.cap + (a.rows < a.E ? a.rows : a.E);
    const int64_t most = parts * a.f_tiles;
    const int64_t grid = most < sm_count() ? most : sm_count();
    if (launch_pdl(expert_mx_kernel<GATE_UP>, dim3((unsigned)grid), dim3(kXThreads), smem,
                   as_cuda(stream), mw0, mw1, mw0s, mw1s, mx, mxs, a) != cudaSuccess) {
        cudaGetLastError();
        return MOE_ERR_CUDA;
    }
    return launch_status();
}

moe_status check_ffn_mx(const void *x, const void *xs, int32_t x_fmt, int32_t w_fmt,
                        const int32_t *offsets, int32_t E, int32_t d, int32_t F, int64_t rows) {
    if (E < 1 || E > kXMaxE || d < 8 || d % 8 != 0 || F < 8 || F % 8 != 0 || rows < 0 ||
        !mx_format_ok(x_fmt) || !mx_format_ok(w_fmt))
        return MOE_ERR_INVALID_ARG;
    if (rows == 0) return MOE_OK;
    if (!x || !xs || !offsets || !mx_aligned(x, xs)) return MOE_ERR_INVALID_ARG;
    if (d > kMxMaxK || F > kMxMaxK || rows >= (int64_t)INT32_MAX - 512 ||
        (int64_t)E * (d > F ? d : F) >= (int64_t)INT32_MAX - 512)
        return MOE_ERR_UNSUPPORTED;
    return MOE_OK;
}

}  // namespace
}  // namespace moe

extern "C" moe_status moe_expert_gate_up_mx(const uint8_t *xq, const uint8_t *xs, int32_t x_format,
                                            const int32_t *offsets, const uint8_t *w1,
                                            const uint8_t *w1_scales, const uint8_t *w3,
                                            const uint8_t *w3_scales, int32_t w_format,
                                            const float *b1, const float *b3, int32_t E, int32_t d,
                                            int32_t F, int64_t rows, int32_t act, uint8_t *h,
                                            uint8_t *h_scales, int32_t h_format, int32_t *d_status,
                                            moe_stream_t stream) {
    using namespace moe;
    const moe_status st = check_ffn_mx(xq, xs, x_format, w_format, offsets, E, d, F, rows);
    if (st != MOE_OK) return st;
    if ((act != MOE_ACT_SWIGLU && act != MOE_ACT_SWIGLU_OAI) || !mx_format_ok(h_format))
        return MOE_ERR_INVALID_ARG;
    if (rows == 0) return MOE_OK;
    if (!w1 || !w1_scales || !w3 || !w3_scales || !h || !h_scales || !mx_aligned(w1, w1_scales) ||
        !mx_aligned(w3, w3_scales) || !mx_aligned(h, h_scales) || !aligned16(b1) || !aligned16(b3))
        return MOE_ERR_INVALID_ARG;
    MxFfnArgs a{};
    a.offsets = offsets;
    a.bias0 = b1;
    a.bias1 = b3;
    a.hq = h;
    a.hs = h_scales;
    a.h_row = mx_row_bytes(F, h_format);
    a.h_scale = mx_scale_bytes(F);
    a.h_fmt = h_format;
    a.status = d_status;
    a.rows = rows;
    a.E = E;
    a.N = F;
    a.act = act;
    return launch_expert_mx<true>(xq, xs, x_format, w1, w1_scales, w3, w3_scales, w_format, d, a,
                                  stream);
}

extern "C" moe_status moe_expert_down_mx(const uint8_t *h, const uint8_t *h_scales,
                                         int32_t h_format, const int32_t *offsets,
                                         const uint8_t *w2, const uint8_t *w2_scales,
                                         int32_t w_format, const float *b2, int32_t E, int32_t d,
                                         int32_t F, int64_t rows, moe_bf16_t *y, int32_t *d_status,
                                         moe_stream_t stream) {
    using namespace moe;
    const moe_status st = check_ffn_mx(h, h_scales, h_format, w_format, offsets, E, d, F, rows);
    if (st != MOE_OK || rows == 0) return st;
    if (!w2 || !w2_scales || !y || !mx_aligned(w2, w2_scales) || !aligned16(y) || !aligned16(b2))
        return MOE_ERR_INVALID_ARG;
    MxFfnArgs a{};
    a.offsets = offsets;
    a.bias0 = b2;
    a.y = y;
    a.status = d_status;
    a.rows = rows;
    a.E = E;
    a.N = d;
    a.act = MOE_ACT_SWIGLU;
    return launch_expert_mx<false>(h, h_scales, h_format, w2, w2_scales, nullptr, nullptr, w_format,
                                   F, a, stream);
}

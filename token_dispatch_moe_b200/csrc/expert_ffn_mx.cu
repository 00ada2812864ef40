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
//   warps 4-11 epilogue: TMEM -> shared memory, transposed to token-major; each
//              thread then takes 8 features of a token: bias, activation, MX
//              block (four lanes) or bf16, and one vector store
// Two accumulators: the epilogue of a tile overlaps the next one's products.
// A gate_up tile has ft gate rows and the ft up rows of the same features in
// its 128 rows; they meet in the epilogue's shared memory.
// Every wait is bounded, as in the bf16 kernels.
#include "mx.cuh"
#include "rows.cuh"
#include "tc.cuh"

namespace moe {
namespace {

constexpr int kXThreads = 384;
constexpr int kXBK = 128;           // K values of a stage
constexpr int kXSuper = 4;          // stages that one load of scales covers
constexpr int kXMaxE = 4096;
constexpr int kXEpiThreads = 256;
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
__device__ __forceinline__ void activate8(float (&g)[8], const float (&u)[8], int act) {
    if (act == MOE_ACT_SWIGLU_OAI) {
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const float gc = fminf(g[k], kXOaiLimit);
            const float uc = fminf(fmaxf(u[k], -kXOaiLimit), kXOaiLimit);
            g[k] = __fdividef(gc, 1.0f + __expf(-kXOaiAlpha * gc)) * (uc + 1.0f);
        }
    } else {
#pragma unroll
        for (int k = 0; k < 8; ++k) g[k] = __fdividef(g[k], 1.0f + __expf(-g[k])) * u[k];
    }
}

__device__ __forceinline__ void load8(const float *p, float (&v)[8]) {
    const float4 x = *reinterpret_cast<const float4 *>(p);
    const float4 y = *reinterpret_cast<const float4 *>(p + 4);
    v[0] = x.x, v[1] = x.y, v[2] = x.z, v[3] = x.w;
    v[4] = y.x, v[5] = y.y, v[6] = y.z, v[7] = y.w;
}

// 8 features of a row of h (four neighbouring lanes hold a block).
__device__ __forceinline__ void store_h(const MxFfnArgs &a, int64_t row, int f, const float (&o)[8],
                                        bool there) {
    uint8_t *qrow = a.hq + row * a.h_row, *srow = a.hs + row * a.h_scale;
    uint32_t byte;
    if (a.h_fmt == MOE_MX_E4M3) {
        const uint2 e = mx_quarter<MOE_MX_E4M3>(o, byte);
        if (there) mx_store<MOE_MX_E4M3>(qrow, srow, f >> 3, e, byte);
    } else {
        const uint2 e = mx_quarter<MOE_MX_E2M1>(o, byte);
        if (there) mx_store<MOE_MX_E2M1>(qrow, srow, f >> 3, e, byte);
    }
}

// Raw scale rows (16 bytes: four stages' words) to the four stages' tiles, `step` bytes apart:
// every second of `pieces` 32-row pieces, rows below `rows`.
__device__ __forceinline__ void turn_scales(const uint8_t *raw, uint8_t *tiles, int step, int first,
                                            int pieces, int rows, int row0, int dst0) {
    for (int i = first; i < pieces; i += 2) {
        const int r = (i >> 2) * 128 + 8 * (i & 3) + row0;
        if (r >= rows) continue;
        const uint4 v = *reinterpret_cast<const uint4 *>(raw + r * 16);
        uint8_t *dst = tiles + (i >> 2) * 512 + (i & 3) * 128 + dst0;
        *reinterpret_cast<uint32_t *>(dst) = v.x;
        *reinterpret_cast<uint32_t *>(dst + step) = v.y;
        *reinterpret_cast<uint32_t *>(dst + 2 * step) = v.z;
        *reinterpret_cast<uint32_t *>(dst + 3 * step) = v.w;
    }
}

struct Tile {
    int e, row0, n, f0;
};

// The tiles of one CTA in order: tile t = part * f_tiles + feature tile, t = blockIdx.x,
// + gridDim.x, ...  Every role of the CTA walks them.  The quotients are carried along:
// a runtime division in a role's loop costs as much as issuing a stage.
struct Walk {
    const int32_t *off, *parts;
    int E, ft, f_tiles, step_p, step_f;
    int p, f, e;

    __device__ __forceinline__ Walk(const MxFfnArgs &a, const int32_t *o, const int32_t *q)
        : off(o), parts(q), E(a.E), ft(a.ft), f_tiles(a.f_tiles) {
        step_p = (int)gridDim.x / f_tiles;
        step_f = (int)gridDim.x - step_p * f_tiles;
        p = (int)blockIdx.x / f_tiles;
        f = (int)blockIdx.x - p * f_tiles;
        e = 0;
    }
    __device__ __forceinline__ void next() {
        p += step_p;
        f += step_f;
        if (f >= f_tiles) {
            f -= f_tiles;
            ++p;
        }
    }
    // False behind the last tile.  The expert by bisection of the part counts before each
    // expert, its share of the block's rows a multiple of 8 but for the last part's.
    __device__ __forceinline__ bool tile(Tile &w) {
        if (p >= parts[E]) return false;
        if (parts[e + 1] <= p) {
            int lo = e + 1, hi = E - 1;
            while (lo < hi) {  // the last e with parts[e] <= p
                const int mid = (lo + hi + 1) >> 1;
                if (parts[mid] <= p) lo = mid; else hi = mid - 1;
            }
            e = lo;
        }
        const int first = off[e], m = off[e + 1] - first;
        const int of = parts[e + 1] - parts[e];
        const int share = of == 1 ? m : ((m + of - 1) / of + 7) & ~7;  // <= cap: no part is empty
        w.e = e;
        w.row0 = first + (p - parts[e]) * share;
        w.n = min(share, first + m - w.row0);
        w.f0 = f * ft;
        return true;
    }
};

// A place in a ring of `size` buffers and the parity of the pass over it.
struct Ring {
    int at = 0;
    uint32_t pass = 0;
    __device__ __forceinline__ void next(int size) {
        if (++at == size) {
            at = 0;
            pass ^= 1u;
        }
    }
};

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
            mbar_init(tempty_bar(b), 8);  // one arrival per epilogue warp
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
    if (any_bad && threadIdx.x == 0) parts[a.E] = 0;  // no tiles
    __syncthreads();
    if (any_bad && threadIdx.x == 0 && blockIdx.x == 0) report(a.status, MOE_ERR_DEVICE_INDEX);
    volatile int *abort_v = &abort_s;
    griddep_launch_dependents();

    // Warps 0 and 1 run their loops whole, so that addresses and descriptors are uniform over
    // the warp; one elected lane issues.
    if (warp == 0) {
        const bool leader = elect_one();
        Walk walk(a, off, parts);
        Tile w;
        Ring st, sf;
        uint32_t its = 0, sits = 0;
        bool ok = true;
        for (; ok && !*abort_v && walk.tile(w); walk.next()) {
            const int boxes = w.n <= a.box ? 1 : (w.n + a.box - 1) / a.box;
            const int wrow = w.e * a.N + w.f0;
            const uint32_t w_rows = (uint32_t)((GATE_UP ? 2 : 1) * a.ft);
            const uint32_t x_rows = (uint32_t)(boxes * a.box);
            const uint32_t sf_bytes = (w_rows + x_rows) * 16u;
            const uint32_t st_bytes = w_rows * a.w_count + x_rows * a.x_count;
            for (int kb = 0; kb < a.num_kb; ++kb) {
                if (kb % kXSuper == 0) {
                    ok = mbar_wait(free_bar(sf.at), sf.pass ^ 1u, a.status);
                    if (!ok) break;
                    if (leader) {
                        const uint32_t sl = base + a.sf + (uint32_t)sf.at * a.slot_bytes;
                        const uint32_t bar = raw_bar(sf.at);
                        const int x = kb / kXSuper * 16;
                        mbar_arrive_expect_tx(bar, sf_bytes);
                        tma_load_2d(sl, &map_w0s, bar, x, wrow);
                        if (GATE_UP)
                            tma_load_2d(sl + (uint32_t)a.ft * 16u, &map_w1s, bar, x, wrow);
                        for (int i = 0; i < boxes; ++i)
                            tma_load_2d(sl + 2048u + (uint32_t)(i * a.box) * 16u, &map_xs, bar, x,
                                        w.row0 + i * a.box);
                    }
                    sf.next(R);
                    ++sits;
                }
                ok = mbar_wait(empty_bar(st.at), st.pass ^ 1u, a.status);
                if (!ok) break;
                if (leader) {
                    const uint32_t dst = base + a.ring + (uint32_t)st.at * a.stage_bytes;
                    const uint32_t bar = full_bar(st.at);
                    const int x = kb * kXBK;
                    mbar_arrive_expect_tx(bar, st_bytes);
                    tma_load_2d(dst, &map_w0, bar, x, wrow);
                    if (GATE_UP) tma_load_2d(dst + (uint32_t)a.ft * 128u, &map_w1, bar, x, wrow);
                    for (int i = 0; i < boxes; ++i)
                        tma_load_2d(dst + a.a_bytes + (uint32_t)(i * a.box) * 128u, &map_x, bar, x,
                                    w.row0 + i * a.box);
                }
                st.next(S);
                ++its;
            }
        }
        if (!ok) *abort_v = 1;
        // Drain: the last loads into every stage and slot have landed before the CTA exits.
        for (uint32_t i = 0, n = min(its, (uint32_t)S); i < n; ++i) {
            if (st.at == 0) st.pass ^= 1u;
            st.at = st.at == 0 ? S - 1 : st.at - 1;
            if (!mbar_wait(full_bar(st.at), st.pass, a.status)) break;
        }
        for (uint32_t i = 0, n = min(sits, (uint32_t)R); i < n; ++i) {
            if (sf.at == 0) sf.pass ^= 1u;
            sf.at = sf.at == 0 ? R - 1 : sf.at - 1;
            if (!mbar_wait(raw_bar(sf.at), sf.pass, a.status)) break;
        }
    } else if (warp == 1) {
        const bool leader = elect_one();
        Walk walk(a, off, parts);
        Tile w;
        Ring st, sf, acc;
        bool ok = true;
        const uint32_t sf_col = tmem_base + 2u * (uint32_t)a.acc_cols;
        // descriptors: only the start address differs
        const uint64_t desc0 = sw128_desc(base + a.ring), sdesc0 = scales_desc(base + a.sf);
        const uint32_t a16 = a.a_bytes >> 4, stage16 = a.stage_bytes >> 4;
        for (; ok && !*abort_v && walk.tile(w); walk.next()) {
            const uint32_t n8 = (uint32_t)(w.n + 7) & ~7u;
            const uint32_t idesc = mx_idesc_at(a.idesc, n8, 0);
            ok = mbar_wait(tempty_bar(acc.at), acc.pass ^ 1u, a.status);
            if (!ok) break;
            tc_fence_after();
            const uint32_t d = tmem_base + (uint32_t)(acc.at * a.acc_cols);
            for (int kb = 0; kb < a.num_kb; ++kb) {
                if (kb % kXSuper == 0) {
                    ok = mbar_wait(ready_bar(sf.at), sf.pass, a.status);
                    if (!ok) break;
                }
                ok = mbar_wait(full_bar(st.at), st.pass, a.status);
                if (!ok) break;
                tc_fence_after();
                const uint32_t q = (uint32_t)(kb % kXSuper);
                const bool last = q == kXSuper - 1 || kb + 1 == a.num_kb;
                if (leader) {
                    const uint64_t sd = sdesc0 + (((uint32_t)sf.at * a.slot_bytes + 2048u + a.raw_b) >> 4);
                    const uint32_t sfa = sf_col + 16u * (q & 1u), sfb = sfa + 4u;
                    tmem_cp_scales(sfa, sd + q * 32u);
                    const uint64_t sdb = sd + 128u + ((q * a.tiled_b) >> 4);
                    tmem_cp_scales(sfb, sdb);
                    if (n8 > 128u) tmem_cp_scales(sfb + 4u, sdb + 32u);
                    const uint64_t ad = desc0 + (uint32_t)st.at * stage16, bd = ad + a16;
                    umma_mx(d, ad, bd, idesc, sfa, sfb, kb > 0 ? 1u : 0u);
                    umma_mx(d, ad + 2u, bd + 2u, mx_idesc_at(idesc, 0, 1), sfa, sfb, 1u);
                    umma_mx(d, ad + 4u, bd + 4u, mx_idesc_at(idesc, 0, 2), sfa, sfb, 1u);
                    umma_mx(d, ad + 6u, bd + 6u, mx_idesc_at(idesc, 0, 3), sfa, sfb, 1u);
                    umma_commit(empty_bar(st.at));
                    if (last) umma_commit(free_bar(sf.at));
                    if (kb + 1 == a.num_kb) umma_commit(tfull_bar(acc.at));
                }
                st.next(S);
                if (last) sf.next(R);
            }
            acc.next(2);
        }
        if (!ok) *abort_v = 1;
        // Every MMA and copy issued above has completed before the columns are freed.
        if (leader) umma_commit(drain_bar);
        mbar_wait(drain_bar, 0u, a.status);
    } else if (warp == 2 || warp == 3) {
        Walk walk(a, off, parts);
        Tile w;
        Ring sf;
        const int supers = (a.num_kb + kXSuper - 1) / kXSuper;
        bool ok = true;
        // The row of a lane in a 32-row piece i of 128 rows, and its place in the 512-byte tile:
        // a quarter-warp's 8 rows lie 32 rows from the next one's, so that the warp's 32 words
        // fill 128 contiguous bytes.
        const int row0 = (lane & 7) + 32 * (lane >> 3);
        const int dst0 = (lane & 7) * 16 + (lane >> 3) * 4;
        for (; ok && walk.tile(w); walk.next()) {
            const int pb = w.n <= 128 ? 4 : 8;
            for (int c = 0; c < supers; ++c) {
                ok = __all_sync(MOE_FULL_MASK,
                                !*abort_v && mbar_wait(raw_bar(sf.at), sf.pass, a.status));
                if (!ok) break;
                uint8_t *sl = gbase + a.sf + (size_t)sf.at * a.slot_bytes;
                // warp 2 turns the pieces 0, 2, .. and warp 3 the others
                turn_scales(sl, sl + 2048 + a.raw_b, 512, warp - 2, 4, 128, row0, dst0);
                turn_scales(sl + 2048, sl + 4096 + a.raw_b, (int)a.tiled_b, warp - 2, pb, a.cap,
                            row0, dst0);
                fence_async_shared();
                __syncwarp();
                if (lane == 0) mbar_arrive(ready_bar(sf.at));
                sf.next(R);
            }
        }
        if (!ok) *abort_v = 1;
    } else if (warp >= 4) {
        // Two warps share a quarter of the TMEM lanes, half of a chunk's columns each.
        const int q = warp & 3, half = (warp - 4) >> 2;
        const int tid = (int)threadIdx.x - 128;
        float *stg = reinterpret_cast<float *>(gbase + a.stg);
        Walk walk(a, off, parts);
        Tile w;
        Ring acc;
        // 8-feature groups of a token: a thread keeps its group (8 or 16 of them a tile).
        const int shift = a.ft == 128 ? 4 : a.ft == 64 ? 3 : 2;
        const int grp = tid & ((1 << shift) - 1), tok0 = tid >> shift, tok_step = kXEpiThreads >> shift;
        for (; walk.tile(w); walk.next()) {
            // Every epilogue thread goes by the same answer: they meet at the barriers below.
            int ok = !*abort_v && mbar_wait(tfull_bar(acc.at), acc.pass, a.status);
            asm volatile(
                "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %0, 0;\n\t"
                "barrier.red.and.pred q, 1, %1, p;\n\tselp.b32 %0, 1, 0, q;\n\t}"
                : "+r"(ok)
                : "n"(kXEpiThreads)
                : "memory");
            if (!ok) {
                *abort_v = 1;
                break;
            }
            tc_fence_after();
            const uint32_t trow = tmem_base + (uint32_t)(acc.at * a.acc_cols) +
                                  ((uint32_t)(q * 32) << 16) + (uint32_t)(16 * half);
            const int f = w.f0 + 8 * grp;
            const bool real_f = f < a.N;
            float b0[8], b1[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) b0[k] = b1[k] = 0.0f;
            if (real_f && a.bias0) load8(a.bias0 + (int64_t)w.e * a.N + f, b0);
            if (GATE_UP && real_f && a.bias1) load8(a.bias1 + (int64_t)w.e * a.N + f, b1);
            for (int c0 = 0; c0 < w.n; c0 += kXChunk) {
                uint32_t v[16];
                tmem_ld16(trow + (uint32_t)c0, v);
                if (c0 + kXChunk >= w.n) {  // the accumulator is free for the tile after next
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(tempty_bar(acc.at));
                }
                epi_sync();  // the last chunk's readers are done
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    stg[(16 * half + i) * kXPitch + 32 * q + lane] = __uint_as_float(v[i]);
                epi_sync();
                const int left = w.n - c0;
                // whole warps go on while any of their tokens is there (the block's shuffles)
                for (int tok = tok0; tok < kXChunk; tok += tok_step) {
                    const bool there = tok < left;
                    if (!__any_sync(MOE_FULL_MASK, there)) break;
                    const int64_t row = (int64_t)w.row0 + c0 + tok;
                    const float *src = stg + tok * kXPitch + 8 * grp;
                    float o[8];
                    load8(src, o);
#pragma unroll
                    for (int k = 0; k < 8; ++k) o[k] += b0[k];
                    if (GATE_UP) {
                        float u[8];
                        load8(src + a.ft, u);
#pragma unroll
                        for (int k = 0; k < 8; ++k) u[k] += b1[k];
                        activate8(o, u, a.act);
                        // features behind N: zeros of the row's padding
#pragma unroll
                        for (int k = 0; k < 8; ++k) o[k] = real_f && there ? o[k] : 0.0f;
                        store_h(a, row, f, o, there);
                    } else if (there && real_f) {
                        *reinterpret_cast<uint4 *>(a.y + row * a.N + f) = pack_bf16x8(o);
                    }
                }
            }
            // The last feature tile's tokens get what is left of their rows' padding.
            if (GATE_UP && w.f0 + a.ft >= a.N) {
                for (int i = tid; i < w.n; i += kXEpiThreads) {
                    const int64_t row = (int64_t)w.row0 + i;
                    uint8_t *qrow = a.hq + row * a.h_row, *srow = a.hs + row * a.h_scale;
                    const int64_t from = a.h_fmt == MOE_MX_E4M3 ? w.f0 + a.ft : (w.f0 + a.ft) / 2;
                    for (int64_t k = from; k < a.h_row; k += 16)
                        *reinterpret_cast<uint4 *>(qrow + k) = make_uint4(0u, 0u, 0u, 0u);
                    for (int64_t k = (w.f0 + a.ft) / kMxBlock; k < a.h_scale; ++k) srow[k] = 0;
                }
            }
            acc.next(2);
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
    a.box = a.cap / 2;  // one or two loads a stage
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
    // Row coordinates stay below 2^31 with a tile's overhang (E rows of weights: at most 2^30).
    if (d > kMxMaxK || F > kMxMaxK || rows >= (int64_t)INT32_MAX - 512) return MOE_ERR_UNSUPPORTED;
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

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
//   warp 0     TMA: weight and token tiles of 128 K values into a stage ring
//   warp 2     TMA: scale rows, 16 bytes (512 K values) at a time, into a second ring
//   warp 3     turns raw scale rows [row][16 bytes] into the tiles that TMEM
//              wants (32 x 16 bytes, four rows' words side by side)
//   warp 1     scale tiles to TMEM (tcgen05.cp) and four MMAs for every 128 K values
//   warp 16    walks the tiles and hands them to the other roles through a ring
//   warps 4-15 epilogue: TMEM -> shared memory, transposed to token-major; each
//              thread then takes 8 features of a token: bias, activation, MX
//              block (four lanes) or bf16, and one vector store
// Two accumulators: the epilogue of a tile overlaps the next one's products.
// A gate_up tile has ft gate rows and the ft up rows of the same features in
// its 128 rows; they meet in the epilogue's shared memory.
//
// PAIR: two CTAs on two SMs (cta_group::2) hold one token tile: each has its
// own 128 weight rows, half of the tokens' rows, and all of the tokens' scales.
// Every wait is bounded, as in the bf16 kernels.
//
// What bounds it.  Few rows: the weights' bytes (128 experts of 2880 x 2880, 64
// tokens of 4 slots: gate_up 158 to 166 us for 0.98 GB, 5.9 to 6.2 TB/s).  Inside an SM a K
// block costs 32 KB of shared memory traffic (16 KB of widened weights written
// and read), 256 clocks at least and 290 measured, under HBM's share.  Many
// rows: tensor pipe, L2 reads and the power cap together (131,072 rows: gate_up
// 1.75 to 2.0 ms, 2.2 to 2.5 PFLOP/s, at 1.2 to 1.6 GHz with sw_power_cap;
// 32,768 rows at 1.5 GHz: tensor pipe 64 % busy, 13.8 TB/s of L2 reads).
// Before, the issuing threads were the bound: with addresses, ring places and
// waits spelled out for every load and MMA a K block took 1660 clocks (4.03 ms).
#include <math.h>

#include "mx.cuh"
#include "tc.cuh"

namespace moe {
namespace {

constexpr int kXThreads = 544;  // 4 warps, 12 of the epilogue (128 .. 511), 1
constexpr int kXBK = 128;           // K values of a stage
constexpr int kXSuper = 4;          // stages that one load of scales covers
constexpr int kXMaxE = 4096;
constexpr int kXMaxDynamic = 227 * 1024 - 64;  // of a CTA on sm_100, without the static part
constexpr int kXMaxCap = 224;  // tokens of a tile: two accumulators and the scales fill TMEM
constexpr int kXMaxStages = 12;
constexpr int kXSlots = 4;  // loads of scales in flight
constexpr uint32_t kXWeightBytes = 128 * kXBK;  // a K block's weight tile in shared memory
constexpr int kXBars = 512;  // bytes of barriers, the TMEM address and the tile ring
constexpr int kXEpiThreads = 384;
constexpr int kXParts = 3;          // warps that share a quarter of the TMEM lanes
constexpr int kXPart = 16;          // token columns of a chunk that each of them takes
constexpr int kXChunk = kXParts * kXPart;
// Floats of a staged token: 16-byte aligned, the rows of eight reading lanes on different banks.
// gate_up: 32 gate and 32 up values, a buffer of 16 tokens for each of the 6 pairs of warps;
// down: 32 values, a buffer for each of the 12 warps.
constexpr int kXPitch[2] = {36, 68};
constexpr int kXStageBytes[2] = {4 * kXParts * kXPart * 36 * 4, 2 * kXParts * kXPart * 68 * 4};
constexpr float kXOaiAlpha = 1.702f;
constexpr float kXOaiLimit = 7.0f;

// Features of a CTA's tile: its 128 weight rows, halved where each feature has a gate and an up.
template <bool GATE_UP>
constexpr int kXFeatures = GATE_UP ? 64 : 128;

struct MxFfnArgs {
    const int32_t *offsets;  // [E+1], ascending
    const float *bias0;      // gate_up: b1 [E][N]; down: b2 [E][N]
    const float *bias1;      // gate_up: b3 [E][N]
    moe_bf16_t *y;           // down: [rows][N]
    uint8_t *hq, *hs;        // gate_up: MX rows of N values
    int64_t h_row, h_scale;  // bytes of those rows
    int32_t *status;
    int64_t rows;
    int E, N;
    int f_tiles;             // tiles (of a CTA or a pair) that cover the features
    int cap;                 // most tokens of a tile; also the columns of an accumulator
    int num_kb, stages, tmem_cols, act, h_fmt;
    uint32_t stage_bytes;          // a K block's weight and token tile in shared memory
    uint32_t stage_tx, slot_tx;    // bytes their barriers count: 4-bit values packed
    uint32_t raw_b, tiled_b, slot_bytes, idesc;
    uint32_t sf, stg, bars, tables;  // offsets in shared memory (the stages come first)
};

// e^-x to a few units of fp32, two at a time: 2^t with t = -x log2(e) rounded, times what the
// rounding of t and of log2(e) lost (to first order).  Without that factor the error grows with
// |x|, to 1e-6 at |x| = 10: no matter to the value of h, but ten times as many of its roundings
// (and of its blocks' powers of two) would fall on the other side than the exact sum's.  x is
// held between -200 and 200, where the result is infinite and 0: past 2.36e38 the product with
// log2(e) would overflow.  BELOW: x is at most 200 by itself.
template <bool BELOW>
__device__ __forceinline__ f32x2 exp_neg(f32x2 x) {
    constexpr float kL = 1.44269504f, kLLow = 1.92596299e-8f, kLn2 = 0.693147181f, kFar = 200.0f;
    const float2 v = halves(x);
    const float a = fmaxf(BELOW ? v.x : fminf(v.x, kFar), -kFar);
    const float b = fmaxf(BELOW ? v.y : fminf(v.y, kFar), -kFar);
    const float ta = -a * kL, tb = -b * kL;
    const f32x2 lost = fma2(pair_of(a, b), pair_of(-kLLow, -kLLow),
                            pair_of(fmaf(-a, kL, -ta), fmaf(-b, kL, -tb)));
    float pa, pb;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(pa) : "f"(ta));
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(pb) : "f"(tb));
    return mul2(pair_of(pa, pb), fma2(lost, pair_of(kLn2, kLn2), pair_of(1.0f, 1.0f)));
}

// 1 / x by the hardware's estimate (one unit of fp32; 0 for an infinite x).
__device__ __forceinline__ f32x2 reciprocal2(f32x2 x) {
    float2 v = halves(x);
    asm("rcp.approx.ftz.f32 %0, %0;" : "+f"(v.x));
    asm("rcp.approx.ftz.f32 %0, %0;" : "+f"(v.y));
    return pair_of(v.x, v.y);
}

// The clamps keep a NaN (fminf and fmaxf would put the limit in its place).
__device__ __forceinline__ float at_most(float v, float limit) {
    float r;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(v), "f"(limit));
    return r;
}
__device__ __forceinline__ float at_least(float v, float limit) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(v), "f"(limit));
    return r;
}

// g becomes act(g, u); a very negative gate gives 0, its limit: the reciprocal of 1 + e^-g is
// flushed to 0 below 2^-126, which is off by less than |g u| 2^-126.
__device__ __forceinline__ void activate8(f32x2 (&g)[4], const f32x2 (&u)[4], int act) {
    const f32x2 one = pair_of(1.0f, 1.0f);
    if (act == MOE_ACT_SWIGLU_OAI) {
        const f32x2 alpha = pair_of(kXOaiAlpha, kXOaiAlpha);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const float2 a = halves(g[k]), b = halves(u[k]);
            const f32x2 gc = pair_of(at_most(a.x, kXOaiLimit), at_most(a.y, kXOaiLimit));
            const f32x2 uc = pair_of(at_most(at_least(b.x, -kXOaiLimit), kXOaiLimit),
                                     at_most(at_least(b.y, -kXOaiLimit), kXOaiLimit));
            const f32x2 rc = reciprocal2(add2(exp_neg<true>(mul2(gc, alpha)), one));
            g[k] = mul2(mul2(gc, rc), add2(uc, one));
        }
    } else {
#pragma unroll
        for (int k = 0; k < 4; ++k)
            g[k] = mul2(mul2(g[k], reciprocal2(add2(exp_neg<false>(g[k]), one))), u[k]);
    }
}

__device__ __forceinline__ void load8(const float *p, f32x2 (&v)[4]) {
    const ulonglong2 x = *reinterpret_cast<const ulonglong2 *>(p);
    const ulonglong2 y = *reinterpret_cast<const ulonglong2 *>(p + 4);
    v[0] = x.x, v[1] = x.y;
    v[2] = y.x, v[3] = y.y;
}

// 8 features of a row of h (four neighbouring lanes hold a block).
__device__ __forceinline__ void store_h(const MxFfnArgs &a, int64_t row, int f, const f32x2 (&o)[4],
                                        bool there, bool real) {
    uint8_t *qrow = a.hq + row * a.h_row, *srow = a.hs + row * a.h_scale;
    uint32_t byte;
    if (a.h_fmt == MOE_MX_E4M3) {
        const uint2 e = mx_quarter<MOE_MX_E4M3>(o, real, byte);
        if (there) mx_store<MOE_MX_E4M3>(qrow, srow, f >> 3, e, byte);
    } else {
        const uint2 e = mx_quarter<MOE_MX_E2M1>(o, real, byte);
        if (there) mx_store<MOE_MX_E2M1>(qrow, srow, f >> 3, e, byte);
    }
}

// Raw scale rows of up to 128 operand rows (16 bytes each: four K blocks' words) to the four
// blocks' 512-byte tiles, `step` bytes apart.  A lane's row in piece i is 8 i + lane % 8 +
// 32 (lane / 8): the warp's 32 words of a block then fill 128 contiguous bytes.
__device__ __forceinline__ void turn_scales(const uint8_t *raw, uint8_t *tiles, uint32_t step,
                                            int lane) {
    const uint4 *src = reinterpret_cast<const uint4 *>(raw) + (lane & 7) + 32 * (lane >> 3);
    uint4 v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = src[8 * i];
    uint8_t *dst = tiles + (lane & 7) * 16 + (lane >> 3) * 4;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        *reinterpret_cast<uint32_t *>(dst + 128 * i) = v[i].x;
        *reinterpret_cast<uint32_t *>(dst + 128 * i + step) = v[i].y;
        *reinterpret_cast<uint32_t *>(dst + 128 * i + 2 * step) = v[i].z;
        *reinterpret_cast<uint32_t *>(dst + 128 * i + 3 * step) = v[i].w;
    }
}

struct Tile {
    int e, row0, n, f0;
};

// The tiles of a CTA (or pair) in order: tile t = part * f_tiles + feature tile, t = its number,
// + their number, ...  One warp walks them ahead of the others: a step (a bisection and a
// division) takes about 1000 clocks, a tenth of a tile.
struct Walk {
    const int32_t *off, *parts;
    int E, f_step, f_first, f_tiles, step_p, step_f;
    int p, f, e;

    // ctas: CTAs that walk as one (1, or 2 of which this is number `rank`), each with `ft` features.
    __device__ __forceinline__ Walk(const MxFfnArgs &a, const int32_t *o, const int32_t *q,
                                    int ctas, int rank, int ft)
        : off(o), parts(q), E(a.E), f_step(ctas * ft), f_first(rank * ft), f_tiles(a.f_tiles) {
        const int unit = (int)blockIdx.x / ctas, units = (int)gridDim.x / ctas;
        step_p = units / f_tiles;
        step_f = units - step_p * f_tiles;
        p = unit / f_tiles;
        f = unit - p * f_tiles;
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
        w.f0 = f * f_step + f_first;
        return true;
    }
};

// Tiles come from the walking warp in a ring of kXTiles; a role takes the next one as its own
// copy and frees the place.  n = 0: no more tiles.
constexpr int kXTiles = 4;
struct TileRing {
    const int4 *slots;
    uint32_t there, taken;  // barriers of place 0
    int32_t *status;
    int at = 0;
    uint32_t pass = 0;

    __device__ __forceinline__ bool wait() {
        return mbar_wait(there + 8u * (uint32_t)at, pass, status);
    }
    __device__ __forceinline__ Tile read() const {
        const int4 v = slots[at];
        return Tile{v.x, v.y, v.z, v.w};
    }
    __device__ __forceinline__ void free() {  // by every thread that counts as a reader
        mbar_arrive(taken + 8u * (uint32_t)at);
    }
    __device__ __forceinline__ void next() {
        at = (at + 1) & (kXTiles - 1);
        if (at == 0) pass ^= 1u;
    }
    // For a role of one thread.
    __device__ __forceinline__ bool take(Tile &w) {
        if (!wait()) return false;
        w = read();
        free();
        next();
        return true;
    }
};

// A K block's tile of an operand's rows.
template <bool PAIR>
__device__ __forceinline__ void load_tile(uint32_t dst, const CUtensorMap *map, uint32_t bar,
                                          int row, int kb) {
    if (PAIR)
        tma_load_3d_pair(dst, map, bar, 0, row, kb);
    else
        tma_load_3d(dst, map, bar, 0, row, kb);
}

template <bool PAIR>
__device__ __forceinline__ void commit(uint32_t bar) {
    if (PAIR)
        umma_commit_pair(bar);
    else
        umma_commit(bar);
}

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
    __device__ __forceinline__ void back(int size) {
        if (at-- == 0) {
            at = size - 1;
            pass ^= 1u;
        }
    }
};

template <bool GATE_UP, bool PAIR>
__global__ void __launch_bounds__(kXThreads, 1)
    expert_mx_kernel(const __grid_constant__ CUtensorMap map_w0,
                     const __grid_constant__ CUtensorMap map_w1,
                     const __grid_constant__ CUtensorMap map_w0s,
                     const __grid_constant__ CUtensorMap map_w1s,
                     const __grid_constant__ CUtensorMap map_x,
                     const __grid_constant__ CUtensorMap map_xs, const MxFfnArgs a) {
    extern __shared__ __align__(16) uint8_t smem_mx[];
    __shared__ int abort_s;
    constexpr int kCtas = PAIR ? 2 : 1, kFt = kXFeatures<GATE_UP>, R = kXSlots;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = PAIR ? (int)cluster_cta_rank() : 0;
    const uint32_t raw = smem_u32(smem_mx);
    const uint32_t base = (raw + 1023u) & ~1023u;
    uint8_t *const gbase = smem_mx + (base - raw);
    const int S = a.stages;
    const uint32_t bar0 = base + a.bars;
    auto full_bar = [&](int s) { return bar0 + 8u * s; };                   // the leader's
    auto empty_bar = [&](int s) { return bar0 + 8u * (S + s); };
    auto raw_bar = [&](int r) { return bar0 + 8u * (2 * S + r); };
    auto ready_bar = [&](int r) { return bar0 + 8u * (2 * S + R + r); };    // the leader's
    auto free_bar = [&](int r) { return bar0 + 8u * (2 * S + 2 * R + r); };
    auto tfull_bar = [&](int b) { return bar0 + 8u * (2 * S + 3 * R + b); };
    auto tempty_bar = [&](int b) { return bar0 + 8u * (2 * S + 3 * R + 2 + b); };  // the leader's
    const uint32_t drain_bar = bar0 + 8u * (2 * S + 3 * R + 4);
    const uint32_t there_bar = bar0 + 8u * (2 * S + 3 * R + 5);  // [kXTiles]
    const uint32_t taken_bar = there_bar + 8u * kXTiles;         // [kXTiles]
    uint32_t *tmem_slot =
        reinterpret_cast<uint32_t *>(gbase + a.bars + 8u * (2 * S + 3 * R + 5 + 2 * kXTiles));
    int4 *tile_slots = reinterpret_cast<int4 *>(gbase + a.bars + kXBars - 16 * kXTiles);
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
            mbar_init(ready_bar(r), kCtas);  // each CTA's turning warp
            mbar_init(free_bar(r), 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(tfull_bar(b), 1);
            mbar_init(tempty_bar(b), kXEpiThreads / 32 * kCtas);  // each CTA's epilogue warps
        }
        mbar_init(drain_bar, 1);
        for (int i = 0; i < kXTiles; ++i) {
            mbar_init(there_bar + 8u * i, 1);
            // readers: the two loading threads, the turning warp, the epilogue's warps, and in
            // the leader the thread that issues the products
            mbar_init(taken_bar + 8u * i, 3 + kXEpiThreads / 32 + (rank == 0 ? 1 : 0));
        }
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 2) {
        if (PAIR) {
            asm volatile(
                "tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                    smem_u32(tmem_slot)),
                "r"(a.tmem_cols)
                : "memory");
            asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
        } else {
            asm volatile(
                "tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                    smem_u32(tmem_slot)),
                "r"(a.tmem_cols)
                : "memory");
            asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
        }
    }
    griddep_wait();  // offsets and tokens come from the kernels before this one
    for (int i = threadIdx.x; i <= a.E; i += blockDim.x) off[i] = __ldg(a.offsets + i);
    tc_fence_before();
    if (PAIR)
        cluster_sync();
    else
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
    TileRing tiles{tile_slots, there_bar, taken_bar, a.status};

    // The producers and the MMA issuer are one thread each, and their loops are unrolled over
    // the K blocks that a load of scales covers: what bounds them is the length of the chain
    // of instructions between two issues.
    if (warp == 0) {
        if (elect_one()) {
            Tile w;
            Ring st;
            uint32_t filled = 0;
            bool ok = true;
            const uint32_t lead_full = PAIR ? cluster_map(full_bar(0), 0) : full_bar(0);
            constexpr uint32_t up = (uint32_t)kFt * kXBK;
            while (ok && !*abort_v) {
                ok = tiles.take(w);
                if (!ok || w.n == 0) break;
                const int wrow = w.e * a.N + w.f0;
                // a pair's tokens in multiples of 16: each CTA holds one half's rows
                const int xrow = w.row0 + (PAIR ? rank * (((w.n + 15) & ~15) >> 1) : 0);
                for (int kb = 0; kb < a.num_kb; ++kb) {
                    ok = mbar_wait(empty_bar(st.at), st.pass ^ 1u, a.status);
                    if (!ok) break;
                    const uint32_t dst = base + (uint32_t)st.at * a.stage_bytes;
                    const uint32_t bar = lead_full + 8u * (uint32_t)st.at;
                    if (rank == 0) mbar_arrive_expect_tx(full_bar(st.at), a.stage_tx);
                    load_tile<PAIR>(dst, &map_w0, bar, wrow, kb);
                    if (GATE_UP) load_tile<PAIR>(dst + up, &map_w1, bar, wrow, kb);
                    load_tile<PAIR>(dst + kXWeightBytes, &map_x, bar, xrow, kb);
                    st.next(S);
                    ++filled;
                }
            }
            if (!ok) *abort_v = 1;
            // Drain: the last loads into every stage have landed before the CTAs exit (the leader's
            // barriers count both CTAs' bytes).  In a pair also the arrivals that tell of the
            // stages' last use: they come from the leader's commits, over the cluster's network.
            // (A CTA by itself waits for its last commit, in warp 1; these waits as well made one
            // token's down 10.6 us from 9.6.)
            for (uint32_t i = 0, n = min(filled, (uint32_t)S); i < n; ++i) {
                st.back(S);
                if (rank == 0 && !mbar_wait(full_bar(st.at), st.pass, a.status)) {
                    *abort_v = 1;
                    break;
                }
                if (PAIR && !*abort_v && !mbar_wait(empty_bar(st.at), st.pass, a.status)) *abort_v = 1;
            }
            // The leader's last commit arrives here too, on every path, after a wait that gave
            // up as well: so the limit is above that of the leader's own waits.
            if (PAIR && rank != 0) mbar_wait_for(drain_bar, 0u, a.status, 3 * kWaitLimitNs);
        }
    } else if (warp == 1) {
        if (rank == 0 && elect_one()) {
            Tile w;
            Ring st, sf, acc;
            bool ok = true;
            const uint32_t sf_col = tmem_base + 2u * (uint32_t)a.cap;
            // descriptors: only the start address, in the low word, differs
            const uint64_t d0 = sw128_desc(base), s0 = scales_desc(base + a.sf + 2048u + a.raw_b);
            const uint32_t d_hi = (uint32_t)(d0 >> 32), s_hi = (uint32_t)(s0 >> 32);
            constexpr uint32_t a16 = kXWeightBytes >> 4;
            const uint32_t stage16 = a.stage_bytes >> 4, slot16 = a.slot_bytes >> 4;
            const uint32_t tiled16 = a.tiled_b >> 4;
            uint32_t d_lo = (uint32_t)d0, s_lo = (uint32_t)s0;  // of the ring places in use
            while (ok && !*abort_v) {
                ok = tiles.take(w);
                if (!ok || w.n == 0) break;
                const uint32_t n = PAIR ? (uint32_t)(w.n + 15) & ~15u : (uint32_t)(w.n + 7) & ~7u;
                uint32_t idesc[4];
#pragma unroll
                for (uint32_t k = 0; k < 4; ++k) idesc[k] = mx_idesc_at(a.idesc, n, k);
                const bool wide = n > 128u;
                ok = mbar_wait(tempty_bar(acc.at), acc.pass ^ 1u, a.status);
                if (!ok) break;
                tc_fence_after();
                const uint32_t d = tmem_base + (uint32_t)(acc.at * a.cap);
                uint32_t more = 0;
                // The four K blocks of a load of scales (fewer behind K's end); false if a wait
                // gave up.
                auto super = [&](int blocks) -> bool {
                    if (!mbar_wait(ready_bar(sf.at), sf.pass, a.status)) return false;
                    tc_fence_after();
#pragma unroll
                    for (int q = 0; q < kXSuper; ++q) {
                        if (q >= blocks) break;
                        if (!mbar_wait(full_bar(st.at), st.pass, a.status)) return false;
                        tc_fence_after();
                        // scales' columns begin at multiples of four
                        const uint32_t sfa = sf_col + 16u * (q & 1), sfb = sfa + 4u;
                        const uint32_t sb = s_lo + 128u + (uint32_t)q * tiled16;
                        tmem_cp_scales<PAIR>(sfa, s_lo + 32u * q, s_hi);
                        tmem_cp_scales<PAIR>(sfb, sb, s_hi);
                        if (wide) tmem_cp_scales<PAIR>(sfb + 4u, sb + 32u, s_hi);
                        const uint32_t b_lo = d_lo + a16;
#pragma unroll
                        for (uint32_t k = 0; k < 4; ++k) {
                            umma_mx<PAIR>(d, d_lo + 2u * k, b_lo + 2u * k, d_hi, idesc[k], sfa, sfb,
                                          more);
                            more = 1u;
                        }
                        commit<PAIR>(empty_bar(st.at));
                        st.next(S);
                        d_lo = st.at == 0 ? (uint32_t)d0 : d_lo + stage16;
                    }
                    commit<PAIR>(free_bar(sf.at));
                    sf.next(R);
                    s_lo = sf.at == 0 ? (uint32_t)s0 : s_lo + slot16;
                    return true;
                };
                int left = a.num_kb;
                for (; ok && left >= kXSuper; left -= kXSuper) ok = super(kXSuper);
                if (ok && left > 0) ok = super(left);
                if (!ok) break;
                commit<PAIR>(tfull_bar(acc.at));
                acc.next(2);
            }
            if (!ok) *abort_v = 1;
            // Every MMA and copy issued above has completed before the columns are freed.
            commit<PAIR>(drain_bar);
            mbar_wait(drain_bar, 0u, a.status);
        }
    } else if (warp == 2) {
        if (elect_one()) {
            Tile w;
            Ring sf;
            uint32_t filled = 0;
            bool ok = true;
            while (ok && !*abort_v) {
                ok = tiles.take(w);
                if (!ok || w.n == 0) break;
                const int wrow = w.e * a.N + w.f0;
                for (int c = 0; c < a.num_kb; c += kXSuper) {
                    ok = mbar_wait(free_bar(sf.at), sf.pass ^ 1u, a.status);
                    if (!ok) break;
                    const uint32_t sl = base + a.sf + (uint32_t)sf.at * a.slot_bytes;
                    const uint32_t bar = raw_bar(sf.at);
                    mbar_arrive_expect_tx(bar, a.slot_tx);
                    tma_load_2d(sl, &map_w0s, bar, 4 * c, wrow);
                    if (GATE_UP) tma_load_2d(sl + (uint32_t)kFt * 16u, &map_w1s, bar, 4 * c, wrow);
                    tma_load_2d(sl + 2048u, &map_xs, bar, 4 * c, w.row0);
                    sf.next(R);
                    ++filled;
                }
            }
            if (!ok) *abort_v = 1;
            for (uint32_t i = 0, n = min(filled, (uint32_t)R); i < n; ++i) {  // as warp 0 does
                sf.back(R);
                if (!mbar_wait(raw_bar(sf.at), sf.pass, a.status)) {
                    *abort_v = 1;
                    break;
                }
                if (PAIR && !*abort_v && !mbar_wait(free_bar(sf.at), sf.pass, a.status)) *abort_v = 1;
            }
        }
    } else if (warp == 3) {
        Ring sf;
        const int supers = (a.num_kb + kXSuper - 1) / kXSuper;
        bool ok = true;
        const uint32_t lead_ready = PAIR ? cluster_map(ready_bar(0), 0) : ready_bar(0);
        while (ok && !*abort_v) {
            ok = __all_sync(MOE_FULL_MASK, tiles.wait());
            if (!ok) break;
            const Tile w = tiles.read();
            __syncwarp();
            if (lane == 0) tiles.free();
            tiles.next();
            if (w.n == 0) break;
            for (int c = 0; c < supers; ++c) {
                ok = __all_sync(MOE_FULL_MASK, mbar_wait(raw_bar(sf.at), sf.pass, a.status));
                if (!ok) break;
                uint8_t *sl = gbase + a.sf + (size_t)sf.at * a.slot_bytes;
                uint8_t *turned = sl + 2048 + a.raw_b;
                turn_scales(sl, turned, 512u, lane);
                turn_scales(sl + 2048, turned + 2048, a.tiled_b, lane);
                if (w.n > 128) turn_scales(sl + 4096, turned + 2560, a.tiled_b, lane);
                fence_async_shared();
                __syncwarp();
                if (lane == 0) {
                    if (PAIR)
                        mbar_arrive_cluster(lead_ready + 8u * (uint32_t)sf.at);
                    else
                        mbar_arrive(ready_bar(sf.at));
                }
                sf.next(R);
            }
        }
        if (!ok) *abort_v = 1;
    } else if (warp == 16) {
        if (lane == 0) {
            Walk walk(a, off, parts, kCtas, rank, kFt);
            Tile w;
            Ring to;
            for (bool any = true; any && !*abort_v; walk.next(), to.next(kXTiles)) {
                any = walk.tile(w);
                if (!mbar_wait(taken_bar + 8u * (uint32_t)to.at, to.pass ^ 1u, a.status)) {
                    *abort_v = 1;
                    break;
                }
                tile_slots[to.at] = make_int4(w.e, w.row0, any ? w.n : 0, w.f0);
                mbar_arrive(there_bar + 8u * (uint32_t)to.at);
            }
        }
    } else {
        // Three warps share a quarter of the TMEM lanes, a third of a chunk's token columns each
        // (with two the epilogue's latencies held up tiles of few K blocks: qwen3 gate_up 390
        // against 376 us, 509 ragged rows' down 108 against 103).
        // gate_up: the 32 gate features of quarter q and the same up features, two quarters
        // on, are an MX block; the two warps that hold them meet in a staging buffer of their
        // own.  down: a warp's 32 features are its own affair.
        const int q = warp & 3, part = (warp - 4) >> 2;
        const int duo = GATE_UP ? q & 1 : q;  // block of 32 features
        const int member = GATE_UP ? q >> 1 : 0;
        const int bar_id = 2 + kXParts * duo + part;
        constexpr int kPitch = kXPitch[GATE_UP];
        float *stg = reinterpret_cast<float *>(gbase + a.stg) +
                     (kXParts * duo + part) * (kXPart * kPitch);
        Ring acc;
        const int grp = lane & 3;  // 8 of the block's features
        const int cover = a.f_tiles * kCtas * kFt;  // features of all tiles, N or a little more
        const uint32_t lead_tempty = PAIR ? cluster_map(tempty_bar(0), 0) : tempty_bar(0);
        for (;;) {
            // One thread polls; the others wait at the barrier that carries its answer.
            int ok = threadIdx.x != 128 || (!*abort_v && tiles.wait() &&
                                            (tiles.read().n == 0 ||
                                             mbar_wait(tfull_bar(acc.at), acc.pass, a.status)));
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
            const Tile w = tiles.read();
            __syncwarp();
            if (lane == 0) tiles.free();
            tiles.next();
            if (w.n == 0) break;
            tc_fence_after();
            const uint32_t trow = tmem_base + (uint32_t)(acc.at * a.cap) +
                                  ((uint32_t)(q * 32) << 16) + (uint32_t)(kXPart * part);
            const int f = w.f0 + 32 * duo + 8 * grp;
            const bool real_f = f < a.N;
            const int mine = w.n - kXPart * part;  // tokens from this part's first on
            uint32_t v[kXPart];
            if (mine > 0) tmem_ld16_nowait(trow, v);
            f32x2 b0[4], b1[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) b0[k] = b1[k] = 0ull;
            if (real_f && a.bias0) load8(a.bias0 + (int64_t)w.e * a.N + f, b0);
            if (GATE_UP && real_f && a.bias1) load8(a.bias1 + (int64_t)w.e * a.N + f, b1);
            for (int c0 = 0; c0 < mine; c0 += kXChunk) {
                auto meet = [&] {  // the warps that share the buffer
                    if (GATE_UP)
                        asm volatile("bar.sync %0, 64;" ::"r"(bar_id) : "memory");
                    else
                        __syncwarp();
                };
                tmem_wait_ld();
                if (c0 > 0) meet();  // the last chunk has been read
#pragma unroll
                for (int i = 0; i < kXPart; ++i)
                    stg[i * kPitch + 32 * member + lane] = __uint_as_float(v[i]);
                if (c0 + kXChunk < mine) tmem_ld16_nowait(trow + (uint32_t)(c0 + kXChunk), v);
                meet();
                // 16 tokens, four lanes each: 8 a warp (gate_up), or both eights (down)
#pragma unroll
                for (int i = 0; i < (GATE_UP ? 1 : 2); ++i) {
                    const int t8 = 8 * (GATE_UP ? member : i);
                    if (c0 + t8 >= mine) break;
                    const int tok = t8 + (lane >> 2);
                    const bool there = c0 + tok < mine;
                    const int64_t row = (int64_t)w.row0 + kXPart * part + c0 + tok;
                    const float *src = stg + tok * kPitch + 8 * grp;
                    f32x2 o[4];
                    load8(src, o);
#pragma unroll
                    for (int k = 0; k < 4; ++k) o[k] = add2(o[k], b0[k]);
                    if (GATE_UP) {
                        f32x2 u[4];
                        load8(src + 32, u);
#pragma unroll
                        for (int k = 0; k < 4; ++k) u[k] = add2(u[k], b1[k]);
                        activate8(o, u, a.act);
                        // features behind N are zeros of the row's padding
                        store_h(a, row, f, o, there, real_f && there);
                    } else if (there && real_f) {
                        uint32_t p[4];
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const float2 v2 = halves(o[k]);
                            const __nv_bfloat162 two = __floats2bfloat162_rn(v2.x, v2.y);
                            p[k] = *reinterpret_cast<const uint32_t *>(&two);
                        }
                        *reinterpret_cast<uint4 *>(a.y + row * a.N + f) =
                            make_uint4(p[0], p[1], p[2], p[3]);
                    }
                }
            }
            // The buffer's last readers before the next tile's writers.
            if (GATE_UP && mine > 0) asm volatile("bar.sync %0, 64;" ::"r"(bar_id) : "memory");
            // This warp's reads are done: the accumulator is free for the tile after next.
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                if (PAIR)
                    mbar_arrive_cluster(lead_tempty + 8u * (uint32_t)acc.at);
                else
                    mbar_arrive(tempty_bar(acc.at));
            }
            // The last feature tile's tokens get what is left of their rows' padding.
            if (GATE_UP && w.f0 + kFt == cover) {
                for (int i = (int)threadIdx.x - 128; i < w.n; i += kXEpiThreads) {
                    const int64_t row = (int64_t)w.row0 + i;
                    uint8_t *qrow = a.hq + row * a.h_row, *srow = a.hs + row * a.h_scale;
                    for (int64_t k = a.h_fmt == MOE_MX_E4M3 ? cover : cover / 2; k < a.h_row; k += 16)
                        *reinterpret_cast<uint4 *>(qrow + k) = make_uint4(0u, 0u, 0u, 0u);
                    for (int64_t k = cover / kMxBlock; k < a.h_scale; k += 2)
                        *reinterpret_cast<uint16_t *>(srow + k) = 0;
                }
            }
            acc.next(2);
        }
    }

    tc_fence_before();
    if (PAIR)
        cluster_sync();  // with the drains above: no CTA leaves while the other, or a commit of
                         // the leader's on its way, may use its memory or barriers
    else
        __syncthreads();
    if (warp == 2) {
        tc_fence_after();
        if (PAIR)
            asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem_base),
                         "r"(a.tmem_cols)
                         : "memory");
        else
            asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem_base),
                         "r"(a.tmem_cols)
                         : "memory");
    }
}

template <bool GATE_UP, bool PAIR>
moe_status launch_expert_mx(const uint8_t *xq, const uint8_t *xs, int32_t x_fmt, const uint8_t *w0,
                            const uint8_t *w0s, const uint8_t *w1, const uint8_t *w1s,
                            int32_t w_fmt, int32_t K, MxFfnArgs a, moe_stream_t stream) {
    constexpr int kCtas = PAIR ? 2 : 1, kFt = kXFeatures<GATE_UP>;
    const bool w4 = w_fmt == MOE_MX_E2M1, x4 = x_fmt == MOE_MX_E2M1;
    a.f_tiles = (a.N + kCtas * kFt - 1) / (kCtas * kFt);
    a.num_kb = mx_padded(K) / kXBK;
    const int b_rows = a.cap / kCtas;
    const uint32_t b_bytes = (uint32_t)b_rows * kXBK;
    a.stage_bytes = kXWeightBytes + b_bytes;
    a.stage_tx =
        (uint32_t)kCtas * ((w4 ? kXWeightBytes / 2 : kXWeightBytes) + (x4 ? b_bytes / 2 : b_bytes));
    a.slot_tx = (uint32_t)(128 + a.cap) * 16u;
    a.raw_b = a.cap > 128 ? 4096u : 2048u;
    a.tiled_b = a.cap > 128 ? 1024u : 512u;
    a.slot_bytes = 2048u + a.raw_b + 2048u + 4u * a.tiled_b;
    a.idesc = mx_idesc(w4 ? 5u : 0u, x4 ? 5u : 0u, 128u * kCtas);
    int cols = 32;
    while (cols < 2 * a.cap + 32) cols *= 2;
    a.tmem_cols = cols;
    const uint32_t stg = kXStageBytes[GATE_UP], bars = kXBars;
    const uint32_t tables = ((uint32_t)(2 * (a.E + 1)) * 4u + 15u) / 16u * 16u;
    const int64_t rest = (int64_t)kXMaxDynamic - 1024 /* alignment slack */ - stg - bars - tables -
                         (int64_t)kXSlots * a.slot_bytes;
    int64_t stages = rest / a.stage_bytes;
    if (stages > kXMaxStages) stages = kXMaxStages;
    if (stages < 2) return MOE_ERR_UNSUPPORTED;
    a.stages = (int)stages;
    a.sf = (uint32_t)a.stages * a.stage_bytes;
    a.stg = a.sf + (uint32_t)kXSlots * a.slot_bytes;
    a.bars = a.stg + stg;
    a.tables = a.bars + bars;
    const size_t smem = 1024 + (size_t)a.tables + tables;
    if (allow_smem(expert_mx_kernel<GATE_UP, PAIR>, kXMaxDynamic) != MOE_OK) return MOE_ERR_CUDA;
    CUtensorMap mw0, mw1, mw0s, mw1s, mx, mxs;
    const int64_t wrows = (int64_t)a.E * a.N;
    const int64_t Kp = mx_padded(K), sp = mx_scale_bytes(K);
    if (!make_mx_map(&mw0, w0, wrows, Kp, w4, kFt) ||
        !make_byte_map(&mw0s, w0s, wrows, sp, kFt) ||
        !make_mx_map(&mx, xq, a.rows, Kp, x4, b_rows) ||
        !make_byte_map(&mxs, xs, a.rows, sp, a.cap))
        return MOE_ERR_CUDA;
    mw1 = mw0;
    mw1s = mw0s;
    if (GATE_UP && (!make_mx_map(&mw1, w1, wrows, Kp, w4, kFt) ||
                    !make_byte_map(&mw1s, w1s, wrows, sp, kFt)))
        return MOE_ERR_CUDA;
    // Never more CTAs than the most tiles these rows can make.
    const int64_t parts = a.rows / a.cap + (a.rows < a.E ? a.rows : a.E);
    const int64_t most = parts * a.f_tiles, slots = sm_count() / kCtas;
    const unsigned grid = (unsigned)(kCtas * (most < slots ? most : slots));
    cudaLaunchAttribute attr[2];
    cudaLaunchConfig_t cfg = pdl_config(dim3(grid), dim3(kXThreads), smem, as_cuda(stream), attr);
    if (PAIR) {
        attr[1].id = cudaLaunchAttributeClusterDimension;
        attr[1].val.clusterDim.x = 2;
        attr[1].val.clusterDim.y = 1;
        attr[1].val.clusterDim.z = 1;
        cfg.numAttrs = 2;
    }
    if (cudaLaunchKernelEx(&cfg, expert_mx_kernel<GATE_UP, PAIR>, mw0, mw1, mw0s, mw1s, mx, mxs,
                           a) != cudaSuccess) {
        cudaGetLastError();
        return MOE_ERR_CUDA;
    }
    return launch_status();
}

// Tile shape by the rows an expert has on average.  The token tile should just hold them, and
// their spread (1.4 of its standard deviation: routing is near a draw), in as few equal parts
// as fit: wider, it takes shared memory from the weights in flight and loads tokens that are
// not there (a tile's boxes hold cap rows, however few it has); narrower, more blocks are cut into parts, each of which
// reads the weights again.  From 33 rows on pairs of CTAs, each with half of the tokens' bytes.
// Measured with 128 experts of 2880 x 2880, e2m1 weights, gate_up in us, by rows an expert:
//    8, 20, 32 (one CTA):  cap 16: 189 289 393,  32: 197 203 261,  48: -   202 211,  64: 217 218 238
//   40, 64, 80 (pairs):    cap 64: 218 332 365,  80: 225 253 316,  96: 226 259 258, 112: 228 275 256
//   40, 64, 80 (one CTA):  cap 64: 230 339 409,  80: 233 257 339,  96: 251 290 281
//  128, 256, 512 (pairs):  cap 128: 424 717 1243,  144: 331 622 1192,  192: 380 686 1184,
//                          224: 386 724 1215
template <bool GATE_UP>
moe_status run_expert_mx(const uint8_t *xq, const uint8_t *xs, int32_t x_fmt, const uint8_t *w0,
                         const uint8_t *w0s, const uint8_t *w1, const uint8_t *w1s, int32_t w_fmt,
                         int32_t K, MxFfnArgs a, moe_stream_t stream) {
    const int64_t share = (a.rows + a.E - 1) / a.E;
    const double need = (double)share + 1.4 * sqrt((double)share);
    const double parts = ceil(need / kXMaxCap);
    a.cap = ((int)ceil(need / parts) + 15) / 16 * 16;
    if (share <= 32)
        return launch_expert_mx<GATE_UP, false>(xq, xs, x_fmt, w0, w0s, w1, w1s, w_fmt, K, a,
                                                stream);
    return launch_expert_mx<GATE_UP, true>(xq, xs, x_fmt, w0, w0s, w1, w1s, w_fmt, K, a, stream);
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
    return run_expert_mx<true>(xq, xs, x_format, w1, w1_scales, w3, w3_scales, w_format, d, a,
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
    return run_expert_mx<false>(h, h_scales, h_format, w2, w2_scales, nullptr, nullptr, w_format,
                                   F, a, stream);
}

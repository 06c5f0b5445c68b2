// Causal softmax attention over packed sequences, backward, on the 5th-generation tensor cores.
//
// With p the softmax (recomputed as exp2(s c - lse) from the forward's cache), delta_i = do_i . o_i:
//     dv_j = sum_i p_ij do_i,   ds_ij = p_ij (do_i . v_j - delta_i),
//     dq_i = scale sum_j ds_ij k_j,   dk_j = scale sum_i ds_ij q_i.
// Two kernels, each the owner of the rows it sums, so that no sum is taken by atomics and the order of
// every one is fixed (a single pass over the scores would save 2 of 7 products, and would have to add
// one of the three gradients up across CTAs):
//   dkdv: one CTA per (128 keys, key head); it walks the group's query heads and the query tiles that see
//         these keys.  S^T = K Q^T, dP^T = V dO^T, dV += P^T dO, dK += dS^T Q.
//   dq:   one CTA per (128 queries, query head) over the key tiles.  S = Q K^T, dP = dO V^T, dQ += dS K.
// P and dS go to tensor memory as bf16, over the columns of S and dP that their own thread has read, and
// are the A operands of the second products; the row tiles in shared memory serve as K-major operands of
// the first products and as MN-major ones of the second.
//
// The products of one item overlap the element-wise work of the next (issue order, dkdv):
//     S(i) dP(i) | P(i) ready: dV(i) S(i+1) | dS(i) ready: dK(i) dP(i+1) | ...
// so the tensor pipe runs dV(i), S(i+1) while dS(i) is formed, and dK(i), dP(i+1) while P(i+1) is.
// 8 warps do the element-wise work (thread = row and half of the columns), one thread of a ninth issues every
// copy and product; 192 KB of shared memory: the CTA's own two tiles, and two stages of the walked ones.
//
// delta uses o with what its rounding left out (the cache's o_lo): row 0 of a sequence, where do . v - delta
// cancels, keeps a gradient of 0.  ds and p are rounded to bf16 for the products, nothing else is.
#include "attn_tc.cuh"
#include "launch.h"
#include "tma_host.h"

namespace gdn {
namespace attn {
namespace {

constexpr int kThreads = 288;
constexpr int kElem = 256;  // element-wise threads

template <int D>
struct BwdSmem {
    static constexpr uint32_t kTile = kRows * D * 2;
    static constexpr uint32_t kOwn0 = 0, kOwn1 = kTile;                         // the CTA's own two tiles
    static constexpr uint32_t kWalk = 2 * kTile;                                // [2 stages][2 tiles]
    static constexpr uint32_t kStats = 6 * kTile;                               // dkdv: [2 stages][lse, delta][128]
    static constexpr uint32_t kBar = kStats + 2 * 2 * kRows * 4;
    static constexpr uint32_t kBytes = kBar + 128 + 1024;
    static __device__ __forceinline__ uint32_t walk(int stage, int which) { return kWalk + (2 * stage + which) * kTile; }
};
constexpr uint32_t TM_S = 0, TM_DP = 128, TM_ACC0 = 256, TM_ACC1 = 384, TM_COLS = 512;

enum BwdBar { B_OWN = 0, B_W0, B_W1, B_S, B_DP, B_X, B_DS, B_END, B_COUNT };

struct BwdParams {
    AttnIO io;
    int tiles, window;
    float scale_log2;
};

__device__ __forceinline__ void setup(Ctx& cx, uint8_t* bars, const AttnIO& io, uint32_t*& tmem_slot) {
    cx.bars = reinterpret_cast<uint64_t*>(bars);
    tmem_slot = reinterpret_cast<uint32_t*>(bars + 96);
    cx.abort_flag = reinterpret_cast<volatile int*>(bars + 100);
    cx.err = io.err;
    cx.wait_ns = io.wait_ns ? io.wait_ns : kWaitNs;
    if (threadIdx.x == 0) {
        for (int i = 0; i < B_COUNT; ++i) mbar_init(cx.bars + i, i == B_X || i == B_DS ? kElem : 1);
        *cx.abort_flag = 0;
        mbar_fence_init();
    }
    if (threadIdx.x >= kElem) {
        tmem_alloc(tmem_slot, TM_COLS);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
}

// D (+)= A B with A [128 x 128] bf16 in tensor memory as two halves of 32 columns, 64 columns apart, and
// B a row tile taken MN-major.
template <int D>
__device__ __forceinline__ void mma_halves(uint32_t d_tmem, uint32_t a_tmem, uint32_t b_smem, bool accumulate) {
    constexpr uint32_t idesc = idesc_bf16_f32_mn(128, D, false, true);
    const uint64_t db = sdesc_mn_sw128(b_smem, kRows * 128u);
#pragma unroll
    for (int k = 0; k < kRows; k += 16)
        mma_ts(d_tmem, a_tmem + (uint32_t)((k >> 6) * 64 + ((k & 63) >> 1)), db + (uint64_t)((k * 128) >> 4), idesc,
               (accumulate || k > 0) ? 1u : 0u);
}

// 64 floats as bf16 pairs into 32 columns.
__device__ __forceinline__ void st_half(uint32_t taddr, const float (&x)[64]) {
#pragma unroll
    for (int q = 0; q < 2; ++q) {
        uint32_t w[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) w[e] = pack_bf16x2(x[32 * q + 2 * e], x[32 * q + 2 * e + 1]);
        tmem_st16(taddr + 16 * q, w);
    }
}

// This thread's part of an accumulator row (half `h` of D columns), times `f`, to dst.
template <int D>
__device__ __forceinline__ void store_acc(uint32_t taddr, int h, __nv_bfloat16* dst, float f, bool live) {
#pragma unroll
    for (int c = 0; c < D / 2; c += 32) {
        uint32_t r[32];
        tmem_ld32(taddr + h * (D / 2) + c, r);
        tmem_ld_wait();
        float v[32];
#pragma unroll
        for (int e = 0; e < 32; ++e) v[e] = __uint_as_float(r[e]) * f;
        if (live) store32_bf16(dst + h * (D / 2) + c, v);
    }
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
attn_dkdv_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                 const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_do, const BwdParams p) {
    using L = BwdSmem<D>;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* sm = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    const uint32_t sb = smem_u32(sm);
    const int tid = threadIdx.x, warp = tid >> 5;
    const int hk = blockIdx.x % p.io.Hk, G = p.io.Hq / p.io.Hk;
    Seq sq;
    if (!find_tile(p.io.cu, p.io.nseq, p.io.T, (int)(blockIdx.x / p.io.Hk), sq)) return;
    const int key0 = sq.local * kRows;
    const int last_row = sq.len - 1 - key0 - (kRows - 1) < p.window - 1 ? sq.len - 1 : key0 + kRows - 1 + p.window - 1;
    const int nq = last_row / kRows - sq.local + 1, m = G * nq;  // query tiles, items
    Ctx cx;
    uint32_t* tmem_slot;
    setup(cx, sm + L::kBar, p.io, tmem_slot);
    const uint32_t tbase = *tmem_slot;

    if (warp == 8) {
        if ((tid & 31) == 0) {
            int issued = 0, seen = 0;
            auto load = [&](int it) {
                const int head = hk * G + it / nq, tile = it % nq, st = it & 1;
                uint64_t* bar = cx.bars + B_W0 + st;
                mbar_arrive_expect_tx(bar, 2 * L::kTile + 2 * kRows * 4);
                const int row = sq.begin + key0 + tile * kRows;
                load_tile<D>(sb + L::walk(st, 0), &tm_q, bar, head, row);
                load_tile<D>(sb + L::walk(st, 1), &tm_do, bar, head, row);
                const int64_t stat = ((int64_t)head * p.tiles + sq.tile + tile) * kRows;
                bulk_g2s(sb + L::kStats + st * 1024u, p.io.lse + stat, kRows * 4, bar);
                bulk_g2s(sb + L::kStats + st * 1024u + 512u, p.io.delta + stat, kRows * 4, bar);
                ++issued;
            };
            mbar_arrive_expect_tx(cx.bars + B_OWN, 2 * L::kTile);
            load_tile<D>(sb + L::kOwn0, &tm_k, cx.bars + B_OWN, hk, sq.begin + key0);
            load_tile<D>(sb + L::kOwn1, &tm_v, cx.bars + B_OWN, hk, sq.begin + key0);
            load(0);
            bool ok = wait_bar(cx, B_OWN, 0);
            const bool own = ok;
            if (ok && (ok = wait_bar(cx, B_W0, 0))) {
                ++seen;
                mma_ss_rows<D>(tbase + TM_S, sb + L::kOwn0, sb + L::walk(0, 0));
                mma_commit(cx.bars + B_S);
                mma_ss_rows<D>(tbase + TM_DP, sb + L::kOwn1, sb + L::walk(0, 1));
                mma_commit(cx.bars + B_DP);
            }
            for (int it = 0; ok && it < m; ++it) {
                const int st = it & 1, nx = st ^ 1;
                // the item before has left its stage: the next one may land there
                if (it && !(ok = wait_bar(cx, B_END, (it - 1) & 1))) break;
                if (it + 1 < m) load(it + 1);
                if (!(ok = wait_bar(cx, B_X, it & 1))) break;
                tc_fence_after();
                mma_halves<D>(tbase + TM_ACC0, tbase + TM_S, sb + L::walk(st, 1), it > 0);
                if (it + 1 < m) {
                    if (!(ok = wait_bar(cx, B_W0 + nx, ((it + 1) >> 1) & 1))) break;
                    ++seen;
                    mma_ss_rows<D>(tbase + TM_S, sb + L::kOwn0, sb + L::walk(nx, 0));
                    mma_commit(cx.bars + B_S);
                }
                if (!(ok = wait_bar(cx, B_DS, it & 1))) break;
                tc_fence_after();
                mma_halves<D>(tbase + TM_ACC1, tbase + TM_DP, sb + L::walk(st, 0), it > 0);
                mma_commit(cx.bars + B_END);
                if (it + 1 < m) {
                    mma_ss_rows<D>(tbase + TM_DP, sb + L::kOwn1, sb + L::walk(nx, 1));
                    mma_commit(cx.bars + B_DP);
                }
            }
            // after an expired wait: the copies still on their way land before the memory is given up
            if (!own) mbar_wait(cx.bars + B_OWN, 0, cx.wait_ns);
            for (; seen < issued; ++seen) mbar_wait(cx.bars + B_W0 + (seen & 1), (seen >> 1) & 1, cx.wait_ns);
        }
        __syncwarp();
    } else {
        const int lane = tid & 127, h = tid >> 7;
        const uint32_t tl = tbase + ((uint32_t)((warp & 3) * 32) << 16);
        const int key = key0 + lane;  // within the sequence
        bool ok = true;
        for (int it = 0; it < m; ++it) {
            const int st = it & 1, row0 = key0 + (it % nq) * kRows + 64 * h;  // row of this thread's first column
            const float* lse = reinterpret_cast<const float*>(sm + L::kStats + st * 1024) + 64 * h;
            const float* delta = lse + kRows;
            if (!(ok = wait_warp(cx, B_W0 + st, (it >> 1) & 1))) break;  // the statistics have landed
            if (!(ok = wait_warp(cx, B_S, it & 1))) break;
            tc_fence_after();
            uint32_t s[2][32];
            tmem_ld32(tl + TM_S + 64 * h, s[0]);
            tmem_ld32(tl + TM_S + 64 * h + 32, s[1]);
            tmem_ld_wait();
            float x[64];
#pragma unroll
            for (int c = 0; c < 64; c += 4) {
                const float4 l4 = *reinterpret_cast<const float4*>(lse + c);
                const float ls[4] = {l4.x, l4.y, l4.z, l4.w};
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    x[c + e] = exp2_approx(fmaf(__uint_as_float(s[(c + e) >> 5][(c + e) & 31]), p.scale_log2, -ls[e]));
            }
            // rows before the key, past its window or past the sequence
            const int q0 = key0 + (it % nq) * kRows;
            const bool tail = q0 + kRows > sq.len;
            if (q0 == key0 || tail || q0 + kRows - 1 - key0 >= p.window) {
                const int lo = key - row0;  // first visible column
                const int hi = min(p.window - 1 < sq.len ? key + p.window - 1 : sq.len - 1, sq.len - 1) - row0;
#pragma unroll
                for (int c = 0; c < 64; ++c)
                    if (c < lo || c > hi) x[c] = 0.f;
            }
            st_half(tl + TM_S + 64 * h, x);
            if (tail) {
                // rows past the sequence have weight 0, but 0 * NaN is not 0; both first products have read them
                if (!(ok = wait_warp(cx, B_DP, it & 1))) break;
                if (lane >= sq.len - q0) zero_row<D>(sm + L::walk(st, h), lane);
                fence_async_shared();
            }
            tmem_st_wait();
            tc_fence_before();
            mbar_arrive(cx.bars + B_X);
            if (!(ok = wait_warp(cx, B_DP, it & 1))) break;
            tc_fence_after();
            tmem_ld32(tl + TM_DP + 64 * h, s[0]);
            tmem_ld32(tl + TM_DP + 64 * h + 32, s[1]);
            tmem_ld_wait();
#pragma unroll
            for (int c = 0; c < 64; c += 4) {
                const float4 d4 = *reinterpret_cast<const float4*>(delta + c);
                const float de[4] = {d4.x, d4.y, d4.z, d4.w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float t = x[c + e] * (__uint_as_float(s[(c + e) >> 5][(c + e) & 31]) - de[e]);
                    x[c + e] = x[c + e] == 0.f ? 0.f : t;  // a row past the sequence may hold anything
                }
            }
            st_half(tl + TM_DP + 64 * h, x);
            tmem_st_wait();
            tc_fence_before();
            mbar_arrive(cx.bars + B_DS);
            if (it && !(ok = wait_warp(cx, B_END, (it - 1) & 1))) break;  // long past; keeps its phase in step
        }
        if (ok && wait_warp(cx, B_END, (m - 1) & 1)) {
            tc_fence_after();
            const int64_t at = ((int64_t)(sq.begin + key) * p.io.Hk + hk) * D;
            store_acc<D>(tl + TM_ACC0, h, static_cast<__nv_bfloat16*>(p.io.dv) + at, 1.f, key < sq.len);
            store_acc<D>(tl + TM_ACC1, h, static_cast<__nv_bfloat16*>(p.io.dk) + at, p.io.scale, key < sq.len);
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 8) tmem_dealloc(tbase, TM_COLS);
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
attn_dq_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
               const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_do, const BwdParams p) {
    using L = BwdSmem<D>;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* sm = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    const uint32_t sb = smem_u32(sm);
    const int tid = threadIdx.x, warp = tid >> 5;
    const int head = blockIdx.x % p.io.Hq, hk = head / (p.io.Hq / p.io.Hk);
    Seq sq;
    if (!find_tile(p.io.cu, p.io.nseq, p.io.T, p.tiles - 1 - (int)(blockIdx.x / p.io.Hq), sq)) return;
    const int row0 = sq.local * kRows;
    const int lo = max(0, row0 - p.window + 1) / kRows, hi = sq.local, m = hi - lo + 1;
    Ctx cx;
    uint32_t* tmem_slot;
    setup(cx, sm + L::kBar, p.io, tmem_slot);
    const uint32_t tbase = *tmem_slot;

    if (warp == 8) {
        if ((tid & 31) == 0) {
            int issued = 0, seen = 0;
            auto load = [&](int it) {
                const int st = it & 1, row = sq.begin + (hi - it) * kRows;
                uint64_t* bar = cx.bars + B_W0 + st;
                mbar_arrive_expect_tx(bar, 2 * L::kTile);
                load_tile<D>(sb + L::walk(st, 0), &tm_k, bar, hk, row);
                load_tile<D>(sb + L::walk(st, 1), &tm_v, bar, hk, row);
                ++issued;
            };
            mbar_arrive_expect_tx(cx.bars + B_OWN, 2 * L::kTile);
            load_tile<D>(sb + L::kOwn0, &tm_q, cx.bars + B_OWN, head, sq.begin + row0);
            load_tile<D>(sb + L::kOwn1, &tm_do, cx.bars + B_OWN, head, sq.begin + row0);
            load(0);
            bool ok = wait_bar(cx, B_OWN, 0);
            const bool own = ok;
            if (ok && (ok = wait_bar(cx, B_W0, 0))) {
                ++seen;
                mma_ss_rows<D>(tbase + TM_S, sb + L::kOwn0, sb + L::walk(0, 0));
                mma_commit(cx.bars + B_S);
                mma_ss_rows<D>(tbase + TM_DP, sb + L::kOwn1, sb + L::walk(0, 1));
                mma_commit(cx.bars + B_DP);
            }
            for (int it = 0; ok && it < m; ++it) {
                const int st = it & 1, nx = st ^ 1;
                if (it && !(ok = wait_bar(cx, B_END, (it - 1) & 1))) break;
                if (it + 1 < m) load(it + 1);
                if (!(ok = wait_bar(cx, B_X, it & 1))) break;  // S(it) is in registers
                if (it + 1 < m) {
                    if (!(ok = wait_bar(cx, B_W0 + nx, ((it + 1) >> 1) & 1))) break;
                    ++seen;
                    tc_fence_after();
                    mma_ss_rows<D>(tbase + TM_S, sb + L::kOwn0, sb + L::walk(nx, 0));
                    mma_commit(cx.bars + B_S);
                }
                if (!(ok = wait_bar(cx, B_DS, it & 1))) break;
                tc_fence_after();
                mma_halves<D>(tbase + TM_ACC0, tbase + TM_DP, sb + L::walk(st, 0), it > 0);
                mma_commit(cx.bars + B_END);
                if (it + 1 < m) {
                    mma_ss_rows<D>(tbase + TM_DP, sb + L::kOwn1, sb + L::walk(nx, 1));
                    mma_commit(cx.bars + B_DP);
                }
            }
            if (!own) mbar_wait(cx.bars + B_OWN, 0, cx.wait_ns);
            for (; seen < issued; ++seen) mbar_wait(cx.bars + B_W0 + (seen & 1), (seen >> 1) & 1, cx.wait_ns);
        }
        __syncwarp();
    } else {
        const int lane = tid & 127, h = tid >> 7;
        const uint32_t tl = tbase + ((uint32_t)((warp & 3) * 32) << 16);
        const int row = row0 + lane;
        const int64_t stat = ((int64_t)head * p.tiles + sq.tile) * kRows + lane;
        const float lse = __ldg(p.io.lse + stat), delta = __ldg(p.io.delta + stat);
        bool ok = true;
        for (int it = 0; it < m; ++it) {
            const int key0 = (hi - it) * kRows;
            if (!(ok = wait_warp(cx, B_S, it & 1))) break;
            tc_fence_after();
            uint32_t s[2][32];
            tmem_ld32(tl + TM_S + 64 * h, s[0]);
            tmem_ld32(tl + TM_S + 64 * h + 32, s[1]);
            tmem_ld_wait();
            tc_fence_before();
            mbar_arrive(cx.bars + B_X);
            float x[64];
#pragma unroll
            for (int c = 0; c < 64; ++c)
                x[c] = exp2_approx(fmaf(__uint_as_float(s[c >> 5][c & 31]), p.scale_log2, -lse));
            // keys after the row or out of its window
            if (it == 0 || key0 <= row0 + kRows - 1 - p.window) {
                const int last = row - key0 - 64 * h, gone = last - p.window;
#pragma unroll
                for (int c = 0; c < 64; ++c)
                    if (c > last || c <= gone) x[c] = 0.f;
            }
            if (!(ok = wait_warp(cx, B_DP, it & 1))) break;
            tc_fence_after();
            tmem_ld32(tl + TM_DP + 64 * h, s[0]);
            tmem_ld32(tl + TM_DP + 64 * h + 32, s[1]);
            tmem_ld_wait();
#pragma unroll
            for (int c = 0; c < 64; ++c) {
                const float t = x[c] * (__uint_as_float(s[c >> 5][c & 31]) - delta);
                x[c] = x[c] == 0.f ? 0.f : t;  // a key past the sequence may hold anything
            }
            st_half(tl + TM_DP + 64 * h, x);
            if (it == 0 && sq.len - key0 < kRows) {
                // K's rows past the sequence: their ds is 0, but 0 * NaN is not; S(0) and dP(0) are done with them
                if (h == 0 && lane >= sq.len - key0) zero_row<D>(sm + L::walk(0, 0), lane);
                fence_async_shared();
            }
            tmem_st_wait();
            tc_fence_before();
            mbar_arrive(cx.bars + B_DS);
            if (it && !(ok = wait_warp(cx, B_END, (it - 1) & 1))) break;
        }
        if (ok && wait_warp(cx, B_END, (m - 1) & 1)) {
            tc_fence_after();
            const int64_t at = ((int64_t)(sq.begin + row) * p.io.Hq + head) * D;
            store_acc<D>(tl + TM_ACC0, h, static_cast<__nv_bfloat16*>(p.io.dq) + at, p.io.scale, row < sq.len);
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 8) tmem_dealloc(tbase, TM_COLS);
}

// delta = do . (o + o_lo) of every row, tile-aligned like lse (0 for a tile's rows past its sequence).
// D / 8 lanes a row, 8 channels each.  HBM bound: three reads of 2 bytes a channel.
template <int D>
__global__ void __launch_bounds__(256) attn_delta_kernel(const AttnIO io, int tiles) {
    constexpr int LANES = D / 8, RPP = 256 / LANES;
    Seq sq;
    const int head = blockIdx.x % io.Hq;
    if (!find_tile(io.cu, io.nseq, io.T, (int)(blockIdx.x / io.Hq), sq)) return;
    const int c0 = (threadIdx.x % LANES) * 8;
    const int row0 = sq.local * kRows;
#pragma unroll
    for (int r0 = 0; r0 < kRows; r0 += RPP) {
        const int r = r0 + threadIdx.x / LANES;
        float sum = 0.f;
        if (row0 + r < sq.len) {
            const int64_t at = ((int64_t)(sq.begin + row0 + r) * io.Hq + head) * D + c0;
            const uint4 a = __ldg(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(io.grad_o) + at));
            const uint4 b = __ldg(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(io.o) + at));
            const uint4 c = __ldg(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(io.o_lo) + at));
            const uint32_t x[4] = {a.x, a.y, a.z, a.w}, y[4] = {b.x, b.y, b.z, b.w}, z[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                sum = fmaf(__uint_as_float(x[i] << 16), __uint_as_float(y[i] << 16) + __uint_as_float(z[i] << 16), sum);
                sum = fmaf(__uint_as_float(x[i] & 0xFFFF0000u),
                           __uint_as_float(y[i] & 0xFFFF0000u) + __uint_as_float(z[i] & 0xFFFF0000u), sum);
            }
        }
#pragma unroll
        for (int o = LANES / 2; o >= 1; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        if (c0 == 0) io.delta[((int64_t)head * tiles + sq.tile) * kRows + r] = sum;
    }
}

template <int D>
cudaError_t launch(const CUtensorMap* maps, const BwdParams& p, cudaStream_t st) {
    const unsigned q_tiles = (unsigned)p.tiles * (unsigned)p.io.Hq, k_tiles = (unsigned)p.tiles * (unsigned)p.io.Hk;
    attn_delta_kernel<D><<<q_tiles, 256, 0, st>>>(p.io, p.tiles);
    count_launch();
    cudaError_t e = cudaGetLastError();
    if (e == cudaSuccess)
        e = cudaFuncSetAttribute(attn_dkdv_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)BwdSmem<D>::kBytes);
    if (e == cudaSuccess)
        e = cudaFuncSetAttribute(attn_dq_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)BwdSmem<D>::kBytes);
    if (e != cudaSuccess) return e;
    attn_dkdv_kernel<D><<<k_tiles, kThreads, BwdSmem<D>::kBytes, st>>>(maps[0], maps[1], maps[2], maps[3], p);
    count_launch();
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    attn_dq_kernel<D><<<q_tiles, kThreads, BwdSmem<D>::kBytes, st>>>(maps[0], maps[1], maps[2], maps[3], p);
    count_launch();
    return cudaGetLastError();
}

}  // namespace
}  // namespace attn

cudaError_t attn_bwd(const AttnIO& io, int d, cudaStream_t st) {
    CUtensorMap maps[4];
    if (!make_rows_map(&maps[0], io.q.p, io.T, io.Hq, d, io.q.stride) ||
        !make_rows_map(&maps[1], io.k.p, io.T, io.Hk, d, io.k.stride) ||
        !make_rows_map(&maps[2], io.v.p, io.T, io.Hk, d, io.v.stride) ||
        !make_rows_map(&maps[3], io.grad_o, io.T, io.Hq, d, (long)io.Hq * d))
        return cudaErrorInvalidValue;
    attn::BwdParams p{};
    p.io = io;
    p.tiles = (int)attn_tiles(io.T, io.nseq);
    p.window = io.window > 0 && io.window < INT32_MAX ? (int)io.window : INT32_MAX;
    p.scale_log2 = io.scale * 1.4426950408889634f;
    return d == 128 ? attn::launch<128>(maps, p, st) : attn::launch<64>(maps, p, st);
}

}  // namespace gdn

// Causal softmax attention over packed sequences, forward, on the 5th-generation tensor cores.
//
// One CTA per (128 query rows, query head), keys in tiles of 128 from the diagonal down to the
// window's edge (the diagonal first: every row then has a finite maximum from the first tile on).
//     S = Q K^T            tcgen05, Q and K row tiles in shared memory, 128 columns of tensor memory
//     P = exp2(S c - m)    thread t owns row t: c = scale log2(e), running reference m and sum l
//     O += P V             tcgen05, P as bf16 over S's columns (A in tensor memory), V as MN-major B
// m is not moved for every new maximum: any reference within 2^8 of it serves as well (p stays below
// 2^8, sums stay fp32, and bf16's relative rounding does not depend on it), so the O accumulator is
// rescaled only when a row's maximum has outgrown m by more than 8.
// P is rounded to bf16 because that is what the tensor cores multiply with bf16 V; l sums the unrounded p.
//
// Two CTAs share an SM (96 KB of shared memory and 256 columns of tensor memory each): while one's
// softmax warps work, the other's products run.  Warps 0-3 are the softmax, one thread of warp 4 issues
// every copy and product.  Every wait is bounded.
#include "attn_tc.cuh"
#include "launch.h"
#include "tma_host.h"

namespace gdn {
namespace attn {
namespace {

constexpr int kThreads = 160;
enum FwdBar { B_K = 0, B_V, B_S, B_P, B_O, B_COUNT };

template <int D>
struct FwdSmem {
    static constexpr uint32_t kTile = kRows * D * 2;
    static constexpr uint32_t kQ = 0, kK = kTile, kV = 2 * kTile, kBar = 3 * kTile;
    static constexpr uint32_t kBytes = kBar + 128 + 1024;  // + alignment slack
};
constexpr uint32_t TM_S = 0, TM_O = 128, TM_COLS = 256;

struct FwdParams {
    AttnIO io;
    int tiles;         // bound on the row tiles
    int window;        // INT_MAX: none
    float scale_log2;
};

template <int D, bool SAVE>
__global__ void __launch_bounds__(kThreads, 2)
attn_fwd_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                const __grid_constant__ CUtensorMap tm_v, const FwdParams p) {
    using L = FwdSmem<D>;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* sm = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    const uint32_t sb = smem_u32(sm);
    const int tid = threadIdx.x, warp = tid >> 5;
    const int head = blockIdx.x % p.io.Hq;
    Seq sq;
    TileMap map(p.io.cu, p.io.nseq, p.io.T);
    if (!map.find((int)(blockIdx.x / p.io.Hq), true, sq)) return;
    const int hk = head / (p.io.Hq / p.io.Hk);
    const int row0 = sq.local * kRows;  // first row, within the sequence
    const int first_key = max(0, row0 - p.window + 1);
    const int hi = sq.local, lo = first_key / kRows, n = hi - lo + 1;

    Ctx cx;
    cx.bars = reinterpret_cast<uint64_t*>(sm + L::kBar);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sm + L::kBar + 64);
    cx.abort_flag = reinterpret_cast<volatile int*>(sm + L::kBar + 68);
    cx.err = p.io.err;
    cx.wait_ns = p.io.wait_ns ? p.io.wait_ns : kWaitNs;
    if (tid == 0) {
        mbar_init(cx.bars + B_K, 1);
        mbar_init(cx.bars + B_V, 1);
        mbar_init(cx.bars + B_S, 1);
        mbar_init(cx.bars + B_P, 128);
        mbar_init(cx.bars + B_O, 1);
        *cx.abort_flag = 0;
        mbar_fence_init();
    }
    if (warp == 4) {
        tmem_alloc(tmem_slot, TM_COLS);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tbase = *tmem_slot;

    if (warp == 4) {
        if ((tid & 31) == 0) {
            int k_issued = 0, v_issued = 0, k_seen = 0, v_seen = 0;
            auto load_k = [&](int i) {
                mbar_arrive_expect_tx(cx.bars + B_K, i == 0 ? 2 * L::kTile : L::kTile);
                if (i == 0) load_tile<D>(sb + L::kQ, &tm_q, cx.bars + B_K, head, sq.begin + row0);
                load_tile<D>(sb + L::kK, &tm_k, cx.bars + B_K, hk, sq.begin + (hi - i) * kRows);
                ++k_issued;
            };
            auto load_v = [&](int i) {
                mbar_arrive_expect_tx(cx.bars + B_V, L::kTile);
                load_tile<D>(sb + L::kV, &tm_v, cx.bars + B_V, hk, sq.begin + (hi - i) * kRows);
                ++v_issued;
            };
            load_k(0);
            load_v(0);
            bool ok = wait_bar(cx, B_K, 0);
            if (ok) {
                ++k_seen;
                mma_ss_rows<D>(tbase + TM_S, sb + L::kQ, sb + L::kK);
                mma_commit(cx.bars + B_S);
            }
            for (int i = 0; ok && i < n; ++i) {
                if (!(ok = wait_bar(cx, B_S, i & 1))) break;  // S(i) done: the K tile is free
                if (i + 1 < n) load_k(i + 1);
                if (!(ok = wait_bar(cx, B_V, i & 1))) break;
                ++v_seen;
                if (!(ok = wait_bar(cx, B_P, i & 1))) break;
                tc_fence_after();
                mma_ts_rows<D>(tbase + TM_O, tbase + TM_S, sb + L::kV, i > 0);
                mma_commit(cx.bars + B_O);
                if (i + 1 == n) break;
                if (!(ok = wait_bar(cx, B_K, (i + 1) & 1))) break;
                ++k_seen;
                // runs after P V (products run in issue order), so it may write over P
                mma_ss_rows<D>(tbase + TM_S, sb + L::kQ, sb + L::kK);
                mma_commit(cx.bars + B_S);
                if (!(ok = wait_bar(cx, B_O, i & 1))) break;  // the V tile is free
                load_v(i + 1);
            }
            // after an expired wait: the copies still on their way land before the memory is given up
            if (k_seen < k_issued) mbar_wait(cx.bars + B_K, (k_issued - 1) & 1, cx.wait_ns);
            if (v_seen < v_issued) mbar_wait(cx.bars + B_V, (v_issued - 1) & 1, cx.wait_ns);
        }
        __syncwarp();
    } else {
        const uint32_t tl = tbase + ((uint32_t)(warp * 32) << 16);
        const int row = row0 + tid;  // within the sequence
        float m = -INFINITY, l = 0.f;
        bool ok = true;
        for (int i = 0; i < n; ++i) {
            if (!(ok = wait_warp(cx, B_S, i & 1))) break;
            // P V of the tile before finished earlier (S was issued after it): its phase is seen here, so
            // that this thread is never two phases behind
            if (i && !(ok = wait_warp(cx, B_O, (i - 1) & 1))) break;
            tc_fence_after();
            uint32_t s[4][32];
#pragma unroll
            for (int c = 0; c < 4; ++c) tmem_ld32(tl + TM_S + 32 * c, s[c]);
            tmem_ld_wait();
            const int key0 = (hi - i) * kRows;
            // keys after the row, or out of its window, leave the softmax
            if (i == 0 || key0 <= row0 + kRows - 1 - p.window) {
                const int last = row - key0, gone = last - p.window;
#pragma unroll
                for (int c = 0; c < 4; ++c)
#pragma unroll
                    for (int e = 0; e < 32; ++e) {
                        const int j = 32 * c + e;
                        if (j > last || j <= gone) s[c][e] = 0xFF800000u;  // -inf
                    }
            }
            float x[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
            for (int c = 0; c < 4; ++c)
#pragma unroll
                for (int e = 0; e < 32; e += 2)
                    x[c] = fmaxf(x[c], fmaxf(__uint_as_float(s[c][e]), __uint_as_float(s[c][e + 1])));
            const float mx = fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3])) * p.scale_log2;
            if (__any_sync(0xffffffffu, mx > m + 8.f)) {
                const float mn = fmaxf(m, mx), f = i ? exp2_approx(m - mn) : 0.f;
                m = mn;
                l *= f;
                if (i) {
#pragma unroll
                    for (int c = 0; c < D / 32; ++c) {
                        uint32_t o[32];
                        tmem_ld32(tl + TM_O + 32 * c, o);
                        tmem_ld_wait();
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            uint32_t w[16];
#pragma unroll
                            for (int e = 0; e < 16; ++e)
                                w[e] = __float_as_uint(__uint_as_float(o[16 * h + e]) * f);
                            tmem_st16(tl + TM_O + 32 * c + 16 * h, w);
                        }
                    }
                }
            }
            float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                uint32_t w[16];
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    const float a = exp2_approx(fmaf(__uint_as_float(s[c][2 * e]), p.scale_log2, -m));
                    const float b = exp2_approx(fmaf(__uint_as_float(s[c][2 * e + 1]), p.scale_log2, -m));
                    sum[e & 3] += a + b;
                    w[e] = pack_bf16x2(a, b);
                }
                tmem_st16(tl + TM_S + 16 * c, w);
            }
            l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
            if (i == 0 && sq.len - key0 < kRows) {
                // V's rows past the sequence: p is 0 there, but 0 * NaN is not
                if (!(ok = wait_warp(cx, B_V, 0))) break;
                if (tid >= sq.len - key0) zero_row<D>(sm + L::kV, tid);
                fence_async_shared();
            }
            tmem_st_wait();
            tc_fence_before();
            mbar_arrive(cx.bars + B_P);
        }
        if (ok && wait_warp(cx, B_O, (n - 1) & 1)) {
            tc_fence_after();
            const bool live = row < sq.len;
            const float inv = 1.f / l;
            const int64_t at = ((int64_t)(sq.begin + row) * p.io.Hq + head) * D;
#pragma unroll
            for (int c = 0; c < D / 32; ++c) {
                uint32_t o[32];
                tmem_ld32(tl + TM_O + 32 * c, o);
                tmem_ld_wait();
                float v[32];
#pragma unroll
                for (int e = 0; e < 32; ++e) v[e] = __uint_as_float(o[e]) * inv;
                if (live) {
                    store32_bf16(static_cast<__nv_bfloat16*>(p.io.o) + at + 32 * c, v);
                    if (SAVE) {
#pragma unroll
                        for (int e = 0; e < 32; ++e) v[e] -= __bfloat162float(__float2bfloat16_rn(v[e]));
                        store32_bf16(static_cast<__nv_bfloat16*>(p.io.o_lo) + at + 32 * c, v);
                    }
                }
            }
            // every row of the tile, so that the backward's copies of it read no uninitialised memory
            if (SAVE) p.io.lse[((int64_t)head * p.tiles + sq.tile) * kRows + tid] = live ? -(m + log2f(l)) : 0.f;
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 4) tmem_dealloc(tbase, TM_COLS);
}

template <int D, bool SAVE>
cudaError_t launch(const CUtensorMap* maps, const FwdParams& p, cudaStream_t st) {
    auto kernel = attn_fwd_kernel<D, SAVE>;
    cudaError_t e =
        cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)FwdSmem<D>::kBytes);
    if (e != cudaSuccess) return e;
    kernel<<<(unsigned)p.tiles * (unsigned)p.io.Hq, kThreads, FwdSmem<D>::kBytes, st>>>(maps[0], maps[1], maps[2], p);
    count_launch();
    return cudaGetLastError();
}

}  // namespace
}  // namespace attn

cudaError_t attn_fwd(const AttnIO& io, int d, cudaStream_t st) {
    CUtensorMap maps[3];
    if (!make_rows_map(&maps[0], io.q.p, io.T, io.Hq, d, io.q.stride) ||
        !make_rows_map(&maps[1], io.k.p, io.T, io.Hk, d, io.k.stride) ||
        !make_rows_map(&maps[2], io.v.p, io.T, io.Hk, d, io.v.stride))
        return cudaErrorInvalidValue;
    attn::FwdParams p{};
    p.io = io;
    p.tiles = (int)attn_tiles(io.T, io.nseq);
    p.window = io.window > 0 && io.window < INT32_MAX ? (int)io.window : INT32_MAX;
    p.scale_log2 = io.scale * 1.4426950408889634f;
    if (d == 128) return io.lse ? attn::launch<128, true>(maps, p, st) : attn::launch<128, false>(maps, p, st);
    return io.lse ? attn::launch<64, true>(maps, p, st) : attn::launch<64, false>(maps, p, st);
}

}  // namespace gdn

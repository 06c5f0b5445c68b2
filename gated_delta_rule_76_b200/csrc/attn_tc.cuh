// What the tensor-core attention kernels share: the tile map of packed sequences, bounded warp-wide
// waits, TMA loads of row tiles, and the product loops over their shared-memory tiles.
//
// Tiles: every sequence is cut into tiles of 128 rows from its own start, and the tiles of all
// sequences are numbered in order; T / 128 + nseq bounds their number on the host, and a CTA finds
// its sequence by a scan over cu_seqlens, 32 sequences a step.  A tile's rows past the end of its
// sequence belong to others (or to nobody): they are loaded, never stored, and kept out of every
// sum (masked scores; zeroed rows of operands that a zero weight would multiply, since 0 * NaN is
// not 0).
//
// A row tile in shared memory is D / 64 boxes of [128 rows][64 channels], 128-byte swizzled: a K-major
// operand (rows x channels) and an MN-major one (channels x rows) at once.
#pragma once
#include <cuda.h>
#include <cuda_bf16.h>

#include "attn.h"
#include "umma.cuh"

namespace gdn {
namespace attn {

using namespace gdn::tc;

constexpr uint64_t kWaitNs = 4000000000ull;
constexpr int kRows = 128;

struct Seq {
    int begin, len;   // first token, tokens
    int tile, local;  // global tile number, tile within the sequence
};

// Warp-collective: the sequence and local tile of global tile `g`, false past the last one.
__device__ __forceinline__ bool find_tile(const int32_t* cu, int nseq, int T, int g, Seq& out) {
    const int lane = threadIdx.x & 31;
    int before = 0;
    for (int s0 = 0; s0 < nseq; s0 += 32) {
        const int s = s0 + lane;
        int b = 0, e = 0;
        if (s < nseq) {
            b = min(max(__ldg(cu + s), 0), T);
            e = min(max(__ldg(cu + s + 1), b), T);
        }
        const int tiles = (e - b + kRows - 1) / kRows;
        int incl = tiles;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int x = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += x;
        }
        const int start = before + incl - tiles;
        const uint32_t hit = __ballot_sync(0xffffffffu, g >= start && g < start + tiles);
        if (hit) {
            const int src = __ffs(hit) - 1;
            out.begin = __shfl_sync(0xffffffffu, b, src);
            out.len = __shfl_sync(0xffffffffu, e, src) - out.begin;
            out.local = g - __shfl_sync(0xffffffffu, start, src);
            out.tile = g;
            return true;
        }
        before += __shfl_sync(0xffffffffu, incl, 31);
    }
    return false;
}

struct Ctx {
    uint64_t* bars;
    volatile int* abort_flag;
    int* err;
    uint64_t wait_ns;
};

// Bounded wait of one thread; on expiry the error word and the CTA's abort flag are set.
__device__ __forceinline__ bool wait_bar(const Ctx& cx, int bar, uint32_t parity) {
    uint64_t* b = cx.bars + bar;
    if (mbar_try_wait(b, parity)) return true;
    const uint64_t t0 = globaltimer_ns();
    while (!mbar_try_wait_sleep(b, parity, 1000u)) {
        if (*cx.abort_flag) return false;
        if (globaltimer_ns() - t0 > cx.wait_ns) {
            *cx.abort_flag = 1;
            atomicOr(cx.err, 1);
            return false;
        }
    }
    return true;
}
// The same by a whole warp, with one answer: tensor-memory instructions that follow need all lanes.
__device__ __forceinline__ bool wait_warp(const Ctx& cx, int bar, uint32_t parity) {
    return __all_sync(0xffffffffu, wait_bar(cx, bar, parity));
}

__device__ __forceinline__ void tma3(uint32_t dst, const CUtensorMap* map, uint64_t* bar, int c0, int c1, int c2) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
        "[%0], [%1, {%3, %4, %5}], [%2];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(c0), "r"(c1), "r"(c2)
        : "memory");
}
// 128 rows of one head from token `row` on.
template <int D>
__device__ __forceinline__ void load_tile(uint32_t dst, const CUtensorMap* map, uint64_t* bar, int head, int row) {
#pragma unroll
    for (int c = 0; c < D; c += 64) tma3(dst + (uint32_t)(c >> 6) * (kRows * 128u), map, bar, c, head, row);
}

// D[tmem] (+)= A[tmem, bf16, 128 columns of K] * B with B a row tile taken MN-major (K = its 128
// rows, N = its D channels).
template <int D>
__device__ __forceinline__ void mma_ts_rows(uint32_t d_tmem, uint32_t a_tmem, uint32_t b_smem, bool accumulate) {
    constexpr uint32_t idesc = idesc_bf16_f32_mn(128, D, false, true);
    const uint64_t db = sdesc_mn_sw128(b_smem, kRows * 128u);
#pragma unroll
    for (int k = 0; k < kRows; k += 16)
        mma_ts(d_tmem, a_tmem + (uint32_t)(k >> 1), db + (uint64_t)((k * 128) >> 4), idesc,
               (accumulate || k > 0) ? 1u : 0u);
}
// D[tmem] = A * B^T for two row tiles (K = channels).
template <int D>
__device__ __forceinline__ void mma_ss_rows(uint32_t d_tmem, uint32_t a_smem, uint32_t b_smem) {
    mma_ss_u<D, kRows, kRows>(d_tmem, a_smem, b_smem, idesc_bf16_f32(128, 128), false);
}

// Zeroes row `row` of a row tile (whole 128-byte lines, so the swizzle does not matter).
template <int D>
__device__ __forceinline__ void zero_row(uint8_t* tile, int row) {
#pragma unroll
    for (int c = 0; c < D; c += 64) {
        uint4* p = reinterpret_cast<uint4*>(tile + (c >> 6) * (kRows * 128) + row * 128);
#pragma unroll
        for (int i = 0; i < 8; ++i) p[i] = make_uint4(0u, 0u, 0u, 0u);
    }
}

__device__ __forceinline__ float exp2_approx(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// 32 floats of a row into 64 bytes of bf16.
__device__ __forceinline__ void store32_bf16(__nv_bfloat16* dst, const float (&x)[32]) {
#pragma unroll
    for (int i = 0; i < 32; i += 8) {
        uint4 u;
        u.x = pack_bf16x2(x[i], x[i + 1]);
        u.y = pack_bf16x2(x[i + 2], x[i + 3]);
        u.z = pack_bf16x2(x[i + 4], x[i + 5]);
        u.w = pack_bf16x2(x[i + 6], x[i + 7]);
        *reinterpret_cast<uint4*>(dst + i) = u;
    }
}

}  // namespace attn
}  // namespace gdn

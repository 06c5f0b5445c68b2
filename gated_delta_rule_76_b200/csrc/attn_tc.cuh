// What the tensor-core attention kernels share: the tile map of packed sequences, bounded warp-wide
// waits, TMA loads of row tiles, and the product loops over their shared-memory tiles.
//
// Tiles: every sequence is cut into tiles of 128 rows from its own start, and the tiles of all
// sequences are numbered in order; T / 128 + nseq bounds their number on the host.  CTAs stay for the whole
// call and find their units of work themselves (TileMap), from cu_seqlens, which the host does not see.  A tile's rows past the end of its
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
    int tile, local;  // global number of its (first) 128-row tile, tile within the sequence
};

// The map from a CTA's units of work to tiles of R rows (128 or 256), one per warp (every call is
// warp-collective).  With up to 32 sequences the tiles come in descending order of their work: a tile of a
// causal sequence of t tiles has 1, 2, .. or t tiles to look at, one tile of each (a window caps the larger
// ones, which keeps the order), so the r-th heaviest is found by counting.  With more sequences they come in the
// sequences' order.
template <int R>
struct TileMap {
    const int32_t* cu;
    int nseq, T;
    int b, e, t;         // up to 32 sequences: this lane's one, its tiles,
    int first, first128;  // and the tiles before them, of R and of 128 rows
    int total;           // tiles

    static __device__ __forceinline__ int scan(int x) {  // inclusive
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, x, o);
            if ((int)(threadIdx.x & 31) >= o) x += y;
        }
        return x;
    }
    // The 32 sequences from s0 on, `before` and `before128` tiles into the batch.
    __device__ __forceinline__ void load(int s0, int& before, int& before128) {
        const int s = s0 + (int)(threadIdx.x & 31);
        b = e = 0;
        if (s < nseq) {
            b = min(max(__ldg(cu + s), 0), T);
            e = min(max(__ldg(cu + s + 1), b), T);
        }
        t = (e - b + R - 1) / R;
        int incl = scan(t);
        first = before + incl - t;
        before += __shfl_sync(0xffffffffu, incl, 31);
        if (R == kRows) {
            first128 = first;
            before128 = before;
        } else {
            const int t128 = (e - b + kRows - 1) / kRows;
            incl = scan(t128);
            first128 = before128 + incl - t128;
            before128 += __shfl_sync(0xffffffffu, incl, 31);
        }
    }
    __device__ __forceinline__ TileMap(const int32_t* cu_, int nseq_, int T_) : cu(cu_), nseq(nseq_), T(T_) {
        int before = 0, before128 = 0;
        for (int s0 = 0; s0 < nseq; s0 += 32) load(s0, before, before128);
        total = before;
    }
    __device__ __forceinline__ void take(Seq& out, int src, int local) const {
        out.begin = __shfl_sync(0xffffffffu, b, src);
        out.len = __shfl_sync(0xffffffffu, e, src) - out.begin;
        out.local = local;
        out.tile = __shfl_sync(0xffffffffu, first128, src) + local * (R / kRows);
    }
    // Tile `rank` of the order; up: the work grows with the tile's place in its sequence (query tiles, which
    // see the keys before them), else it falls (key tiles).  False past the last one.
    __device__ __forceinline__ bool find(int rank, bool up, Seq& out) {
        if (rank >= total) return false;
        const int lane = threadIdx.x & 31;
        if (nseq <= 32) {
            // the largest work x that more than `rank` tiles reach
            int lo = 1, hi = __reduce_max_sync(0xffffffffu, t);
            while (lo < hi) {
                const int mid = (lo + hi + 1) >> 1;
                if ((int)__reduce_add_sync(0xffffffffu, max(0, t - mid + 1)) > rank) lo = mid;
                else hi = mid - 1;
            }
            const int among = rank - (int)__reduce_add_sync(0xffffffffu, max(0, t - lo));
            const uint32_t have = __ballot_sync(0xffffffffu, t >= lo);
            const bool me = t >= lo && __popc(have & ((1u << lane) - 1u)) == among;
            const int src = __ffs(__ballot_sync(0xffffffffu, me)) - 1;
            const int n = __shfl_sync(0xffffffffu, t, src);
            take(out, src, up ? lo - 1 : n - lo);
            return true;
        }
        const int g = up ? total - 1 - rank : rank;
        int before = 0, before128 = 0;
        for (int s0 = 0;; s0 += 32) {
            load(s0, before, before128);
            const uint32_t hit = __ballot_sync(0xffffffffu, g >= first && g < first + t);
            if (hit) {
                const int src = __ffs(hit) - 1;
                take(out, src, g - __shfl_sync(0xffffffffu, first, src));
                return true;
            }
        }
    }
    // Unit k of this CTA's share of `heads` times the tiles: rows of the grid's width in the order above,
    // every second one backwards, so that the CTAs' sums even out.  0: unit found, 1: none in this row, 2: no more.
    __device__ __forceinline__ int unit(int k, int heads, bool up, Seq& sq, int& head) {
        const int64_t at = (int64_t)k * gridDim.x;
        if (at >= (int64_t)total * heads) return 2;
        const int64_t u = at + ((k & 1) ? gridDim.x - 1 - blockIdx.x : blockIdx.x);
        if (u >= (int64_t)total * heads) return 1;
        const uint32_t rank = (uint32_t)u / (uint32_t)heads;  // u < 2^31: the host checks
        head = (int)((uint32_t)u - rank * (uint32_t)heads);
        return find((int)rank, up, sq) ? 0 : 2;
    }
};

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

// ---- pairs of fp32 in one 64-bit register ------------------------------------------------------
typedef unsigned long long f2;
__device__ __forceinline__ f2 f2_of(float lo, float hi) {
    f2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ f2 f2_of(uint32_t lo, uint32_t hi) {
    f2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "r"(lo), "r"(hi));
    return r;
}
__device__ __forceinline__ void f2_get(f2 v, float& lo, float& hi) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ f2 f2_add(f2 a, f2 b) {
    f2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ f2 f2_mul(f2 a, f2 b) {
    f2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ f2 f2_fma(f2 a, f2 b, f2 c) {
    f2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
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

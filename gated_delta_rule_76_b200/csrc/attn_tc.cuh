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

// Bounded wait of one thread; on expiry the error word and the CTA's abort flag are set.  A try waits in
// hardware for a while, and most phases complete within the first few: the clock is read only after those.
__device__ __forceinline__ bool wait_bar(const Ctx& cx, int bar, uint32_t parity) {
    uint64_t* b = cx.bars + bar;
    uint64_t t0 = 0;
#pragma unroll 1
    for (uint32_t i = 0;; ++i) {
        if (mbar_try_wait(b, parity)) return true;
        if (i < 16) continue;
        if (*cx.abort_flag) return false;
        const uint64_t now = globaltimer_ns();
        if (!t0) t0 = now;
        if (now - t0 > cx.wait_ns) {
            *cx.abort_flag = 1;
            atomicOr(cx.err, 1);
            return false;
        }
    }
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

// Shared-memory descriptors of a row tile, as the low word that a tile's address decides and a constant high
// word (umma.cuh has the fields): K-major, and MN-major with 64-channel groups a box apart.  The issuing thread
// forms one 32-bit sum a product slice.
constexpr uint32_t kDescHi = (1024u >> 4) | (1u << 14) | (2u << 29);
__device__ __forceinline__ uint32_t desc_k(uint32_t tile) { return (tile >> 4) | (1u << 16); }
__device__ __forceinline__ uint32_t desc_mn(uint32_t tile) { return (tile >> 4) | ((kRows * 128u >> 4) << 16); }
__device__ __forceinline__ uint64_t desc_of(uint32_t lo) {
    uint64_t d;
    asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "r"(lo), "r"(kDescHi));
    return d;
}
// D[tmem] (+)= A[tmem, bf16] * B with B a row tile taken MN-major (desc_mn; K = its 128 rows, N = its D
// channels), for the rows K0 .. K1 - 1; a_tmem is A's column of row 0.
template <int D, int K0, int K1>
__device__ __forceinline__ void mma_ts_rows(uint32_t d_tmem, uint32_t a_tmem, uint32_t b_desc, bool accumulate) {
    constexpr uint32_t idesc = idesc_bf16_f32_mn(128, D, false, true);
#pragma unroll
    for (int k = K0; k < K1; k += 16)
        mma_ts(d_tmem, a_tmem + (uint32_t)(k >> 1), desc_of(b_desc + (uint32_t)((k * 128) >> 4)), idesc,
               (accumulate || k > K0) ? 1u : 0u);
}
// D[tmem] = A * B^T for two row tiles (desc_k; K = channels).
template <int D>
__device__ __forceinline__ void mma_ss_rows(uint32_t d_tmem, uint32_t a_desc, uint32_t b_desc) {
    constexpr uint32_t idesc = idesc_bf16_f32(128, 128);
#pragma unroll
    for (int k = 0; k < D; k += 16) {
        const uint32_t o = ((uint32_t)(k >> 6) * kRows * 128u + (uint32_t)(k & 63) * 2u) >> 4;
        mma_ss(d_tmem, desc_of(a_desc + o), desc_of(b_desc + o), idesc, k > 0 ? 1u : 0u);
    }
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

// 2^x of a pair on the FMA pipe, for x <= 100 or so: x = n + f with n the nearest integer (found by adding
// 1.5 * 2^23) and |f| <= 1/2, 2^f by a polynomial, n added to the exponent field.  The polynomial is the
// minimax one of degree 4 for the relative error with the constant 1 (2^0 = 1 exactly), fitted by reweighted
// least squares: 2.9e-6 in fp32, far below the 2^-8 of the bf16 weight that the result becomes.  From -127 down the
// result is 0 (the exponent field of 1, 127, less 127); NaN gives NaN or infinity.
// The exponential unit computes 16 a cycle and SM, which is as long as the products take: the kernels send a part
// of the exponentials this way (kPoly).
__device__ __forceinline__ f2 exp2_poly(f2 x) {
    float lo, hi;
    f2_get(x, lo, hi);
    asm("max.NaN.f32 %0, %0, %1;" : "+f"(lo) : "f"(-127.f));
    asm("max.NaN.f32 %0, %0, %1;" : "+f"(hi) : "f"(-127.f));
    x = f2_of(lo, hi);
    const f2 t = f2_add(x, f2_of(12582912.f, 12582912.f));
    const f2 f = f2_fma(f2_add(t, f2_of(-12582912.f, -12582912.f)), f2_of(-1.f, -1.f), x);
    f2 y = f2_fma(f, f2_of(0.009582852945f, 0.009582852945f), f2_of(0.05590642616f, 0.05590642616f));
    y = f2_fma(f, y, f2_of(0.2402409911f, 0.2402409911f));
    y = f2_fma(f, y, f2_of(0.6931241751f, 0.6931241751f));
    y = f2_fma(f, y, f2_of(1.f, 1.f));
    float n0, n1;
    f2_get(t, n0, n1);
    f2_get(y, lo, hi);
    return f2_of(__float_as_uint(lo) + (__float_as_uint(n0) << 23), __float_as_uint(hi) + (__float_as_uint(n1) << 23));
}
// 2^x of a pair, by polynomial or on the exponential unit.
template <bool POLY>
__device__ __forceinline__ f2 exp2_pair(f2 x) {
    if (POLY) return exp2_poly(x);
    float a, b;
    f2_get(x, a, b);
    return f2_of(exp2_approx(a), exp2_approx(b));
}

// One arrival for a warp, after all its lanes' tensor-memory and shared-memory work.
__device__ __forceinline__ void arrive_warp(const Ctx& cx, int bar) {
    tc_fence_before();
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(cx.bars + bar);
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

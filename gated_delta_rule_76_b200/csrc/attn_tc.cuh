// What the tensor-core attention kernels share: the tile map of packed sequences, bounded warp-wide
// waits, TMA loads of row tiles, and the product loops over their shared-memory tiles.
//
// Tiles: every sequence is cut into tiles of 128 rows from its own start, and the tiles of all
// sequences are numbered in order; T / 128 + nseq bounds their number on the host.  CTAs stay for the whole
// call and find their units of work themselves (TileMap, UnitQueue), from cu_seqlens, which the host does not
// see.  A tile's rows past the end of its sequence belong to others (or to nobody): they are loaded, never stored, and kept out of every
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

constexpr uint64_t kWaitNs = 4000000000ull;  // limit of one bounded wait
constexpr int kRows = 128;
constexpr int kNoWindow = 1 << 30;  // more than any sequence has; differences with it stay within 32 bits

struct Seq {
    int begin, len;   // first token, tokens
    int tile, local;  // global number of its (first) 128-row tile, tile within the sequence
};

// The map from a CTA's units of work to tiles of R rows (128 or 256), one per warp (every call is
// warp-collective).  With up to 32 sequences the tiles come in descending order of their work: a tile of a
// causal sequence of t tiles has 1, 2, .. or t tiles to look at, one tile of each (a window caps the larger
// ones, which keeps the order), so the r-th heaviest is found by counting.  With more sequences they come in the
// sequences' order, the heaviest of a sequence first; a warp asks for them in that order, and reads the array on from
// where it was.
template <int R>
struct TileMap {
    const int32_t* cu;
    int nseq, T;
    int s0;                   // the 32 sequences held, from this one on:
    int b, e, t;              // this lane's one, its tiles,
    int first, first128;      // and the tiles before them, of R and of 128 rows
    int upto, upto128, end;   // tiles up to the 32's end, their last token
    int total;                // tiles of all

    static __device__ __forceinline__ int scan(int x) {  // inclusive
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, x, o);
            if ((int)(threadIdx.x & 31) >= o) x += y;
        }
        return x;
    }
    // Entry `i` of the array, within [0, T].
    __device__ __forceinline__ int at(int i) const { return i <= nseq ? min(max(__ldg(cu + i), 0), T) : 0; }
    // Takes the next 32 sequences, this lane's from entry x to entry y.  Entries count as the largest so far: whatever
    // the array holds, the sequences do not overlap, and their tiles stay within the host's bound.
    __device__ __forceinline__ void load(int x, int y) {
        b = max(x, end);
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int z = __shfl_up_sync(0xffffffffu, b, o);
            if ((int)(threadIdx.x & 31) >= o) b = max(b, z);
        }
        e = max(y, b);
        end = __shfl_sync(0xffffffffu, e, 31);
        t = (e - b + R - 1) / R;
        int incl = scan(t);
        first = upto + incl - t;
        upto += __shfl_sync(0xffffffffu, incl, 31);
        if (R == kRows) {
            first128 = first;
            upto128 = upto;
        } else {
            const int t128 = (e - b + kRows - 1) / kRows;
            incl = scan(t128);
            first128 = upto128 + incl - t128;
            upto128 += __shfl_sync(0xffffffffu, incl, 31);
        }
    }
    __device__ __forceinline__ TileMap(const int32_t* cu_, int nseq_, int T_) : cu(cu_), nseq(nseq_), T(T_) {
        const int lane = threadIdx.x & 31;
        s0 = upto = upto128 = end = 0;
        int x = at(lane), y = at(lane + 1);
        load(x, y);
        if (nseq > 32) {
            const int x0 = x, y0 = y;
            x = at(lane + 32);
            y = at(lane + 33);
            for (int s = 32; s < nseq; s += 32) {
                const int xn = at(s + lane + 32), yn = at(s + lane + 33);  // on their way during the sums
                load(x, y);
                x = xn;
                y = yn;
            }
            total = upto;
            upto = upto128 = end = 0;
            load(x0, y0);
        } else {
            total = upto;
        }
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
        while (rank >= upto && s0 < nseq) {
            s0 += 32;
            load(at(s0 + lane), at(s0 + lane + 1));
        }
        const uint32_t hit = __ballot_sync(0xffffffffu, rank >= first && rank < first + t);
        if (!hit) return false;  // an array that changes meanwhile
        const int src = __ffs(hit) - 1;
        const int n = __shfl_sync(0xffffffffu, t, src), i = rank - __shfl_sync(0xffffffffu, first, src);
        take(out, src, up ? n - 1 - i : i);
        return true;
    }
};

struct Ctx {
    uint64_t* bars;
    volatile int* abort_flag;
    int* err;
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
        if (now - t0 > kWaitNs) {
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

// Kernels launched ahead of the end of the one before them in the stream: that one lets it happen, once its CTAs
// are all running; this one waits until it is complete and its writes are visible.
__device__ __forceinline__ void grid_launch_next() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void grid_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// Units of work (a tile of the order, and a head), drawn from a counter in the caller's workspace, which the call
// has cleared, so that whoever is free takes the heaviest one left.  Results do not depend on who computes them.  The copying warp draws (it runs ahead), finds the tile and
// passes it on through four slots in shared memory.
struct Unit {
    int begin, len;   // the sequence's first token, its tokens
    int tile, local;  // global number of its (first) 128-row tile, tile within the sequence
    int head;
};
struct UnitQueue {
    static constexpr uint32_t kBytes = 4 * 32;
    static constexpr int kBars = 8;  // [4] passed on (an arrival), [4] read (an arrival a reading warp)
    volatile int* slots;  // [4][8] shared: a Unit, and whether there is one
    int bar;              // the first of the barriers
    bool own;             // whether the CTA's first unit is its own number: not where a grid's CTAs start late, one by
                          // one, and would find the heaviest units still waiting for them
    int n;                // units so far
    // Drawing side, the whole warp (counter: NULL where there is a unit a CTA at most): the next unit; false past the last one, or after an expired wait (then ok is
    // false too).  The heads of a tile are next to one another; `up` as in TileMap::find.
    template <int R>
    __device__ __forceinline__ bool draw(const Ctx& cx, TileMap<R>& map, int heads, bool up, int* counter, Unit& x,
                                         bool& ok) {
        if (n >= 4 && !(ok = wait_warp(cx, bar + 4 + (n & 3), ((n >> 2) - 1) & 1))) return false;
        const bool lead = (threadIdx.x & 31) == 0;
        int64_t u = blockIdx.x;
        if (n || !own) {
            u = INT32_MAX;
            if (lead && counter) u = (own ? (int64_t)gridDim.x : 0) + atomicAdd(counter, 1);
        }
        u = __shfl_sync(0xffffffffu, u, 0);
        bool have = u < (int64_t)map.total * heads;  // below 2^31: the host checks
        if (have) {
            Seq sq{};
            const uint32_t rank = (uint32_t)u / (uint32_t)heads;
            have = map.find((int)rank, up, sq);
            x = Unit{sq.begin, sq.len, sq.tile, sq.local, (int)((uint32_t)u - rank * (uint32_t)heads)};
        }
        if (lead) {
            volatile int* s = slots + 8 * (n & 3);
            s[0] = x.begin; s[1] = x.len; s[2] = x.tile; s[3] = x.local; s[4] = x.head; s[5] = have;
            mbar_arrive(cx.bars + bar + (n & 3));
        }
        ++n;
        return have;
    }
    // Reading side, a whole warp: false past the last unit, or after an expired wait (then ok is false too).
    __device__ __forceinline__ bool take(const Ctx& cx, Unit& x, bool& ok) {
        if (!(ok = wait_warp(cx, bar + (n & 3), (n >> 2) & 1))) return false;
        const volatile int* s = slots + 8 * (n & 3);
        x = Unit{s[0], s[1], s[2], s[3], s[4]};
        const bool have = s[5] != 0;
        __syncwarp();
        if ((threadIdx.x & 31) == 0) mbar_arrive(cx.bars + bar + 4 + (n & 3));
        ++n;
        return have;
    }
};

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

__device__ __forceinline__ f2 exp2_pair(f2 x) {
    float a, b;
    f2_get(x, a, b);
    return f2_of(exp2_approx(a), exp2_approx(b));
}

// The columns lo .. hi of 32, as bits.
__device__ __forceinline__ uint32_t columns(int lo, int hi) {
    if (hi < 0 || lo > 31 || lo > hi) return 0u;
    return (0xFFFFFFFFu << max(lo, 0)) & (0xFFFFFFFFu >> (31 - min(hi, 31)));
}
// Entries without their bit to `fill`.  A warp that has them all skips it.
__device__ __forceinline__ void mask_columns(uint32_t (&s)[32], uint32_t bits, uint32_t fill) {
    if (__all_sync(0xffffffffu, bits == 0xFFFFFFFFu)) return;
#pragma unroll
    for (int e = 0; e < 32; ++e)
        if (!(bits & (1u << e))) s[e] = fill;
}
constexpr uint32_t kMinusInf = 0xFF800000u;

// One arrival for a warp, after all its lanes' tensor-memory and shared-memory work.
__device__ __forceinline__ void arrive_warp(const Ctx& cx, int bar) {
    tc_fence_before();
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(cx.bars + bar);
}

// Four lanes' 16-byte pieces exchanged, w[lane][piece] for w[piece][lane]: rows and columns 1 apart, then 2.  All lanes.
__device__ __forceinline__ void exchange4(uint32_t (&w)[4][4]) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int o = 1; o <= 2; ++o) {
        const bool odd = lane & o;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            if (c & o) continue;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const uint32_t got = __shfl_xor_sync(0xffffffffu, odd ? w[c][j] : w[c + o][j], o);
                if (odd) w[c][j] = got;
                else w[c + o][j] = got;
            }
        }
    }
}
// 32 columns of 32 consecutive rows, a row a lane, as bf16 to dst (the first lane's row; rows `stride` elements apart),
// for the rows below `rows`.  Four lanes exchange their 16-byte pieces first, so that a store writes 64 bytes each of
// 8 rows: a store of 16 bytes each of 32 rows takes the load/store unit 32 cycles, which the whole CTA waits for at
// the end of its unit of work.  All lanes.
__device__ __forceinline__ void store_rows(__nv_bfloat16* dst, int64_t stride, const float (&x)[32], int rows) {
    const int lane = threadIdx.x & 31;
    uint32_t w[4][4];  // piece, word
#pragma unroll
    for (int i = 0; i < 16; ++i) w[i >> 2][i & 3] = pack_bf16x2(x[2 * i], x[2 * i + 1]);
    exchange4(w);
    dst += (lane & ~3) * stride + 8 * (lane & 3);
    rows -= lane & ~3;
#pragma unroll
    for (int i = 0; i < 4; ++i, dst += stride)
        if (i < rows) *reinterpret_cast<uint4*>(dst) = make_uint4(w[i][0], w[i][1], w[i][2], w[i][3]);
}
// The same of 32 columns as they are, fp32.
__device__ __forceinline__ void store_rows_f32(float* dst, int64_t stride, const uint32_t (&x)[32], int rows) {
    const int lane = threadIdx.x & 31;
    dst += (lane & ~3) * stride + 4 * (lane & 3);
    rows -= lane & ~3;
#pragma unroll
    for (int c = 0; c < 32; c += 16) {
        uint32_t w[4][4];
#pragma unroll
        for (int i = 0; i < 16; ++i) w[i >> 2][i & 3] = x[c + i];
        exchange4(w);
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (i < rows) *reinterpret_cast<uint4*>(dst + i * stride + c) = make_uint4(w[i][0], w[i][1], w[i][2], w[i][3]);
    }
}

}  // namespace attn
}  // namespace gdn

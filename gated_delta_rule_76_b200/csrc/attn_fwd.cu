// Causal softmax attention over packed sequences, forward, on the 5th-generation tensor cores.
//
// A unit of work is two tiles of 128 query rows that look at the same keys: the same rows of two query heads
// of one key head (PAIR_HEADS, where the group is even: their key tiles are the same), or else 256 rows of one
// head.  Keys come in tiles of 128 from the diagonal down to the window's edge (the diagonal first: every row
// then has a finite maximum from the first tile on).  For each of the two:
//     S = Q K^T            tcgen05, Q and K row tiles in shared memory, 128 columns of tensor memory
//     P = exp2(S c - m)    a thread a row: c = scale log2(e), running reference m and sum l
//     O += P V             tcgen05, P as bf16 over S's columns (A in tensor memory), V as MN-major B
// m is not moved for every new maximum: any reference within 2^8 of it serves as well (p stays below
// 2^8, sums stay fp32, and bf16's relative rounding is no larger for it), so a row's part of the O accumulator is
// rescaled only when its own maximum has outgrown m by more than 8.
// P is rounded to bf16 because that is what the tensor cores multiply with bf16 V; l sums the unrounded p.
//
// One CTA an SM stays for the whole call and walks its units as one stream.  Warps 0-3 and 4-7 are the
// softmax of either tile, warp 8 copies, warp 9 issues the products, in the order
//     P0(j) ready: P0 V (j), S0(j+1) | P1(j) ready: P1 V (j), S1(j+1) | ...
// so the tensor pipe works on one tile while the other's softmax runs.  (One issuer: two let the tiles' products
// interleave, which lengthens both chains: 381 us against 300 for 8192 tokens, 16 heads.)  P goes over in two halves, so
// that the first half of P V runs under the second half's exponentials.  Every wait is bounded.
//
// What bounds: a tile's own chain, about 3400 cycles an item on the timestamps: softmax 1750, then until the next S is
// seen 1650 (the second half of P V 256, S 512, about 490 from a product's last instruction to its barrier, and the
// waits).  Products alone take 2048 a pair of items (an S product reads shared memory at its full 128 bytes a cycle;
// the two tiles share each copy of K and V), the exponentials as long (16 a cycle and SM).  A prompt of 16384
// tokens, 8 heads of 128 on one: 440 us, 1250 TFLOP/s, the tensor pipe active 57% of the time.  At a unit's end the CTA
// waits about 3500 cycles more for the last P V, the rows on their way out and the first masked tile.
// Of the kernels only those of heads of 128 that keep the cache, whole, spill: 4 bytes (pairs of heads) and 40.
// Where units are few, each is cut into parts of its key tiles (attn.h), whose sums against their own references go through
// the workspace in fp32 and are joined by a second kernel.
// Tried and slower: 3 of 8 exponentials by a polynomial on the FMA pipe (514 us instead of 447: the softmax's
// instructions are in the chain, the exponential unit is not what it waits for); S in steps of 64 keys with two
// buffers each (636 us: the narrow product takes 386 cycles instead of 256, and every step its own waits); units of one
// tile where there are few (2600 tokens, 8 heads: 57 us instead of 55).
#include "attn_tc.cuh"
#include "launch.h"
#include "tma_host.h"

namespace gdn {
namespace attn {
namespace {

constexpr int kThreads = 384;
constexpr int kCopyWarp = 8, kMmaWarp = 9;  // warps 10 and 11 complete their warpgroup
// Registers a thread: the launch's, and what the softmax warpgroups and the third take of them
constexpr int kRegs = 168, kSoftmaxRegs = 200, kOtherRegs = 88;
static_assert(256 * kSoftmaxRegs + 128 * kOtherRegs <= kThreads * kRegs, "the split waits forever above the launch's total");

template <int D>
struct FwdSmem {
    static constexpr int kStages = D == 128 ? 5 : 10;  // ring of K and V tiles, K(0) V(0) K(1) V(1) ..
    static constexpr uint32_t kTile = kRows * D * 2;
    static constexpr uint32_t kQ = 0, kRing = 2 * kTile, kBar = kRing + kStages * kTile;
    static constexpr uint32_t kBytes = kBar + 320 + UnitQueue::kBytes;  // the dynamic array starts on 1024 bytes
    static __device__ __forceinline__ uint32_t ring(int i) { return kRing + (uint32_t)(i % kStages) * kTile; }
};
static_assert(FwdSmem<128>::kBytes <= 232448, "227 KB");
enum FwdBar {
    B_Q = 0, B_Q_FREE,
    B_S,                  // [2 tiles] S done
    B_PA = B_S + 2,       // [2] first half of P written (an arrival a warp)
    B_PB = B_PA + 2,      // [2] second half
    B_O = B_PB + 2,       // [2] the unit's last P V done
    B_U = B_O + 2,        // UnitQueue
    B_R = B_U + UnitQueue::kBars,  // [stages] landed
    // [8] ring tiles 2q + 1 and 2q + 2 read for the last time (q mod 8).  A barrier must not complete again before the
    // copying warp has waited for it: with 10 stages tile 2q + 10 is loaded once pair q - 1 is free, so that pairs
    // q to q + 4 may be freed in a row.
    B_R_FREE = B_R + 10,
    B_COUNT = B_R_FREE + 8
};
static_assert(B_COUNT * 8 <= 304, "barriers");
// tensor memory: S of either tile, O of either tile
constexpr uint32_t TM_S = 0, TM_O = 256, TM_COLS = 512;

struct FwdParams {
    AttnIO io;
    int tiles;         // bound on the 128-row tiles
    int window;        // kNoWindow: none
    int parts;         // of a unit's key tiles
    float scale_log2;
};

// The two tiles of a unit: first row within the sequence, its own key tile, query head, and key tiles hi down to lo
// (hi < lo: there is nothing to do, or no such tile).
struct Tile {
    int row0, diag, head, hi, lo;
};
struct Pair {
    Tile a, b;
    int top, bottom;  // key tiles of either; top < bottom: none
    int part;
};
template <bool PAIR_HEADS>
__device__ __forceinline__ Tile tile_of(const Unit& un, int unit_head, int window, int s) {
    Tile t;
    t.row0 = PAIR_HEADS ? un.local * kRows : (2 * un.local + s) * kRows;
    t.head = PAIR_HEADS ? 2 * unit_head + s : unit_head;
    t.diag = t.hi = t.row0 / kRows;
    t.lo = t.row0 < un.len ? max(0, t.row0 - window + 1) / kRows : t.hi + 1;
    return t;
}
template <bool PAIR_HEADS, bool PARTS>
__device__ __forceinline__ Pair pair_of(const Unit& un, const FwdParams& p) {
    Pair pr;
    const int unit_head = PARTS ? un.head / p.parts : un.head;
    pr.part = un.head - (PARTS ? unit_head * p.parts : un.head);
    pr.a = tile_of<PAIR_HEADS>(un, unit_head, p.window, 0);
    pr.b = tile_of<PAIR_HEADS>(un, unit_head, p.window, 1);
    pr.top = pr.b.hi >= pr.b.lo ? pr.b.hi : pr.a.hi;
    pr.bottom = pr.a.lo;  // the first tile exists, and sees at least as far back
    if (PARTS) {
        const int64_t n = pr.top - pr.bottom + 1;
        const int from = (int)(n * pr.part / p.parts), to = (int)(n * (pr.part + 1) / p.parts);
        pr.bottom = pr.top - to + 1;
        pr.top -= from;
        pr.a.hi = min(pr.a.hi, pr.top);
        pr.b.hi = min(pr.b.hi, pr.top);
        pr.a.lo = max(pr.a.lo, pr.bottom);
        pr.b.lo = max(pr.b.lo, pr.bottom);
    }
    return pr;
}

// The issuing thread's place in the stream of ring tiles.
template <int D>
struct RingAt {
    uint32_t slot = 0, phase = 0;
    __device__ __forceinline__ void next() {
        if (++slot == (uint32_t)FwdSmem<D>::kStages) {
            slot = 0;
            phase ^= 1u;
        }
    }
    __device__ __forceinline__ bool landed(const Ctx& cx) const { return wait_bar(cx, B_R + slot, phase); }
};

// S of tile S against the K tile in ring slot `slot`.
template <int D, int S>
__device__ __forceinline__ void s_product(const Ctx& cx, uint32_t tbase, uint32_t q_desc, uint32_t ring_k, uint32_t slot) {
    constexpr uint32_t step = FwdSmem<D>::kTile >> 4;
    mma_ss_rows<D>(tbase + TM_S + 128 * S, q_desc + S * step, ring_k + slot * step);
    mma_commit(cx.bars + B_S + S);
}
// Tile S's part of key tile kt: P V with V in ring slot v, then S of the next key tile with K in slot k.
template <int D, int S>
__device__ __forceinline__ bool tile_step(const Ctx& cx, uint32_t tbase, const Tile& t, int kt, uint32_t q_desc,
                                          uint32_t ring_k, uint32_t ring_mn, uint32_t v, const RingAt<D>& k,
                                          uint32_t& parity) {
    constexpr uint32_t step = FwdSmem<D>::kTile >> 4;
    if (kt <= t.hi && kt >= t.lo) {
        const uint32_t vd = ring_mn + v * step;
        if (!wait_bar(cx, B_PA + S, parity)) return false;
        tc_fence_after();
        mma_ts_rows<D, 0, 64>(tbase + TM_O + 128 * S, tbase + TM_S + 128 * S, vd, kt < t.hi);
        if (!wait_bar(cx, B_PB + S, parity)) return false;
        tc_fence_after();
        mma_ts_rows<D, 64, 128>(tbase + TM_O + 128 * S, tbase + TM_S + 128 * S, vd, true);
        if (kt == t.lo) mma_commit(cx.bars + B_O + S);
        parity ^= 1u;
    }
    if (kt - 1 <= t.hi && kt - 1 >= t.lo) {
        if (!k.landed(cx)) return false;
        s_product<D, S>(cx, tbase, q_desc, ring_k, k.slot);  // runs after P V, so it may write over P
    }
    return true;
}

__device__ __forceinline__ float max3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

// PARTS: units are cut into parts of their key tiles (attn.h).
template <int D, bool SAVE, bool PAIR_HEADS, bool PARTS>
__global__ void __launch_bounds__(kThreads, 1)
attn_fwd_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                const __grid_constant__ CUtensorMap tm_v, const FwdParams p) {
    using L = FwdSmem<D>;
    constexpr int NS = L::kStages;
    extern __shared__ __align__(1024) uint8_t sm[];
    const uint32_t sb = smem_u32(sm);
    const int tid = threadIdx.x, warp = tid >> 5;
    const int G = p.io.Hq / p.io.Hk, heads = (PAIR_HEADS ? p.io.Hq / 2 : p.io.Hq) * (PARTS ? p.parts : 1);

    Ctx cx;
    cx.bars = reinterpret_cast<uint64_t*>(sm + L::kBar);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sm + L::kBar + 304);
    cx.abort_flag = reinterpret_cast<volatile int*>(sm + L::kBar + 308);
    cx.err = p.io.err;
    if (blockIdx.x == 0 && tid == 0) *cx.err = 0;  // every CTA is running, and none gives up a wait within microseconds
    if (sb & 1023u) {
        if (tid == 0) atomicOr(cx.err, 1);
        return;
    }
    if (tid == 0) {
        for (int i = 0; i < B_COUNT; ++i) mbar_init(cx.bars + i, i >= B_U + 4 && i < B_R ? kCopyWarp + 1 : i >= B_PA && i < B_O ? 4 : 1);
        *cx.abort_flag = 0;
        mbar_fence_init();
    }
    if (warp == kMmaWarp) {
        tmem_alloc(tmem_slot, TM_COLS);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tbase = *tmem_slot;
    UnitQueue units{reinterpret_cast<volatile int*>(sm + L::kBar + 320), B_U, true, 0};
    Unit un{};
    bool ok = true;

    if (warp >= 8) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
        if (warp == kCopyWarp) {
            int owns = 0, ri = 0;  // Q loads and ring loads issued
            TileMap<PAIR_HEADS ? kRows : 2 * kRows> map(p.io.cu, p.io.nseq, p.io.T);
            while (units.draw(cx, map, heads, true, p.io.counters, un, ok)) {
                const Pair pr = pair_of<PAIR_HEADS, PARTS>(un, p);
                if (PARTS && pr.top < pr.bottom) continue;
                const int hk = pr.a.head / G;
                if ((tid & 31) == 0) {
                    auto load = [&](const CUtensorMap* map_, int kt) -> bool {
                        if (ri >= NS) {  // the slot's last tile, ri - NS, is free with its pair
                            const int q = ri > NS ? (ri - NS - 1) >> 1 : 0;
                            if (!wait_bar(cx, B_R_FREE + (q & 7), (q >> 3) & 1)) return false;
                        }
                        uint64_t* bar = cx.bars + B_R + ri % NS;
                        mbar_arrive_expect_tx(bar, L::kTile);
                        load_tile<D>(sb + L::ring(ri), map_, bar, hk, un.begin + kt * kRows);
                        ++ri;
                        return true;
                    };
                    ok = load(&tm_k, pr.top);  // need not wait for the unit before
                    if (ok && owns) ok = wait_bar(cx, B_Q_FREE, (owns - 1) & 1);
                    if (ok) {
                        const bool two = pr.b.hi >= pr.b.lo;
                        mbar_arrive_expect_tx(cx.bars + B_Q, two ? 2 * L::kTile : L::kTile);
                        load_tile<D>(sb + L::kQ, &tm_q, cx.bars + B_Q, pr.a.head, un.begin + pr.a.row0);
                        if (two) load_tile<D>(sb + L::kQ + L::kTile, &tm_q, cx.bars + B_Q, pr.b.head, un.begin + pr.b.row0);
                        ++owns;
                    }
                    ok = ok && load(&tm_v, pr.top);
                    for (int kt = pr.top - 1; ok && kt >= pr.bottom; --kt) ok = load(&tm_k, kt) && load(&tm_v, kt);
                }
                if (!(ok = __shfl_sync(0xffffffffu, (int)ok, 0) != 0)) break;
            }
            if ((tid & 31) == 0 && *cx.abort_flag) {
                // after an expired wait: the copies still on their way land before the memory is given up
                if (owns) mbar_wait(cx.bars + B_Q, (owns - 1) & 1, kWaitNs);
                for (int i = ri < NS ? 0 : ri - NS; i < ri; ++i) mbar_wait(cx.bars + B_R + i % NS, (i / NS) & 1, kWaitNs);
            }
            __syncwarp();
        } else if (warp == kMmaWarp) {
            // The stream of ring tiles: K, V K, V K, .., V and the next unit's K, ..; a V and the K after it are freed
            // together, after the K's products.
            uint32_t q_parity = 0, p0 = 0, p1 = 0, pairs = 0;
            RingAt<D> at;
            const uint32_t q_desc = desc_k(sb + L::kQ), ring_k = desc_k(sb + L::kRing), ring_mn = desc_mn(sb + L::kRing);
            bool first = true;
            while (units.take(cx, un, ok)) {
                const Pair pr = pair_of<PAIR_HEADS, PARTS>(un, p);
                if (PARTS && pr.top < pr.bottom) continue;
                if ((tid & 31) == 0) {
                    ok = wait_bar(cx, B_Q, q_parity) && at.landed(cx);
                    q_parity ^= 1u;
                    if (ok) {
                        if (pr.top <= pr.a.hi && (!PARTS || pr.top >= pr.a.lo)) s_product<D, 0>(cx, tbase, q_desc, ring_k, at.slot);
                        if (pr.b.hi >= pr.b.lo) s_product<D, 1>(cx, tbase, q_desc, ring_k, at.slot);
                        if (!first) mma_commit(cx.bars + B_R_FREE + (pairs++ & 7));
                        first = false;
                        if (pr.top == pr.bottom) mma_commit(cx.bars + B_Q_FREE);
                    }
                    for (int kt = pr.top; ok && kt >= pr.bottom; --kt) {
                        at.next();
                        const uint32_t v = at.slot;
                        if (!(ok = at.landed(cx))) break;
                        at.next();  // the next K, of this unit or of the one after
                        ok = tile_step<D, 0>(cx, tbase, pr.a, kt, q_desc, ring_k, ring_mn, v, at, p0) &&
                             tile_step<D, 1>(cx, tbase, pr.b, kt, q_desc, ring_k, ring_mn, v, at, p1);
                        if (ok && kt > pr.bottom) {
                            mma_commit(cx.bars + B_R_FREE + (pairs++ & 7));
                            if (kt - 1 == pr.bottom) mma_commit(cx.bars + B_Q_FREE);
                        }
                    }
                }
                if (!(ok = __shfl_sync(0xffffffffu, (int)ok, 0) != 0)) break;
            }
            __syncwarp();
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
        const int s_ = warp >> 2, lane = tid & 127;  // tile of the pair, row within it
        const uint32_t tl = tbase + ((uint32_t)((warp & 3) * 32) << 16);
        const uint32_t t_s = tl + TM_S + 128 * s_, t_o = tl + TM_O + 128 * s_;
        const f2 scale2 = f2_of(p.scale_log2, p.scale_log2);
        int gi = 0, done = 0;  // items and units of this tile so far
        int ri = 0;            // ring tiles so far
        while (units.take(cx, un, ok)) {
            const Pair pr = pair_of<PAIR_HEADS, PARTS>(un, p);
            const Tile me = s_ ? pr.b : pr.a;
            const int row0 = me.row0, hi = me.hi, lo = me.lo;
            const int row = row0 + lane;
            float m = -INFINITY, l = 0.f;
            for (int kt = hi; kt >= lo; --kt, ++gi) {
                if (!(ok = wait_warp(cx, B_S + s_, gi & 1))) break;
                tc_fence_after();  // P V of the tile before is complete as well: S was issued after it
                uint32_t s[4][32];
#pragma unroll
                for (int c = 0; c < 4; ++c) tmem_ld32(t_s + 32 * c, s[c]);
                tmem_ld_wait();
                const int key0 = kt * kRows;
                // keys after the row, or out of its window, leave the softmax
                if (kt == (PARTS ? me.diag : hi) || key0 <= row0 + kRows - 1 - p.window) {
                    const int last = row - key0;
#pragma unroll
                    for (int c = 0; c < 4; ++c) mask_columns(s[c], columns(last - p.window + 1 - 32 * c, last - 32 * c), kMinusInf);
                }
                float x[4];
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    x[c] = fmaxf(__uint_as_float(s[c][0]), __uint_as_float(s[c][1]));
#pragma unroll
                    for (int e = 2; e < 32; e += 2) x[c] = max3(x[c], __uint_as_float(s[c][e]), __uint_as_float(s[c][e + 1]));
                }
                const float mx = fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3])) * p.scale_log2;
                // Each row decides for itself; the vote only skips the work.  p's rounding goes by m, so that a row that moved
                // with its warp's others would get other bits from padding, the next sequence's rows or later queries.
                const bool move = mx > m + 8.f;
                if (__any_sync(0xffffffffu, move)) {
                    const float f = !move ? 1.f : m == -INFINITY ? 0.f : exp2_approx(m - mx);
                    if (move) m = mx;
                    l *= f;
                    if (kt < hi) {
#pragma unroll
                        for (int c = 0; c < D / 16; ++c) {
                            uint32_t o[16];
                            tmem_ld16(t_o + 16 * c, o);
                            tmem_ld_wait();
#pragma unroll
                            for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                            tmem_st16(t_o + 16 * c, o);
                        }
                    }
                }
                // a row that sees none of the keys so far (in a part that starts at the window's edge) keeps p = 0
                const float nm1 = PARTS && m == -INFINITY ? 0.f : -m;
                const f2 nm = f2_of(nm1, nm1);
                f2 sum[2] = {f2_of(0.f, 0.f), f2_of(0.f, 0.f)};
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    uint32_t w[16];
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        const f2 y = f2_fma(f2_of(s[c][2 * e], s[c][2 * e + 1]), scale2, nm);
                        const f2 x = exp2_pair(y);
                        sum[e & 1] = f2_add(sum[e & 1], x);
                        float a, b;
                        f2_get(x, a, b);
                        w[e] = pack_bf16x2(a, b);
                    }
                    tmem_st16(t_s + 16 * c, w);
                    if (c == 1) {
                        if (kt == (PARTS ? me.diag : hi) && un.len - key0 < kRows && (!PAIR_HEADS || s_ == 0)) {
                            // V's rows past the sequence: p is 0 there, but 0 * NaN is not.  Two heads share the
                            // tile, whose product with P1 follows the one with P0.
                            const int slot = ri + 2 * (pr.top - kt) + 1;
                            if (!(ok = wait_warp(cx, B_R + slot % NS, (slot / NS) & 1))) break;
                            if (lane >= un.len - key0) zero_row<D>(sm + L::ring(slot), lane);
                            fence_async_shared();
                        }
                        tmem_st_wait();
                        arrive_warp(cx, B_PA + s_);
                    }
                }
                if (!ok) break;
                tmem_st_wait();
                arrive_warp(cx, B_PB + s_);
                float a, b;
                f2_get(f2_add(sum[0], sum[1]), a, b);
                l += a + b;
            }
            ri += 2 * (pr.top - pr.bottom + 1);
            if (!ok) break;
            const bool live = row < un.len;
            if (PARTS && live) p.io.part_ml[((int64_t)pr.part * p.io.T + un.begin + row) * p.io.Hq + me.head] = make_float2(m, l);
            if (hi < lo) continue;
            if (!(ok = wait_warp(cx, B_O + s_, done & 1))) break;
            ++done;
            tc_fence_after();
            // the next unit's first product into O waits for its P, which follows this
            const int64_t stride = (int64_t)p.io.Hq * D;
            const int first = row - (lane & 31), rows = un.len - first;  // of the warp
            const int64_t at = (int64_t)(un.begin + first) * stride + me.head * D;
            if (PARTS) {
#pragma unroll
                for (int c = 0; c < D; c += 32) {
                    uint32_t o[32];
                    tmem_ld32(t_o + c, o);
                    tmem_ld_wait();
                    store_rows_f32(p.io.part_o + (int64_t)pr.part * p.io.T * stride + at + c, stride, o, rows);
                }
                continue;
            }
            const float inv = 1.f / l;
#pragma unroll
            for (int c0 = 0; c0 < D; c0 += 64) {
                uint32_t o[2][32];
                tmem_ld32(t_o + c0, o[0]);
                tmem_ld32(t_o + c0 + 32, o[1]);
                tmem_ld_wait();
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    float v[32];
#pragma unroll
                    for (int e = 0; e < 32; ++e) v[e] = __uint_as_float(o[c][e]) * inv;
                    store_rows(static_cast<__nv_bfloat16*>(p.io.o) + at + c0 + 32 * c, stride, v, rows);
                    if (SAVE) {
#pragma unroll
                        for (int e = 0; e < 32; ++e) v[e] -= __bfloat162float(__float2bfloat16_rn(v[e]));
                        store_rows(static_cast<__nv_bfloat16*>(p.io.o_lo) + at + c0 + 32 * c, stride, v, rows);
                    }
                }
            }
            // every row of the tile, so that the backward's copies of it read no uninitialised memory
            if (SAVE) {
                const int tile = un.tile + (PAIR_HEADS ? 0 : s_);
                p.io.lse[((int64_t)me.head * p.tiles + tile) * kRows + lane] = live ? -(m + log2f(l)) : 0.f;
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == kMmaWarp) tmem_dealloc(tbase, TM_COLS);
}

// o of a tile of rows and a head from its parts: each has the sums of its keys against its own reference m.
// D / 4 lanes a row, a row a lane.
template <int D, bool SAVE>
__global__ void __launch_bounds__(256) attn_fwd_join_kernel(const FwdParams p) {
    constexpr int LANES = D / 4;
    Seq sq{};
    const int head = blockIdx.x % p.io.Hq;
    TileMap<kRows> map(p.io.cu, p.io.nseq, p.io.T);
    const bool have = map.find((int)(blockIdx.x / p.io.Hq), true, sq);
    const int r = blockIdx.y * (256 / LANES) + threadIdx.x / LANES, row = sq.local * kRows + r, c = (threadIdx.x % LANES) * 4;
    grid_wait();
    if (!have) return;
    float nlse = 0.f;  // of rows past the sequence
    if (row < sq.len) {
        const int64_t rows = (int64_t)p.io.T * p.io.Hq, at = (int64_t)(sq.begin + row) * p.io.Hq + head;
        float m = -INFINITY;
#pragma unroll 4
        for (int s = 0; s < p.parts; ++s) m = fmaxf(m, __ldcg(p.io.part_ml + s * rows + at).x);
        float l = 0.f, v[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
        for (int s = 0; s < p.parts; ++s) {
            const float2 ml = __ldcg(p.io.part_ml + s * rows + at);
            const bool sees = ml.x != -INFINITY;  // else nothing was written
            const float f = sees ? exp2_approx(ml.x - m) : 0.f;
            const float4 o = sees ? __ldcg(reinterpret_cast<const float4*>(p.io.part_o + (s * rows + at) * D + c))
                                  : make_float4(0.f, 0.f, 0.f, 0.f);
            l = fmaf(f, ml.y, l);
            v[0] = fmaf(f, o.x, v[0]);
            v[1] = fmaf(f, o.y, v[1]);
            v[2] = fmaf(f, o.z, v[2]);
            v[3] = fmaf(f, o.w, v[3]);
        }
        const float inv = 1.f / l;
        uint32_t hi[2], lo[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const float x = v[2 * i] * inv, y = v[2 * i + 1] * inv;
            hi[i] = pack_bf16x2(x, y);
            lo[i] = pack_bf16x2(x - __uint_as_float(hi[i] << 16), y - __uint_as_float(hi[i] & 0xFFFF0000u));
        }
        *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.io.o) + at * D + c) = make_uint2(hi[0], hi[1]);
        if (SAVE) *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.io.o_lo) + at * D + c) = make_uint2(lo[0], lo[1]);
        nlse = -(m + log2f(l));
    }
    if (SAVE && c == 0) p.io.lse[((int64_t)head * p.tiles + sq.tile) * kRows + r] = nlse;
}

template <int D, bool SAVE, bool PAIR_HEADS, bool PARTS>
cudaError_t launch(const CUtensorMap* maps, FwdParams p, cudaStream_t st) {
    auto kernel = attn_fwd_kernel<D, SAVE, PAIR_HEADS, PARTS>;
    cudaError_t e =
        cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)FwdSmem<D>::kBytes);
    cudaFuncAttributes attr;
    if (e == cudaSuccess) e = cudaFuncGetAttributes(&attr, kernel);
    if (e != cudaSuccess) return e;
    if (attr.numRegs < kRegs) return cudaErrorInvalidConfiguration;  // setmaxnreg counts on them
    const int64_t units = (int64_t)p.tiles * p.io.Hq / (PAIR_HEADS ? 2 : 1) * p.parts;
    if (units <= 148) p.io.counters = nullptr;  // a unit a CTA
    else if ((e = cudaMemsetAsync(p.io.counters, 0, sizeof(int), st)) != cudaSuccess) return e;
    kernel<<<(unsigned)(units < 148 ? units : 148), kThreads, FwdSmem<D>::kBytes, st>>>(maps[0], maps[1], maps[2], p);
    count_launch();
    if ((e = cudaGetLastError()) != cudaSuccess || !PARTS) return e;
    cudaLaunchAttribute early{};
    early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    early.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)p.tiles * (unsigned)p.io.Hq, kRows * (D / 4) / 256);
    cfg.blockDim = dim3(256);
    cfg.stream = st;
    cfg.attrs = &early;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, attn_fwd_join_kernel<D, SAVE>, p);
    count_launch();
    return e;
}
template <int D, bool SAVE>
cudaError_t launch_s(const CUtensorMap* maps, const FwdParams& p, cudaStream_t st) {
    const bool pairs = p.io.Hq / p.io.Hk % 2 == 0;
    if (p.parts > 1) return pairs ? launch<D, SAVE, true, true>(maps, p, st) : launch<D, SAVE, false, true>(maps, p, st);
    return pairs ? launch<D, SAVE, true, false>(maps, p, st) : launch<D, SAVE, false, false>(maps, p, st);
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
    p.parts = attn_fwd_parts(io.T, io.nseq, io.Hq, d, io.window);
    p.window = io.window > 0 && io.window < attn::kNoWindow ? (int)io.window : attn::kNoWindow;
    p.scale_log2 = io.scale * 1.4426950408889634f;
    if (d == 128) return io.lse ? attn::launch_s<128, true>(maps, p, st) : attn::launch_s<128, false>(maps, p, st);
    return io.lse ? attn::launch_s<64, true>(maps, p, st) : attn::launch_s<64, false>(maps, p, st);
}

}  // namespace gdn

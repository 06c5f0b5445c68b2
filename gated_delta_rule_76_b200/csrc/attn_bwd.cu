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
// Each CTA stays for the whole call and walks its units (a tile and a head), and their items (a pair of
// tiles), as one stream: warp 8 copies, warp 9 issues the products, warps 0-7 do the element-wise work
// (thread = row and half of the columns).  The products of one item overlap the element-wise work of the
// next (issue order, dkdv):
//     S(i) dP(i) | P(i) ready: dV(i) S(i+1) | dS(i) ready: dK(i) dP(i+1) | ...
// so the tensor pipe runs dV(i), S(i+1) while dS(i) is formed, and dK(i), dP(i+1) while P(i+1) is.
// Shared memory (226 KB): the unit's own two tiles, three stages of the walked tile that S and the last product
// read (a copy takes about as long as an item, and a stage is held for one and a half), two of the other.
//
// Where the key tiles' units are few, each is cut into parts (attn.h), whose fp32 sums go through the workspace and are
// joined in their order by a last kernel.
//
// The first kernel forms delta; dkdv is set up while it runs, and waits for it.  dq needs nothing from dkdv: its CTAs
// start as dkdv's end, and fill the SMs that have run out of key tiles.
//
// What bounds: dkdv's chain of P, dV, S (about 2980 cycles an item in a long call, of which the products take 2048) and
// dq's element-wise work (2660 and 1536).  Forward and backward of 4 sequences of 2048, 16 heads of 128 on 4: 338 us, 712
// TFLOP/s of the formula's 7 products (the kernels compute 9), the tensor pipe active 51% of dkdv and 48% of dq.
// Tried and slower: dkdv with S in halves, one of them ahead of dV (8%: the narrow products' time); 16 element-wise warps
// (no difference).
//
// delta uses o with what its rounding left out (the cache's o_lo): row 0 of a sequence, where do . v - delta
// cancels, keeps a gradient of 0.  ds and p are rounded to bf16 for the products, nothing else is.
#include "attn_tc.cuh"
#include "launch.h"
#include "tma_host.h"

namespace gdn {
namespace attn {
namespace {

constexpr int kThreads = 320;
constexpr int kElem = 256;  // element-wise threads
constexpr int kCopyWarp = 8, kMmaWarp = 9;

template <int D>
struct BwdSmem {
    static constexpr uint32_t kTile = kRows * D * 2;
    static constexpr uint32_t kOwn0 = 0, kOwn1 = kTile;
    static constexpr uint32_t kA = 2 * kTile, kB = 5 * kTile;  // [3] and [2] stages
    static constexpr uint32_t kStats = 7 * kTile;              // dkdv: [2][-lse, -delta][128]
    static constexpr uint32_t kBar = kStats + 2 * 1024;
    static constexpr uint32_t kBytes = kBar + 240 + UnitQueue::kBytes;  // the dynamic array starts on 1024 bytes
    static __device__ __forceinline__ uint32_t a(int i) { return kA + (uint32_t)(i % 3) * kTile; }
    static __device__ __forceinline__ uint32_t b(int i) { return kB + (uint32_t)(i & 1) * kTile; }
};
static_assert(BwdSmem<128>::kBytes <= 232448, "227 KB");
constexpr uint32_t TM_S = 0, TM_DP = 128, TM_ACC0 = 256, TM_ACC1 = 384, TM_DS = 384, TM_COLS = 512;

enum BwdBar {
    B_OWN = 0, B_OWN_FREE,      // own tiles landed; read for the last time
    B_A, B_B = B_A + 3,         // stages of A and B landed
    B_FREE = B_B + 2,           // [4] item's stages (dq: A's) read for the last time (item mod 4)
    B_V_FREE = B_FREE + 4,      // [2] dq: stages of B read for the last time
    B_S = B_V_FREE + 2, B_DP,   // products done
    B_X, B_Y, B_DS,             // element-wise steps done (an arrival a warp)
    B_END,                      // the unit's accumulators are complete
    B_U,                        // UnitQueue
    B_COUNT = B_U + UnitQueue::kBars
};
static_assert(B_COUNT * 8 <= 224, "barriers");

struct BwdParams {
    AttnIO io;
    int tiles, window;
    int parts;  // of a key tile's unit
    float scale_log2;
};

// Barriers, tensor memory; false if the shared array does not start where the tiles need it.
__device__ __forceinline__ bool setup(Ctx& cx, uint8_t* sm, uint8_t* bars, const AttnIO& io, uint32_t*& tmem_slot) {
    cx.bars = reinterpret_cast<uint64_t*>(bars);
    tmem_slot = reinterpret_cast<uint32_t*>(bars + 224);
    cx.abort_flag = reinterpret_cast<volatile int*>(bars + 228);
    cx.err = io.err;
    if (smem_u32(sm) & 1023u) {
        if (threadIdx.x == 0) atomicOr(cx.err, 1);
        return false;
    }
    if (threadIdx.x == 0) {
        for (int i = 0; i < B_COUNT; ++i) mbar_init(cx.bars + i, i >= B_U + 4 ? kElem / 32 + 1 : i >= B_X && i <= B_DS ? kElem / 32 : 1);
        *cx.abort_flag = 0;
        mbar_fence_init();
    }
    if (threadIdx.x >> 5 == kMmaWarp) {
        tmem_alloc(tmem_slot, TM_COLS);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    return true;
}

// After an expired wait: the copies still on their way land before the memory is given up.  owns, items: how
// many of each were issued.
__device__ __forceinline__ void drain(const Ctx& cx, int owns, int a_items, int b_items) {
    if (!*cx.abort_flag) return;
    if (owns) mbar_wait(cx.bars + B_OWN, (owns - 1) & 1, kWaitNs);
    for (int i = a_items < 3 ? 0 : a_items - 3; i < a_items; ++i)
        mbar_wait(cx.bars + B_A + i % 3, (i / 3) & 1, kWaitNs);
    for (int i = b_items < 2 ? 0 : b_items - 2; i < b_items; ++i)
        mbar_wait(cx.bars + B_B + (i & 1), (i >> 1) & 1, kWaitNs);
}

// D (+)= A B with A [128 x 128] bf16 in tensor memory as two halves of 32 columns, 64 columns apart, and
// B a row tile taken MN-major; of either half the quarters Q0 .. Q1 - 1 (16 of its 64 rows of B each).
template <int D, int Q0, int Q1>
__device__ __forceinline__ void mma_halves(uint32_t d_tmem, uint32_t a_tmem, uint32_t b_desc, bool accumulate) {
    constexpr uint32_t idesc = idesc_bf16_f32_mn(128, D, false, true);
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int q = Q0; q < Q1; ++q)
            mma_ts(d_tmem, a_tmem + (uint32_t)(h * 64 + q * 8), desc_of(b_desc + (uint32_t)(((h * 64 + q * 16) * 128) >> 4)),
                   idesc, (accumulate || h > 0 || q > Q0) ? 1u : 0u);
}

// The issuing thread's place in the stream of items: stages of A and B, and the phase bits of the barriers.
template <int D>
struct ItemAt {
    static constexpr uint32_t kStep = BwdSmem<D>::kTile >> 4;
    uint32_t a = 0, a_phase = 0, b = 0, b_phase = 0, phase = 0, mod4 = 0;
    __device__ __forceinline__ void next() {
        if (++a == 3) {
            a = 0;
            a_phase ^= 1u;
        }
        b ^= 1u;
        b_phase ^= b ^ 1u;  // flips when b returns to 0
        phase ^= 1u;
        mod4 = (mod4 + 1) & 3;
    }
};

// 32 floats (16 pairs) as bf16 pairs into 16 columns.
__device__ __forceinline__ void st_quarter(uint32_t taddr, const f2* x) {
    uint32_t w[16];
#pragma unroll
    for (int e = 0; e < 16; ++e) {
        float lo, hi;
        f2_get(x[e], lo, hi);
        w[e] = pack_bf16x2(lo, hi);
    }
    tmem_st16(taddr, w);
}
// Half `h` of the D columns of an accumulator's rows, times `f`, to dst (the warp's first row; rows `stride` elements
// apart) for the rows below `rows`.
template <int D>
__device__ __forceinline__ void store_acc(uint32_t taddr, int h, __nv_bfloat16* dst, int64_t stride, float f, int rows) {
#pragma unroll
    for (int c = 0; c < D / 2; c += 32) {
        uint32_t r[32];
        tmem_ld32(taddr + h * (D / 2) + c, r);
        tmem_ld_wait();
        float v[32];
#pragma unroll
        for (int e = 0; e < 32; ++e) v[e] = __uint_as_float(r[e]) * f;
        store_rows(dst + h * (D / 2) + c, stride, v, rows);
    }
}

// The same half of this thread's row as fp32, to dst.
template <int D>
__device__ __forceinline__ void store_part(uint32_t taddr, int h, float* dst, bool live) {
#pragma unroll
    for (int c = 0; c < D / 2; c += 32) {
        uint32_t r[32];
        tmem_ld32(taddr + h * (D / 2) + c, r);
        tmem_ld_wait();
        if (!live) continue;
#pragma unroll
        for (int e = 0; e < 32; e += 4)
            *reinterpret_cast<uint4*>(dst + h * (D / 2) + c + e) = make_uint4(r[e], r[e + 1], r[e + 2], r[e + 3]);
    }
}

// Items of a key tile's unit: G heads times the query tiles local .. last that see it.
__device__ __forceinline__ int query_tiles(const Unit& un, int window) {
    const int key0 = un.local * kRows, reach = un.len - key0 - kRows;  // rows after the tile
    const int last = reach < window - 1 ? un.len - 1 : key0 + kRows - 1 + window - 1;
    return last / kRows - un.local + 1;
}

// Part `part` of a key tile's unit: its items from `first` on, m of them.
struct Part {
    int nq, first, m;
};
__device__ __forceinline__ Part part_of(const Unit& un, int part, int parts, int G, int window) {
    const int nq = query_tiles(un, window);
    const int64_t all = (int64_t)G * nq;
    const int first = (int)(all * part / parts);
    return Part{nq, first, (int)(all * (part + 1) / parts) - first};
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
attn_dkdv_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                 const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_do, const BwdParams p) {
    using L = BwdSmem<D>;
    extern __shared__ __align__(1024) uint8_t sm[];
    const uint32_t sb = smem_u32(sm);
    const int tid = threadIdx.x, warp = tid >> 5;
    const int G = p.io.Hq / p.io.Hk;
    Ctx cx;
    uint32_t* tmem_slot;
    if (!setup(cx, sm, sm + L::kBar, p.io, tmem_slot)) return;
    grid_wait();  // for delta, and the counters
    grid_launch_next();
    const uint32_t tbase = *tmem_slot;
    UnitQueue units{reinterpret_cast<volatile int*>(sm + L::kBar + 240), B_U, true, 0};
    Unit un{};
    bool ok = true;
    int gi = 0;  // items so far, over all units: the stages' and barriers' phases go by it

    if (warp == kCopyWarp) {
        int owns = 0, a_items = 0, b_items = 0;  // issued
        TileMap<kRows> map(p.io.cu, p.io.nseq, p.io.T);
        while (units.draw(cx, map, p.io.Hk * p.parts, false, p.io.counters, un, ok)) {
            const int hk = un.head / p.parts, key0 = un.begin + un.local * kRows;
            const Part pt = part_of(un, un.head - hk * p.parts, p.parts, G, p.window);
            if ((tid & 31) == 0) {
                for (int it = 0; ok && it < pt.m; ++it, ++gi) {
                    const int head = hk * G + (pt.first + it) / pt.nq, tile = (pt.first + it) % pt.nq;
                    // A's stage was freed with item gi - 3, which the load before this one has waited for
                    uint64_t* bar = cx.bars + B_A + gi % 3;
                    mbar_arrive_expect_tx(bar, L::kTile);
                    load_tile<D>(sb + L::a(gi), &tm_q, bar, head, key0 + tile * kRows);
                    ++a_items;
                    if (gi >= 2 && !(ok = wait_bar(cx, B_FREE + ((gi - 2) & 3), ((gi - 2) >> 2) & 1))) break;
                    bar = cx.bars + B_B + (gi & 1);
                    mbar_arrive_expect_tx(bar, L::kTile + 2 * kRows * 4);
                    load_tile<D>(sb + L::b(gi), &tm_do, bar, head, key0 + tile * kRows);
                    const int64_t stat = ((int64_t)head * p.tiles + un.tile + tile) * kRows;
                    bulk_g2s(sb + L::kStats + (gi & 1) * 1024u, p.io.lse + stat, kRows * 4, bar);
                    bulk_g2s(sb + L::kStats + (gi & 1) * 1024u + 512u, p.io.delta + stat, kRows * 4, bar);
                    ++b_items;
                    if (it == 0) {  // the first walked tiles need not wait for the unit before
                        if (owns && !(ok = wait_bar(cx, B_OWN_FREE, (owns - 1) & 1))) break;
                        mbar_arrive_expect_tx(cx.bars + B_OWN, 2 * L::kTile);
                        load_tile<D>(sb + L::kOwn0, &tm_k, cx.bars + B_OWN, hk, key0);
                        load_tile<D>(sb + L::kOwn1, &tm_v, cx.bars + B_OWN, hk, key0);
                        ++owns;
                    }
                }
            }
            if (!(ok = __shfl_sync(0xffffffffu, (int)ok, 0) != 0)) break;
        }
        if ((tid & 31) == 0) drain(cx, owns, a_items, b_items);
        __syncwarp();
    } else if (warp == kMmaWarp) {
        using At = ItemAt<D>;
        At at, nx;  // the item, and the one after it
        nx.next();
        uint32_t own_phase = 0;
        const uint32_t own0 = desc_k(sb + L::kOwn0), own1 = desc_k(sb + L::kOwn1);
        const uint32_t ak = desc_k(sb + L::kA), bk = desc_k(sb + L::kB), am = desc_mn(sb + L::kA), bm = desc_mn(sb + L::kB);
        while (units.take(cx, un, ok)) {
            const int m = part_of(un, un.head % p.parts, p.parts, G, p.window).m;
            if (m == 0) continue;
            if ((tid & 31) == 0) {
                auto s_product = [&](const At& i) -> bool {
                    if (!wait_bar(cx, B_A + i.a, i.a_phase)) return false;
                    mma_ss_rows<D>(tbase + TM_S, own0, ak + i.a * At::kStep);
                    mma_commit(cx.bars + B_S);
                    return true;
                };
                auto dp_product = [&](const At& i, bool last) -> bool {
                    if (!wait_bar(cx, B_B + i.b, i.b_phase)) return false;
                    mma_ss_rows<D>(tbase + TM_DP, own1, bk + i.b * At::kStep);
                    mma_commit(cx.bars + B_DP);
                    if (last) mma_commit(cx.bars + B_OWN_FREE);
                    return true;
                };
                ok = wait_bar(cx, B_OWN, own_phase) && s_product(at) && dp_product(at, m == 1);
                own_phase ^= 1u;
                for (int it = 0; ok && it < m; ++it) {
                    if (!(ok = wait_bar(cx, B_X, at.phase))) break;
                    tc_fence_after();
                    mma_halves<D, 0, 2>(tbase + TM_ACC0, tbase + TM_S, bm + at.b * At::kStep, it > 0);
                    if (!(ok = wait_bar(cx, B_Y, at.phase))) break;
                    tc_fence_after();
                    mma_halves<D, 2, 4>(tbase + TM_ACC0, tbase + TM_S, bm + at.b * At::kStep, true);
                    if (it + 1 < m && !(ok = s_product(nx))) break;  // runs after dV, so it may write over P
                    if (!(ok = wait_bar(cx, B_DS, at.phase))) break;
                    tc_fence_after();
                    mma_halves<D, 0, 4>(tbase + TM_ACC1, tbase + TM_DP, am + at.a * At::kStep, it > 0);
                    mma_commit(cx.bars + B_FREE + at.mod4);
                    if (it + 1 == m) mma_commit(cx.bars + B_END);
                    else if (!(ok = dp_product(nx, it + 2 == m))) break;
                    at = nx;
                    nx.next();
                }
            }
            if (!(ok = __shfl_sync(0xffffffffu, (int)ok, 0) != 0)) break;
        }
        __syncwarp();
    } else {
        const int lane = tid & 127, h = tid >> 7;
        const uint32_t tl = tbase + ((uint32_t)((warp & 3) * 32) << 16);
        const f2 scale2 = f2_of(p.scale_log2, p.scale_log2);
        int done = 0;
        while (units.take(cx, un, ok)) {
            const int hk = un.head / p.parts, part = un.head - hk * p.parts;
            const Part pt = part_of(un, part, p.parts, G, p.window);
            if (pt.m == 0) continue;
            const int key0 = un.local * kRows, key = key0 + lane;  // within the sequence
            for (int it = 0, tile = pt.first % pt.nq; it < pt.m; ++it, ++gi, tile = tile + 1 == pt.nq ? 0 : tile + 1) {
                const int q0 = key0 + tile * kRows;
                const float* nlse = reinterpret_cast<const float*>(sm + L::kStats + (gi & 1) * 1024) + 64 * h;
                const float* ndelta = nlse + kRows;
                if (!(ok = wait_warp(cx, B_B + (gi & 1), (gi >> 1) & 1))) break;  // the statistics have landed
                if (!(ok = wait_warp(cx, B_S, gi & 1))) break;
                tc_fence_after();
                uint32_t s[2][32];
                tmem_ld32(tl + TM_S + 64 * h, s[0]);
                tmem_ld32(tl + TM_S + 64 * h + 32, s[1]);
                tmem_ld_wait();
                // rows before the key, past its window or past the sequence
                const bool tail = q0 + kRows > un.len;
                const bool masked = tile == 0 || tail || q0 + kRows - 1 - key0 >= p.window;
                const int row0 = q0 + 64 * h;
                uint32_t see[2] = {0xFFFFFFFFu, 0xFFFFFFFFu};
                if (masked) {
                    const int last = min(p.window - 1 < un.len ? key + p.window - 1 : un.len - 1, un.len - 1) - row0;
#pragma unroll
                    for (int q = 0; q < 2; ++q) {
                        see[q] = columns(key - row0 - 32 * q, last - 32 * q);
                        mask_columns(s[q], see[q], kMinusInf);
                    }
                }
                if (tail) {
                    // rows past the sequence have weight 0, but 0 * NaN is not 0; both first products have read them
                    if (!(ok = wait_warp(cx, B_DP, gi & 1))) break;
                    if (lane >= un.len - q0) zero_row<D>(sm + (h ? L::b(gi) : L::a(gi)), lane);
                    fence_async_shared();
                }
                f2 x[32];
#pragma unroll
                for (int q = 0; q < 2; ++q) {
#pragma unroll
                    for (int c = 0; c < 16; c += 2) {
                        const float4 l4 = *reinterpret_cast<const float4*>(nlse + 32 * q + 2 * c);
                        const f2 a = f2_fma(f2_of(s[q][2 * c], s[q][2 * c + 1]), scale2, f2_of(l4.x, l4.y));
                        const f2 b = f2_fma(f2_of(s[q][2 * c + 2], s[q][2 * c + 3]), scale2, f2_of(l4.z, l4.w));
                        x[16 * q + c] = exp2_pair(a);
                        x[16 * q + c + 1] = exp2_pair(b);
                    }
                    st_quarter(tl + TM_S + 64 * h + 16 * q, x + 16 * q);
                    tmem_st_wait();
                    arrive_warp(cx, q ? B_Y : B_X);
                }
                if (!(ok = wait_warp(cx, B_DP, gi & 1))) break;
                tc_fence_after();
                tmem_ld32(tl + TM_DP + 64 * h, s[0]);
                tmem_ld32(tl + TM_DP + 64 * h + 32, s[1]);
                tmem_ld_wait();
                if (masked) {  // where the weight is 0, do . v may be anything
                    mask_columns(s[0], see[0], 0u);
                    mask_columns(s[1], see[1], 0u);
                }
#pragma unroll
                for (int c = 0; c < 32; c += 2) {
                    const float4 d4 = *reinterpret_cast<const float4*>(ndelta + 2 * c);
                    x[c] = f2_mul(x[c], f2_add(f2_of(s[c >> 4][(2 * c) & 31], s[c >> 4][(2 * c + 1) & 31]), f2_of(d4.x, d4.y)));
                    x[c + 1] = f2_mul(x[c + 1],
                                      f2_add(f2_of(s[c >> 4][(2 * c + 2) & 31], s[c >> 4][(2 * c + 3) & 31]), f2_of(d4.z, d4.w)));
                }
                st_quarter(tl + TM_DP + 64 * h, x);
                st_quarter(tl + TM_DP + 64 * h + 16, x + 16);
                tmem_st_wait();
                arrive_warp(cx, B_DS);
            }
            if (!ok || !(ok = wait_warp(cx, B_END, done & 1))) break;
            ++done;
            tc_fence_after();
            // the next unit's first product into these accumulators waits for its P, which follows this
            const int first = key - (lane & 31);
            const int64_t stride = (int64_t)p.io.Hk * D, at = (un.begin + first) * stride + hk * D;
            if (p.parts == 1) {
                store_acc<D>(tl + TM_ACC0, h, static_cast<__nv_bfloat16*>(p.io.dv) + at, stride, 1.f, un.len - first);
                store_acc<D>(tl + TM_ACC1, h, static_cast<__nv_bfloat16*>(p.io.dk) + at, stride, p.io.scale, un.len - first);
            } else {
                const int64_t all = (int64_t)p.io.T * stride, row = at + (lane & 31) * stride;
                store_part<D>(tl + TM_ACC0, h, p.io.part_dv + part * all + row, key < un.len);
                store_part<D>(tl + TM_ACC1, h, p.io.part_dk + part * all + row, key < un.len);
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == kMmaWarp) tmem_dealloc(tbase, TM_COLS);
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
attn_dq_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
               const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_do, const BwdParams p) {
    using L = BwdSmem<D>;
    extern __shared__ __align__(1024) uint8_t sm[];
    const uint32_t sb = smem_u32(sm);
    const int tid = threadIdx.x, warp = tid >> 5;
    const int G = p.io.Hq / p.io.Hk;
    Ctx cx;
    uint32_t* tmem_slot;
    if (!setup(cx, sm, sm + L::kBar, p.io, tmem_slot)) {
        grid_wait();
        return;
    }
    const uint32_t tbase = *tmem_slot;
    UnitQueue units{reinterpret_cast<volatile int*>(sm + L::kBar + 240), B_U, false, 0};
    Unit un{};
    bool ok = true;
    int gi = 0;
    // key tiles of a unit, from the diagonal down to the window's edge
    auto key_tiles = [&]() { return un.local - max(0, un.local * kRows - p.window + 1) / kRows + 1; };

    if (warp == kCopyWarp) {
        int owns = 0, a_items = 0, b_items = 0;  // issued
        TileMap<kRows> map(p.io.cu, p.io.nseq, p.io.T);
        while (units.draw(cx, map, p.io.Hq, true, p.io.counters + 1, un, ok)) {
            const int m = key_tiles(), head = un.head, hk = head / G, row0 = un.begin + un.local * kRows;
            if ((tid & 31) == 0) {
                for (int it = 0; ok && it < m; ++it, ++gi) {
                    const int row = row0 - it * kRows;
                    if (gi >= 3 && !(ok = wait_bar(cx, B_FREE + ((gi - 3) & 3), ((gi - 3) >> 2) & 1))) break;
                    uint64_t* bar = cx.bars + B_A + gi % 3;
                    mbar_arrive_expect_tx(bar, L::kTile);
                    load_tile<D>(sb + L::a(gi), &tm_k, bar, hk, row);
                    ++a_items;
                    if (gi >= 2 && !(ok = wait_bar(cx, B_V_FREE + (gi & 1), ((gi >> 1) - 1) & 1))) break;
                    bar = cx.bars + B_B + (gi & 1);
                    mbar_arrive_expect_tx(bar, L::kTile);
                    load_tile<D>(sb + L::b(gi), &tm_v, bar, hk, row);
                    ++b_items;
                    if (it == 0) {
                        if (owns && !(ok = wait_bar(cx, B_OWN_FREE, (owns - 1) & 1))) break;
                        mbar_arrive_expect_tx(cx.bars + B_OWN, 2 * L::kTile);
                        load_tile<D>(sb + L::kOwn0, &tm_q, cx.bars + B_OWN, head, row0);
                        load_tile<D>(sb + L::kOwn1, &tm_do, cx.bars + B_OWN, head, row0);
                        ++owns;
                    }
                }
            }
            if (!(ok = __shfl_sync(0xffffffffu, (int)ok, 0) != 0)) break;
        }
        if ((tid & 31) == 0) drain(cx, owns, a_items, b_items);
        __syncwarp();
    } else if (warp == kMmaWarp) {
        using At = ItemAt<D>;
        At at, nx;  // the item, and the one after it
        nx.next();
        uint32_t own_phase = 0;
        const uint32_t own0 = desc_k(sb + L::kOwn0), own1 = desc_k(sb + L::kOwn1);
        const uint32_t ak = desc_k(sb + L::kA), bk = desc_k(sb + L::kB), am = desc_mn(sb + L::kA);
        while (units.take(cx, un, ok)) {
            const int m = key_tiles();
            if ((tid & 31) == 0) {
                auto s_product = [&](const At& i) -> bool {
                    if (!wait_bar(cx, B_A + i.a, i.a_phase)) return false;
                    tc_fence_after();
                    mma_ss_rows<D>(tbase + TM_S, own0, ak + i.a * At::kStep);
                    mma_commit(cx.bars + B_S);
                    return true;
                };
                auto dp_product = [&](const At& i, bool last) -> bool {
                    if (!wait_bar(cx, B_B + i.b, i.b_phase)) return false;
                    tc_fence_after();
                    mma_ss_rows<D>(tbase + TM_DP, own1, bk + i.b * At::kStep);
                    mma_commit(cx.bars + B_DP);
                    mma_commit(cx.bars + B_V_FREE + i.b);
                    if (last) mma_commit(cx.bars + B_OWN_FREE);
                    return true;
                };
                ok = wait_bar(cx, B_OWN, own_phase) && s_product(at) && dp_product(at, m == 1);
                own_phase ^= 1u;
                for (int it = 0; ok && it < m; ++it) {
                    if (!(ok = wait_bar(cx, B_X, at.phase))) break;  // S is in registers
                    if (it + 1 < m && !(ok = s_product(nx))) break;
                    if (!(ok = wait_bar(cx, B_Y, at.phase))) break;  // so is dP
                    if (it + 1 < m && !(ok = dp_product(nx, it + 2 == m))) break;
                    if (!(ok = wait_bar(cx, B_DS, at.phase))) break;
                    tc_fence_after();
                    mma_ts_rows<D, 0, 128>(tbase + TM_ACC0, tbase + TM_DS, am + at.a * At::kStep, it > 0);
                    mma_commit(cx.bars + B_FREE + at.mod4);
                    if (it + 1 == m) mma_commit(cx.bars + B_END);
                    at = nx;
                    nx.next();
                }
            }
            if (!(ok = __shfl_sync(0xffffffffu, (int)ok, 0) != 0)) break;
        }
        __syncwarp();
    } else {
        const int lane = tid & 127, h = tid >> 7;
        const uint32_t tl = tbase + ((uint32_t)((warp & 3) * 32) << 16);
        const f2 scale2 = f2_of(p.scale_log2, p.scale_log2);
        int done = 0;
        while (units.take(cx, un, ok)) {
            const int m = key_tiles(), row0 = un.local * kRows, row = row0 + lane;
            const int64_t stat = ((int64_t)un.head * p.tiles + un.tile) * kRows + lane;
            const float nlse = __ldcg(p.io.lse + stat), ndelta = __ldcg(p.io.delta + stat);
            const f2 nlse2 = f2_of(nlse, nlse), ndelta2 = f2_of(ndelta, ndelta);
            for (int it = 0; it < m; ++it, ++gi) {
                const int key0 = row0 - it * kRows;
                if (!(ok = wait_warp(cx, B_S, gi & 1))) break;
                tc_fence_after();
                uint32_t s[2][32];
                tmem_ld32(tl + TM_S + 64 * h, s[0]);
                tmem_ld32(tl + TM_S + 64 * h + 32, s[1]);
                tmem_ld_wait();
                arrive_warp(cx, B_X);
                // keys after the row or out of its window
                const bool masked = it == 0 || key0 <= row0 + kRows - 1 - p.window;
                uint32_t see[2] = {0xFFFFFFFFu, 0xFFFFFFFFu};
                if (masked) {
                    const int last = row - key0 - 64 * h;
#pragma unroll
                    for (int q = 0; q < 2; ++q) {
                        see[q] = columns(last - p.window + 1 - 32 * q, last - 32 * q);
                        mask_columns(s[q], see[q], kMinusInf);
                    }
                }
                f2 x[32];
#pragma unroll
                for (int c = 0; c < 32; ++c)
                    x[c] = exp2_pair(f2_fma(f2_of(s[c >> 4][(2 * c) & 31], s[c >> 4][(2 * c + 1) & 31]), scale2, nlse2));
                if (!(ok = wait_warp(cx, B_DP, gi & 1))) break;
                tc_fence_after();
                tmem_ld32(tl + TM_DP + 64 * h, s[0]);
                tmem_ld32(tl + TM_DP + 64 * h + 32, s[1]);
                tmem_ld_wait();
                arrive_warp(cx, B_Y);
                if (masked) {  // where the weight is 0, do . v may be anything
                    mask_columns(s[0], see[0], 0u);
                    mask_columns(s[1], see[1], 0u);
                }
#pragma unroll
                for (int c = 0; c < 32; ++c)
                    x[c] = f2_mul(x[c], f2_add(f2_of(s[c >> 4][(2 * c) & 31], s[c >> 4][(2 * c + 1) & 31]), ndelta2));
                // dQ of the item before has read its dS
                if (gi && !(ok = wait_warp(cx, B_FREE + ((gi - 1) & 3), ((gi - 1) >> 2) & 1))) break;
                st_quarter(tl + TM_DS + 32 * h, x);
                st_quarter(tl + TM_DS + 32 * h + 16, x + 16);
                if (it == 0 && un.len - key0 < kRows) {
                    // K's rows past the sequence: their ds is 0, but 0 * NaN is not; S is done with them
                    if (h == 0 && lane >= un.len - key0) zero_row<D>(sm + L::a(gi), lane);
                    fence_async_shared();
                }
                tmem_st_wait();
                arrive_warp(cx, B_DS);
            }
            if (!ok || !(ok = wait_warp(cx, B_END, done & 1))) break;
            ++done;
            tc_fence_after();
            const int first = row - (lane & 31);
            const int64_t stride = (int64_t)p.io.Hq * D, at = (un.begin + first) * stride + un.head * D;
            store_acc<D>(tl + TM_ACC0, h, static_cast<__nv_bfloat16*>(p.io.dq) + at, stride, p.io.scale, un.len - first);
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == kMmaWarp) tmem_dealloc(tbase, TM_COLS);
    if (tid == 0) grid_wait();  // what follows this kernel follows dkdv as well
}

// -delta = -do . (o + o_lo) of every row, tile-aligned like lse (0 for a tile's rows past its sequence).
// D / 8 lanes a row, 8 channels each.  HBM bound: three reads of 2 bytes a channel.  A CTA walks its tiles in order.
template <int D>
__global__ void __launch_bounds__(256) attn_delta_kernel(const AttnIO io, int tiles) {
    constexpr int LANES = D / 8, RPP = 256 / LANES;
    grid_launch_next();
    if (blockIdx.x == 0 && threadIdx.x < 2) {
        if (threadIdx.x == 0) *io.err = 0;
        io.counters[threadIdx.x] = 0;
    }
    TileMap<kRows> map(io.cu, io.nseq, io.T);
    const int c0 = (threadIdx.x % LANES) * 8;
    const int64_t units = (int64_t)map.total * io.Hq;
    for (int64_t u = blockIdx.x; u < units; u += gridDim.x) {
        Seq sq{};
        const int rank = (int)(u / io.Hq), head = (int)(u - (int64_t)rank * io.Hq);
        if (!map.find(rank, false, sq)) return;
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
            if (c0 == 0) io.delta[((int64_t)head * tiles + sq.tile) * kRows + r] = -sum;
        }
    }
}

// dk and dv of a key tile and head from the parts' sums, in their order.  D / 4 lanes a row, a row a lane.
template <int D>
__global__ void __launch_bounds__(256) attn_join_kernel(const BwdParams p) {
    constexpr int LANES = D / 4;
    Seq sq{};
    const int hk = blockIdx.x % p.io.Hk, G = p.io.Hq / p.io.Hk;
    TileMap<kRows> map(p.io.cu, p.io.nseq, p.io.T);
    const bool have = map.find((int)(blockIdx.x / p.io.Hk), false, sq);
    const int row = sq.local * kRows + blockIdx.y * (256 / LANES) + threadIdx.x / LANES;
    grid_wait();
    if (!have || row >= sq.len) return;
    const Unit un{sq.begin, sq.len, sq.tile, sq.local, hk};
    // with fewer items than parts some are empty, and nothing was written for them
    const bool all = (int64_t)G * query_tiles(un, p.window) >= p.parts;
    const int64_t stride = (int64_t)p.io.Hk * D, step = (int64_t)p.io.T * stride;
    const int64_t at = (sq.begin + row) * stride + hk * D + (threadIdx.x % LANES) * 4;
    float4 k = make_float4(0.f, 0.f, 0.f, 0.f), v = k;
#pragma unroll 4
    for (int s = 0; s < p.parts; ++s) {
        const bool there = all || part_of(un, s, p.parts, G, p.window).m;
        const float4 zero = make_float4(0.f, 0.f, 0.f, 0.f);
        const float4 a = there ? __ldcg(reinterpret_cast<const float4*>(p.io.part_dk + s * step + at)) : zero;
        const float4 b = there ? __ldcg(reinterpret_cast<const float4*>(p.io.part_dv + s * step + at)) : zero;
        k.x += a.x; k.y += a.y; k.z += a.z; k.w += a.w;
        v.x += b.x; v.y += b.y; v.z += b.z; v.w += b.w;
    }
    const float f = p.io.scale;
    *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.io.dk) + at) =
        make_uint2(pack_bf16x2(k.x * f, k.y * f), pack_bf16x2(k.z * f, k.w * f));
    *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.io.dv) + at) =
        make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w));
}

template <int D>
cudaError_t launch(const CUtensorMap* maps, const BwdParams& p, cudaStream_t st) {
    const unsigned q_tiles = (unsigned)p.tiles * (unsigned)p.io.Hq, k_tiles = (unsigned)p.tiles * (unsigned)p.io.Hk;
    const unsigned k_units = k_tiles * (unsigned)p.parts;
    // more sequences than a warp holds: few CTAs, which read the array on
    const unsigned walkers = p.io.nseq > 32 && q_tiles > 148 * 6 ? 148 * 6 : q_tiles;
    attn_delta_kernel<D><<<walkers, 256, 0, st>>>(p.io, p.tiles);
    count_launch();
    cudaError_t e = cudaGetLastError();
    if (e == cudaSuccess)
        e = cudaFuncSetAttribute(attn_dkdv_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)BwdSmem<D>::kBytes);
    if (e == cudaSuccess)
        e = cudaFuncSetAttribute(attn_dq_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)BwdSmem<D>::kBytes);
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute early{};
    early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    early.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(k_units < 148 ? k_units : 148);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = BwdSmem<D>::kBytes;
    cfg.stream = st;
    cfg.attrs = &early;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, attn_dkdv_kernel<D>, maps[0], maps[1], maps[2], maps[3], p);
    count_launch();
    if (e != cudaSuccess) return e;
    cfg.gridDim = dim3(q_tiles < 148 ? q_tiles : 148);
    e = cudaLaunchKernelEx(&cfg, attn_dq_kernel<D>, maps[0], maps[1], maps[2], maps[3], p);
    count_launch();
    if (e != cudaSuccess || p.parts == 1) return e;
    cfg.gridDim = dim3(k_tiles, kRows * (D / 4) / 256);
    cfg.blockDim = dim3(256);
    cfg.dynamicSmemBytes = 0;
    e = cudaLaunchKernelEx(&cfg, attn_join_kernel<D>, p);
    count_launch();
    return e;
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
    p.window = io.window > 0 && io.window < attn::kNoWindow ? (int)io.window : attn::kNoWindow;
    p.parts = attn_bwd_parts(io.T, io.nseq, io.Hq, io.Hk, io.window);
    p.scale_log2 = io.scale * 1.4426950408889634f;
    return d == 128 ? attn::launch<128>(maps, p, st) : attn::launch<64>(maps, p, st);
}

}  // namespace gdn

// Single-token attention over the paged cache: o = softmax(scale q K^T) V for one query token a
// sequence, with the query heads of a key head (up to 16 a CTA) as the rows of the products.
//
// Bound: HBM, each cached k and v read once (2 d bf16 a token and key head against 4 d flops a query
// head: below the tensor-core ridge for any group that fits 16 rows).  What has to be kept is bytes in
// flight, so each warp runs its own pipeline: tiles of 16 tokens, k and v rows copied by cp.async into
// a private ring of shared memory, the page of the tile after looked up meanwhile, no barrier
// between the warps of a CTA.  The products are 16-row mma.sync: the 128-row tcgen05 tile would be
// mostly padding here, and the tensor pipe is not what bounds.  One pass: running reference and
// sum per row (the reference follows the maximum only when that has outgrown it by 2^8), scores and
// output accumulators in registers.
//
// Tiles start at positions that are multiples of 16.  Where 16 divides the page size (PAGED16) a tile lies in
// one page and its rows are evenly spaced; otherwise every row is looked up by itself.
//
// A context is split over CTAs in chunks of tokens that the host chooses from the sizes alone
// (plan_decode_attn); the warps of a CTA are joined in shared memory and the chunks of a sequence by
// combine_kernel, both in index order, so results do not depend on timing.
//
// The compiler reports spills of 8 (pages of 16s) and 36 bytes at d = 128 with up to 8 heads a group, whose 168 registers
// are what three CTAs an SM leave.
//
// Measured, d = 128: 256 sequences of 64 to 4500 tokens, 16 heads on 2: 58.6 us, 4.7 TB/s (a copy: 6.5); one sequence of 8191
// tokens: 8.7 us, two kernels' latency (8.4 MB would take 1.3).
#include <cuda_bf16.h>

#include "attn.h"
#include "launch.h"
#include "umma.cuh"

namespace gdn {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kTile = 16;    // tokens of a warp's tile

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool valid) {
    // with source size 0 nothing is read and the 16 bytes are zeros
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(valid ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Tokens of sequence n that are read: [first, len); base: the tile that first lies in.
struct Context {
    int first, base, len;
};
__device__ __forceinline__ Context context_of(const DecodeAttnParams& p, int n) {
    const int c = __ldg(p.context + n);
    Context x;
    x.len = c < 0 ? 0 : (c > p.max_context ? (int)p.max_context : c);
    x.first = p.window > 0 && x.len > p.window ? x.len - (int)p.window : 0;
    x.base = x.first & ~(kTile - 1);
    return x;
}

// A warp's ring holds kStages tiles, kStages - 1 of them on their way while one is read.  With up to 8 query
// heads a group the registers allow three CTAs an SM, two stages each (64 KB at d = 128): 58.6 us for 256
// sequences of 64 to 4500 tokens, against 64.1 us for two CTAs of three stages.  With more than 8 heads the registers
// allow two.
template <int D, bool ROWS16>
struct Smem {
    static constexpr int kStages = ROWS16 ? 3 : 2, kCtas = ROWS16 ? 2 : 3;
    static constexpr int kBox = kTile * 128;                 // 64 channels of a tile's rows, 128-byte swizzled
    static constexpr int kHalf = D / 64 * kBox;              // the tile's k (or v)
    static constexpr int kStage = 2 * kHalf;
    static constexpr int kRing = kWarps * kStages * kStage;  // also the join's [warps][16][D] fp32
    static constexpr int kBytes = kRing + kWarps * 16 * 2 * 4;
    static_assert(kRing >= kWarps * 16 * D * 4, "the join fits the ring");
};

// ROWS16: the group has more than 8 query heads; otherwise rows 8-15 of the products are padding.
template <int D, bool PAGED16, bool ROWS16>
__global__ void __launch_bounds__(kThreads, Smem<D, ROWS16>::kCtas) decode_attn_kernel(const DecodeAttnParams p, float scale_log2) {
    using S = Smem<D, ROWS16>;
    constexpr int kStages = S::kStages;
    extern __shared__ __align__(1024) uint8_t smem[];
    // lets the joining kernel be set up while this one runs; it waits for this one's results itself
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int G = p.Hq / p.Hk, blocks = (G + 15) / 16;
    uint32_t b = blockIdx.x;
    const int split = (int)(b % (uint32_t)p.splits);
    b /= (uint32_t)p.splits;
    const int rb = (int)(b % (uint32_t)blocks);
    b /= (uint32_t)blocks;
    const int hk = (int)(b % (uint32_t)p.Hk), n = (int)(b / (uint32_t)p.Hk);
    const int rows = min(16, G - rb * 16), hq0 = hk * G + rb * 16;
    const Context cx = context_of(p, n);
    if (split > 0 && (int64_t)cx.base + (int64_t)split * p.chunk >= cx.len) return;
    const int begin = cx.base + split * p.chunk;
    const int count = cx.len - begin < p.chunk ? max(cx.len - begin, 0) : p.chunk;  // tokens from begin on
    const bool whole = cx.len - cx.base <= p.chunk;  // one split: the result goes straight to o

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int g = lane >> 2, c = lane & 3;
    uint8_t* ring_p = smem + warp * kStages * S::kStage;
    const uint32_t ring = tc::smem_u32(ring_p);
    const int tiles = (count + kTile - 1) / kTile;
    const int mine = tiles > warp ? (tiles - warp + kWarps - 1) / kWarps : 0;  // tiles warp, warp + kWarps, ...
    const int64_t row_elems = (int64_t)p.Hk * D;
    const __nv_bfloat16* kc = static_cast<const __nv_bfloat16*>(p.k_cache) + (int64_t)hk * D;
    const __nv_bfloat16* vc = static_cast<const __nv_bfloat16*>(p.v_cache) + (int64_t)hk * D;
    const int32_t* table = p.table + (int64_t)n * p.max_pages;
    auto pos_of = [&](int i) { return begin + (i * kWarps + warp) * kTile; };

    // The cache row of the tile's first token (PAGED16) or of its token lane % 16; -1 where there is none.
    auto find_row = [&](int i) -> int64_t {
        if (i >= mine) return -1;
        const uint32_t pos = (uint32_t)pos_of(i) + (PAGED16 ? 0 : lane & 15);
        const uint32_t page_no = (uint32_t)(((uint64_t)pos * p.page_mul) >> p.page_shift);
        if (page_no >= (uint64_t)p.max_pages) return -1;
        const int page = __ldg(table + page_no);
        if (page < 0 || page >= p.num_pages) return -1;
        return (int64_t)page * p.page_size + (pos - page_no * (uint32_t)p.page_size);
    };
    constexpr int CH = D / 8, RPI = 32 / CH;  // 16-byte pieces a row, rows a warp instruction
    const int my_row = lane / CH, my_ch = lane % CH;
    const uint32_t my_box = (uint32_t)((my_ch >> 3) * S::kBox);
    auto issue = [&](int i, int64_t row) {
        const uint32_t kb = ring + (uint32_t)((i % kStages) * S::kStage) + my_box, vb = kb + S::kHalf;
        const int lo = cx.first - pos_of(i), hi = cx.len - pos_of(i);  // the tile's tokens that exist
        const __nv_bfloat16 *ks = kc + my_ch * 8, *vs = vc + my_ch * 8;
        if (PAGED16) {
            const int64_t at = (row < 0 ? 0 : row + my_row) * row_elems;
            ks += at;
            vs += at;
        }
        const int64_t step = row < 0 ? 0 : RPI * row_elems;
#pragma unroll
        for (int r0 = 0; r0 < kTile; r0 += RPI) {
            const int r = r0 + my_row;
            const uint32_t dst = (uint32_t)(r * 128 + (((my_ch & 7) ^ (r & 7)) << 4));
            if (PAGED16) {
                const bool ok = row >= 0 && r >= lo && r < hi;
                cp_async16(kb + dst, ks, ok);
                cp_async16(vb + dst, vs, ok);
                ks += step;
                vs += step;
            } else {
                const int64_t at = __shfl_sync(0xffffffffu, row, r);
                const bool ok = at >= 0 && r >= lo && r < hi;
                const int64_t off = (ok ? at : 0) * row_elems;
                cp_async16(kb + dst, ks + off, ok);
                cp_async16(vb + dst, vs + off, ok);
            }
        }
    };
    // Bit t: token t of tile i, whose rows are `row`, exists.
    auto exists = [&](int i, int64_t row) -> uint32_t {
        const int lo = cx.first - pos_of(i), hi = cx.len - pos_of(i);
        if (PAGED16) {
            if (row < 0) return 0u;
            const uint32_t upto = hi >= kTile ? 0xFFFFu : (hi <= 0 ? 0u : (1u << hi) - 1u);
            return lo > 0 ? upto & ~((1u << lo) - 1u) : upto;
        }
        const int t = lane & 15;
        return __ballot_sync(0xffffffffu, row >= 0 && t >= lo && t < hi) & 0xFFFFu;
    };

    // ring prologue: tiles 0 .. kStages - 2 on their way, the row of the one after looked up
    uint32_t valid[kStages - 1];
    int64_t next;
    {
        int64_t rows_of[kStages];
#pragma unroll
        for (int i = 0; i < kStages; ++i) rows_of[i] = find_row(i);
#pragma unroll
        for (int i = 0; i < kStages - 1; ++i) {
            if (i < mine) issue(i, rows_of[i]);
            cp_commit();
            valid[i] = exists(i, rows_of[i]);
        }
        next = rows_of[kStages - 1];
    }

    // q as the A operand: row g (and g + 8), channels 2c, 2c + 1 (and + 8) of each 16
    uint32_t qa[D / 16][4];
    {
        const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(p.q) + (int64_t)n * p.q_stride + (int64_t)hq0 * D;
        auto pair = [&](int r, int ch) -> uint32_t {
            if (r >= rows) return 0u;
            const __nv_bfloat16* s = q + r * D + ch;
            if (p.q_vec) return __ldg(reinterpret_cast<const uint32_t*>(s));
            return (uint32_t)__bfloat16_as_ushort(s[0]) | ((uint32_t)__bfloat16_as_ushort(s[1]) << 16);
        };
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
            qa[k][0] = pair(g, k * 16 + 2 * c);
            qa[k][1] = ROWS16 ? pair(g + 8, k * 16 + 2 * c) : 0u;
            qa[k][2] = pair(g, k * 16 + 2 * c + 8);
            qa[k][3] = ROWS16 ? pair(g + 8, k * 16 + 2 * c + 8) : 0u;
        }
    }

    float o[D / 8][4];
#pragma unroll
    for (int j = 0; j < D / 8; ++j) o[j][0] = o[j][1] = o[j][2] = o[j][3] = 0.f;
    // rows g and g + 8: reference (in units of log 2) and this lane's share of the sum
    float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;
    // ldmatrix: this lane's row of the k and v matrices, and its four swizzled places in a 128-byte row
    const int lr = lane & 7, lm = lane >> 3;
    uint32_t k_at[4], v_at[4];
#pragma unroll
    for (int x = 0; x < 4; ++x) {
        k_at[x] = (uint32_t)((((lm >> 1) << 3) + lr) * 128 + (((2 * x + (lm & 1)) ^ lr) << 4));
        v_at[x] = (uint32_t)((((lm & 1) << 3) + lr) * 128 + (((2 * x + (lm >> 1)) ^ lr) << 4)) + S::kHalf;
    }
#pragma unroll 1
    for (int i = 0; i < mine; ++i) {
        // the tile kStages - 1 ahead takes the slot that the last iteration read
        const int64_t row = next;
        const int ahead = i + kStages - 1;
        next = find_row(ahead + 1);
        if (ahead < mine) issue(ahead, row);
        cp_commit();
        const uint32_t mask = valid[0];
#pragma unroll
        for (int s = 0; s + 1 < kStages - 1; ++s) valid[s] = valid[s + 1];
        valid[kStages - 2] = ahead < mine ? exists(ahead, row) : 0u;
        cp_wait<kStages - 1>();
        __syncwarp();
        if (mask == 0u) continue;  // nothing of this tile exists; the slot is not read

        const uint32_t kb = ring + (uint32_t)((i % kStages) * S::kStage);
        float s0[4] = {}, s1[4] = {};  // tokens 0-7 and 8-15
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
            uint32_t kf[4];
            ldsm4(kb + (uint32_t)((k >> 2) * S::kBox) + k_at[k & 3], kf);
            mma16816(s0, qa[k], kf[0], kf[1]);
            mma16816(s1, qa[k], kf[2], kf[3]);
        }
        if (mask != 0xFFFFu) {  // tokens that do not exist leave the softmax
            const uint32_t mm = mask >> (2 * c);
            if (!(mm & 1u)) s0[0] = s0[2] = -INFINITY;
            if (!(mm & 2u)) s0[1] = s0[3] = -INFINITY;
            if (!(mm & 256u)) s1[0] = s1[2] = -INFINITY;
            if (!(mm & 512u)) s1[1] = s1[3] = -INFINITY;
        }
        float x0 = fmaxf(fmaxf(s0[0], s0[1]), fmaxf(s1[0], s1[1]));
        x0 = fmaxf(x0, __shfl_xor_sync(0xffffffffu, x0, 1));
        x0 = fmaxf(x0, __shfl_xor_sync(0xffffffffu, x0, 2)) * scale_log2;
        float x1 = -INFINITY;
        if (ROWS16) {
            x1 = fmaxf(fmaxf(s0[2], s0[3]), fmaxf(s1[2], s1[3]));
            x1 = fmaxf(x1, __shfl_xor_sync(0xffffffffu, x1, 1));
            x1 = fmaxf(x1, __shfl_xor_sync(0xffffffffu, x1, 2)) * scale_log2;
        }
        // each row decides for itself, the vote only skips the work: a head's rounding of p, which goes by its reference,
        // does not depend on the other heads of its group
        const bool up0 = x0 > m0 + 8.f, up1 = ROWS16 && x1 > m1 + 8.f;
        if (__any_sync(0xffffffffu, up0 || up1)) {
            const float f0 = up0 ? ex2(m0 - x0) : 1.f, f1 = up1 ? ex2(m1 - x1) : 1.f;
            if (up0) m0 = x0;
            if (up1) m1 = x1;
            l0 *= f0;
            l1 *= f1;
#pragma unroll
            for (int j = 0; j < D / 8; ++j) {
                o[j][0] *= f0;
                o[j][1] *= f0;
                o[j][2] *= f1;
                o[j][3] *= f1;
            }
        }
        // a row whose every score so far is -inf keeps p = 0
        const float z0 = m0 == -INFINITY ? 0.f : m0;
        s0[0] = ex2(fmaf(s0[0], scale_log2, -z0)); s0[1] = ex2(fmaf(s0[1], scale_log2, -z0));
        s1[0] = ex2(fmaf(s1[0], scale_log2, -z0)); s1[1] = ex2(fmaf(s1[1], scale_log2, -z0));
        l0 += (s0[0] + s0[1]) + (s1[0] + s1[1]);
        // p rounded to bf16, the tensor cores' operand type; the sum keeps fp32
        uint32_t pa[4] = {tc::pack_bf16x2(s0[0], s0[1]), 0u, tc::pack_bf16x2(s1[0], s1[1]), 0u};
        if (ROWS16) {
            const float z1 = m1 == -INFINITY ? 0.f : m1;
            s0[2] = ex2(fmaf(s0[2], scale_log2, -z1)); s0[3] = ex2(fmaf(s0[3], scale_log2, -z1));
            s1[2] = ex2(fmaf(s1[2], scale_log2, -z1)); s1[3] = ex2(fmaf(s1[3], scale_log2, -z1));
            l1 += (s0[2] + s0[3]) + (s1[2] + s1[3]);
            pa[1] = tc::pack_bf16x2(s0[2], s0[3]);
            pa[3] = tc::pack_bf16x2(s1[2], s1[3]);
        }
#pragma unroll
        for (int j = 0; j < D / 16; ++j) {
            uint32_t vf[4];
            ldsm4_t(kb + (uint32_t)((j >> 2) * S::kBox) + v_at[j & 3], vf);
            mma16816(o[2 * j], pa, vf[0], vf[1]);
            mma16816(o[2 * j + 1], pa, vf[2], vf[3]);
        }
        __syncwarp();
    }
    cp_wait<0>();
    l0 += __shfl_xor_sync(0xffffffffu, l0, 1);
    l0 += __shfl_xor_sync(0xffffffffu, l0, 2);
    if (ROWS16) {
        l1 += __shfl_xor_sync(0xffffffffu, l1, 1);
        l1 += __shfl_xor_sync(0xffffffffu, l1, 2);
    }

    // join the warps: [warp][16][D] accumulators in the ring, references and sums behind it
    __syncthreads();
    float* acc = reinterpret_cast<float*>(smem);
    float* ms = reinterpret_cast<float*>(smem + S::kRing);
    float* ls = ms + kWarps * 16;
#pragma unroll
    for (int j = 0; j < D / 8; ++j) {
        float* r0 = acc + (warp * 16 + g) * D + j * 8 + 2 * c;
        *reinterpret_cast<float2*>(r0) = make_float2(o[j][0], o[j][1]);
        if (ROWS16) *reinterpret_cast<float2*>(r0 + 8 * D) = make_float2(o[j][2], o[j][3]);
    }
    if (c == 0) {
        ms[warp * 16 + g] = m0;
        ms[warp * 16 + g + 8] = m1;
        ls[warp * 16 + g] = l0;
        ls[warp * 16 + g + 8] = l1;
    }
    __syncthreads();
    const int64_t out_rows = (int64_t)p.N * p.Hq;
    for (int e = threadIdx.x; e < rows * (D / 4); e += kThreads) {
        const int r = e / (D / 4), ch = (e - r * (D / 4)) * 4;
        float m = ms[r];
#pragma unroll
        for (int w = 1; w < kWarps; ++w) m = fmaxf(m, ms[w * 16 + r]);
        float l = 0.f;
        float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            const float mw = ms[w * 16 + r], f = mw == -INFINITY ? 0.f : ex2(mw - m);
            const float4 a = *reinterpret_cast<const float4*>(acc + (w * 16 + r) * D + ch);
            l = fmaf(f, ls[w * 16 + r], l);
            x.x = fmaf(f, a.x, x.x);
            x.y = fmaf(f, a.y, x.y);
            x.z = fmaf(f, a.z, x.z);
            x.w = fmaf(f, a.w, x.w);
        }
        const int64_t out = (int64_t)n * p.Hq + hq0 + r;
        if (whole) {
            const float inv = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);  // no token: 0; NaN stays
            *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.o) + out * D + ch) =
                make_uint2(tc::pack_bf16x2(x.x * inv, x.y * inv), tc::pack_bf16x2(x.z * inv, x.w * inv));
        } else {
            // accumulators [split][row][D], then references and sums [split][row][2]
            *reinterpret_cast<float4*>(p.part + ((int64_t)split * out_rows + out) * D + ch) = x;
            if (ch == 0)
                *reinterpret_cast<float2*>(p.part + (int64_t)p.splits * out_rows * D +
                                           ((int64_t)split * out_rows + out) * 2) = make_float2(m, l);
        }
    }
}

// Joins the chunks of one (sequence, query head): a CTA a row, four warps that take every fourth chunk, D / 32
// channels a lane.
template <int D>
__global__ void __launch_bounds__(128) combine_kernel(const DecodeAttnParams p) {
    constexpr int C = D / 32;
    __shared__ float red[4][D];
    __shared__ float red_l[4], red_m[4];
    asm volatile("griddepcontrol.wait;" ::: "memory");  // the partial results are written
    const int64_t row = blockIdx.x, out_rows = (int64_t)p.N * p.Hq;
    const Context cx = context_of(p, (int)(row / p.Hq));
    const int used = (cx.len - cx.base + p.chunk - 1) / p.chunk;
    if (used <= 1) return;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const float* part = p.part + row * D + lane * C;
    const float2* ml = reinterpret_cast<const float2*>(p.part + (int64_t)p.splits * out_rows * D) + row;
    float m = -INFINITY;
    for (int s = threadIdx.x; s < used; s += 128) m = fmaxf(m, ml[s * out_rows].x);
#pragma unroll
    for (int off = 16; off; off >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
    if (lane == 0) red_m[warp] = m;
    __syncthreads();
    m = fmaxf(fmaxf(red_m[0], red_m[1]), fmaxf(red_m[2], red_m[3]));
    float l = 0.f, x[C] = {};
#pragma unroll 4
    for (int s = warp; s < used; s += 4) {
        const float2 v = ml[s * out_rows];
        const float f = v.x == -INFINITY ? 0.f : ex2(v.x - m);
        l = fmaf(f, v.y, l);
        const float* a = part + (int64_t)s * out_rows * D;
#pragma unroll
        for (int i = 0; i < C; i += 2) {
            const float2 y = *reinterpret_cast<const float2*>(a + i);
            x[i] = fmaf(f, y.x, x[i]);
            x[i + 1] = fmaf(f, y.y, x[i + 1]);
        }
    }
#pragma unroll
    for (int i = 0; i < C; ++i) red[warp][lane * C + i] = x[i];
    if (lane == 0) red_l[warp] = l;
    __syncthreads();
    if (threadIdx.x >= D) return;
    const int ch = threadIdx.x;
    const float sum = (red[0][ch] + red[1][ch]) + (red[2][ch] + red[3][ch]);
    l = (red_l[0] + red_l[1]) + (red_l[2] + red_l[3]);
    static_cast<__nv_bfloat16*>(p.o)[row * D + ch] = __float2bfloat16_rn(l == 0.f ? 0.f : sum / l);
}

template <int D, bool PAGED16, bool ROWS16>
cudaError_t launch(const DecodeAttnParams& p, cudaStream_t st) {
    using S = Smem<D, ROWS16>;
    auto kernel = decode_attn_kernel<D, PAGED16, ROWS16>;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kBytes);
    if (e != cudaSuccess) return e;
    const int64_t blocks = (p.Hq / p.Hk + 15) / 16;
    kernel<<<(unsigned)(p.N * p.Hk * blocks * p.splits), kThreads, S::kBytes, st>>>(p, p.scale * 1.4426950408889634f);
    count_launch();
    if ((e = cudaGetLastError()) != cudaSuccess || p.splits == 1) return e;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)((int64_t)p.N * p.Hq));
    cfg.blockDim = dim3(128);
    cfg.stream = st;
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, combine_kernel<D>, p);
    count_launch();
    return e;
}

template <int D>
cudaError_t launch_d(DecodeAttnParams p, cudaStream_t st) {
    // pos / page_size as (pos * page_mul) >> page_shift, exact for pos < 2^31: page_mul = ceil(2^page_shift / page_size)
    // with 2^(page_shift - 31) >= page_size
    p.page_shift = 31;
    while ((int64_t(1) << (p.page_shift - 31)) < p.page_size) ++p.page_shift;
    p.page_mul = (uint32_t)(((uint64_t(1) << p.page_shift) + (uint64_t)p.page_size - 1) / (uint64_t)p.page_size);
    const bool paged = p.page_size % kTile == 0, rows16 = p.Hq / p.Hk > 8;
    if (paged) return rows16 ? launch<D, true, true>(p, st) : launch<D, true, false>(p, st);
    return rows16 ? launch<D, false, true>(p, st) : launch<D, false, false>(p, st);
}

}  // namespace

// Chunk length and number of chunks for contexts of up to `reach` tokens (and the tile before a window's
// start).  Eight CTAs' worth of work an SM evens out ragged lengths; chunks of at most 512 tokens keep a long
// sequence from being the tail (256 sequences of 64 to 4500 tokens: 58.6 us; 59.1 us with 1024, 78 us with 256, whose
// joins cost more); at least 64 give every warp a tile, and at least 128 where 64 would make more than a CTA an
// SM, since a chunk's start, end and join take longer than its second 64 tokens (one sequence of 8191, 2 key heads:
// 8.7 us, 10.1 with 64, 9.4 with 192; 4 of 8000: 9.8 and 14.9; one of 2000, 1 key head: 6.8 us with 64, 7.0 with 128).
// The partial results are bounded at 64 MB and 512 chunks, whatever the table's reach: beyond them, chunks grow.
// The contexts are not known here, so that a reach far above them costs chunks that are too long and CTAs that find
// nothing to do, which max_context avoids.  Tables for 4500, 32768 and 131072 tokens under the 256 sequences of up to
// 4500: 58.4, 70.6 and 101.7 us, with max_context 58 us each; one sequence of 8191 under 8192, 131072 and 2^20: 8.6, 10.4
// and 28.7 us, with it 8.6 us each.
void plan_decode_attn(int64_t N, int64_t Hq, int64_t Hk, int64_t reach, int* chunk, int* splits) {
    const int64_t units = N * Hk * ((Hq / Hk + 15) / 16);
    reach += kTile;
    int64_t c = (units * reach + 148 * 8 - 1) / (148 * 8);
    const int64_t least = units * reach <= 148 * 64 ? 64 : 128;
    c = c < least ? least : (c > 512 ? 512 : c);
    int64_t most = (int64_t(1) << 24) / (N * Hq * 130);
    most = most < 1 ? 1 : (most > 512 ? 512 : most);
    if (c * most < reach) c = (reach + most - 1) / most;
    c = (c + 63) / 64 * 64;
    *chunk = (int)c;
    *splits = (int)((reach + c - 1) / c);
}

size_t decode_attn_part_floats(int64_t N, int64_t Hq, int64_t d, int splits) {
    return splits > 1 ? (size_t)splits * N * Hq * (d + 2) : 0;
}

cudaError_t decode_attn(const DecodeAttnParams& p, int d, cudaStream_t st) {
    return d == 128 ? launch_d<128>(p, st) : launch_d<64>(p, st);
}

}  // namespace gdn

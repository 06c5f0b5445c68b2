// Single-token attention over the paged cache: o = softmax(scale q K^T) V for one query token a
// sequence, with the query heads of a key head (up to 16 a CTA) as the rows of the products.
//
// Bound: HBM, each cached k and v read once (2 d bf16 a token and key head against 4 d flops a query
// head: below the tensor-core ridge for any group that fits 16 rows).  What has to be kept is bytes in
// flight, so each warp runs its own pipeline: tiles of 16 tokens, k and v rows copied by cp.async into
// a private ring of shared memory (the page of each row is looked up one tile ahead), no barrier
// between the warps of a CTA.  The products are 16-row mma.sync: the 128-row tcgen05 tile would be
// mostly padding here, and the tensor pipe is not what bounds.  One pass: running maximum and
// sum per row, scores and output accumulators in registers.
//
// A context is split over CTAs in chunks of tokens that the host chooses from the sizes alone
// (plan_decode_attn); the warps of a CTA are joined in shared memory and the chunks of a sequence by
// combine_kernel, both in index order, so results do not depend on timing.
#include <cuda_bf16.h>

#include "attn.h"
#include "launch.h"
#include "umma.cuh"

namespace gdn {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kTile = 16;    // tokens of a warp's tile
constexpr int kStages = 3;   // tiles of a warp's ring: 2 in flight while one is read
constexpr int kSplitSlices = 4;

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

// Tokens of sequence n that are read: [first, len).
__device__ __forceinline__ void context_range(const DecodeAttnParams& p, int n, int64_t& first, int64_t& len) {
    int64_t c = __ldg(p.context + n);
    len = c < 0 ? 0 : (c > p.max_context ? p.max_context : c);
    first = p.window > 0 && len > p.window ? len - p.window : 0;
}

template <int D>
struct Smem {
    static constexpr int kRow = D * 2;                       // bytes of a k or v row
    static constexpr int kStage = 2 * kTile * kRow;          // k rows, then v rows
    static constexpr int kRing = kWarps * kStages * kStage;  // also the join's [warps][16][D] fp32
    static constexpr int kBytes = kRing + kWarps * 16 * 2 * 4;
    static_assert(kRing >= kWarps * 16 * D * 4, "the join fits the ring");
};

template <int D>
__global__ void __launch_bounds__(kThreads) decode_attn_kernel(DecodeAttnParams p, float scale_log2) {
    using S = Smem<D>;
    extern __shared__ __align__(128) uint8_t smem[];
    const int G = p.Hq / p.Hk, blocks = (G + 15) / 16;
    int64_t b = blockIdx.x;
    const int split = (int)(b % p.splits);
    b /= p.splits;
    const int rb = (int)(b % blocks);
    b /= blocks;
    const int hk = (int)(b % p.Hk), n = (int)(b / p.Hk);
    const int rows = min(16, G - rb * 16), hq0 = hk * G + rb * 16;
    int64_t first, len;
    context_range(p, n, first, len);
    const int64_t begin = first + (int64_t)split * p.chunk;
    if (begin >= len && split > 0) return;
    const int count = (int)(len - begin < p.chunk ? (len > begin ? len - begin : 0) : p.chunk);
    const bool whole = len - first <= p.chunk;  // one split: the result goes straight to o

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int g = lane >> 2, c = lane & 3;
    const uint32_t ring = tc::smem_u32(smem) + (uint32_t)(warp * kStages * S::kStage);
    const int tiles = (count + kTile - 1) / kTile;
    const int mine = tiles > warp ? (tiles - warp + kWarps - 1) / kWarps : 0;  // tiles warp, warp + kWarps, ...
    const int64_t row_elems = (int64_t)p.Hk * D;
    const __nv_bfloat16* kc = static_cast<const __nv_bfloat16*>(p.k_cache) + (int64_t)hk * D;
    const __nv_bfloat16* vc = static_cast<const __nv_bfloat16*>(p.v_cache) + (int64_t)hk * D;
    const int32_t* table = p.table + (int64_t)n * p.max_pages;

    // The cache row of token lane % 16 of this warp's tile i, or -1 where there is none.
    auto find_row = [&](int i) -> int64_t {
        const int off = (i * kWarps + warp) * kTile + (lane & 15);
        if (i >= mine || off >= count) return -1;
        const int64_t pos = begin + off, page_no = pos / p.page_size;
        if (page_no >= p.max_pages) return -1;
        const int page = __ldg(table + page_no);
        if (page < 0 || page >= p.num_pages) return -1;
        return (int64_t)page * p.page_size + (pos - page_no * p.page_size);
    };
    auto issue = [&](int i, int64_t row) {
        constexpr int CH = D / 8, RPI = 32 / CH;  // 16-byte pieces a row, rows a warp instruction
        const uint32_t kb = ring + (uint32_t)((i % kStages) * S::kStage), vb = kb + kTile * S::kRow;
        const int ch = lane % CH;
#pragma unroll
        for (int r0 = 0; r0 < kTile; r0 += RPI) {
            const int r = r0 + lane / CH;
            const int64_t at = __shfl_sync(0xffffffffu, row, r);
            const bool ok = at >= 0;
            const int64_t off = (ok ? at : 0) * row_elems + ch * 8;
            const uint32_t dst = (uint32_t)(r * S::kRow + ((ch ^ (r & 7)) << 4));
            cp_async16(kb + dst, kc + off, ok);
            cp_async16(vb + dst, vc + off, ok);
        }
    };

    // ring prologue: tiles 0 .. kStages - 2 on their way, the row of the one after looked up
    uint32_t valid[kStages];  // bit t: token t of the tile in that slot exists
    int64_t next = -1;
    {
        int64_t rows_of[kStages];
#pragma unroll
        for (int i = 0; i < kStages; ++i) rows_of[i] = find_row(i);
#pragma unroll
        for (int i = 0; i < kStages - 1; ++i) {
            if (i < mine) issue(i, rows_of[i]);
            cp_commit();
            valid[i] = __ballot_sync(0xffffffffu, rows_of[i] >= 0) & 0xFFFFu;
        }
        valid[kStages - 1] = 0;
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
            qa[k][1] = pair(g + 8, k * 16 + 2 * c);
            qa[k][2] = pair(g, k * 16 + 2 * c + 8);
            qa[k][3] = pair(g + 8, k * 16 + 2 * c + 8);
        }
    }

    float o[D / 8][4];
#pragma unroll
    for (int j = 0; j < D / 8; ++j) o[j][0] = o[j][1] = o[j][2] = o[j][3] = 0.f;
    float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;  // rows g and g + 8 (l: this lane's share)
    const int lr = lane & 7, lm = lane >> 3;                   // ldmatrix: row and matrix of this lane
#pragma unroll 1
    for (int i = 0; i < mine; ++i) {
        // the tile kStages - 1 ahead takes the slot that the last iteration read
        const int64_t row = next;
        const int ahead = i + kStages - 1;
        next = find_row(ahead + 1);
        __syncwarp();
        if (ahead < mine) issue(ahead, row);
        cp_commit();
        const uint32_t ahead_valid = __ballot_sync(0xffffffffu, row >= 0) & 0xFFFFu;
        cp_wait<kStages - 1>();
        __syncwarp();
        const uint32_t mask = valid[0];
#pragma unroll
        for (int s = 0; s + 1 < kStages - 1; ++s) valid[s] = valid[s + 1];
        valid[kStages - 2] = ahead_valid;

        const uint32_t kb = ring + (uint32_t)((i % kStages) * S::kStage), vb = kb + kTile * S::kRow;
        float s0[4] = {}, s1[4] = {};  // tokens 0-7 and 8-15
        {
            const int t = ((lm >> 1) << 3) + lr;
#pragma unroll
            for (int k = 0; k < D / 16; ++k) {
                uint32_t kf[4];
                ldsm4(kb + (uint32_t)(t * S::kRow + (((2 * k + (lm & 1)) ^ lr) << 4)), kf);
                mma16816(s0, qa[k], kf[0], kf[1]);
                mma16816(s1, qa[k], kf[2], kf[3]);
            }
        }
        // scores in units of log 2; tokens that do not exist leave the softmax
        const uint32_t mm = mask >> (2 * c);
        const bool t0 = mm & 1u, t1 = mm & 2u, t2 = mm & 256u, t3 = mm & 512u;
        s0[0] = t0 ? s0[0] * scale_log2 : -INFINITY;
        s0[1] = t1 ? s0[1] * scale_log2 : -INFINITY;
        s0[2] = t0 ? s0[2] * scale_log2 : -INFINITY;
        s0[3] = t1 ? s0[3] * scale_log2 : -INFINITY;
        s1[0] = t2 ? s1[0] * scale_log2 : -INFINITY;
        s1[1] = t3 ? s1[1] * scale_log2 : -INFINITY;
        s1[2] = t2 ? s1[2] * scale_log2 : -INFINITY;
        s1[3] = t3 ? s1[3] * scale_log2 : -INFINITY;
        float x0 = fmaxf(fmaxf(s0[0], s0[1]), fmaxf(s1[0], s1[1]));
        float x1 = fmaxf(fmaxf(s0[2], s0[3]), fmaxf(s1[2], s1[3]));
        x0 = fmaxf(x0, __shfl_xor_sync(0xffffffffu, x0, 1));
        x1 = fmaxf(x1, __shfl_xor_sync(0xffffffffu, x1, 1));
        x0 = fmaxf(x0, __shfl_xor_sync(0xffffffffu, x0, 2));
        x1 = fmaxf(x1, __shfl_xor_sync(0xffffffffu, x1, 2));
        if (__any_sync(0xffffffffu, x0 > m0 || x1 > m1)) {
            const float n0 = fmaxf(m0, x0), n1 = fmaxf(m1, x1);
            const float f0 = n0 == -INFINITY ? 1.f : exp2f(m0 - n0), f1 = n1 == -INFINITY ? 1.f : exp2f(m1 - n1);
            m0 = n0;
            m1 = n1;
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
        const float z0 = m0 == -INFINITY ? 0.f : m0, z1 = m1 == -INFINITY ? 0.f : m1;
        s0[0] = exp2f(s0[0] - z0); s0[1] = exp2f(s0[1] - z0);
        s1[0] = exp2f(s1[0] - z0); s1[1] = exp2f(s1[1] - z0);
        s0[2] = exp2f(s0[2] - z1); s0[3] = exp2f(s0[3] - z1);
        s1[2] = exp2f(s1[2] - z1); s1[3] = exp2f(s1[3] - z1);
        l0 += (s0[0] + s0[1]) + (s1[0] + s1[1]);
        l1 += (s0[2] + s0[3]) + (s1[2] + s1[3]);
        // p rounded to bf16, the tensor cores' operand type; the sum above keeps fp32
        const uint32_t pa[4] = {tc::pack_bf16x2(s0[0], s0[1]), tc::pack_bf16x2(s0[2], s0[3]),
                                tc::pack_bf16x2(s1[0], s1[1]), tc::pack_bf16x2(s1[2], s1[3])};
        {
            const int t = ((lm & 1) << 3) + lr;
#pragma unroll
            for (int j = 0; j < D / 16; ++j) {
                uint32_t vf[4];
                ldsm4_t(vb + (uint32_t)(t * S::kRow + (((2 * j + (lm >> 1)) ^ lr) << 4)), vf);
                mma16816(o[2 * j], pa, vf[0], vf[1]);
                mma16816(o[2 * j + 1], pa, vf[2], vf[3]);
            }
        }
        __syncwarp();
    }
    cp_wait<0>();
    l0 += __shfl_xor_sync(0xffffffffu, l0, 1);
    l1 += __shfl_xor_sync(0xffffffffu, l1, 1);
    l0 += __shfl_xor_sync(0xffffffffu, l0, 2);
    l1 += __shfl_xor_sync(0xffffffffu, l1, 2);

    // join the warps: [warp][16][D] accumulators in the ring, maxima and sums behind it
    __syncthreads();
    float* acc = reinterpret_cast<float*>(smem);
    float* ms = reinterpret_cast<float*>(smem + S::kRing);
    float* ls = ms + kWarps * 16;
#pragma unroll
    for (int j = 0; j < D / 8; ++j) {
        float* r0 = acc + (warp * 16 + g) * D + j * 8 + 2 * c;
        *reinterpret_cast<float2*>(r0) = make_float2(o[j][0], o[j][1]);
        *reinterpret_cast<float2*>(r0 + 8 * D) = make_float2(o[j][2], o[j][3]);
    }
    if (c == 0) {
        ms[warp * 16 + g] = m0;
        ms[warp * 16 + g + 8] = m1;
        ls[warp * 16 + g] = l0;
        ls[warp * 16 + g + 8] = l1;
    }
    __syncthreads();
    const int64_t out_rows = (int64_t)p.N * p.Hq;
    for (int e = threadIdx.x; e < rows * D; e += kThreads) {
        const int r = e / D, ch = e - r * D;
        float m = -INFINITY;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) m = fmaxf(m, ms[w * 16 + r]);
        float l = 0.f, x = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            const float mw = ms[w * 16 + r], f = mw == -INFINITY ? 0.f : exp2f(mw - m);
            l += f * ls[w * 16 + r];
            x = fmaf(f, acc[(w * 16 + r) * D + ch], x);
        }
        const int64_t out = (int64_t)n * p.Hq + hq0 + r;
        if (whole) {
            static_cast<__nv_bfloat16*>(p.o)[out * D + ch] = __float2bfloat16_rn(l > 0.f ? x / l : 0.f);
        } else {
            float* part = p.part + ((int64_t)split * out_rows + out) * (D + 2);
            part[2 + ch] = x;
            if (ch == 0) {
                part[0] = m;
                part[1] = l;
            }
        }
    }
}

// Joins the chunks of one (sequence, query head): one CTA a row, a thread a channel and slice of the
// chunks.
template <int D>
__global__ void __launch_bounds__(D* kSplitSlices) combine_kernel(DecodeAttnParams p) {
    __shared__ float red[kSplitSlices][D];
    __shared__ float red_l[kSplitSlices], red_m[D * kSplitSlices / 32];
    const int64_t row = blockIdx.x, out_rows = (int64_t)p.N * p.Hq;
    int64_t first, len;
    context_range(p, (int)(row / p.Hq), first, len);
    const int used = (int)((len - first + p.chunk - 1) / p.chunk);
    if (used <= 1) return;
    const int ch = threadIdx.x % D, slice = threadIdx.x / D;
    const float* part = p.part + row * (D + 2);
    const int64_t step = out_rows * (D + 2);
    float m = -INFINITY;
    for (int s = threadIdx.x; s < used; s += D * kSplitSlices) m = fmaxf(m, part[s * step]);
#pragma unroll
    for (int off = 16; off; off >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
    if ((threadIdx.x & 31) == 0) red_m[threadIdx.x >> 5] = m;
    __syncthreads();
    m = red_m[0];
#pragma unroll
    for (int w = 1; w < D * kSplitSlices / 32; ++w) m = fmaxf(m, red_m[w]);
    float l = 0.f, x = 0.f;
    for (int s = slice; s < used; s += kSplitSlices) {
        const float ms = part[s * step], f = ms == -INFINITY ? 0.f : exp2f(ms - m);
        l = fmaf(f, part[s * step + 1], l);
        x = fmaf(f, part[s * step + 2 + ch], x);
    }
    red[slice][ch] = x;
    if (ch == 0) red_l[slice] = l;
    __syncthreads();
    if (slice) return;
    x = 0.f;
    l = 0.f;
#pragma unroll
    for (int s = 0; s < kSplitSlices; ++s) {
        x += red[s][ch];
        l += red_l[s];
    }
    static_cast<__nv_bfloat16*>(p.o)[row * D + ch] = __float2bfloat16_rn(l > 0.f ? x / l : 0.f);
}

template <int D>
cudaError_t launch(const DecodeAttnParams& p, cudaStream_t st) {
    using S = Smem<D>;
    cudaError_t e = cudaFuncSetAttribute(decode_attn_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kBytes);
    if (e != cudaSuccess) return e;
    const int64_t blocks = (p.Hq / p.Hk + 15) / 16;
    decode_attn_kernel<D><<<(unsigned)(p.N * p.Hk * blocks * p.splits), kThreads, S::kBytes, st>>>(
        p, p.scale * 1.4426950408889634f);
    count_launch();
    if (p.splits > 1) {
        combine_kernel<D><<<(unsigned)((int64_t)p.N * p.Hq), D * kSplitSlices, 0, st>>>(p);
        count_launch();
    }
    return cudaGetLastError();
}

}  // namespace

// Chunk length and number of chunks for contexts of up to `reach` tokens.  Two CTAs fit on an SM;
// eight CTAs' worth of work an SM evens out ragged lengths, chunks of at most 512 tokens keep a long sequence
// from being the tail, and at least 64 give every warp a tile.  The partial results are bounded at
// 64 MB and 512 chunks, whatever the table's reach.
void plan_decode_attn(int64_t N, int64_t Hq, int64_t Hk, int64_t reach, int* chunk, int* splits) {
    const int64_t units = N * Hk * ((Hq / Hk + 15) / 16);
    int64_t c = (units * reach + 148 * 8 - 1) / (148 * 8);
    c = c < 64 ? 64 : (c > 512 ? 512 : c);
    int64_t most = (int64_t(1) << 24) / (N * Hq * 130);
    most = most < 1 ? 1 : (most > 512 ? 512 : most);
    if (c * most < reach) c = (reach + most - 1) / most;
    c = (c + 63) / 64 * 64;
    *chunk = (int)c;
    *splits = (int)((reach + c - 1) / c);
    if (*splits < 1) *splits = 1;
}

size_t decode_attn_part_floats(int64_t N, int64_t Hq, int64_t d, int splits) {
    return splits > 1 ? (size_t)splits * N * Hq * (d + 2) : 0;
}

cudaError_t decode_attn(const DecodeAttnParams& p, int d, cudaStream_t st) {
    return d == 128 ? launch<128>(p, st) : launch<64>(p, st);
}

}  // namespace gdn

// Per-head RMS norm of q and k with the rotation by position (forward, backward), and the paged
// cache's append, which does the same on the way into the cache (the formulas stand at gdn_qk_norm
// in gdn.h).
//
// A head row of d channels is held by d / 8 lanes, 8 channels (one 16-byte bf16 vector) each, so a warp
// holds 2 rows of 128 or 4 of 64.  The mean of squares is a butterfly over those lanes.  In the half
// layout the partner of channel i is i +- rot / 2, the same register of another lane (rot / 2 is a
// multiple of 8): one shuffle a channel.  In the interleaved layout it is the neighbouring register.
//
// A CTA takes a tile of tokens and all their heads, flattened to rows.  cos and sin of the tile's
// tokens are formed once, in shared memory, and shared by every head: the angle p * f in turns is
// a product in 64 bits, of which only the fraction is kept, so that positions of millions lose
// nothing; fp32 sincospi then sees an argument in [-1, 1].
//
// Bound: HBM, each row read once and written once (backward: two rows read, one written).
#include <cuda_bf16.h>

#include "attn.h"
#include "common.cuh"
#include "launch.h"

namespace gdn {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxTile = 8;   // tokens a CTA at most
constexpr int kHalfMax = 64;  // rot / 2 at most

__device__ __forceinline__ void load8(const float* p, bool vec, float (&x)[8]) {
    if (vec) {
        const float4 a = __ldg(reinterpret_cast<const float4*>(p)), b = __ldg(reinterpret_cast<const float4*>(p) + 1);
        x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
        x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = __ldg(p + i);
    }
}
__device__ __forceinline__ void load8(const __nv_bfloat16* p, bool vec, float (&x)[8]) {
    if (vec) {
        const uint4 v = __ldg(reinterpret_cast<const uint4*>(p));
        const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[2 * i] = __uint_as_float(u[i] << 16);
            x[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = __bfloat162float(p[i]);
    }
}
__device__ __forceinline__ void store8(float* p, const float (&x)[8]) {
    reinterpret_cast<float4*>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float (&x)[8]) {
    uint32_t u[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
        u[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    *reinterpret_cast<uint4*>(p) = make_uint4(u[0], u[1], u[2], u[3]);
}

// Sum over the d / 8 lanes of a row.
template <int D>
__device__ __forceinline__ float row_sum(float x) {
#pragma unroll
    for (int o = D / 16; o >= 1; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

struct Table {
    float c[kMaxTile][kHalfMax];
    float s[kMaxTile][kHalfMax];
};

// cos and sin of `n` tokens' angles; pos(i): the position of the tile's token i.
template <class POS>
__device__ __forceinline__ void fill_table(Table& tb, const RopeParams& r, int n, POS pos) {
    const int half = r.rot >> 1;
    for (int i = threadIdx.x; i < n * half; i += kThreads) {
        const int t = i / half, j = i - t * half;
        const double turns = (double)pos(t) * (double)__ldg(r.inv_freq + j) * 0.15915494309189533577;
        float sn, cs;
        sincospif((float)(2.0 * (turns - rint(turns))), &sn, &cs);
        tb.c[t][j] = cs * r.rot_scale;
        tb.s[t][j] = sn * r.rot_scale;
    }
}

// The rotation (or, with inverse, its transpose) of a row's first rot channels; c0: this lane's
// first channel.  Every lane of the warp calls it.
template <int D>
__device__ __forceinline__ void rotate(float (&x)[8], const Table& tb, int t, int c0, const RopeParams& r,
                                       bool inverse) {
    if (r.rot == 0) return;
    const int half = r.rot >> 1;
    const bool in = c0 < r.rot;
    if (r.interleaved) {
        if (!in) return;
        const float4 c = *reinterpret_cast<const float4*>(&tb.c[t][c0 >> 1]);
        float4 s = *reinterpret_cast<const float4*>(&tb.s[t][c0 >> 1]);
        const float cc[4] = {c.x, c.y, c.z, c.w}, ss[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float sn = inverse ? -ss[i] : ss[i], a = x[2 * i], b = x[2 * i + 1];
            x[2 * i] = a * cc[i] - b * sn;
            x[2 * i + 1] = b * cc[i] + a * sn;
        }
    } else {
        const bool lower = c0 < half;
        const int lane = threadIdx.x & 31, hop = half >> 3;
        const int src = in ? (lower ? lane + hop : lane - hop) : lane;
        float y[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = __shfl_sync(0xffffffffu, x[i], src);
        if (!in) return;
        const int j = lower ? c0 : c0 - half;
        const bool minus = lower != inverse;
#pragma unroll
        for (int g = 0; g < 2; ++g) {
            const float4 c = *reinterpret_cast<const float4*>(&tb.c[t][j + 4 * g]);
            const float4 s = *reinterpret_cast<const float4*>(&tb.s[t][j + 4 * g]);
            const float cc[4] = {c.x, c.y, c.z, c.w}, ss[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) x[4 * g + i] = x[4 * g + i] * cc[i] + (minus ? -ss[i] : ss[i]) * y[4 * g + i];
        }
    }
}

// Where the cache takes a token: its position, and its slot (page * page_size + offset), kNoSlot if
// the table has none for it, or kOutside for a token of no sequence.
constexpr int64_t kNoSlot = -1, kOutside = -2;
__device__ __forceinline__ void find_token(const AppendParams& a, int T, int t, int& pos, int64_t& slot) {
    int s = t, i = 0;
    pos = 0;
    slot = kOutside;
    if (a.cu) {
        // the last sequence that starts at or before t
        int lo = 0, hi = a.nseq;
        while (lo < hi) {
            const int mid = (lo + hi) >> 1;
            if (__ldg(a.cu + mid + 1) > t) hi = mid;
            else lo = mid + 1;
        }
        s = lo;
        if (s >= a.nseq) return;
        const int begin = __ldg(a.cu + s);
        if (begin < 0 || begin > t) return;
        i = t - begin;
    }
    slot = kNoSlot;
    const int64_t p = (int64_t)__ldg(a.context + s) + i;
    if (p < 0 || p > 2147483647) return;
    pos = (int)p;
    const int64_t page_no = p / a.page_size;
    if (page_no >= a.max_pages) return;
    const int page = __ldg(a.table + (int64_t)s * a.max_pages + page_no);
    if (page < 0 || page >= a.num_pages) return;
    slot = (int64_t)page * a.page_size + (p - page_no * a.page_size);
}

// Rows of a tile: token-major, a token's q heads, then its k heads (append: then its v heads).
template <class T, int D, bool APPEND>
__global__ void __launch_bounds__(kThreads) rope_fwd_kernel(QkParams p, int tile) {
    constexpr int LANES = D / 8, RPC = kThreads / LANES;  // lanes a row, rows a pass of the CTA
    __shared__ Table tb;
    __shared__ int s_pos[kMaxTile];
    __shared__ int64_t s_slot[kMaxTile];
    const int t0 = blockIdx.x * tile, n = min(tile, p.T - t0);
    const int per = p.Hq + (APPEND ? 2 : 1) * p.Hk, rows = n * per;
    const int c0 = (threadIdx.x % LANES) * 8;
    if (APPEND) {
        if ((int)threadIdx.x < n) find_token(p.app, p.T, t0 + threadIdx.x, s_pos[threadIdx.x], s_slot[threadIdx.x]);
        __syncthreads();
        fill_table(tb, p.rope, n, [&](int t) { return s_pos[t]; });
    } else {
        fill_table(tb, p.rope, n, [&](int t) { return __ldg(p.positions + t0 + t); });
    }
    __syncthreads();
    float wq[8], wk[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) wq[i] = wk[i] = 1.f;
    if (p.rope.q_w) load8(static_cast<const T*>(p.rope.q_w) + c0, true, wq);
    if (p.rope.k_w) load8(static_cast<const T*>(p.rope.k_w) + c0, true, wk);
    for (int base = 0; base < rows; base += RPC) {
        const int row = base + threadIdx.x / LANES;
        const bool live = row < rows;  // whole warps stay in step: the shuffles need every lane
        const int t = live ? row / per : 0, h = live ? row - t * per : 0;
        const int64_t tok = t0 + t;
        const bool is_q = h < p.Hq, is_v = APPEND && h >= p.Hq + p.Hk;
        const int hk = is_q ? h : (is_v ? h - p.Hq - p.Hk : h - p.Hq);
        const Rows& src = is_q ? p.q : (is_v ? p.v : p.k);
        float x[8] = {};
        if (live) load8(static_cast<const T*>(src.p) + tok * src.stride + (int64_t)hk * D + c0, src.vec != 0, x);
        float y[8], ss = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) ss = fmaf(x[i], x[i], ss);
        // a warp's rows may be of different kinds: every lane takes part in the shuffles, and the
        // results are used where they apply
        ss = row_sum<D>(ss);
        const bool norm = is_q ? p.rope.q_w != nullptr : p.rope.k_w != nullptr;
        const float r = norm ? 1.f / sqrtf(ss * (1.f / D) + p.rope.eps) : 1.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = x[i] * r * (is_q ? wq[i] : wk[i]);
        rotate<D>(y, tb, t, c0, p.rope, false);
        if (!live) continue;
        if constexpr (APPEND) {
            const int64_t slot = s_slot[t];
            if (slot == kOutside) continue;
            if (is_q) {
                store8(static_cast<T*>(p.q_out) + (tok * p.Hq + hk) * D + c0, y);
            } else {
                const int64_t at = (slot * p.Hk + hk) * D + c0;
                if (is_v) {
                    if (slot >= 0) store8(static_cast<T*>(p.app.v_cache) + at, x);
                } else {
                    if (slot >= 0) store8(static_cast<T*>(p.app.k_cache) + at, y);
                    if (p.k_out) store8(static_cast<T*>(p.k_out) + (tok * p.Hk + hk) * D + c0, y);
                }
            }
        } else {
            store8(is_q ? static_cast<T*>(p.q_out) + (tok * p.Hq + hk) * D + c0
                        : static_cast<T*>(p.k_out) + (tok * p.Hk + hk) * D + c0,
                   y);
        }
    }
}

// The reverse mode.  With n = x r w, r = 1 / sqrt(mean x^2 + eps), and gn the gradient of n (the
// rotation's transpose applied to the gradient of y):
//     dw = sum over rows of gn x r,     dx = r (gn w - x r^2 mean(gn w x)).
// The CTAs walk the tiles in a fixed stride and keep dw in registers, 8 channels of q's and of k's
// weights a lane; at the end a CTA adds its rows in shared memory and stores one partial, and
// rope_dw_kernel adds the CTAs' partials.  Every order is fixed by the sizes.
template <class T, int D>
__global__ void __launch_bounds__(kThreads) rope_bwd_kernel(QkParams p, T* __restrict__ dq, T* __restrict__ dk,
                                                            int tile, int tiles) {
    constexpr int LANES = D / 8, RPC = kThreads / LANES;
    __shared__ Table tb;
    __shared__ float red[2][RPC][D];
    const int per = p.Hq + p.Hk;
    const int c0 = (threadIdx.x % LANES) * 8;
    float wq[8], wk[8], aq[8], ak[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        wq[i] = wk[i] = 1.f;
        aq[i] = ak[i] = 0.f;
    }
    if (p.rope.q_w) load8(static_cast<const T*>(p.rope.q_w) + c0, true, wq);
    if (p.rope.k_w) load8(static_cast<const T*>(p.rope.k_w) + c0, true, wk);
    for (int it = blockIdx.x; it < tiles; it += gridDim.x) {
        const int t0 = it * tile, n = min(tile, p.T - t0), rows = n * per;
        __syncthreads();
        fill_table(tb, p.rope, n, [&](int t) { return __ldg(p.positions + t0 + t); });
        __syncthreads();
        for (int base = 0; base < rows; base += RPC) {
            const int row = base + threadIdx.x / LANES;
            const bool live = row < rows;
            const int t = live ? row / per : 0, h = live ? row - t * per : 0;
            const int64_t tok = t0 + t;
            const bool is_q = h < p.Hq;
            const int hk = is_q ? h : h - p.Hq;
            const Rows& src = is_q ? p.q : p.k;
            const int64_t at = is_q ? (tok * p.Hq + hk) * D + c0 : (tok * p.Hk + hk) * D + c0;
            float x[8] = {}, g[8] = {};
            if (live) {
                load8(static_cast<const T*>(src.p) + tok * src.stride + (int64_t)hk * D + c0, src.vec != 0, x);
                load8(static_cast<const T*>(is_q ? p.gq : p.gk) + at, true, g);
            }
            rotate<D>(g, tb, t, c0, p.rope, true);
            float ss = 0.f, gx = 0.f;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                ss = fmaf(x[i], x[i], ss);
                gx = fmaf(g[i] * (is_q ? wq[i] : wk[i]), x[i], gx);
            }
            ss = row_sum<D>(ss);
            gx = row_sum<D>(gx);
            if (!live) continue;
            if (is_q ? p.rope.q_w != nullptr : p.rope.k_w != nullptr) {
                const float r = 1.f / sqrtf(ss * (1.f / D) + p.rope.eps), m = r * r * gx * (1.f / D);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float dw = g[i] * x[i] * r;
                    if (is_q) aq[i] += dw;
                    else ak[i] += dw;
                    g[i] = r * (g[i] * (is_q ? wq[i] : wk[i]) - x[i] * m);
                }
            }
            store8((is_q ? dq : dk) + at, g);
        }
    }
    if (!p.partials) return;
    const int row = threadIdx.x / LANES;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        red[0][row][c0 + i] = aq[i];
        red[1][row][c0 + i] = ak[i];
    }
    __syncthreads();
    if (threadIdx.x < 2 * D) {
        const int w = threadIdx.x / D, c = threadIdx.x % D;
        float s = 0.f;
        for (int r = 0; r < RPC; ++r) s += red[w][r][c];
        p.partials[((int64_t)blockIdx.x * 2 + w) * D + c] = s;
    }
}

// dw[c] = sum over the CTAs' partials, 32 channels a CTA, 32 strided slices of the partials each.
__global__ void __launch_bounds__(1024) rope_dw_kernel(const float* __restrict__ partials, int ctas, int d,
                                                       float* __restrict__ dq_w, float* __restrict__ dk_w) {
    __shared__ float red[32][33];
    const int c = blockIdx.x * 32 + threadIdx.x;  // channel of [2][d]
    float s = 0.f;
    for (int i = threadIdx.y; i < ctas; i += 32) s += partials[(int64_t)i * 2 * d + c];
    red[threadIdx.y][threadIdx.x] = s;
    __syncthreads();
    if (threadIdx.y) return;
    s = 0.f;
    for (int i = 0; i < 32; ++i) s += red[i][threadIdx.x];
    float* out = c < d ? dq_w : dk_w;
    if (out) out[c < d ? c : c - d] = s;
}

// Tokens a CTA: enough CTAs to fill the GPU several times over (8 of 256 threads fit on an SM), and
// as many tokens each as that leaves, which shares a CTA's start over more rows.
int tile_of(int T) {
    const int t = T / (148 * 8);
    return t < 1 ? 1 : (t > kMaxTile ? kMaxTile : t);
}
// The backward's CTAs stay for the whole call: four a SM.
int bwd_ctas(int T) {
    const int tiles = (T + tile_of(T) - 1) / tile_of(T);
    return tiles < 148 * 4 ? tiles : 148 * 4;
}

template <class T, int D, bool APPEND>
cudaError_t launch_fwd(const QkParams& p, cudaStream_t st) {
    const int tile = tile_of(p.T);
    rope_fwd_kernel<T, D, APPEND><<<(p.T + tile - 1) / tile, kThreads, 0, st>>>(p, tile);
    count_launch();
    return cudaGetLastError();
}

template <class T, int D>
cudaError_t launch_bwd(const QkParams& p, float* dq_w, float* dk_w, void* dq, void* dk, cudaStream_t st) {
    const int tile = tile_of(p.T), ctas = bwd_ctas(p.T);
    if (ctas) {
        rope_bwd_kernel<T, D><<<ctas, kThreads, 0, st>>>(p, static_cast<T*>(dq), static_cast<T*>(dk), tile,
                                                         (p.T + tile - 1) / tile);
        count_launch();
    }
    if (p.partials) {
        rope_dw_kernel<<<2 * D / 32, dim3(32, 32), 0, st>>>(p.partials, ctas, D, dq_w, dk_w);
        count_launch();
    }
    return cudaGetLastError();
}

}  // namespace

cudaError_t qk_norm_rope_fwd(const QkParams& p, int d, bool bf16, cudaStream_t st) {
    if (p.T == 0) return cudaSuccess;
    if (bf16) return d == 128 ? launch_fwd<__nv_bfloat16, 128, false>(p, st) : launch_fwd<__nv_bfloat16, 64, false>(p, st);
    return d == 128 ? launch_fwd<float, 128, false>(p, st) : launch_fwd<float, 64, false>(p, st);
}

size_t qk_norm_rope_bwd_partials(int T, int d) { return (size_t)bwd_ctas(T) * 2 * d; }

cudaError_t qk_norm_rope_bwd(const QkParams& p, int d, bool bf16, void* dq, void* dk, float* dq_w, float* dk_w,
                             cudaStream_t st) {
    if (bf16)
        return d == 128 ? launch_bwd<__nv_bfloat16, 128>(p, dq_w, dk_w, dq, dk, st)
                        : launch_bwd<__nv_bfloat16, 64>(p, dq_w, dk_w, dq, dk, st);
    return d == 128 ? launch_bwd<float, 128>(p, dq_w, dk_w, dq, dk, st) : launch_bwd<float, 64>(p, dq_w, dk_w, dq, dk, st);
}

cudaError_t kv_append(const QkParams& p, int d, cudaStream_t st) {
    if (p.T == 0) return cudaSuccess;
    return d == 128 ? launch_fwd<__nv_bfloat16, 128, true>(p, st) : launch_fwd<__nv_bfloat16, 64, true>(p, st);
}

}  // namespace gdn

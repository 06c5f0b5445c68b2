// Per-head RMS norm of q and k with the rotation by position (forward, backward), and the paged
// cache's append, which does the same on the way into the cache (the formulas stand at gdn_qk_norm
// in gdn.h).
//
// A head row of d channels is held by d / 8 lanes, 8 channels (one 16-byte bf16 vector) each, so a warp
// holds 2 rows of 128 or 4 of 64.  A warp takes one token and walks (a part of) its heads, so that all
// that depends on the token and the channel alone is formed once, in registers:
//     y_i = r (x_i A_i + x_p(i) B_i),   A_i = w_i cos, B_i = -+ w_p(i) sin,   r = 1 / sqrt(mean x^2 + eps)
// with p(i) the partner of channel i in its pair.  In the half layout the partner is i +- rot / 2, the same
// register of another lane (rot / 2 is a multiple of 8), and the raw words are exchanged, before
// the row's reduction ends; in the interleaved layout it is the neighbouring register.
//
// Angles: p * f in turns is a product in 64 bits, of which only the fraction is kept, so that positions
// of millions lose nothing; fp32 sincospi then sees an argument in [-1, 1].  A warp forms its token's
// rot / 2 angles once, two a lane.
//
// Bound: HBM, each row read once and written once (backward: two rows read, one written).  What it
// takes is enough loads in flight and few instructions a channel: the rows of a batch of kBatch are all
// loaded before the first is used.
#include <cuda_bf16.h>

#include "attn.h"
#include "common.cuh"
#include "launch.h"

namespace gdn {
namespace {

constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;
constexpr int kHalfMax = 64;  // rot / 2 at most

// Eight channels as they lie in memory.
template <class T> struct Raw;
template <> struct Raw<__nv_bfloat16> { uint32_t w[4]; };
template <> struct Raw<float> { uint32_t w[8]; };

template <class T>
__device__ __forceinline__ Raw<T> load_raw(const T* p, bool vec) {
    constexpr int W = sizeof(Raw<T>) / 4;
    Raw<T> r;
    if (vec) {
#pragma unroll
        for (int i = 0; i < W; i += 4) {
            const uint4 v = __ldg(reinterpret_cast<const uint4*>(p) + i / 4);
            r.w[i] = v.x; r.w[i + 1] = v.y; r.w[i + 2] = v.z; r.w[i + 3] = v.w;
        }
    } else if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int i = 0; i < 8; ++i) r.w[i] = __float_as_uint(__ldg(p + i));
    } else {
        const unsigned short* u = reinterpret_cast<const unsigned short*>(p);
#pragma unroll
        for (int i = 0; i < 4; ++i) r.w[i] = (uint32_t)__ldg(u + 2 * i) | ((uint32_t)__ldg(u + 2 * i + 1) << 16);
    }
    return r;
}
__device__ __forceinline__ void unpack(const Raw<__nv_bfloat16>& r, float (&x)[8]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(r.w[i] << 16);
        x[2 * i + 1] = __uint_as_float(r.w[i] & 0xFFFF0000u);
    }
}
__device__ __forceinline__ void unpack(const Raw<float>& r, float (&x)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = __uint_as_float(r.w[i]);
}
template <class T>
__device__ __forceinline__ void store_raw(T* p, const Raw<T>& r) {
#pragma unroll
    for (int i = 0; i < (int)(sizeof(Raw<T>) / 4); i += 4)
        reinterpret_cast<uint4*>(p)[i / 4] = make_uint4(r.w[i], r.w[i + 1], r.w[i + 2], r.w[i + 3]);
}
__device__ __forceinline__ Raw<float> pack(const float (&x)[8], float) {
    Raw<float> r;
#pragma unroll
    for (int i = 0; i < 8; ++i) r.w[i] = __float_as_uint(x[i]);
    return r;
}
__device__ __forceinline__ Raw<__nv_bfloat16> pack(const float (&x)[8], __nv_bfloat16) {
    Raw<__nv_bfloat16> r;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
        r.w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    return r;
}

// Sum over the d / 8 lanes of a row.
template <int D>
__device__ __forceinline__ float row_sum(float x) {
#pragma unroll
    for (int o = D / 16; o >= 1; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

// Where this lane's eight channels stand in the rotation.
struct Place {
    int c0;        // first channel
    bool in;       // among the rotated ones
    bool lower;    // half layout: first of its pairs
    int src;       // half layout: the lane that holds the partners
    int pc0;       // half layout: the partners' first channel
};
template <int D>
__device__ __forceinline__ Place place_of(const RopeParams& r) {
    Place pl;
    const int lane = threadIdx.x & 31, half = r.rot >> 1;
    pl.c0 = (lane % (D / 8)) * 8;
    pl.in = pl.c0 < r.rot;
    pl.lower = pl.c0 < half;
    const bool swap = pl.in && !r.interleaved;
    pl.src = swap ? (pl.lower ? lane + (half >> 3) : lane - (half >> 3)) : lane;
    pl.pc0 = swap ? (pl.lower ? pl.c0 + half : pl.c0 - half) : pl.c0;
    return pl;
}

// cos and signed sin of this lane's channels at position pos (1 and 0 where nothing is rotated):
//     y_i = x_i c_i + x_p(i) s_i.  Warp-collective; tb: the warp's [2][kHalfMax] floats.
__device__ __forceinline__ void angles(const RopeParams& r, const Place& pl, int pos, float* tb, float (&c)[8],
                                       float (&s)[8]) {
    const int half = r.rot >> 1;
    __syncwarp();
    for (int j = threadIdx.x & 31; j < half; j += 32) {
        const double turns = (double)pos * (double)__ldg(r.inv_freq + j) * 0.15915494309189533577;
        float sn, cs;
        sincospif((float)(2.0 * (turns - rint(turns))), &sn, &cs);
        tb[j] = cs * r.rot_scale;
        tb[kHalfMax + j] = sn * r.rot_scale;
    }
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        c[i] = 1.f;
        s[i] = 0.f;
    }
    if (!pl.in) return;
    if (r.interleaved) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            c[i] = tb[(pl.c0 + i) >> 1];
            s[i] = (i & 1) ? tb[kHalfMax + ((pl.c0 + i) >> 1)] : -tb[kHalfMax + ((pl.c0 + i) >> 1)];
        }
    } else {
        const int j = pl.lower ? pl.c0 : pl.pc0;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            c[i] = tb[j + i];
            s[i] = pl.lower ? -tb[kHalfMax + j + i] : tb[kHalfMax + j + i];
        }
    }
}

// The partners of x (whose words are r).  Every lane of the warp calls it.
template <class T>
__device__ __forceinline__ void partners(const Raw<T>& r, const float (&x)[8], const Place& pl, bool interleaved,
                                         float (&y)[8]) {
    if (interleaved) {
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = x[i ^ 1];
    } else {
        Raw<T> o;
#pragma unroll
        for (int i = 0; i < (int)(sizeof(Raw<T>) / 4); ++i) o.w[i] = __shfl_sync(0xffffffffu, r.w[i], pl.src);
        unpack(o, y);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = pl.in ? y[i] : 0.f;  // not x: 0 times an infinity is not 0
}

// The norm weights of this lane's channels and of their partners (1 without a norm).
template <class T>
__device__ __forceinline__ void weights(const void* w, const Place& pl, bool interleaved, float (&own)[8],
                                        float (&partner)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) own[i] = partner[i] = 1.f;
    if (!w) return;
    unpack(load_raw(static_cast<const T*>(w) + pl.c0, true), own);
    if (interleaved) {
#pragma unroll
        for (int i = 0; i < 8; ++i) partner[i] = own[i ^ 1];
    } else {
        unpack(load_raw(static_cast<const T*>(w) + pl.pc0, true), partner);
    }
}

// Where the cache takes a token: its position, and its slot (page * page_size + offset), kNoSlot if
// the table has none for it, or kOutside for a token of no sequence.
constexpr int64_t kNoSlot = -1, kOutside = -2;
__device__ __forceinline__ void find_token(const AppendParams& a, int t, int& pos, int64_t& slot) {
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

// Rows of one kind (q, k or v) that a warp takes of its token: heads part * RPW + (lane's row), step
// parts * RPW.  batch(n, ...) sees kBatch of them at a time, loaded together.
constexpr int kBatch = 4;

// One kind's rows, normalised and rotated, to dst (and dst2), rows of D elements from there on.
template <class T, int D>
__device__ __forceinline__ void rope_rows(const T* src, bool vec, int H, T* dst, T* dst2, bool norm, float eps,
                                          bool interleaved, const Place& pl, const float (&A)[8], const float (&B)[8],
                                          int part, int parts) {
    constexpr int RPW = 256 / D;
    const int r0 = (threadIdx.x & 31) / (D / 8), step = parts * RPW;
    for (int base = part * RPW; base < H; base += kBatch * step) {
        Raw<T> raw[kBatch];
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            const int h = base + u * step + r0;
            if (h < H) raw[u] = load_raw(src + (int64_t)h * D + pl.c0, vec);
            else raw[u] = Raw<T>{};
        }
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            const int h = base + u * step + r0;
            if (base + u * step >= H) break;  // the whole warp
            float x[8], y[8];
            unpack(raw[u], x);
            partners(raw[u], x, pl, interleaved, y);
            float r = 1.f;
            if (norm) {
                float ss = 0.f;
#pragma unroll
                for (int i = 0; i < 8; ++i) ss = fmaf(x[i], x[i], ss);
                r = rsqrtf(row_sum<D>(ss) * (1.f / D) + eps);
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) y[i] = r * fmaf(x[i], A[i], y[i] * B[i]);
            if (h < H) {
                const Raw<T> out = pack(y, T{});
                if (dst) store_raw(dst + (int64_t)h * D + pl.c0, out);
                if (dst2) store_raw(dst2 + (int64_t)h * D + pl.c0, out);
            }
        }
    }
}

template <class T, int D, bool APPEND>
__global__ void __launch_bounds__(kThreads) rope_fwd_kernel(const QkParams p, int parts) {
    constexpr int RPW = 256 / D;
    __shared__ float tb[kWarps][2 * kHalfMax];
    const int warp = threadIdx.x >> 5;
    const int64_t unit = (int64_t)blockIdx.x * kWarps + warp;
    const int64_t t = unit / parts;
    const int part = (int)(unit - t * parts);
    if (t >= p.T) return;
    int pos = 0;
    int64_t slot = 0;
    if (APPEND) {
        find_token(p.app, (int)t, pos, slot);
        if (slot == kOutside) return;
    } else if (p.positions) {
        pos = __ldg(p.positions + t);
    }
    const Place pl = place_of<D>(p.rope);
    const bool il = p.rope.interleaved != 0;
    float c[8], s[8];
    angles(p.rope, pl, pos, tb[warp], c, s);
    auto rows = [&](const Rows& src, const void* w, int H, T* dst, T* dst2) {
        float own[8], partner[8];
        weights<T>(w, pl, il, own, partner);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            own[i] *= c[i];
            partner[i] *= s[i];
        }
        rope_rows<T, D>(static_cast<const T*>(src.p) + t * src.stride, src.vec != 0, H, dst, dst2, w != nullptr,
                        p.rope.eps, il, pl, own, partner, part, parts);
    };
    if (p.Hq) rows(p.q, p.rope.q_w, p.Hq, static_cast<T*>(p.q_out) + t * p.Hq * D, static_cast<T*>(nullptr));
    T* k_out = p.k_out ? static_cast<T*>(p.k_out) + t * p.Hk * D : nullptr;
    if constexpr (APPEND) {
        const int64_t at = slot * p.Hk * D;
        T* kc = slot >= 0 ? static_cast<T*>(p.app.k_cache) + at : nullptr;
        if (kc || k_out) rows(p.k, p.rope.k_w, p.Hk, k_out, kc);
        if (slot >= 0) {
            const T* v = static_cast<const T*>(p.v.p) + t * p.v.stride;
            T* vc = static_cast<T*>(p.app.v_cache) + at;
            for (int h = part * RPW + (threadIdx.x & 31) / (D / 8); h < p.Hk; h += parts * RPW)
                store_raw(vc + (int64_t)h * D + pl.c0, load_raw(v + (int64_t)h * D + pl.c0, p.v.vec != 0));
        }
    } else if (p.Hk) {
        rows(p.k, p.rope.k_w, p.Hk, k_out, static_cast<T*>(nullptr));
    }
}

// The reverse mode.  With n = x r w, r = 1 / sqrt(mean x^2 + eps), and gn the gradient of n (the
// rotation's transpose applied to the gradient of y):
//     dw = sum over rows of gn x r,     dx = r (gn w - x r^2 mean(gn w x)).
// The warps walk the tokens in a fixed stride and keep dw in registers, 8 channels of q's and of k's
// weights a lane; at the end a CTA adds its warps' in shared memory and stores one partial, and
// rope_dw_kernel adds the CTAs' partials.  Every order is fixed by the sizes.
template <class T, int D>
__device__ __forceinline__ void rope_grad_rows(const T* src, bool vec, const T* grad, int H, T* dst, bool norm, float eps,
                                               bool interleaved, const Place& pl, const float (&w)[8], const float (&c)[8],
                                               const float (&s)[8], float (&acc)[8]) {
    constexpr int RPW = 256 / D, BATCH = 2;
    const int r0 = (threadIdx.x & 31) / (D / 8);
    for (int base = 0; base < H; base += BATCH * RPW) {
        Raw<T> rx[BATCH], rg[BATCH];
#pragma unroll
        for (int u = 0; u < BATCH; ++u) {
            const int h = base + u * RPW + r0;
            rx[u] = rg[u] = Raw<T>{};
            if (h < H) {
                rx[u] = load_raw(src + (int64_t)h * D + pl.c0, vec);
                rg[u] = load_raw(grad + (int64_t)h * D + pl.c0, true);
            }
        }
#pragma unroll
        for (int u = 0; u < BATCH; ++u) {
            const int h = base + u * RPW + r0;
            if (base + u * RPW >= H) break;
            float g[8], y[8];
            unpack(rg[u], g);
            partners(rg[u], g, pl, interleaved, y);
#pragma unroll
            for (int i = 0; i < 8; ++i) g[i] = fmaf(g[i], c[i], -(y[i] * s[i]));  // the transpose turns back
            if (norm) {
                float x[8], ss = 0.f, gx = 0.f;
                unpack(rx[u], x);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    ss = fmaf(x[i], x[i], ss);
                    gx = fmaf(g[i] * w[i], x[i], gx);
                }
                ss = row_sum<D>(ss);
                gx = row_sum<D>(gx);
                // a lane without a row adds nothing, whatever eps is
                const float r = h < H ? rsqrtf(ss * (1.f / D) + eps) : 0.f, m = r * r * gx * (1.f / D);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    acc[i] = fmaf(g[i] * x[i], r, acc[i]);
                    g[i] = r * fmaf(g[i], w[i], -(x[i] * m));
                }
            }
            if (h < H) store_raw(dst + (int64_t)h * D + pl.c0, pack(g, T{}));
        }
    }
}

template <class T, int D>
__global__ void __launch_bounds__(kThreads) rope_bwd_kernel(const QkParams p, T* __restrict__ dq, T* __restrict__ dk) {
    constexpr int RPW = 256 / D;
    __shared__ float tb[kWarps][2 * kHalfMax];
    __shared__ float red[2][kWarps * RPW][D];
    const int warp = threadIdx.x >> 5;
    const Place pl = place_of<D>(p.rope);
    const bool il = p.rope.interleaved != 0;
    float wq[8], wk[8], aq[8], ak[8], c[8], s[8];
    {
        float unused[8];
        weights<T>(p.rope.q_w, pl, il, wq, unused);
        weights<T>(p.rope.k_w, pl, il, wk, unused);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) aq[i] = ak[i] = 0.f;
    for (int64_t t = (int64_t)blockIdx.x * kWarps + warp; t < p.T; t += (int64_t)gridDim.x * kWarps) {
        angles(p.rope, pl, p.positions ? __ldg(p.positions + t) : 0, tb[warp], c, s);
        rope_grad_rows<T, D>(static_cast<const T*>(p.q.p) + t * p.q.stride, p.q.vec != 0,
                             static_cast<const T*>(p.gq) + t * p.Hq * D, p.Hq, dq + t * p.Hq * D, p.rope.q_w != nullptr,
                             p.rope.eps, il, pl, wq, c, s, aq);
        if (p.Hk)
            rope_grad_rows<T, D>(static_cast<const T*>(p.k.p) + t * p.k.stride, p.k.vec != 0,
                                 static_cast<const T*>(p.gk) + t * p.Hk * D, p.Hk, dk + t * p.Hk * D,
                                 p.rope.k_w != nullptr, p.rope.eps, il, pl, wk, c, s, ak);
    }
    if (!p.partials) return;
    const int row = threadIdx.x / (D / 8);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        red[0][row][pl.c0 + i] = aq[i];
        red[1][row][pl.c0 + i] = ak[i];
    }
    __syncthreads();
    for (int e = threadIdx.x; e < 2 * D; e += kThreads) {
        const int w = e / D, ch = e % D;
        float sum = 0.f;
#pragma unroll
        for (int r = 0; r < kWarps * RPW; ++r) sum += red[w][r][ch];
        p.partials[(int64_t)blockIdx.x * 2 * D + e] = sum;
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

// Warps that share a token's heads: one where the tokens alone fill the GPU (148 SMs of 16 CTAs), more for
// the few tokens of a serving step, down to one batch of rows a warp.
int parts_of(int T, int heads, int d) {
    const int rpw = 256 / d, most = (heads + rpw - 1) / rpw;
    const int want = T ? (148 * 16 * kWarps + T - 1) / T : 1;
    return want < 1 ? 1 : (want > most ? most : want);
}
// The backward's CTAs stay for the whole call: eight a SM.
int bwd_ctas(int T) {
    const int64_t c = ((int64_t)T + kWarps - 1) / kWarps;
    return (int)(c < 148 * 8 ? c : 148 * 8);
}

template <class T, int D, bool APPEND>
cudaError_t launch_fwd(const QkParams& p, cudaStream_t st) {
    const int parts = parts_of(p.T, p.Hq > p.Hk ? p.Hq : p.Hk, D);
    rope_fwd_kernel<T, D, APPEND><<<(unsigned)(((int64_t)p.T * parts + kWarps - 1) / kWarps), kThreads, 0, st>>>(p, parts);
    count_launch();
    return cudaGetLastError();
}

template <class T, int D>
cudaError_t launch_bwd(const QkParams& p, float* dq_w, float* dk_w, void* dq, void* dk, cudaStream_t st) {
    const int ctas = bwd_ctas(p.T);
    if (ctas) {
        rope_bwd_kernel<T, D><<<ctas, kThreads, 0, st>>>(p, static_cast<T*>(dq), static_cast<T*>(dk));
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

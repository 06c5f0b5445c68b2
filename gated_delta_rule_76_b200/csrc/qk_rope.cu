// Per-head RMS norm of q and k with the rotation by position (forward, backward), and the paged
// cache's append, which does the same on the way into the cache (the formulas stand at gdn_qk_norm
// in gdn.h).
//
// A lane holds 16 channels of a head row, two 16-byte vectors (of bf16), chosen so that both channels of each
// of its 8 pairs are its own: in the half layout vectors v and v + rot / 16 (rot / 2 is a multiple of
// 8 channels), in the interleaved layout neighbouring ones; vectors that are not rotated pair up among themselves.
// a and b are the first and second channels of the pairs, and only loading and storing know the layout.
// Eight lanes hold a row of 128, four a row of 64: a warp 4 or 8 rows.
//
// A warp takes one token and walks (a part of) its heads of one kind (q, k or v), so that all that depends on the
// token and the channel alone is formed once, in registers:
//     y_a = r (a (w_a cos) - b (w_b sin)),  y_b = r (b (w_b cos) + a (w_a sin)),  r = 1 / sqrt(mean x^2 + eps).
// Angles: p * f in turns is a product in 64 bits, of which only the fraction is kept, so that positions
// of millions lose nothing; fp32 sincospi then sees an argument in [-1, 1].  A warp forms its token's
// rot / 2 angles once, two a lane at most.
//
// Bound: HBM, each row read once and written once (backward: two rows read, one written).  What it
// takes is enough loads in flight (the rows of a batch are all loaded before the first is used) and few
// instructions a channel (no exchange between lanes but the row's sum; packed fp32 pairs).
// Measured, d = 128 in bf16: 32768 tokens of 16 + 4 heads forward and backward 177 us, 4.7 TB/s (a copy: 6.5);
// 4099 tokens of 128 + 16 heads forward 57 us, 5.2 TB/s; two tokens 3.2 us.  In fp32, the 32768 tokens: forward 122 us, 5.5
// TB/s, backward 214 us, 4.7 TB/s, the latter with 48 to 52 bytes of spills at its 128 registers.  Tried and slower: five CTAs an SM (262 us:
// spills), batches of 2 rows (186 us), the backward's rows through a private ring in shared memory (189 us).
#include <cuda_bf16.h>

#include "attn.h"
#include "common.cuh"
#include "launch.h"

namespace gdn {
namespace {

constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;
constexpr int kHalfMax = 64;  // rot / 2 at most

// ---- pairs of fp32 in one 64-bit register ------------------------------------------------------
typedef unsigned long long f2;
__device__ __forceinline__ f2 f2_of(float lo, float hi) {
    f2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ void f2_get(f2 v, float& lo, float& hi) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
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

// ---- eight channels as they lie in memory ----------------------------------------------------
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
template <class T>
__device__ __forceinline__ void store_raw(T* p, const Raw<T>& r) {
#pragma unroll
    for (int i = 0; i < (int)(sizeof(Raw<T>) / 4); i += 4)
        reinterpret_cast<uint4*>(p)[i / 4] = make_uint4(r.w[i], r.w[i + 1], r.w[i + 2], r.w[i + 3]);
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
__device__ __forceinline__ void pack(const float (&x)[8], Raw<float>& r) {
#pragma unroll
    for (int i = 0; i < 8; ++i) r.w[i] = __float_as_uint(x[i]);
}
__device__ __forceinline__ void pack(const float (&x)[8], Raw<__nv_bfloat16>& r) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
        r.w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
}

// ---- a lane's 16 channels ---------------------------------------------------------------------
// Where they stand: the first channels of its two vectors, and the first of its 8 angles (-1: not rotated).
struct Place {
    int c0, c1, angle;
};
template <int D, bool IL>
__device__ __forceinline__ Place place_of(int rot) {
    const int l = (threadIdx.x & 31) % (D / 16);
    if (IL) return Place{16 * l, 16 * l + 8, 16 * l < rot ? 8 * l : -1};
    const int hv = rot >> 4;  // vectors of a half
    if (l < hv) return Place{8 * l, 8 * (l + hv), 8 * l};
    return Place{8 * (2 * hv + 2 * (l - hv)), 8 * (2 * hv + 2 * (l - hv)) + 8, -1};
}

template <class T> struct Raw2 { Raw<T> v0, v1; };
template <class T>
__device__ __forceinline__ Raw2<T> load_row(const T* p, const Place& pl, bool vec) {
    return Raw2<T>{load_raw(p + pl.c0, vec), load_raw(p + pl.c1, vec)};
}
template <class T>
__device__ __forceinline__ void store_row(T* p, const Place& pl, const Raw2<T>& r) {
    store_raw(p + pl.c0, r.v0);
    store_raw(p + pl.c1, r.v1);
}
// The 8 pairs as 4 + 4 packed registers, and back.
template <bool IL, class T>
__device__ __forceinline__ void split(const Raw2<T>& r, f2 (&a)[4], f2 (&b)[4]) {
    float x[8], y[8];
    unpack(r.v0, x);
    unpack(r.v1, y);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (IL) {
            const int e = 4 * (i & 1);
            a[i] = i < 2 ? f2_of(x[e], x[e + 2]) : f2_of(y[e], y[e + 2]);
            b[i] = i < 2 ? f2_of(x[e + 1], x[e + 3]) : f2_of(y[e + 1], y[e + 3]);
        } else {
            a[i] = f2_of(x[2 * i], x[2 * i + 1]);
            b[i] = f2_of(y[2 * i], y[2 * i + 1]);
        }
    }
}
template <bool IL, class T>
__device__ __forceinline__ Raw2<T> join(const f2 (&a)[4], const f2 (&b)[4]) {
    float x[8], y[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float a0, a1, b0, b1;
        f2_get(a[i], a0, a1);
        f2_get(b[i], b0, b1);
        if (IL) {
            const int e = 4 * (i & 1);
            float(&o)[8] = i < 2 ? x : y;
            o[e] = a0; o[e + 1] = b0; o[e + 2] = a1; o[e + 3] = b1;
        } else {
            x[2 * i] = a0; x[2 * i + 1] = a1;
            y[2 * i] = b0; y[2 * i + 1] = b1;
        }
    }
    Raw2<T> r;
    pack(x, r.v0);
    pack(y, r.v1);
    return r;
}

// Sum over the d / 16 lanes of a row.
template <int D>
__device__ __forceinline__ float row_sum(float x) {
#pragma unroll
    for (int o = D / 32; o >= 1; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}
__device__ __forceinline__ float f2_sum(f2 v) {
    float a, b;
    f2_get(v, a, b);
    return a + b;
}

// cos and sin of this lane's pairs at position pos (1 and 0 where nothing is rotated).
// Warp-collective; tb: the warp's [2][kHalfMax] floats.
__device__ __forceinline__ void angles(const RopeParams& r, const Place& pl, int pos, float* tb, f2 (&c)[4], f2 (&s)[4]) {
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
    for (int i = 0; i < 4; ++i) {
        c[i] = f2_of(1.f, 1.f);
        s[i] = f2_of(0.f, 0.f);
        if (pl.angle >= 0) {
            const float2 x = *reinterpret_cast<const float2*>(tb + pl.angle + 2 * i);
            const float2 y = *reinterpret_cast<const float2*>(tb + kHalfMax + pl.angle + 2 * i);
            c[i] = f2_of(x.x, x.y);
            s[i] = f2_of(y.x, y.y);
        }
    }
}

template <bool IL, class T>
__device__ __forceinline__ void weights(const void* w, const Place& pl, f2 (&wa)[4], f2 (&wb)[4]) {
    if (w) {
        split<IL>(load_row(static_cast<const T*>(w), pl, true), wa, wb);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) wa[i] = wb[i] = f2_of(1.f, 1.f);
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

constexpr int kBatch = 4;  // rows a lane loads before it uses the first

// A warp's rows of one kind, from src to dst and dst2 (either may be NULL), heads head0, head0 + step, ...;
// ROPE: normalised (with w) and rotated by c, s, else copied.  `before` runs while the first rows are on
// their way: it forms c and s.
template <class T, int D, bool IL, bool ROPE, class F>
__device__ __forceinline__ void fwd_rows(const T* src, bool vec, int H, T* dst, T* dst2, const void* w, float eps,
                                         const Place& pl, f2 (&c)[4], f2 (&s)[4], int base, int step, F before) {
    const int r0 = (threadIdx.x & 31) / (D / 16);
    f2 ca[4], sb[4], cb[4], sa[4];  // w_a cos, -w_b sin, w_b cos, w_a sin
    bool ready = false;
    for (; base < H; base += kBatch * step) {
        Raw2<T> raw[kBatch];
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            const int h = base + u * step + r0;
            raw[u] = Raw2<T>{};
            if (h < H) raw[u] = load_row(src + (int64_t)h * D, pl, vec);
        }
        if (ROPE && !ready) {
            f2 wa[4], wb[4];
            weights<IL, T>(w, pl, wa, wb);
            before();
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                ca[i] = f2_mul(wa[i], c[i]);
                cb[i] = f2_mul(wb[i], c[i]);
                sa[i] = f2_mul(wa[i], s[i]);
                sb[i] = f2_mul(f2_mul(wb[i], s[i]), f2_of(-1.f, -1.f));
            }
            ready = true;
        }
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            const int h = base + u * step + r0;
            if (base + u * step >= H) break;  // the whole warp
            Raw2<T> out = raw[u];
            if (ROPE) {
                f2 a[4], b[4];
                split<IL>(raw[u], a, b);
                f2 r = f2_of(1.f, 1.f);
                if (w) {
                    f2 ss = f2_mul(a[0], a[0]);
#pragma unroll
                    for (int i = 1; i < 4; ++i) ss = f2_fma(a[i], a[i], ss);
#pragma unroll
                    for (int i = 0; i < 4; ++i) ss = f2_fma(b[i], b[i], ss);
                    const float x = rsqrtf(row_sum<D>(f2_sum(ss)) * (1.f / D) + eps);
                    r = f2_of(x, x);
                }
                if (pl.angle >= 0) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const f2 ya = f2_fma(a[i], ca[i], f2_mul(b[i], sb[i]));
                        const f2 yb = f2_fma(b[i], cb[i], f2_mul(a[i], sa[i]));
                        a[i] = f2_mul(r, ya);
                        b[i] = f2_mul(r, yb);
                    }
                } else {  // not 0 times the partner, which may be infinite
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        a[i] = f2_mul(r, f2_mul(a[i], ca[i]));
                        b[i] = f2_mul(r, f2_mul(b[i], cb[i]));
                    }
                }
                out = join<IL, T>(a, b);
            }
            if (h < H) {
                if (dst) store_row(dst + (int64_t)h * D, pl, out);
                if (dst2) store_row(dst2 + (int64_t)h * D, pl, out);
            }
        }
    }
}

// 2^parts_log warps share a token's heads.
template <class T, int D, bool IL, bool APPEND>
__global__ void __launch_bounds__(kThreads) rope_fwd_kernel(const QkParams p, int parts_log) {
    constexpr int RPW = 512 / D;
    __shared__ __align__(16) float tb[kWarps][2 * kHalfMax];
    const int64_t unit = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
    const int t = (int)(unit >> parts_log);
    if (unit >> parts_log >= p.T) return;
    const int base = ((int)unit & ((1 << parts_log) - 1)) * RPW, step = RPW << parts_log;
    int pos = 0;
    int64_t slot = kNoSlot;
    if (APPEND) {
        find_token(p.app, t, pos, slot);
        if (slot == kOutside) return;
    } else if (p.positions) {
        pos = __ldg(p.positions + t);
    }
    const Place pl = place_of<D, IL>(p.rope.rot);
    f2 c[4], s[4];
    bool have = false;
    auto turn = [&]() {
        if (!have) angles(p.rope, pl, pos, tb[threadIdx.x >> 5], c, s);
        have = true;
    };
    T* none = nullptr;
    const int64_t q_at = (int64_t)t * p.Hq * D, k_at = (int64_t)t * p.Hk * D;
    if (p.Hq)
        fwd_rows<T, D, IL, true>(static_cast<const T*>(p.q.p) + t * p.q.stride, p.q.vec != 0, p.Hq,
                                 static_cast<T*>(p.q_out) + q_at, none, p.rope.q_w, p.rope.eps, pl, c, s, base, step, turn);
    T* k_out = p.k_out ? static_cast<T*>(p.k_out) + k_at : none;
    T* kc = APPEND && slot >= 0 ? static_cast<T*>(p.app.k_cache) + slot * p.Hk * D : none;
    if (k_out || kc)
        fwd_rows<T, D, IL, true>(static_cast<const T*>(p.k.p) + t * p.k.stride, p.k.vec != 0, p.Hk, k_out, kc, p.rope.k_w,
                                 p.rope.eps, pl, c, s, base, step, turn);
    if (APPEND && slot >= 0)
        fwd_rows<T, D, IL, false>(static_cast<const T*>(p.v.p) + t * p.v.stride, p.v.vec != 0, p.Hk,
                                  static_cast<T*>(p.app.v_cache) + slot * p.Hk * D, none, nullptr, 0.f, pl, c, s, base, step,
                                  turn);
}

// The reverse mode.  With n = x r w, r = 1 / sqrt(mean x^2 + eps), and gn the gradient of n (the
// rotation's transpose applied to the gradient of y):
//     dw = sum over rows of gn x r,     dx = r (gn w - x r^2 mean(gn w x)).
// The first `ctas_q` CTAs take q's rows, the others k's, each walking the tokens in a fixed stride; dw stays in
// registers, 16 channels a lane, until a CTA adds its warps' in shared memory and stores one
// partial; rope_dw_kernel adds the CTAs'.  Every order is fixed by the sizes.  All in fp32: a lane's own sum runs over its
// rows of the tokens its warp takes (32768 tokens of 16 + 4 heads: 84 rows of q), and the chains behind it over 16 rows,
// 13 partials and 32 slices, so that no term takes part in more than about 150 roundings.
// A token's heads are one warp's: 64 tokens of 64 + 8 heads take 12.5 us (fp32: 17.8), the forward, which shares them, 3.7.
template <class T, int D, bool IL>
__global__ void __launch_bounds__(kThreads, 4) rope_bwd_kernel(const QkParams p, T* __restrict__ dq, T* __restrict__ dk,
                                                               int ctas_q) {
    constexpr int RPW = 512 / D, BATCH = 2;
    __shared__ __align__(16) float tb[kWarps][2 * kHalfMax];
    __shared__ float red[kWarps * RPW][D];
    const int warp = threadIdx.x >> 5, r0 = (threadIdx.x & 31) / (D / 16);
    const bool is_q = (int)blockIdx.x < ctas_q;
    const int cta = is_q ? blockIdx.x : blockIdx.x - ctas_q, ctas = is_q ? ctas_q : gridDim.x - ctas_q;
    const int H = is_q ? p.Hq : p.Hk;
    const Rows& in = is_q ? p.q : p.k;
    const void* w = is_q ? p.rope.q_w : p.rope.k_w;
    const bool vec = in.vec != 0;
    const Place pl = place_of<D, IL>(p.rope.rot);
    f2 wa[4], wb[4], acca[4], accb[4];
    weights<IL, T>(w, pl, wa, wb);
#pragma unroll
    for (int i = 0; i < 4; ++i) acca[i] = accb[i] = f2_of(0.f, 0.f);
    const f2 minus = f2_of(-1.f, -1.f);
    for (int64_t t = (int64_t)cta * kWarps + warp; t < p.T; t += (int64_t)ctas * kWarps) {
        const T* src = static_cast<const T*>(in.p) + t * in.stride;
        const T* grad = static_cast<const T*>(is_q ? p.gq : p.gk) + t * H * D;
        T* dst = (is_q ? dq : dk) + t * H * D;
        f2 c[4], s[4];
        for (int base = 0; base < H; base += BATCH * RPW) {
            Raw2<T> rx[BATCH], rg[BATCH];
#pragma unroll
            for (int u = 0; u < BATCH; ++u) {
                const int h = base + u * RPW + r0;
                rx[u] = rg[u] = Raw2<T>{};
                if (h < H) {
                    rg[u] = load_row(grad + (int64_t)h * D, pl, true);
                    rx[u] = load_row(src + (int64_t)h * D, pl, vec);
                }
            }
            // while the first rows are on their way
            if (base == 0) angles(p.rope, pl, p.positions ? __ldg(p.positions + t) : 0, tb[warp], c, s);
#pragma unroll
            for (int u = 0; u < BATCH; ++u) {
                const int h = base + u * RPW + r0;
                if (base + u * RPW >= H) break;
                f2 ga[4], gb[4];
                split<IL>(rg[u], ga, gb);
                if (pl.angle >= 0) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {  // the transpose turns back
                        const f2 a = f2_fma(ga[i], c[i], f2_mul(gb[i], s[i]));
                        gb[i] = f2_fma(gb[i], c[i], f2_mul(f2_mul(ga[i], minus), s[i]));
                        ga[i] = a;
                    }
                }
                if (w) {
                    f2 a[4], b[4];
                    split<IL>(rx[u], a, b);
                    f2 ss = f2_mul(a[0], a[0]), gx = f2_mul(f2_mul(ga[0], wa[0]), a[0]);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        if (i) {
                            ss = f2_fma(a[i], a[i], ss);
                            gx = f2_fma(f2_mul(ga[i], wa[i]), a[i], gx);
                        }
                        ss = f2_fma(b[i], b[i], ss);
                        gx = f2_fma(f2_mul(gb[i], wb[i]), b[i], gx);
                    }
                    const float s1 = row_sum<D>(f2_sum(ss)), g1 = row_sum<D>(f2_sum(gx));
                    // a lane without a row adds nothing, whatever eps is
                    const float r1 = h < H ? rsqrtf(s1 * (1.f / D) + p.rope.eps) : 0.f;
                    const float m1 = -r1 * r1 * g1 * (1.f / D);
                    const f2 r = f2_of(r1, r1), m = f2_of(m1, m1);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        acca[i] = f2_fma(f2_mul(ga[i], a[i]), r, acca[i]);
                        accb[i] = f2_fma(f2_mul(gb[i], b[i]), r, accb[i]);
                        ga[i] = f2_mul(r, f2_fma(ga[i], wa[i], f2_mul(a[i], m)));
                        gb[i] = f2_mul(r, f2_fma(gb[i], wb[i], f2_mul(b[i], m)));
                    }
                }
                if (h < H) store_row(dst + (int64_t)h * D, pl, join<IL, T>(ga, gb));
            }
        }
    }
    if (!p.partials || !w) return;
    const int row = threadIdx.x / (D / 16);
    const Raw2<float> acc = join<IL, float>(acca, accb);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        red[row][pl.c0 + i] = __uint_as_float(acc.v0.w[i]);
        red[row][pl.c1 + i] = __uint_as_float(acc.v1.w[i]);
    }
    __syncthreads();
    if (threadIdx.x < D) {
        float sum = 0.f;
#pragma unroll
        for (int r = 0; r < kWarps * RPW; ++r) sum += red[r][threadIdx.x];
        p.partials[(int64_t)blockIdx.x * D + threadIdx.x] = sum;
    }
}

// dw[c] = sum over the CTAs' partials of one kind (blockIdx.y), 32 channels a CTA, 32 strided slices of the
// partials each.
__global__ void __launch_bounds__(1024) rope_dw_kernel(const float* __restrict__ partials, int ctas_q, int ctas_k, int d,
                                                       float* __restrict__ dq_w, float* __restrict__ dk_w) {
    __shared__ float red[32][33];
    float* out = blockIdx.y ? dk_w : dq_w;
    if (!out) return;
    const int c = blockIdx.x * 32 + threadIdx.x;
    const int first = blockIdx.y ? ctas_q : 0, n = blockIdx.y ? ctas_k : ctas_q;
    float s = 0.f;
#pragma unroll 8
    for (int i = threadIdx.y; i < n; i += 32) s += partials[(int64_t)(first + i) * d + c];
    red[threadIdx.y][threadIdx.x] = s;
    __syncthreads();
    if (threadIdx.y) return;
    s = 0.f;
#pragma unroll
    for (int i = 0; i < 32; ++i) s += red[i][threadIdx.x];
    out[c] = s;
}

// Warps that share a token's heads, as a power of 2: one where the tokens alone fill the GPU (148 SMs of 16
// warps, twice over), more for the few tokens of a serving step, down to one pass over a warp's rows.
int parts_log_of(int T, int heads, int d) {
    const int rpw = 512 / d;
    int log = 0;
    while (((int64_t)T << log) < 148 * 16 * 2 && (rpw << log) < heads) ++log;
    return log;
}
// The backward's CTAs stay for the whole call, four a SM, shared out by what a token costs either kind: its
// passes of a warp, and about two more for the angles.
void bwd_ctas(int T, int Hq, int Hk, int d, int* q, int* k) {
    const int rpw = 512 / d;
    const int64_t most = ((int64_t)T + kWarps - 1) / kWarps, all = 148 * 4;
    const int64_t cq = (Hq + rpw - 1) / rpw + 2, ck = Hk ? (Hk + rpw - 1) / rpw + 2 : 0;
    const int64_t nk = all * ck / (cq + ck), nq = all - nk;
    *q = (int)(nq < most ? nq : most);
    *k = (int)(nk < most ? nk : most);
}

template <class T, int D, bool APPEND>
cudaError_t launch_fwd(const QkParams& p, cudaStream_t st) {
    const int log = parts_log_of(p.T, p.Hq > p.Hk ? p.Hq : p.Hk, D);
    const unsigned ctas = (unsigned)((((int64_t)p.T << log) + kWarps - 1) / kWarps);
    if (p.rope.interleaved) rope_fwd_kernel<T, D, true, APPEND><<<ctas, kThreads, 0, st>>>(p, log);
    else rope_fwd_kernel<T, D, false, APPEND><<<ctas, kThreads, 0, st>>>(p, log);
    count_launch();
    return cudaGetLastError();
}

template <class T, int D>
cudaError_t launch_bwd(const QkParams& p, float* dq_w, float* dk_w, void* dq, void* dk, cudaStream_t st) {
    int nq, nk;
    bwd_ctas(p.T, p.Hq, p.Hk, D, &nq, &nk);
    if (nq + nk) {
        if (p.rope.interleaved)
            rope_bwd_kernel<T, D, true><<<nq + nk, kThreads, 0, st>>>(p, static_cast<T*>(dq), static_cast<T*>(dk), nq);
        else
            rope_bwd_kernel<T, D, false><<<nq + nk, kThreads, 0, st>>>(p, static_cast<T*>(dq), static_cast<T*>(dk), nq);
        count_launch();
    }
    if (p.partials) {
        rope_dw_kernel<<<dim3(D / 32, 2), dim3(32, 32), 0, st>>>(p.partials, nq, nk, D, dq_w, dk_w);
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

size_t qk_norm_rope_bwd_partials(int T, int Hq, int Hk, int d) {
    int nq, nk;
    bwd_ctas(T, Hq, Hk, d, &nq, &nk);
    return (size_t)(nq + nk) * d;
}

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

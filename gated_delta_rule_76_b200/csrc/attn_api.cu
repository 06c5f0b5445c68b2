// C ABI of the softmax-attention layer (include/gdn.h): argument validation on the host, workspace
// carving and launches.  Nothing here allocates device memory or synchronises.
#include <cmath>

#include "api_util.h"
#include "attn.h"
#include "gdn.h"
#include "launch.h"

using namespace gdn;

namespace {

constexpr int64_t kMaxTokens = int64_t(1) << 30;

// Sizes shared by every call; `kinds`: the dtypes it takes (bf16 only, or fp32 too).
gdn_status check_sizes(int64_t T, int64_t Hq, int64_t Hk, int64_t d, int32_t dtype, bool f32_too, bool need_q = true) {
    if (T < 0 || Hq < (need_q ? 1 : 0) || Hk < 0)
        return fail(GDN_ERR_INVALID_ARG, "bad sizes T=%lld Hq=%lld Hk=%lld", (long long)T, (long long)Hq, (long long)Hk);
    if (d != 64 && d != 128) return fail(GDN_ERR_UNSUPPORTED, "d=%lld: supported are 64 and 128", (long long)d);
    if (dtype != GDN_BF16 && dtype != GDN_F32) return fail(GDN_ERR_INVALID_ARG, "unknown dtype %d", dtype);
    if (dtype == GDN_F32 && !f32_too) return fail(GDN_ERR_UNSUPPORTED, "this call takes bf16 only");
    if (T >= kMaxTokens || Hq > 4096 || Hk > 4096) return fail(GDN_ERR_UNSUPPORTED, "problem too large: T < 2^30, heads <= 4096");
    return GDN_OK;
}
gdn_status check_groups(int64_t Hq, int64_t Hk) {
    if (Hk < 1 || Hq % Hk != 0)
        return fail(GDN_ERR_INVALID_ARG, "Hq=%lld is not a multiple of Hk=%lld", (long long)Hq, (long long)Hk);
    return GDN_OK;
}
gdn_status check_unused(const gdn_strides& s, bool k, bool v) {
    if (s.alpha || s.b || s.w || s.z || (!k && s.k) || (!v && s.v))
        return fail(GDN_ERR_INVALID_ARG, "a stride is given for a tensor this call does not take");
    return GDN_OK;
}
gdn_status check_norm(const gdn_qk_norm& n, int64_t d) {
    if (n.rot_dim < 0 || n.rot_dim > d || n.rot_dim % 16)
        return fail(GDN_ERR_INVALID_ARG, "rot_dim=%lld: a multiple of 16 up to d=%lld is needed", (long long)n.rot_dim,
                    (long long)d);
    if ((n.rot_dim != 0) != (n.inv_freq != nullptr))
        return fail(GDN_ERR_INVALID_ARG, "inv_freq is needed exactly when rot_dim > 0");
    if (n.interleaved != 0 && n.interleaved != 1) return fail(GDN_ERR_INVALID_ARG, "interleaved must be 0 or 1");
    if (!(n.norm_eps >= 0.f)) return fail(GDN_ERR_INVALID_ARG, "norm_eps must be >= 0");
    return GDN_OK;
}
gdn_status check_scale(float scale, int64_t window) {
    if (!(scale > 0.f) || std::isinf(scale)) return fail(GDN_ERR_INVALID_ARG, "scale must be positive and finite");
    if (window < 0) return fail(GDN_ERR_INVALID_ARG, "window must be >= 0");
    return GDN_OK;
}

Rows rows_of(const void* p, int64_t row, int64_t stride, size_t es) {
    const int64_t st = stride ? stride : row;
    return Rows{p, st, ((reinterpret_cast<uintptr_t>(p) | (uintptr_t)(st * (int64_t)es)) & 15u) == 0};
}
RopeParams rope_of(const gdn_qk_norm& n) {
    return RopeParams{n.q_norm_w, n.k_norm_w, n.inv_freq, (int)n.rot_dim, n.interleaved, n.norm_eps, n.rot_scale};
}
Buf freq_buf(const gdn_qk_norm& n) { return {n.inv_freq, (size_t)(n.rot_dim / 2) * 4, "inv_freq"}; }

// Sizes of a paged cache (Hk and d are checked before).
gdn_status check_cache(int64_t num_pages, int64_t page_size, int64_t max_pages, int64_t Hk, int64_t d) {
    if (num_pages < 1 || page_size < 1 || max_pages < 1 || num_pages > INT32_MAX || page_size > INT32_MAX ||
        max_pages > INT32_MAX)
        return fail(GDN_ERR_INVALID_ARG, "num_pages, page_size and max_pages must be in [1, 2^31)");
    if (num_pages > (int64_t(1) << 46) / (page_size * Hk * d))  // byte offsets stay within 64 bits
        return fail(GDN_ERR_UNSUPPORTED, "problem too large: a cache must stay below 2^46 elements");
    return GDN_OK;
}

// Shared by the norm-and-rotation calls; k may be absent with Hk = 0.
template <class A>
gdn_status check_qk(const A* a) {
    if (!a) return fail(GDN_ERR_INVALID_ARG, "args is NULL");
    gdn_status s = check_sizes(a->T, a->Hq, a->Hk, a->d, a->dtype, true);
    if (s || (s = check_norm(a->norm, a->d)) || (s = check_unused(a->strides, true, false)) ||
        (s = check_stride(a->strides.q, a->Hq * a->d, "q")) || (s = check_stride(a->strides.k, a->Hk * a->d, "k")))
        return s;
    if (a->T > 0 && (!a->q || (a->Hk > 0) != (a->k != nullptr)))
        return fail(GDN_ERR_INVALID_ARG, "q is required, and k exactly when Hk > 0");
    if (a->T > 0 && (a->norm.rot_dim > 0) != (a->positions != nullptr))
        return fail(GDN_ERR_INVALID_ARG, "positions are needed exactly when rot_dim > 0");
    if (a->norm.k_norm_w && a->Hk == 0) return fail(GDN_ERR_INVALID_ARG, "k_norm_w is given without k");
    return GDN_OK;
}
template <class A>
QkParams qk_params(const A* a) {
    QkParams p{};
    const size_t es = elem_size(a->dtype);
    p.q = rows_of(a->q, a->Hq * a->d, a->strides.q, es);
    p.k = rows_of(a->k, a->Hk * a->d, a->strides.k, es);
    p.T = (int)a->T;
    p.Hq = (int)a->Hq;
    p.Hk = (int)a->Hk;
    p.rope = rope_of(a->norm);
    return p;
}

// The tensor-core calls read rows whose address and stride are multiples of 16 bytes in place; other
// strided inputs are copied into the workspace.
bool in_place(const void* p, int64_t row, int64_t stride) { return rows_of(p, row, stride, 2).vec != 0; }
template <class A>
int attn_copies(A* a, StridedIn* in) {
    int n = 0;
    if (a->q && !in_place(a->q, a->Hq * a->d, a->strides.q)) in[n++] = {&a->q, a->Hq * a->d, a->strides.q, 2};
    if (a->k && !in_place(a->k, a->Hk * a->d, a->strides.k)) in[n++] = {&a->k, a->Hk * a->d, a->strides.k, 2};
    if (a->v && !in_place(a->v, a->Hk * a->d, a->strides.v)) in[n++] = {&a->v, a->Hk * a->d, a->strides.v, 2};
    return n;
}
template <class A>
size_t attn_copy_bytes(const A* a) {
    A p = *a;
    StridedIn in[3];
    return pack_bytes(in, attn_copies(&p, in), (size_t)a->T);
}
// Copies what has to be dense to `dst` and points *p at it.
template <class A>
cudaError_t attn_copy(A* p, char* dst, cudaStream_t st) {
    StridedIn in[3];
    const int n = attn_copies(p, in);
    const void *q = p->q, *k = p->k, *v = p->v;
    cudaError_t e = pack_inputs(in, n, (size_t)p->T, dst, st);
    if (p->q != q) p->strides.q = 0;
    if (p->k != k) p->strides.k = 0;
    if (p->v != v) p->strides.v = 0;
    return e;
}

size_t lse_bytes(int64_t T, int64_t nseq, int64_t Hq) { return align256((size_t)(attn_tiles(T, nseq) * Hq) * 128 * 4); }
size_t cache_bytes(int64_t T, int64_t nseq, int64_t Hq, int64_t d) {
    return T > 0 && nseq > 0 ? lse_bytes(T, nseq, Hq) + (size_t)(T * Hq * d) * 2 : 0;
}

// The forward's partial sums (none where a unit is one part): the rows' o, then their references and weights.
size_t fwd_part_o_bytes(const gdn_attn_fwd_args* a, int parts) {
    return align256((size_t)parts * (size_t)(a->T * a->Hq * a->d) * sizeof(float));
}
size_t fwd_part_bytes(const gdn_attn_fwd_args* a) {
    const int parts = attn_fwd_parts(a->T, a->nseq, a->Hq, a->d, a->window);
    return parts > 1 ? fwd_part_o_bytes(a, parts) + align256((size_t)parts * (size_t)(a->T * a->Hq) * sizeof(float2)) : 0;
}
// One of the backward's two arrays of partial sums (none where a unit is one part).
size_t part_bytes(const gdn_attn_bwd_args* a) {
    const int parts = attn_bwd_parts(a->T, a->nseq, a->Hq, a->Hk, a->window);
    return parts > 1 ? align256((size_t)parts * (size_t)(a->T * a->Hk * a->d) * sizeof(float)) : 0;
}

template <class A>
gdn_status check_attn(const A* a, Buf* in) {
    if (!a) return fail(GDN_ERR_INVALID_ARG, "args is NULL");
    gdn_status s = check_sizes(a->T, a->Hq, a->Hk, a->d, a->dtype, false);
    if (s || (s = check_groups(a->Hq, a->Hk)) || (s = check_scale(a->scale, a->window)) ||
        (s = check_unused(a->strides, true, true)) || (s = check_stride(a->strides.q, a->Hq * a->d, "q")) ||
        (s = check_stride(a->strides.k, a->Hk * a->d, "k")) || (s = check_stride(a->strides.v, a->Hk * a->d, "v")))
        return s;
    if (a->nseq < 0 || a->nseq >= kMaxTokens) return fail(GDN_ERR_INVALID_ARG, "bad nseq=%lld", (long long)a->nseq);
    if (attn_tiles(a->T, a->nseq) * a->Hq >= (int64_t(1) << 31))
        return fail(GDN_ERR_UNSUPPORTED, "problem too large: tiles of 128 rows times heads must stay below 2^31");
    if (a->T > 0 && (!a->q || !a->k || !a->v || !a->cu_seqlens || !a->o))
        return fail(GDN_ERR_INVALID_ARG, "q, k, v, cu_seqlens and o are required");
    const size_t T = (size_t)a->T;
    in[0] = tok(a->q, T, a->Hq * a->d, a->strides.q, 2, "q");
    in[1] = tok(a->k, T, a->Hk * a->d, a->strides.k, 2, "k");
    in[2] = tok(a->v, T, a->Hk * a->d, a->strides.v, 2, "v");
    in[3] = {a->cu_seqlens, (size_t)(a->nseq + 1) * 4, "cu_seqlens", 4};
    return GDN_OK;
}
template <class A>
AttnIO attn_io(const A* a, void* ws) {
    AttnIO io{};
    io.q = rows_of(a->q, a->Hq * a->d, a->strides.q, 2);
    io.k = rows_of(a->k, a->Hk * a->d, a->strides.k, 2);
    io.v = rows_of(a->v, a->Hk * a->d, a->strides.v, 2);
    io.cu = a->cu_seqlens;
    io.T = (int)a->T;
    io.nseq = (int)a->nseq;
    io.Hq = (int)a->Hq;
    io.Hk = (int)a->Hk;
    io.window = a->window;
    io.scale = a->scale;
    io.err = ws_status(ws);
    io.counters = ws_status(ws) + 2;
    return io;
}
void cache_into(AttnIO* io, const void* cache) {
    char* c = static_cast<char*>(const_cast<void*>(cache));
    io->lse = reinterpret_cast<float*>(c);
    io->o_lo = c + lse_bytes(io->T, io->nseq, io->Hq);
}

}  // namespace

extern "C" {

gdn_status gdn_qk_norm_rope_fwd(const gdn_qk_fwd_args* a, gdn_stream stream) {
    gdn_status s = check_qk(a);
    if (s) return s;
    if (a->T > 0 && (!a->q_out || (a->Hk > 0) != (a->k_out != nullptr)))
        return fail(GDN_ERR_INVALID_ARG, "q_out is required, and k_out exactly with k");
    const size_t es = elem_size(a->dtype), T = (size_t)a->T, d = (size_t)a->d;
    const Buf in[] = {
        tok(a->q, T, a->Hq * a->d, a->strides.q, es, "q"), tok(a->k, T, a->Hk * a->d, a->strides.k, es, "k"),
        {a->positions, T * 4, "positions", 4}, {a->norm.q_norm_w, d * es, "q_norm_w"},
        {a->norm.k_norm_w, d * es, "k_norm_w"}, freq_buf(a->norm),
    };
    const Buf out[] = {{a->q_out, T * a->Hq * d * es, "q_out"}, {a->k_out, T * a->Hk * d * es, "k_out"}};
    if ((s = check_buffers(in, 6, out, 2))) return s;
    QkParams p = qk_params(a);
    p.positions = a->positions;
    p.q_out = a->q_out;
    p.k_out = a->k_out;
    cudaError_t e = qk_norm_rope_fwd(p, (int)a->d, a->dtype == GDN_BF16, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? GDN_OK : cuda_fail(e, "gdn_qk_norm_rope_fwd");
}

size_t gdn_qk_norm_rope_bwd_workspace_size(const gdn_qk_bwd_args* a) {
    if (!a || a->T < 0 || a->T >= kMaxTokens || a->Hq < 1 || a->Hk < 0 || a->d < 1 || a->d > 128) return 0;
    if (!a->norm.q_norm_w && !a->norm.k_norm_w) return 0;
    return 256 + align256(qk_norm_rope_bwd_partials((int)a->T, (int)a->Hq, (int)a->Hk, (int)a->d) * sizeof(float));
}

gdn_status gdn_qk_norm_rope_bwd(const gdn_qk_bwd_args* a, void* workspace, size_t workspace_bytes, gdn_stream stream) {
    gdn_status s = check_qk(a);
    if (s) return s;
    if (a->T > 0 && (!a->grad_q_out || !a->grad_q))
        return fail(GDN_ERR_INVALID_ARG, "grad_q_out and grad_q are required");
    if (a->T > 0 && ((a->Hk > 0) != (a->grad_k_out != nullptr) || (a->Hk > 0) != (a->grad_k != nullptr)))
        return fail(GDN_ERR_INVALID_ARG, "grad_k_out and grad_k are needed exactly with k");
    if ((a->norm.q_norm_w != nullptr) != (a->grad_q_norm_w != nullptr) ||
        (a->norm.k_norm_w != nullptr) != (a->grad_k_norm_w != nullptr))
        return fail(GDN_ERR_INVALID_ARG, "grad_q_norm_w and grad_k_norm_w are needed exactly with their norms");
    const size_t es = elem_size(a->dtype), T = (size_t)a->T, d = (size_t)a->d;
    const size_t nq = T * a->Hq * d * es, nk = T * a->Hk * d * es;
    const Buf in[] = {
        tok(a->q, T, a->Hq * a->d, a->strides.q, es, "q"), tok(a->k, T, a->Hk * a->d, a->strides.k, es, "k"),
        {a->positions, T * 4, "positions", 4}, {a->norm.q_norm_w, d * es, "q_norm_w"},
        {a->norm.k_norm_w, d * es, "k_norm_w"}, freq_buf(a->norm), {a->grad_q_out, nq, "grad_q_out"},
        {a->grad_k_out, nk, "grad_k_out"},
    };
    const size_t need = gdn_qk_norm_rope_bwd_workspace_size(a);
    const Buf out[] = {{a->grad_q, nq, "grad_q"}, {a->grad_k, nk, "grad_k"}, {a->grad_q_norm_w, d * 4, "grad_q_norm_w"},
                       {a->grad_k_norm_w, d * 4, "grad_k_norm_w"}};
    if ((s = check_buffers(in, 8, out, 4)) || (s = check_workspace(workspace, workspace_bytes, need))) return s;
    QkParams p = qk_params(a);
    p.positions = a->positions;
    p.gq = a->grad_q_out;
    p.gk = a->grad_k_out;
    p.partials = need ? reinterpret_cast<float*>(static_cast<char*>(workspace) + 256) : nullptr;
    cudaError_t e = qk_norm_rope_bwd(p, (int)a->d, a->dtype == GDN_BF16, a->grad_q, a->grad_k, a->grad_q_norm_w,
                                     a->grad_k_norm_w, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? GDN_OK : cuda_fail(e, "gdn_qk_norm_rope_bwd");
}

size_t gdn_attn_fwd_cache_size(const gdn_attn_fwd_args* a) {
    if (!a || a->T < 0 || a->T >= kMaxTokens || a->nseq < 0 || a->Hq < 1 || a->d < 1) return 0;
    return cache_bytes(a->T, a->nseq, a->Hq, a->d);
}

size_t gdn_attn_fwd_workspace_size(const gdn_attn_fwd_args* a) {
    if (!a || a->T < 1 || a->T >= kMaxTokens || a->Hq < 1 || a->Hk < 1 || a->d < 1) return 0;
    return with_copies(256 + fwd_part_bytes(a), attn_copy_bytes(a));
}

gdn_status gdn_attn_fwd(const gdn_attn_fwd_args* a, void* workspace, size_t workspace_bytes, gdn_stream stream) {
    Buf in[4];
    gdn_status s = check_attn(a, in);
    if (s) return s;
    const Buf out[] = {{a->o, (size_t)(a->T * a->Hq * a->d) * 2, "o"},
                       {a->bwd_cache, a->bwd_cache ? a->bwd_cache_bytes : 0, "bwd_cache"}};
    if (a->bwd_cache && (reinterpret_cast<uintptr_t>(a->bwd_cache) & 255u))
        return fail(GDN_ERR_INVALID_ARG, "bwd_cache is not 256-byte aligned");
    if ((s = check_buffers(in, 4, out, 2))) return s;
    if (a->bwd_cache && a->bwd_cache_bytes < gdn_attn_fwd_cache_size(a))
        return fail(GDN_ERR_WORKSPACE, "bwd_cache has %zu bytes, %zu needed", a->bwd_cache_bytes,
                    gdn_attn_fwd_cache_size(a));
    if (a->T == 0 || a->nseq == 0) return GDN_OK;
    if ((s = check_workspace(workspace, workspace_bytes, gdn_attn_fwd_workspace_size(a)))) return s;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    gdn_attn_fwd_args pa = *a;
    char* ws = static_cast<char*>(workspace);
    cudaError_t e = attn_copy(&pa, ws + 256 + fwd_part_bytes(a), st);
    if (e == cudaSuccess) {
        AttnIO io = attn_io(&pa, workspace);
        io.o = a->o;
        io.part_o = reinterpret_cast<float*>(ws + 256);
        io.part_ml = reinterpret_cast<float2*>(ws + 256 + fwd_part_o_bytes(a, attn_fwd_parts(a->T, a->nseq, a->Hq, a->d, a->window)));
        if (a->bwd_cache) cache_into(&io, a->bwd_cache);
        e = attn_fwd(io, (int)a->d, st);
    }
    return e == cudaSuccess ? GDN_OK : cuda_fail(e, "gdn_attn_fwd");
}

size_t gdn_attn_bwd_workspace_size(const gdn_attn_bwd_args* a) {
    if (!a || a->T < 1 || a->T >= kMaxTokens || a->nseq < 0 || a->Hq < 1 || a->Hk < 1 || a->d < 1) return 0;
    if (a->nseq == 0 || a->Hq < a->Hk) return 0;
    return with_copies(256 + lse_bytes(a->T, a->nseq, a->Hq) + 2 * part_bytes(a), attn_copy_bytes(a));
}

gdn_status gdn_attn_bwd(const gdn_attn_bwd_args* a, void* workspace, size_t workspace_bytes, gdn_stream stream) {
    Buf in[7];
    gdn_status s = check_attn(a, in);
    if (s) return s;
    if (a->T > 0 && (!a->grad_o || !a->grad_q || !a->grad_k || !a->grad_v || !a->fwd_cache))
        return fail(GDN_ERR_INVALID_ARG, "grad_o, fwd_cache, grad_q, grad_k and grad_v are required");
    const size_t nq = (size_t)(a->T * a->Hq * a->d) * 2, nk = (size_t)(a->T * a->Hk * a->d) * 2;
    in[4] = {a->o, nq, "o"};
    in[5] = {a->grad_o, nq, "grad_o"};
    in[6] = {a->fwd_cache, a->fwd_cache ? a->fwd_cache_bytes : 0, "fwd_cache", 256};
    const Buf out[] = {{a->grad_q, nq, "grad_q"}, {a->grad_k, nk, "grad_k"}, {a->grad_v, nk, "grad_v"}};
    if ((s = check_buffers(in, 7, out, 3))) return s;
    const size_t cache = cache_bytes(a->T, a->nseq, a->Hq, a->d);
    if (a->fwd_cache_bytes < cache)
        return fail(GDN_ERR_INVALID_ARG, "fwd_cache has %zu bytes, %zu needed", a->fwd_cache_bytes, cache);
    if (a->T == 0 || a->nseq == 0) return GDN_OK;
    if ((s = check_workspace(workspace, workspace_bytes, gdn_attn_bwd_workspace_size(a)))) return s;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    gdn_attn_bwd_args pa = *a;
    char* ws = static_cast<char*>(workspace);
    const size_t delta = lse_bytes(a->T, a->nseq, a->Hq);
    const size_t parts = part_bytes(a);
    cudaError_t e = attn_copy(&pa, ws + 256 + delta + 2 * parts, st);
    if (e == cudaSuccess) {
        AttnIO io = attn_io(&pa, workspace);
        cache_into(&io, a->fwd_cache);
        io.o = const_cast<void*>(a->o);
        io.grad_o = a->grad_o;
        io.dq = a->grad_q;
        io.dk = a->grad_k;
        io.dv = a->grad_v;
        io.delta = reinterpret_cast<float*>(ws + 256);
        io.part_dk = reinterpret_cast<float*>(ws + 256 + delta);
        io.part_dv = reinterpret_cast<float*>(ws + 256 + delta + parts);
        e = attn_bwd(io, (int)a->d, st);
    }
    return e == cudaSuccess ? GDN_OK : cuda_fail(e, "gdn_attn_bwd");
}

gdn_status gdn_kv_append(const gdn_kv_append_args* a, gdn_stream stream) {
    if (!a) return fail(GDN_ERR_INVALID_ARG, "args is NULL");
    gdn_status s = check_sizes(a->T, a->Hq, a->Hk, a->d, a->dtype, false, false);
    if (s || (s = check_norm(a->norm, a->d)) || (s = check_unused(a->strides, true, true)) ||
        (s = check_stride(a->strides.q, a->Hq * a->d, "q")) || (s = check_stride(a->strides.k, a->Hk * a->d, "k")) ||
        (s = check_stride(a->strides.v, a->Hk * a->d, "v")))
        return s;
    if (a->Hk < 1) return fail(GDN_ERR_INVALID_ARG, "Hk must be at least 1");
    if (a->nseq < 0 || a->nseq >= kMaxTokens || (!a->cu_seqlens && a->nseq != a->T))
        return fail(GDN_ERR_INVALID_ARG, "nseq=%lld: without cu_seqlens it must be T=%lld", (long long)a->nseq, (long long)a->T);
    if ((s = check_cache(a->num_pages, a->page_size, a->max_pages, a->Hk, a->d))) return s;
    if (a->T > 0 && (!a->k || !a->v || !a->context_lens || !a->block_table || !a->k_cache || !a->v_cache))
        return fail(GDN_ERR_INVALID_ARG, "k, v, context_lens, block_table, k_cache and v_cache are required");
    if (a->T > 0 && ((a->Hq > 0) != (a->q != nullptr) || (a->Hq > 0) != (a->q_out != nullptr)))
        return fail(GDN_ERR_INVALID_ARG, "q and q_out are needed exactly when Hq > 0");
    if (a->norm.q_norm_w && a->Hq == 0) return fail(GDN_ERR_INVALID_ARG, "q_norm_w is given without q");
    const size_t T = (size_t)a->T, d = (size_t)a->d;
    const size_t cache = (size_t)(a->num_pages * a->page_size) * (size_t)(a->Hk * a->d) * 2;
    const Buf in[] = {
        tok(a->q, T, a->Hq * a->d, a->strides.q, 2, "q"), tok(a->k, T, a->Hk * a->d, a->strides.k, 2, "k"),
        tok(a->v, T, a->Hk * a->d, a->strides.v, 2, "v"), {a->cu_seqlens, (size_t)(a->nseq + 1) * 4, "cu_seqlens", 4},
        {a->context_lens, (size_t)a->nseq * 4, "context_lens", 4},
        {a->block_table, (size_t)(a->nseq * a->max_pages) * 4, "block_table", 4},
        {a->norm.q_norm_w, d * 2, "q_norm_w"}, {a->norm.k_norm_w, d * 2, "k_norm_w"}, freq_buf(a->norm),
    };
    const Buf out[] = {{a->q_out, T * a->Hq * d * 2, "q_out"}, {a->k_out, T * a->Hk * d * 2, "k_out"},
                       {a->k_cache, cache, "k_cache"}, {a->v_cache, cache, "v_cache"}};
    if ((s = check_buffers(in, 9, out, 4))) return s;
    QkParams p = qk_params(a);
    p.v = rows_of(a->v, a->Hk * a->d, a->strides.v, 2);
    p.q_out = a->q_out;
    p.k_out = a->k_out;
    p.app = AppendParams{a->cu_seqlens, a->context_lens, a->block_table, a->k_cache, a->v_cache,
                         a->num_pages, a->page_size, a->max_pages, (int)a->nseq};
    cudaError_t e = kv_append(p, (int)a->d, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? GDN_OK : cuda_fail(e, "gdn_kv_append");
}

// Tokens a sequence can have, and read: the block table's reach and max_context, and of those the window's.
static int64_t decode_max_context(const gdn_attn_decode_args* a) {
    const int64_t limit = (int64_t(1) << 31) - 4096;  // context_lens are 32-bit
    int64_t m = a->max_pages > limit / a->page_size ? limit : a->max_pages * a->page_size;
    if (a->max_context > 0 && a->max_context < m) m = a->max_context;
    return m;
}
static void decode_plan(const gdn_attn_decode_args* a, int* chunk, int* splits) {
    int64_t reach = decode_max_context(a);
    if (a->window > 0 && a->window < reach) reach = a->window;
    plan_decode_attn(a->N, a->Hq, a->Hk, reach, chunk, splits);
}
static gdn_status check_decode_sizes(const gdn_attn_decode_args* a) {
    if (!a) return fail(GDN_ERR_INVALID_ARG, "args is NULL");
    gdn_status s = check_sizes(a->N, a->Hq, a->Hk, a->d, a->dtype, false);
    if (s || (s = check_groups(a->Hq, a->Hk)) || (s = check_scale(a->scale, a->window)) ||
        (s = check_unused(a->strides, false, false)) || (s = check_stride(a->strides.q, a->Hq * a->d, "q")))
        return s;
    if ((s = check_cache(a->num_pages, a->page_size, a->max_pages, a->Hk, a->d))) return s;
    if (a->max_context < 0) return fail(GDN_ERR_INVALID_ARG, "max_context must be >= 0");
    if (a->N * a->Hq >= (int64_t(1) << 22))
        return fail(GDN_ERR_UNSUPPORTED, "problem too large: sequences times heads must stay below 2^22");
    return GDN_OK;
}

size_t gdn_attn_decode_workspace_size(const gdn_attn_decode_args* a) {
    if (check_decode_sizes(a) || a->N == 0) return 0;
    int chunk, splits;
    decode_plan(a, &chunk, &splits);
    return align256(decode_attn_part_floats(a->N, a->Hq, a->d, splits) * sizeof(float));
}

gdn_status gdn_attn_decode(const gdn_attn_decode_args* a, void* workspace, size_t workspace_bytes, gdn_stream stream) {
    gdn_status s = check_decode_sizes(a);
    if (s) return s;
    if (a->N == 0) return GDN_OK;
    if (!a->q || !a->k_cache || !a->v_cache || !a->block_table || !a->context_lens || !a->o)
        return fail(GDN_ERR_INVALID_ARG, "q, k_cache, v_cache, block_table, context_lens and o are required");
    const size_t N = (size_t)a->N;
    const size_t cache = (size_t)(a->num_pages * a->page_size) * (size_t)(a->Hk * a->d) * 2;
    const Buf in[] = {tok(a->q, N, a->Hq * a->d, a->strides.q, 2, "q"), {a->k_cache, cache, "k_cache"},
                      {a->v_cache, cache, "v_cache"}, {a->block_table, N * (size_t)a->max_pages * 4, "block_table", 4},
                      {a->context_lens, N * 4, "context_lens", 4}};
    const Buf out[] = {{a->o, N * (size_t)(a->Hq * a->d) * 2, "o"}};
    DecodeAttnParams p{};
    decode_plan(a, &p.chunk, &p.splits);
    const size_t need = align256(decode_attn_part_floats(a->N, a->Hq, a->d, p.splits) * sizeof(float));
    if ((s = check_buffers(in, 5, out, 1)) || (s = check_workspace(workspace, workspace_bytes, need))) return s;
    if (a->N * a->Hk * ((a->Hq / a->Hk + 15) / 16) * p.splits >= (int64_t(1) << 31))
        return fail(GDN_ERR_UNSUPPORTED, "problem too large: give max_context");
    const Rows q = rows_of(a->q, a->Hq * a->d, a->strides.q, 2);
    p.q = a->q;
    p.q_stride = q.stride;
    p.q_vec = ((reinterpret_cast<uintptr_t>(a->q) & 3u) == 0 && q.stride % 2 == 0) ? 1 : 0;
    p.k_cache = a->k_cache;
    p.v_cache = a->v_cache;
    p.table = a->block_table;
    p.context = a->context_lens;
    p.o = a->o;
    p.part = static_cast<float*>(workspace);
    p.num_pages = a->num_pages;
    p.max_pages = a->max_pages;
    p.max_context = decode_max_context(a);
    p.window = a->window;
    p.page_size = a->page_size;
    p.N = (int)a->N;
    p.Hq = (int)a->Hq;
    p.Hk = (int)a->Hk;
    p.scale = a->scale;
    cudaError_t e = decode_attn(p, (int)a->d, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? GDN_OK : cuda_fail(e, "gdn_attn_decode");
}

}  // extern "C"

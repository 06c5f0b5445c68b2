// Launchers of the softmax-attention layer's kernels (entry points in attn_api.cu).
#pragma once
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace gdn {

// Norm and rotation of head rows (qk_rope.cu).  A row source or destination of tokens `stride`
// elements apart; vec: every row starts on a 16-byte boundary.
struct Rows {
    const void* p;
    int64_t stride;
    int vec;
};

struct RopeParams {
    const void *q_w, *k_w;   // [d] norm weights or NULL
    const float* inv_freq;   // [rot / 2]
    int rot, interleaved;
    float eps, rot_scale;
};

// What kv_append adds to the forward: the rows of k and v go to the cache.
struct AppendParams {
    const int32_t *cu, *context, *table;  // cu may be NULL: token t is sequence t's
    void *k_cache, *v_cache;
    int64_t num_pages, page_size, max_pages;
    int nseq;
};

struct QkParams {
    Rows q, k, v;              // v: append only
    const int32_t* positions;  // forward and backward
    void *q_out, *k_out;       // dense; NULL: not wanted
    const void *gq, *gk;       // backward: gradients of q_out, k_out (dense)
    int T, Hq, Hk;
    RopeParams rope;
    AppendParams app;
    float* partials;           // backward: [CTAs][d]
};

cudaError_t qk_norm_rope_fwd(const QkParams& p, int d, bool bf16, cudaStream_t st);
size_t qk_norm_rope_bwd_partials(int T, int Hq, int Hk, int d);  // floats
// dq_w, dk_w [d] (NULL without the norm)
cudaError_t qk_norm_rope_bwd(const QkParams& p, int d, bool bf16, void* dq, void* dk, float* dq_w, float* dk_w,
                             cudaStream_t st);
cudaError_t kv_append(const QkParams& p, int d, cudaStream_t st);

// Single-token attention over the paged cache (attn_decode.cu).
struct DecodeAttnParams {
    const void* q;
    int64_t q_stride;
    int q_vec;
    const void *k_cache, *v_cache;
    const int32_t *table, *context;
    void* o;
    float* part;               // split contexts: [split][N * Hq][d], then [split][N * Hq][2]
    int64_t num_pages, max_pages, max_context, window;
    int64_t page_size;
    uint32_t page_mul;         // pos / page_size = (pos * page_mul) >> page_shift
    int page_shift;
    int N, Hq, Hk;
    int chunk, splits;         // tokens a split, splits a sequence
    float scale;
};
void plan_decode_attn(int64_t N, int64_t Hq, int64_t Hk, int64_t reach, int* chunk, int* splits);
size_t decode_attn_part_floats(int64_t N, int64_t Hq, int64_t d, int splits);
cudaError_t decode_attn(const DecodeAttnParams& p, int d, cudaStream_t st);

// Causal attention over packed sequences on the tensor cores (attn_fwd.cu, attn_bwd.cu).
struct AttnIO {
    Rows q, k, v;              // bf16, 16-byte aligned rows (vec)
    const int32_t* cu;
    int T, nseq, Hq, Hk;
    int64_t window;            // 0: none
    float scale;
    void* o;                   // forward: out; backward: the forward's output
    // the forward's cache: rows' -log2 sum exp2 of the scaled scores, tile-aligned [Hq][tiles][128], and
    // o - bf16(o) [T,Hq,d] (NULL in a forward that keeps none)
    float* lse;
    void* o_lo;
    // backward
    const void* grad_o;
    void *dq, *dk, *dv;
    float* delta;              // [Hq][tiles][128]: rows' -sum of grad_o .* o
    // forward, where units are cut into parts: their sums, and each row's reference and sum of weights
    float* part_o;             // [parts][T][Hq][d]
    float2* part_ml;           // [parts][T][Hq]
    float *part_dk, *part_dv;  // [parts][T][Hk][d], where the key tiles' units are cut into parts
    int* err;                  // device error word
    int* counters;             // [2] the units drawn so far (forward and dkdv; dq)
};
// Tiles of 128 rows over all sequences, at most.
inline int64_t attn_tiles(int64_t T, int64_t nseq) { return T / 128 + (nseq < T ? nseq : T); }
// Parts that dkdv cuts a key tile's unit into.  The heaviest unit, the first key tile of a sequence with all the
// group's queries, takes as long as the SMs' average of dkdv's and dq's work together at 160 units (one sequence or
// several equal ones), or at 80 where a window makes the units alike (one shorter than half of the call's tokens is taken
// to: the sequences' lengths are not known here); with fewer it would be what the call waits for
// (backward of 4096 tokens, 16 heads on 2: 515 us whole, 247 us in 3 parts; one sequence of 2600, 8 heads on 1: 344 and
// 86 us).  A part costs its sums' way through memory (4 x 2048 tokens, 16 heads on 4, 272 units: 266 us whole, 314 us in 2
// parts), and is worth it from two items on.  Where the two meet depends on the group: long sequences of 4 and more heads
// on one gain up to the 192 units of the limit, small groups lose from 130 on.  Two parts and whole, us: 161 units of 20480
// tokens, 8 heads on 1 2724 and 3021, 1 on 1 470 and 345; 168 units of 2600 tokens, 32 heads on 8 248 and 244, 8 on 8 104
// and 68.  The limit takes the long calls' side.
inline int attn_bwd_parts(int64_t T, int64_t nseq, int64_t Hq, int64_t Hk, int64_t window) {
    const int64_t units = attn_tiles(T, nseq) * Hk, items = Hq / Hk * ((T + 127) / 128);
    const int64_t want = window > 0 && window < T / 2 ? 80 : 192;
    int64_t parts = (want + units - 1) / units;
    if (parts > 16) parts = 16;
    if (parts > items / 2) parts = items / 2;
    return parts < 1 ? 1 : (int)parts;
}
// Parts that the forward cuts a unit's key tiles into, as the least estimate (us).  Where there are few units, the longest
// row's key tiles, one after the other, are what the call waits for: 2 us a tile, 1.6 with heads of 64.  A part has its own
// start and end, 5 us, and its sums' way through memory and the joining kernel.  The sequences' lengths are not known
// here: the longest is taken as twice what is left for one more (8192 tokens, 4 heads on 1: 124 us whole, 84 us in 2 parts;
// 1783 and 7 tokens, 3 heads: 32 and 25 us; 1777, 16 heads, left whole: 33 us, 47 in 3 parts).  Many short sequences beside
// a long one make it look shorter than it is: the 8192 tokens with 15 sequences of one token are left whole (127 us).
inline int attn_fwd_parts(int64_t T, int64_t nseq, int64_t Hq, int64_t d, int64_t window) {
    if (T < 1 || nseq < 1) return 1;
    const double units = (double)((attn_tiles(T, nseq) * Hq + 1) / 2), sums = (double)(T * Hq * d) * 4.0;
    int64_t tiles = (2 * T / (nseq + 1) + 127) / 128;
    if (window > 0 && window / 128 + 2 < tiles) tiles = window / 128 + 2;
    const double chain = (d == 128 ? 2.0 : 1.6) * (double)tiles;
    double least = 0.0;
    int parts = 1;
    for (int p = 1; p <= 8 && (p == 1 || p * 3 <= tiles); ++p) {
        const double longest = chain / p + 5.0, even = units * (chain / 2.0 + 5.0 * p) / 148.0;
        const double t = (longest > even ? longest : even) + (p > 1 ? 4.0 + p * sums / 2.5e6 : 0.0);
        if (p == 1 || t < 0.95 * least) {
            least = t;
            parts = p;
        }
    }
    return parts;
}
cudaError_t attn_fwd(const AttnIO& io, int d, cudaStream_t st);
cudaError_t attn_bwd(const AttnIO& io, int d, cudaStream_t st);

}  // namespace gdn

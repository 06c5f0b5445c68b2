// Host-side helpers shared by the entry points of the C ABI (gdn_api.cu, attn_api.cu): the
// thread-local error message, checks of buffers, strides and workspaces, and the dense copies of
// strided inputs.
#pragma once
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "gdn.h"
#include "launch.h"

namespace gdn {

// Records the calling thread's error message and returns `code` (gdn_api.cu).
gdn_status fail(gdn_status code, const char* fmt, ...);
gdn_status cuda_fail(cudaError_t e, const char* where);

inline size_t elem_size(int dtype) { return dtype == GDN_F32 ? 4 : 2; }

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

struct Buf {
    const void* p;
    size_t bytes;
    const char* name;
    size_t align = 16;  // required alignment of p (a strided input: its element size)
};

inline bool overlaps(const Buf& a, const Buf& b) {
    if (!a.p || !b.p || !a.bytes || !b.bytes) return false;
    const uintptr_t a0 = reinterpret_cast<uintptr_t>(a.p), b0 = reinterpret_cast<uintptr_t>(b.p);
    return a0 < b0 + b.bytes && b0 < a0 + a.bytes;
}

// Every output against every input and every other output.
inline gdn_status check_buffers(const Buf* in, int nin, const Buf* out, int nout) {
    for (int i = 0; i < nin; ++i)
        if (in[i].p && (reinterpret_cast<uintptr_t>(in[i].p) & (in[i].align - 1)))
            return fail(GDN_ERR_INVALID_ARG, "%s is not %zu-byte aligned", in[i].name, in[i].align);
    for (int i = 0; i < nout; ++i) {
        if (out[i].p && !aligned16(out[i].p))
            return fail(GDN_ERR_INVALID_ARG, "%s is not 16-byte aligned", out[i].name);
        for (int j = 0; j < nin; ++j)
            if (overlaps(out[i], in[j]))
                return fail(GDN_ERR_INVALID_ARG, "output %s overlaps input %s", out[i].name, in[j].name);
        for (int j = 0; j < i; ++j)
            if (overlaps(out[i], out[j]))
                return fail(GDN_ERR_INVALID_ARG, "outputs %s and %s overlap", out[i].name, out[j].name);
    }
    return GDN_OK;
}

inline size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

// ---- token strides (gdn_strides) ---------------------------------------------------------
// A token-major input of `rows` tokens of `row` elements whose tokens are `stride` elements apart
// (0: dense).  One that is not dense is copied into the workspace before the call's kernels run.
inline bool strided(int64_t stride, int64_t row) { return stride != 0 && stride != row; }

// The input as a buffer: from its first to its last element; a strided one needs only the
// alignment of its element type.
inline Buf tok(const void* p, size_t rows, int64_t row, int64_t stride, size_t es, const char* name) {
    const size_t step = (size_t)(stride ? stride : row);
    return Buf{p, p && rows ? ((rows - 1) * step + (size_t)row) * es : 0, name, strided(stride, row) ? es : 16};
}

inline gdn_status check_stride(int64_t stride, int64_t row, const char* name) {
    if (stride != 0 && (stride < row || stride > (int64_t(1) << 31)))
        return fail(GDN_ERR_INVALID_ARG, "token stride of %s is %lld: it must be 0 or in [%lld, 2^31]", name,
                    (long long)stride, (long long)row);
    return GDN_OK;
}

// One input of a call, for the copies: where the call reads its pointer, its row and stride.
struct StridedIn {
    const void** slot;
    int64_t row, stride;
    size_t es;
};

// Bytes of the dense copies of the strided inputs (each 256-byte aligned).
inline size_t pack_bytes(const StridedIn* in, int n, size_t rows) {
    size_t bytes = 0;
    for (int i = 0; i < n; ++i)
        if (*in[i].slot && strided(in[i].stride, in[i].row)) bytes += align256(rows * (size_t)in[i].row * in[i].es);
    return bytes;
}

// Copies every strided input into `dst` (the workspace past the call's own part) and points its
// slot at the copy.
inline cudaError_t pack_inputs(const StridedIn* in, int n, size_t rows, char* dst, cudaStream_t st) {
    for (int i = 0; i < n; ++i) {
        if (!*in[i].slot || !strided(in[i].stride, in[i].row)) continue;
        const long row_bytes = (long)(in[i].row * (int64_t)in[i].es);
        cudaError_t e = pack_rows(*in[i].slot, dst, (long)rows, row_bytes, (long)(in[i].stride * (int64_t)in[i].es), st);
        if (e != cudaSuccess) return e;
        *in[i].slot = dst;
        dst += align256(rows * (size_t)row_bytes);
    }
    return cudaSuccess;
}

// Workspace of a call's own part plus the copies of its strided inputs after it.
inline size_t with_copies(size_t own, size_t copies) { return copies ? align256(own) + copies : own; }


inline gdn_status check_workspace(void* ws, size_t have, size_t need) {
    if (need == 0) return GDN_OK;
    if (!ws) return fail(GDN_ERR_WORKSPACE, "workspace is NULL, %zu bytes needed", need);
    if (have < need) return fail(GDN_ERR_WORKSPACE, "workspace has %zu bytes, %zu needed", have, need);
    if (reinterpret_cast<uintptr_t>(ws) & 255u) return fail(GDN_ERR_WORKSPACE, "workspace is not 256-byte aligned");
    return GDN_OK;
}

// Status word at the start of every workspace, cleared at the start of each call.
inline int* ws_status(void* ws) { return static_cast<int*>(ws); }

}  // namespace gdn

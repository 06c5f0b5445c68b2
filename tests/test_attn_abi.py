"""The attention layer's C calls on the host: struct layouts, refusals before any launch, sizes of caches and
workspaces.  Fake device addresses; no call here reaches a kernel."""
import ctypes
import os
import subprocess

import pytest
import torch

from gated_delta_rule_76_b200 import build as gbuild
from gated_delta_rule_76_b200 import gdn

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 4
MB = 1 << 20
WS = ctypes.c_void_p(1 << 40)
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def lib():
    gbuild.build()
    return gdn.load()


STRUCTS = {"gdn_qk_norm": gdn.QkNorm, "gdn_qk_fwd_args": gdn.QkFwdArgs, "gdn_qk_bwd_args": gdn.QkBwdArgs,
           "gdn_attn_fwd_args": gdn.AttnFwdArgs, "gdn_attn_bwd_args": gdn.AttnBwdArgs,
           "gdn_kv_append_args": gdn.KvAppendArgs, "gdn_attn_decode_args": gdn.AttnDecodeArgs}


def test_ctypes_structs_match_c_layout(tmp_path):
    """A host program prints sizeof and every offsetof."""
    lines = ["#include <stdio.h>", "#include <stddef.h>", '#include "gdn.h"', "int main(void) {"]
    for cname, py in STRUCTS.items():
        lines.append(f'printf("{cname} size %zu\\n", sizeof({cname}));')
        lines += [f'printf("{cname} {f} %zu\\n", offsetof({cname}, {f}));' for f, _ in py._fields_]
    src, exe = tmp_path / "layout.c", tmp_path / "layout"
    src.write_text("\n".join(lines + ["return 0; }"]))
    subprocess.check_call(["gcc", "-std=c99", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)])
    out = subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout
    got = {tuple(line.split()[:2]): int(line.split()[2]) for line in out.splitlines()}
    for cname, py in STRUCTS.items():
        assert got[cname, "size"] == ctypes.sizeof(py), cname
        for f, _ in py._fields_:
            assert got[cname, f] == getattr(py, f).offset, (cname, f)


def norm(**kw):
    return gdn.QkNorm(**{**dict(q_norm_w=MB, k_norm_w=2 * MB, inv_freq=3 * MB, rot_dim=64, interleaved=0, norm_eps=1e-6,
                                rot_scale=1.0), **kw})


def build_args(cls, base, kw):
    n = {k: kw.pop(k) for k in list(kw) if k in ("q_norm_w", "k_norm_w", "inv_freq", "rot_dim", "interleaved", "norm_eps")}
    st = {k[3:]: kw.pop(k) for k in list(kw) if k.startswith("st_")}
    a = cls(**{**base, **kw})
    if hasattr(a, "norm"):
        a.norm = norm(**n)
    for k, v in st.items():
        setattr(a.strides, k, v)
    return a


def qk_fwd(**kw):
    return build_args(gdn.QkFwdArgs, dict(q=10 * MB, k=11 * MB, positions=12 * MB, q_out=13 * MB, k_out=14 * MB, T=8, Hq=4, Hk=2,
                                   d=128, dtype=0), kw)


def qk_bwd(**kw):
    return build_args(gdn.QkBwdArgs, dict(q=10 * MB, k=11 * MB, positions=12 * MB, grad_q_out=13 * MB, grad_k_out=14 * MB,
                                   grad_q=15 * MB, grad_k=16 * MB, grad_q_norm_w=17 * MB, grad_k_norm_w=18 * MB, T=8,
                                   Hq=4, Hk=2, d=128, dtype=0), kw)


def attn_fwd(**kw):
    return build_args(gdn.AttnFwdArgs, dict(q=10 * MB, k=11 * MB, v=12 * MB, cu_seqlens=13 * MB, o=14 * MB, T=8, nseq=2, Hq=4, Hk=2,
                                     d=128, window=0, scale=0.1, dtype=0), kw)


def attn_bwd(**kw):
    return build_args(gdn.AttnBwdArgs, dict(q=10 * MB, k=11 * MB, v=12 * MB, cu_seqlens=13 * MB, o=14 * MB, grad_o=15 * MB,
                                     grad_q=16 * MB, grad_k=17 * MB, grad_v=18 * MB, T=8, nseq=2, Hq=4, Hk=2, d=128,
                                     window=0, scale=0.1, dtype=0, fwd_cache=19 * MB, fwd_cache_bytes=MB), kw)


def append(**kw):
    return build_args(gdn.KvAppendArgs, dict(q=10 * MB, k=11 * MB, v=12 * MB, cu_seqlens=13 * MB, context_lens=14 * MB,
                                      block_table=15 * MB, q_out=16 * MB, k_out=17 * MB, k_cache=20 * MB,
                                      v_cache=30 * MB, T=8, nseq=2, Hq=4, Hk=2, d=128, num_pages=16, page_size=16,
                                      max_pages=8, dtype=0), kw)


def decode(**kw):
    return build_args(gdn.AttnDecodeArgs, dict(q=10 * MB, k_cache=20 * MB, v_cache=30 * MB, block_table=11 * MB, context_lens=12 * MB,
                                        o=13 * MB, N=2, Hq=4, Hk=2, d=128, num_pages=16, page_size=16, max_pages=8,
                                        max_context=0, window=0, scale=0.1, dtype=0), kw)


# name, its arguments, whether it takes a workspace
CALLS = {"gdn_qk_norm_rope_fwd": (qk_fwd, False), "gdn_qk_norm_rope_bwd": (qk_bwd, True), "gdn_attn_fwd": (attn_fwd, True),
         "gdn_attn_bwd": (attn_bwd, True), "gdn_kv_append": (append, False), "gdn_attn_decode": (decode, True)}


def call(lib, name, a, ws=WS, nbytes=1 << 40):
    f = getattr(lib, name)
    ref = None if a is None else ctypes.byref(a)
    return f(ref, ws, nbytes, None) if CALLS[name][1] else f(ref, None)


SIZES = [(dict(d=96), UNSUPPORTED), (dict(d=256), UNSUPPORTED), (dict(dtype=7), INVALID), (dict(Hk=-1), INVALID),
         (dict(Hq=5000, Hk=5000), UNSUPPORTED), (dict(st_alpha=512), INVALID), (dict(st_z=512), INVALID),
         (dict(st_q=511), INVALID), (dict(st_q=(1 << 31) + 1), INVALID), (dict(q=10 * MB + 2), INVALID)]
NORM = [(dict(rot_dim=8), INVALID), (dict(rot_dim=144), INVALID), (dict(rot_dim=-16), INVALID), (dict(rot_dim=0), INVALID),
        (dict(inv_freq=None), INVALID), (dict(interleaved=2), INVALID), (dict(norm_eps=-1.0), INVALID),
        (dict(norm_eps=NAN), INVALID), (dict(q_norm_w=MB + 8), INVALID)]
SCALE = [(dict(scale=0.0), INVALID), (dict(scale=-1.0), INVALID), (dict(scale=NAN), INVALID), (dict(scale=INF), INVALID),
         (dict(window=-1), INVALID), (dict(dtype=1), UNSUPPORTED), (dict(Hk=3), INVALID), (dict(Hk=0), INVALID)]
TOKENS = [(dict(T=-1), INVALID), (dict(T=1 << 30), UNSUPPORTED), (dict(st_k=255), INVALID), (dict(k=11 * MB + 4), INVALID)]
CACHE = [(dict(num_pages=0), INVALID), (dict(page_size=0), INVALID), (dict(max_pages=0), INVALID),
         (dict(num_pages=1 << 31), INVALID), (dict(page_size=1 << 31), INVALID),
         (dict(num_pages=(1 << 31) - 1, page_size=(1 << 31) - 1), UNSUPPORTED), (dict(num_pages=1 << 19, page_size=1 << 20), UNSUPPORTED),
         (dict(k_cache=None), INVALID), (dict(v_cache=30 * MB + 8), INVALID), (dict(block_table=15 * MB + 2), INVALID),
         (dict(block_table=None), INVALID), (dict(context_lens=None), INVALID)]
REFUSED = {
    "gdn_qk_norm_rope_fwd": SIZES + NORM + TOKENS + [
        (dict(q=None), INVALID), (dict(k=None), INVALID), (dict(Hk=0), INVALID), (dict(Hk=0, k=None, k_out=None), INVALID),  # k_norm_w
        (dict(positions=None), INVALID), (dict(positions=12 * MB + 2), INVALID), (dict(q_out=None), INVALID),
        (dict(k_out=None), INVALID), (dict(q_out=10 * MB), INVALID), (dict(q_out=10 * MB + 4096), INVALID),
        (dict(k_out=13 * MB), INVALID), (dict(q_out=13 * MB + 8), INVALID), (dict(st_v=256), INVALID), (dict(Hq=0), INVALID)],
    "gdn_qk_norm_rope_bwd": SIZES + NORM + TOKENS + [
        (dict(grad_q_out=None), INVALID), (dict(grad_k_out=None), INVALID), (dict(grad_q=None), INVALID),
        (dict(grad_k=None), INVALID), (dict(grad_q_norm_w=None), INVALID), (dict(grad_k_norm_w=None), INVALID),
        (dict(q_norm_w=None), INVALID), (dict(grad_q=13 * MB), INVALID), (dict(grad_k=15 * MB), INVALID)],
    "gdn_attn_fwd": SIZES + SCALE + TOKENS + [
        (dict(nseq=-1), INVALID), (dict(nseq=1 << 30), INVALID), (dict(q=None), INVALID), (dict(v=None), INVALID),
        (dict(cu_seqlens=None), INVALID), (dict(cu_seqlens=13 * MB + 2), INVALID), (dict(o=None), INVALID),
        (dict(o=12 * MB), INVALID), (dict(st_v=100), INVALID), (dict(T=(1 << 30) - 1, nseq=1, Hq=4096, Hk=4096), UNSUPPORTED),
        (dict(bwd_cache=20 * MB, bwd_cache_bytes=100), WORKSPACE), (dict(bwd_cache=20 * MB + 16, bwd_cache_bytes=MB), INVALID),
        (dict(bwd_cache=10 * MB, bwd_cache_bytes=MB), INVALID), (dict(bwd_cache=14 * MB, bwd_cache_bytes=MB), INVALID)],
    "gdn_attn_bwd": SIZES + SCALE + TOKENS + [
        (dict(grad_o=None), INVALID), (dict(fwd_cache=None), INVALID), (dict(fwd_cache_bytes=100), INVALID),
        (dict(fwd_cache=19 * MB + 16), INVALID), (dict(grad_q=None), INVALID), (dict(grad_v=None), INVALID),
        (dict(grad_k=18 * MB), INVALID), (dict(grad_v=14 * MB), INVALID), (dict(grad_q=19 * MB), INVALID),
        (dict(o=None), INVALID), (dict(nseq=-1), INVALID)],
    "gdn_kv_append": SIZES + NORM + TOKENS + CACHE + [
        (dict(dtype=1), UNSUPPORTED), (dict(Hk=0), INVALID), (dict(nseq=-1), INVALID), (dict(cu_seqlens=None), INVALID),
        (dict(q=None), INVALID), (dict(q_out=None), INVALID), (dict(Hq=0), INVALID),
        (dict(Hq=0, q=None, q_out=None), INVALID),  # q_norm_w is left
        (dict(v=None), INVALID), (dict(v_cache=20 * MB), INVALID), (dict(k_out=20 * MB), INVALID),
        (dict(k_cache=11 * MB), INVALID), (dict(Hq=-1), INVALID)],
    "gdn_attn_decode": SIZES + SCALE + CACHE + [
        (dict(N=-1), INVALID), (dict(N=1 << 21), UNSUPPORTED), (dict(max_context=-1), INVALID), (dict(o=None), INVALID),
        (dict(o=10 * MB), INVALID), (dict(o=20 * MB), INVALID), (dict(st_k=256), INVALID), (dict(q=None), INVALID)],
}


@pytest.mark.parametrize("name", list(REFUSED))
def test_host_validation_rejects_before_launch(lib, name):
    before = gdn.kernel_launches()
    assert call(lib, name, None) == INVALID
    for kw, code in REFUSED[name]:
        rc = call(lib, name, CALLS[name][0](**kw))
        assert rc == code, (kw, rc, lib.gdn_last_error())
        assert lib.gdn_last_error().decode()
    assert gdn.kernel_launches() == before


@pytest.mark.parametrize("name", [n for n, (_, ws) in CALLS.items() if ws])
def test_workspace_checks(lib, name):
    a = CALLS[name][0](**({"max_pages": 4096, "num_pages": 4096, "k_cache": 1 << 33, "v_cache": 1 << 34} if name == "gdn_attn_decode" else {}))
    need = getattr(lib, name + "_workspace_size")(ctypes.byref(a))
    assert need > 0 and need % 256 == 0
    assert call(lib, name, a, None, need) == WORKSPACE
    assert call(lib, name, a, WS, need - 1) == WORKSPACE
    assert call(lib, name, a, ctypes.c_void_p(WS.value + 16), need) == WORKSPACE
    assert getattr(lib, name + "_workspace_size")(None) == 0


def test_sizes_of_caches_and_workspaces(lib):
    size = lambda f, a: f(ctypes.byref(a))
    # the forward's cache: a float a row of every tile (T / 128 + nseq at most), and T rows of bf16
    for T, nseq, Hq, d in ((1, 1, 1, 64), (128, 1, 4, 128), (1000, 7, 3, 64)):
        a = attn_fwd(T=T, nseq=nseq, Hq=Hq, Hk=1, d=d)
        got = size(lib.gdn_attn_fwd_cache_size, a)
        rows = nseq * 128 + T
        assert T * Hq * d * 2 + T * Hq * 4 <= got <= T * Hq * d * 2 + rows * Hq * 4 + 256
    assert size(lib.gdn_attn_fwd_cache_size, attn_fwd(T=0)) == 0
    assert size(lib.gdn_attn_fwd_cache_size, attn_fwd(T=-1)) == 0
    # a strided input that the copies cannot take in place adds its dense copy
    dense = size(lib.gdn_attn_fwd_workspace_size, attn_fwd())
    assert size(lib.gdn_attn_fwd_workspace_size, attn_fwd(st_q=520)) == dense
    assert size(lib.gdn_attn_fwd_workspace_size, attn_fwd(st_q=514)) == dense + 8 * 512 * 2
    assert size(lib.gdn_attn_fwd_workspace_size, attn_fwd(q=10 * MB + 2, st_q=520)) == dense + 8 * 512 * 2
    assert size(lib.gdn_attn_bwd_workspace_size, attn_bwd(st_k=257)) == size(lib.gdn_attn_bwd_workspace_size, attn_bwd()) + 8 * 256 * 2
    # no norm, no partial sums
    none = dict(q_norm_w=None, k_norm_w=None, grad_q_norm_w=None, grad_k_norm_w=None)
    assert size(lib.gdn_qk_norm_rope_bwd_workspace_size, qk_bwd(**none)) == 0
    # an unsplit context needs no partial results
    assert size(lib.gdn_attn_decode_workspace_size, decode(max_pages=1, page_size=16)) == 0
    assert size(lib.gdn_attn_decode_workspace_size, decode(d=96)) == 0


def test_calls_without_tokens_do_nothing(lib):
    before = gdn.kernel_launches()
    assert call(lib, "gdn_attn_fwd", attn_fwd(T=0, q=None, k=None, v=None, cu_seqlens=None, o=None), None, 0) == 0
    assert call(lib, "gdn_attn_fwd", attn_fwd(nseq=0), None, 0) == 0
    assert call(lib, "gdn_attn_bwd", attn_bwd(nseq=0), None, 0) == 0
    assert call(lib, "gdn_attn_decode", decode(N=0), None, 0) == 0
    assert gdn.kernel_launches() == before


def test_binding_takes_cuda_tensors_only():
    q, k = torch.zeros(4, 2, 64, dtype=torch.bfloat16), torch.zeros(4, 1, 64, dtype=torch.bfloat16)
    cache, table, ctx = torch.zeros(2, 16, 1, 64, dtype=torch.bfloat16), torch.zeros(4, 2, dtype=torch.int32), torch.ones(4, dtype=torch.int32)
    for f in (lambda: gdn.gdn_qk_norm_rope_fwd(q, k), lambda: gdn.gdn_qk_norm_rope_bwd(q, k, grad_q=q, grad_k=k),
              lambda: gdn.gdn_attn_fwd(q, k, k, [0, 4]),
              lambda: gdn.gdn_attn_bwd(q, k, k, [0, 4], q, grad_o=q, fwd_cache=torch.zeros(1, dtype=torch.uint8)),
              lambda: gdn.gdn_kv_append(k, k, cache, cache, table, ctx),
              lambda: gdn.gdn_attn_decode(q, cache, cache, table, ctx)):
        with pytest.raises(gdn.GdnError, match="CUDA tensors only"):
            f()


def test_binding_checks_cu_seqlens_on_the_host():
    for bad in ([], [[0, 4]], [0, 3, 2, 4], [-1, 4], [0, 5], torch.tensor([0, 5])):
        with pytest.raises(gdn.GdnError):
            gdn._cu_seqlens(bad, 0, 4)


def test_public_names():
    import gated_delta_rule_76_b200 as pkg
    for name in ("gdn_qk_norm_rope_fwd", "gdn_qk_norm_rope_bwd", "gdn_attn_fwd", "gdn_attn_bwd", "gdn_attn_fwd_cache_size",
                 "gdn_kv_append", "gdn_attn_decode"):
        assert getattr(pkg, name) is getattr(gdn, name) and name in pkg.__all__

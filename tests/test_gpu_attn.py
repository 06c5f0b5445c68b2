"""Causal attention over packed sequences on the GPU: forward and backward against the plain fp64 form
(bounds in attn_ref.py), sequence edges, windows, grouped heads, strides, rows outside every sequence,
values that must not leak between sequences, streams and graphs."""
import pytest
import torch

import attn_ref as ref
from gated_delta_rule_76_b200 import gdn

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


def make(lens, Hq, Hk, d, seed=0, extra=0, amp=1.0):
    g = torch.Generator().manual_seed(seed)
    T = sum(lens) + extra
    mk = lambda h: (amp * torch.randn(T, h, d, generator=g)).to(BF).cuda()
    cu = [sum(lens[:i]) for i in range(len(lens) + 1)]
    return mk(Hq), mk(Hk), mk(Hk), mk(Hq), cu


def fwd(q, k, v, cu, **kw):
    cache = torch.empty(gdn.gdn_attn_fwd_cache_size(q, k, v, cu), dtype=torch.uint8, device="cuda")
    return gdn.gdn_attn_fwd(q, k, v, cu, bwd_cache=cache, **kw), cache


SHAPES = [
    # lens, Hq, Hk, d, window
    ([1], 1, 1, 128, 0),
    ([2, 1, 1], 2, 1, 64, 0),
    ([127], 2, 2, 128, 0),
    ([128], 2, 1, 128, 0),
    ([129], 2, 1, 64, 0),
    ([5, 0, 64, 130, 1], 4, 2, 128, 0),
    ([257, 384], 3, 1, 128, 0),
    ([300, 71], 5, 1, 64, 0),
    ([700], 2, 2, 128, 0),
    ([400, 129], 2, 1, 128, 1),
    ([400, 129], 2, 1, 64, 2),
    ([640], 2, 1, 128, 128),
    ([640, 33], 2, 1, 128, 129),
    ([513], 1, 1, 64, 100),
    ([513, 90], 2, 2, 128, 5000),
    ([3] * 70, 2, 1, 64, 0),
]


@pytest.mark.parametrize("lens,Hq,Hk,d,window", SHAPES)
def test_forward(lens, Hq, Hk, d, window):
    q, k, v, _, cu = make(lens, Hq, Hk, d)
    o, bound = ref.packed(q, k, v, cu, d ** -0.5, window)
    ref.within(gdn.gdn_attn_fwd(q, k, v, cu, window=window), o, bound, "o")
    ref.within(fwd(q, k, v, cu, window=window)[0], o, bound, "o keeping the cache")


def test_forward_large_scores_and_many_rescales():
    # scores up to ~ +-300: the running reference moves by more than 2^8 many times
    q, k, v, _, cu = make([520], 2, 1, 128, amp=6.0)
    k *= torch.linspace(0.05, 2, 520, device="cuda").to(BF)[:, None, None].flip(0)
    o, _ = ref.packed(q, k, v, cu, 128 ** -0.5, 0)
    # scores of magnitude 300 carry 2^-24 * 300 * a few of absolute error into the exponent: far below U
    _, bound = ref.packed(q, k, v, cu, 128 ** -0.5, 0)
    ref.within(gdn.gdn_attn_fwd(q, k, v, cu), o, bound, "o")


def test_scale_is_taken():
    q, k, v, _, cu = make([90, 140], 2, 1, 64)
    o, bound = ref.packed(q, k, v, cu, 0.02, 0)
    ref.within(gdn.gdn_attn_fwd(q, k, v, cu, scale=0.02), o, bound, "o")


def test_rows_outside_every_sequence_stay_and_never_leak():
    lens = [100, 200]
    q, k, v, _, cu = make(lens, 2, 1, 128, extra=77)
    want = gdn.gdn_attn_fwd(q[:300].contiguous(), k[:300].contiguous(), v[:300].contiguous(), cu)
    for bad in (float("nan"), float("inf")):
        for t in (q, k, v):
            t[300:] = bad
        o = torch.full_like(q, 7.0)
        gdn.gdn_attn_fwd(q, k, v, cu, o=o)
        assert torch.equal(o[:300], want)
        assert (o[300:] == 7.0).all()
    # a sequence of NaN leaves its neighbours alone
    for t in (q, k, v):
        t[100:] = float("nan")
    o = gdn.gdn_attn_fwd(q, k, v, cu)
    assert torch.equal(o[:100], want[:100])
    # sequences need not start at token 0
    q, k, v, _, _ = make([300], 2, 1, 128)
    o = torch.full_like(q, 3.0)
    gdn.gdn_attn_fwd(q, k, v, [50, 250], o=o)
    want, bound = ref.packed(q, k, v, [50, 250], 128 ** -0.5, 0)
    ref.within(o[50:250], want[50:250], bound[50:250], "o")
    assert (o[:50] == 3.0).all() and (o[250:] == 3.0).all()


def test_no_sequences_and_no_tokens():
    q, k, v, _, _ = make([10], 2, 1, 64)
    o = torch.full_like(q, 2.0)
    gdn.gdn_attn_fwd(q, k, v, [0], o=o)
    gdn.gdn_attn_fwd(q, k, v, [0, 0, 0], o=o)
    assert (o == 2.0).all()
    e = q[:0]
    assert gdn.gdn_attn_fwd(e, k[:0], v[:0], [0, 0]).shape == e.shape


def test_malformed_cu_seqlens_on_the_device_stay_in_bounds():
    q, k, v, _, _ = make([256], 2, 1, 64)
    o = torch.full_like(q, 2.0)
    for cu in ([-5, 100, 10 ** 6], [200, 100, 50], [2 ** 31 - 1, -2 ** 31], [0, 256, 0, 256]):
        gdn.gdn_attn_fwd(q, k, v, torch.tensor(cu, dtype=torch.int32, device="cuda"), o=o)
    torch.cuda.synchronize()
    want, bound = ref.packed(q, k, v, [0, 256], 64 ** -0.5, 0)
    ref.within(gdn.gdn_attn_fwd(q, k, v, [0, 256]), want, bound, "o after")


@pytest.mark.parametrize("shift", [0, 8, 1])
def test_strided_inputs(shift):
    """Slices of one projection buffer: aligned ones are read in place, odd ones through a copy."""
    T, Hq, Hk, d = 200, 4, 2, 64
    g = torch.Generator().manual_seed(3)
    buf = torch.randn(T, (Hq + 2 * Hk) * d + 2 * shift, generator=g).to(BF).cuda()
    at = [shift, shift + Hq * d, shift + (Hq + Hk) * d]
    q, k, v = (buf[:, a:a + h * d].view(T, h, d) for a, h in zip(at, (Hq, Hk, Hk)))
    do = torch.randn(T, Hq, d, generator=g).to(BF).cuda()
    cu = [0, 150, 200]
    o, cache = fwd(q, k, v, cu)
    dense = [t.contiguous() for t in (q, k, v)]
    o2, cache2 = fwd(*dense, cu)
    assert torch.equal(o, o2)
    a = gdn.gdn_attn_bwd(q, k, v, cu, o, grad_o=do, fwd_cache=cache)
    b = gdn.gdn_attn_bwd(*dense, cu, o2, grad_o=do, fwd_cache=cache2)
    for x in ("dq", "dk", "dv"):
        assert torch.equal(a[x], b[x])


def test_same_bits_again_on_another_stream_and_in_a_graph():
    q, k, v, do, cu = make([333, 500, 40], 4, 2, 128)
    cu = torch.tensor(cu, dtype=torch.int32, device="cuda")
    o, cache = fwd(q, k, v, cu, window=300)
    want = [o] + list(gdn.gdn_attn_bwd(q, k, v, cu, o, grad_o=do, fwd_cache=cache, window=300).values())

    def step(stream=None):
        o, cache = fwd(q, k, v, cu, window=300, stream=stream)
        return [o] + list(gdn.gdn_attn_bwd(q, k, v, cu, o, grad_o=do, fwd_cache=cache, window=300, stream=stream).values())

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = step()
    torch.cuda.current_stream().wait_stream(side)
    for a, b in zip(want, other):
        assert torch.equal(a, b)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    q2 = q.clone()
    q.normal_()
    graph.replay()
    o2, cache2 = fwd(q, k, v, cu, window=300)
    assert torch.equal(held[0], o2)
    q.copy_(q2)
    graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(want, held):
        assert torch.equal(a, b)


@pytest.mark.parametrize("lens,Hq,Hk,d,window", SHAPES)
def test_backward(lens, Hq, Hk, d, window):
    q, k, v, do, cu = make(lens, Hq, Hk, d, seed=1)
    _, _, grads, bounds = ref.packed(q, k, v, cu, d ** -0.5, window, do)
    o, cache = fwd(q, k, v, cu, window=window)
    got = gdn.gdn_attn_bwd(q, k, v, cu, o, grad_o=do, fwd_cache=cache, window=window)
    for name, g, b in zip(("dq", "dk", "dv"), grads, bounds):
        ref.within(got[name], g, b, name)


def test_backward_rows_outside_every_sequence_stay_and_never_leak():
    lens = [100, 200]
    q, k, v, do, cu = make(lens, 4, 2, 128, extra=77)
    cut = [t[:300].contiguous() for t in (q, k, v, do)]
    o, cache = fwd(*cut[:3], cu)
    want = gdn.gdn_attn_bwd(*cut[:3], cu, o, grad_o=cut[3], fwd_cache=cache)
    for t in (q, k, v, do):
        t[300:] = float("nan")
    o = torch.full_like(q, float("nan"))
    cache = torch.empty(gdn.gdn_attn_fwd_cache_size(q, k, v, cu), dtype=torch.uint8, device="cuda")
    gdn.gdn_attn_fwd(q, k, v, cu, o=o, bwd_cache=cache)
    held = [torch.full_like(t, 5.0) for t in (q, k, v)]
    gdn.gdn_attn_bwd(q, k, v, cu, o, grad_o=do, fwd_cache=cache, dq=held[0], dk=held[1], dv=held[2])
    for x, name in zip(held, ("dq", "dk", "dv")):
        assert torch.equal(x[:300], want[name]), name
        assert (x[300:] == 5.0).all(), name


def test_backward_of_the_first_row_is_exact():
    """Row 0 of a sequence sees itself alone: its score's gradient is 0, and v's row passes through."""
    q, k, v, do, cu = make([1, 1, 1, 1], 2, 2, 64)
    o, cache = fwd(q, k, v, cu)
    g = gdn.gdn_attn_bwd(q, k, v, cu, o, grad_o=do, fwd_cache=cache)
    assert torch.equal(o, v) and torch.equal(g["dv"], do)
    # ds = do . v - do . o, two fp32 sums of 64 products in different orders: 64 * 2^-24 of their magnitude
    lim = 64 ** -0.5 * 64 * 2.0 ** -24 * 2 * (do.float().abs() * v.float().abs()).sum(-1, keepdim=True)
    assert (g["dq"].float().abs() <= lim * k.float().abs()).all()
    assert (g["dk"].float().abs() <= lim * q.float().abs()).all()


def test_workspace_status_is_clean():
    q, k, v, _, cu = make([200], 1, 1, 64)
    ws = torch.empty(1 << 20, dtype=torch.uint8, device="cuda")
    gdn.gdn_attn_fwd(q, k, v, cu, workspace=ws)
    import ctypes
    st = ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    assert gdn.load().gdn_workspace_status(ctypes.c_void_p(ws.data_ptr()), st) == 0

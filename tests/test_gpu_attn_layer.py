"""The attention layer's calls together, as a training step and a server use them, and what single-operator tests
do not reach: many units of work per CTA, more sequences than a warp has lanes, calls on two streams at once,
arrays of sequence starts that no caller should pass."""
import ctypes

import pytest
import torch

import attn_ref as ref
from gated_delta_rule_76_b200 import gdn

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


def rnd(*s, seed=0, dtype=BF):
    return torch.randn(*s, generator=torch.Generator().manual_seed(seed)).to(dtype).cuda()


def starts(lens):
    return [sum(lens[:i]) for i in range(len(lens) + 1)]


def cache_of(q, k, v, cu):
    return torch.empty(gdn.gdn_attn_fwd_cache_size(q, k, v, cu), dtype=torch.uint8, device="cuda")


def host(t):
    return ref.f64(t) if t.is_floating_point() else t.cpu()


@pytest.mark.parametrize("lens,Hq,Hk,d,window,rot,il", [
    ([200, 1, 77], 4, 2, 128, 0, 128, False),
    ([129, 300], 6, 2, 64, 100, 32, True),
])
def test_training_step_of_a_layer(lens, Hq, Hk, d, window, rot, il):
    """One projection buffer's slices through norm and rotation, attention, and both backwards; each stage against
    the fp64 form over what the stage before it returned, so that only its own roundings count."""
    T, cu = sum(lens), starts(lens)
    qkv = rnd(T, (Hq + 2 * Hk) * d, seed=1)
    q, k, v = (t.unflatten(1, (-1, d)) for t in qkv.split([Hq * d, Hk * d, Hk * d], 1))
    assert not q.is_contiguous()
    pos = torch.cat([torch.arange(n) for n in lens]).to(torch.int32).cuda()
    freq = (10000.0 ** (-torch.arange(0, rot, 2).double() / rot)).float().cuda()
    qw, kw = ((1 + 0.2 * torch.randn(d, generator=torch.Generator().manual_seed(s))).to(BF).cuda() for s in (2, 3))
    do = rnd(T, Hq, d, seed=4)
    norm = dict(q_norm_w=qw, k_norm_w=kw, interleaved=il)

    qr, kr = gdn.gdn_qk_norm_rope_fwd(q, k, pos, freq, **norm)
    cache = cache_of(qr, kr, v, cu)
    o = gdn.gdn_attn_fwd(qr, kr, v, cu, window=window, bwd_cache=cache)
    g = gdn.gdn_attn_bwd(qr, kr, v, cu, o, grad_o=do, fwd_cache=cache, window=window)
    gx = gdn.gdn_qk_norm_rope_bwd(q, k, pos, freq, grad_q=g["dq"], grad_k=g["dk"], **norm)

    for got, x, w, grad, name in ((qr, q, qw, "dq", "q"), (kr, k, kw, "dk", "k")):
        a = [host(t) for t in (x, w, pos, freq)]
        y = ref.norm_rope(*a, interleaved=il)
        # fp32 arithmetic of a pair (3e-6 of the row's largest, rotated), then one rounding
        ref.within(got, y, 3e-6 * 2 ** 0.5 * y.abs().amax(-1, keepdim=True) + ref.U * y.abs(), name)
        dx, dw = ref.norm_rope_grad(*a, host(g[grad]), interleaved=il)
        r = 1 / torch.sqrt((a[0] ** 2).mean(-1, keepdim=True) + 1e-6)
        top = host(g[grad]).abs().amax(-1, keepdim=True) * 2 ** 0.5
        mag = r * a[1].abs().max() * top * (1 + r * r * a[0].abs() * a[0].abs().mean(-1, keepdim=True))
        ref.within(gx["d" + name], dx, 6e-6 * mag + ref.U * dx.abs(), "d" + name)
        ref.within(gx[f"d{name}_norm_w"], dw, ref.F * (top * a[0].abs() * r).sum((0, 1)), f"d{name}_norm_w")
    want, bound, grads, bounds = ref.packed(qr, kr, v, cu, d ** -0.5, window, do)
    ref.within(o, want, bound, "o")
    for name, x, b in zip(("dq", "dk", "dv"), grads, bounds):
        ref.within(g[name], x, b, name)


@pytest.mark.parametrize("lens,Hq,Hk,d,window", [
    ([260] * 20, 8, 2, 64, 0),                                   # about five units a CTA
    ([131, 1, 0, 7] * 10 + [400], 12, 4, 64, 0),                 # more than 32 sequences; one tile and two
    ([131, 1, 0, 7] * 10 + [400], 9, 3, 64, 50),                 # an odd group: pairs of tiles, the second often missing
    ([20] * 300, 3, 1, 64, 0),
    ([2] * 500 + [150] + [0, 1] * 40 + [129], 4, 2, 64, 0),      # many runs of 32 sequences, some of them empty
    ([0] * 70 + [5] + [0] * 70, 2, 1, 128, 0),
    # few key tiles: the backward takes them in parts
    ([1800], 2, 1, 128, 0),
    ([1793, 3, 900], 3, 3, 64, 0),                                # pairs of tiles of unequal reach
    ([1500, 640], 1, 1, 128, 700),                                # parts that end at the window's edge
    ([2050], 5, 1, 64, 1100),
    ([1100], 10, 2, 128, 0),
    ([1100, 900], 7, 7, 128, 300),
])
def test_many_units_a_cta(lens, Hq, Hk, d, window):
    T, cu = sum(lens), starts(lens)
    q, k, v, do = (rnd(T, h, d, seed=s) for s, h in enumerate((Hq, Hk, Hk, Hq)))
    cache = cache_of(q, k, v, cu)
    o = gdn.gdn_attn_fwd(q, k, v, cu, window=window, bwd_cache=cache)
    g = gdn.gdn_attn_bwd(q, k, v, cu, o, grad_o=do, fwd_cache=cache, window=window)
    want, bound, grads, bounds = ref.packed(q, k, v, cu, d ** -0.5, window, do)
    ref.within(o, want, bound, "o")
    for name, x, b in zip(("dq", "dk", "dv"), grads, bounds):
        ref.within(g[name], x, b, name)


@pytest.mark.parametrize("Hq,Hk,d,window", [(2, 1, 128, 0), (3, 3, 64, 700)])
def test_a_long_sequence_in_a_padded_batch(Hq, Hk, d, window):
    """Few units, cut into parts: what lies before and behind the sequence is neither read nor written."""
    T, a, b = 2100, 50, 1900
    q, k, v, do = (rnd(T, h, d, seed=s) for s, h in enumerate((Hq, Hk, Hk, Hq)))
    want, bound, grads, bounds = ref.packed(*(t[a:b] for t in (q, k, v)), [0, b - a], d ** -0.5, window, do[a:b])
    for t in (q, k, v, do):
        t[:a] = t[b:] = float("nan")
    cu = [a, b]
    cache = cache_of(q, k, v, cu)
    o = torch.full_like(q, float("nan"))
    gdn.gdn_attn_fwd(q, k, v, cu, window=window, o=o, bwd_cache=cache)
    held = [torch.full_like(t, 5.0) for t in (q, k, v)]
    gdn.gdn_attn_bwd(q, k, v, cu, o, grad_o=do, fwd_cache=cache, window=window, dq=held[0], dk=held[1], dv=held[2])
    assert o[:a].isnan().all() and o[b:].isnan().all()
    ref.within(o[a:b], want, bound, "o")
    for t, x, y, name in zip(held, grads, bounds, ("dq", "dk", "dv")):
        assert (t[:a] == 5.0).all() and (t[b:] == 5.0).all(), name
        ref.within(t[a:b], x, y, name)


def test_short_units_in_a_row_keep_the_copies_in_step():
    """Many units of one or two key tiles at heads of 64, whose ring of key tiles runs five pairs ahead: no wait may
    expire, and every run gives the same bits."""
    lens = [1, 1, 0, 128, 0, 64, 63, 64, 1, 200, 2, 65, 64, 1, 2, 2, 64, 129, 2, 64, 64, 128, 65, 128, 128, 1, 0, 64, 127, 65, 127,
            63, 64, 1, 64, 129, 63, 200, 127, 0, 63, 0, 127, 2]
    st = ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    for Hq, Hk, d, window in ((24, 8, 64, 1), (24, 8, 64, 0), (16, 8, 64, 1), (16, 8, 128, 1)):
        T, cu = sum(lens), torch.tensor(starts(lens), dtype=torch.int32, device="cuda")
        q, k, v = (rnd(T, h, d, seed=s) for s, h in enumerate((Hq, Hk, Hk)))
        want, bound = ref.packed(q, k, v, starts(lens), d ** -0.5, window)
        ws = torch.empty(1 << 16, dtype=torch.uint8, device="cuda")
        first = None
        for _ in range(30):
            o = gdn.gdn_attn_fwd(q, k, v, cu, window=window, workspace=ws)
            assert gdn.load().gdn_workspace_status(ctypes.c_void_p(ws.data_ptr()), st) == 0
            first = o if first is None else first
            assert torch.equal(o, first)
        ref.within(first, want, bound, "o")


def test_calls_on_two_streams_at_once():
    """Two runs of the layer in flight together, each with its own workspace: the same bits as one after the other."""
    lens, Hq, Hk, d = [500, 300, 41], 8, 2, 128
    T, cu = sum(lens), torch.tensor(starts(lens), dtype=torch.int32, device="cuda")
    q, k, v, do = (rnd(T, h, d, seed=s) for s, h in enumerate((Hq, Hk, Hk, Hq)))

    def step(q, stream=None):
        cache = cache_of(q, k, v, cu)
        o = gdn.gdn_attn_fwd(q, k, v, cu, bwd_cache=cache, stream=stream)
        return [o, *gdn.gdn_attn_bwd(q, k, v, cu, o, grad_o=do, fwd_cache=cache, stream=stream).values()]

    inputs = [q, -q]
    want = [step(x) for x in inputs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in inputs]
    for _ in range(5):
        got = []
        for x, s in zip(inputs, streams):
            with torch.cuda.stream(s):
                got.append(step(x))
        torch.cuda.synchronize()
        for a, b in zip(want, got):
            assert all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("cu", [
    [0, 1280] * 6,                   # overlapping sequences: more tiles than the tokens have
    [0, 1280] * 40,
    [0, -7, 900, 300, 1280, 5],
    [2 ** 31 - 1] * 3, [-2 ** 31, 2 ** 31 - 1],
])
def test_malformed_cu_seqlens_write_nothing_but_the_results(cu):
    """Whatever the device array holds: the buffers' neighbours stay as they were, and the calls end."""
    T, Hq, Hk, d, pad = 1280, 2, 1, 64, 4096
    cu = torch.tensor(cu, dtype=torch.int32, device="cuda")
    q, k, v, do = (rnd(T, h, d, seed=s) for s, h in enumerate((Hq, Hk, Hk, Hq)))

    def guarded(nbytes):
        whole = torch.full((nbytes + 2 * pad,), 0x5A, dtype=torch.uint8, device="cuda")
        return whole, whole[pad:pad + nbytes]

    guards = []

    def out(like):
        whole, mid = guarded(like.numel() * 2)
        guards.append(whole)
        return mid.view(BF).view(like.shape)

    whole, cache = guarded(gdn.gdn_attn_fwd_cache_size(q, k, v, cu))
    guards.append(whole)
    cache.zero_()
    o = out(q)
    gdn.gdn_attn_fwd(q, k, v, cu, o=o, bwd_cache=cache)
    o.nan_to_num_()
    ws, room = guarded(1 << 25)
    guards.append(ws)
    gdn.gdn_attn_bwd(q, k, v, cu, o, grad_o=do, fwd_cache=cache, dq=out(q), dk=out(k), dv=out(v), workspace=room)
    torch.cuda.synchronize()
    for t in guards:
        assert (t[:pad] == 0x5A).all() and (t[-pad:] == 0x5A).all()
    st = ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    assert gdn.load().gdn_workspace_status(ctypes.c_void_p(room.data_ptr()), st) == 0


def test_one_workspace_serves_call_after_call():
    """The counters of the call before are cleared: a workspace of any contents, used again and again."""
    lens, Hq, Hk, d = [700, 650], 16, 4, 64
    q, k, v, do = (rnd(sum(lens), h, d, seed=s) for s, h in enumerate((Hq, Hk, Hk, Hq)))
    cu = starts(lens)
    ws = torch.full((1 << 25,), 0xFF, dtype=torch.uint8, device="cuda")
    cache = cache_of(q, k, v, cu)
    o = gdn.gdn_attn_fwd(q, k, v, cu, bwd_cache=cache)
    g = gdn.gdn_attn_bwd(q, k, v, cu, o, grad_o=do, fwd_cache=cache)
    for _ in range(3):
        c2 = cache_of(q, k, v, cu)
        o2 = gdn.gdn_attn_fwd(q, k, v, cu, bwd_cache=c2, workspace=ws)
        g2 = gdn.gdn_attn_bwd(q, k, v, cu, o2, grad_o=do, fwd_cache=c2, workspace=ws)
        assert torch.equal(o, o2) and all(torch.equal(g[n], g2[n]) for n in g)


def test_decode_and_append_in_one_graph_replayed():
    """The captured step of a server: append, attend, advance; replays walk the cache on."""
    N, Hq, Hk, d, page, steps, rot = 3, 4, 2, 64, 16, 20, 64
    kc, vc = rnd(20, page, Hk, d, seed=1), rnd(20, page, Hk, d, seed=2)
    table = torch.randperm(20, generator=torch.Generator().manual_seed(0))[:18].view(N, 6).to(torch.int32).cuda()
    first = torch.tensor([0, 30, 61], dtype=torch.int32, device="cuda")
    freq = (10000.0 ** (-torch.arange(0, rot, 2).double() / rot)).float().cuda()
    toks = [rnd(steps, N, h, d, seed=s) for s, h in ((3, Hq), (4, Hk), (5, Hk))]

    def step(q, k, v, kc, vc, ctx):
        qs, _ = gdn.gdn_kv_append(k, v, kc, vc, table, ctx, q=q, inv_freq=freq)
        ctx += 1
        return gdn.gdn_attn_decode(qs, kc, vc, table, ctx)

    kc1, vc1, ctx1 = kc.clone(), vc.clone(), first.clone()
    want = [step(*(t[i] for t in toks), kc1, vc1, ctx1) for i in range(steps)]
    held, ctx = [t[0].clone() for t in toks], first.clone()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        o = step(*held, kc, vc, ctx)
    for i in range(steps):
        for h, t in zip(held, toks):
            h.copy_(t[i])
        graph.replay()
        assert torch.equal(o, want[i]), i
    assert torch.equal(ctx, ctx1) and torch.equal(kc, kc1) and torch.equal(vc, vc1)


def calls():
    """Every natively marshalled call, with and without its optional arguments: name -> call."""
    T, Hq, Hk, d, page = 70, 4, 2, 64, 16
    q, k, v = (rnd(T, h, d, seed=s) for s, h in enumerate((Hq, Hk, Hk)))
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    pos, cu, freq, w = i32(list(range(T))), i32([0, 3, 70]), rnd(16, seed=7, dtype=torch.float32).abs(), rnd(d, seed=8)
    kc, vc = rnd(12, page, Hk, d, seed=5), rnd(12, page, Hk, d, seed=6)
    table, ctx = torch.arange(12, dtype=torch.int32, device="cuda").view(2, 6), i32([20, 1])
    norm = dict(q_norm_w=w, k_norm_w=w, norm_eps=1e-5, interleaved=True, rot_scale=0.5)

    def append(**kw):
        caches = kc.clone(), vc.clone()
        return [*gdn.gdn_kv_append(k, v, *caches, table, ctx, cu_seqlens=cu, **kw), *caches]

    def train(**kw):
        cache = cache_of(q, k, v, cu)
        cache.zero_()
        o = gdn.gdn_attn_fwd(q, k, v, cu, bwd_cache=cache, **kw)
        return [o, cache, *gdn.gdn_attn_bwd(q, k, v, cu, o, grad_o=-q, fwd_cache=cache, **kw).values()]

    one = lambda t: t[:2].contiguous()
    return {
        "qk grads": lambda: list(gdn.gdn_qk_norm_rope_bwd(q, k, pos, freq, grad_q=-q, grad_k=-k, **norm).values()),
        "qk grads, q alone": lambda: list(gdn.gdn_qk_norm_rope_bwd(q, None, pos, freq, grad_q=-q).values()),
        "train": train,
        "train window": lambda: train(scale=0.3, window=5),
        "qk": lambda: gdn.gdn_qk_norm_rope_fwd(q, k, pos, freq, **norm),
        "qk f32, q alone": lambda: gdn.gdn_qk_norm_rope_fwd(q.float(), None, q_norm_w=w.float()),
        "attn": lambda: [gdn.gdn_attn_fwd(q, k, v, cu)],
        "attn window": lambda: [gdn.gdn_attn_fwd(q, k, v, cu, scale=0.3, window=5)],
        "append": lambda: append(q=q, inv_freq=freq, want_k=True, **norm),
        "append k": lambda: append(inv_freq=freq),
        "append one": lambda: gdn.gdn_kv_append(one(k), one(v), kc.clone(), vc.clone(), table, ctx, q=one(q)),
        "decode": lambda: [gdn.gdn_attn_decode(one(q), kc, vc, table, ctx)],
        "decode window": lambda: [gdn.gdn_attn_decode(one(q), kc, vc, table, ctx, scale=0.2, window=7, max_context=50)],
    }


def test_native_marshalling_is_the_general_one(monkeypatch):
    assert gdn._native is not None, "the native module is not built"
    got = {name: f() for name, f in calls().items()}
    monkeypatch.setattr(gdn, "_native", None)
    for name, f in calls().items():
        want = f()
        assert len(want) == len(got[name])
        for a, b in zip(got[name], want):
            assert (a is None and b is None) or torch.equal(a, b), name


def test_refusals_say_the_same_through_both(monkeypatch):
    q, k = rnd(8, 4, 64), rnd(8, 3, 64)
    cu = torch.tensor([0, 8], dtype=torch.int32, device="cuda")
    kc, table, ctx = rnd(4, 16, 2, 64), torch.zeros(8, 2, dtype=torch.int32, device="cuda"), cu[1:].repeat(8)
    bad = [
        lambda: gdn.gdn_attn_fwd(q, k, k, cu),                                  # 4 heads on 3
        lambda: gdn.gdn_attn_fwd(q, q, q, cu, scale=-1.0),
        lambda: gdn.gdn_attn_fwd(q, q, q, cu, window=-1),
        lambda: gdn.gdn_attn_fwd(q, q, q.float(), cu),
        lambda: gdn.gdn_attn_fwd(q, q, q[:4], cu),
        lambda: gdn.gdn_attn_fwd(q, q, q, cu.long()),
        lambda: gdn.gdn_attn_fwd(q.float(), q.float(), q.float(), cu),          # bf16 only
        lambda: gdn.gdn_qk_norm_rope_fwd(q, k, None, torch.ones(8, device="cuda")),
        lambda: gdn.gdn_qk_norm_rope_fwd(q, k, norm_eps=-1.0),
        lambda: gdn.gdn_qk_norm_rope_fwd(q, k, interleaved=2),
        lambda: gdn.gdn_qk_norm_rope_fwd(q, k, q_norm_w=rnd(32)),
        lambda: gdn.gdn_qk_norm_rope_fwd(rnd(8, 4, 32), None),
        lambda: gdn.gdn_kv_append(q, q, kc, kc, table, ctx),                    # 4 heads into a cache of 2
        lambda: gdn.gdn_kv_append(q[:, :2].contiguous(), q[:, :2].contiguous(), kc, kc, table, ctx),  # one cache for both
        lambda: gdn.gdn_attn_decode(q, kc, kc, table[:4], ctx),
        lambda: gdn.gdn_attn_decode(q, kc, kc, table, ctx, max_context=-1),
        lambda: gdn.gdn_attn_decode(q, kc.float(), kc, table, ctx),
        lambda: gdn.gdn_qk_norm_rope_bwd(q, k, grad_q=q),                       # k without its gradient
        lambda: gdn.gdn_qk_norm_rope_bwd(q, k, grad_q=q, grad_k=k[:4]),
        lambda: gdn.gdn_attn_fwd(q, q, q, cu, bwd_cache=torch.empty(256, dtype=torch.uint8, device="cuda")),
        lambda: gdn.gdn_attn_bwd(q, q, q, cu, q, grad_o=q, fwd_cache=torch.empty(256, dtype=torch.uint8, device="cuda")),
        lambda: gdn.gdn_attn_bwd(q, q, q, cu, q, grad_o=q[:4], fwd_cache=cache_of(q, q, q, cu)),
    ]

    def says(f):
        before = gdn.kernel_launches()
        with pytest.raises(gdn.GdnError) as e:
            f()
        assert gdn.kernel_launches() == before
        return str(e.value)

    got = [says(f) for f in bad]
    monkeypatch.setattr(gdn, "_native", None)
    assert got == [says(f) for f in bad]


def test_offsets_past_32_bits_in_a_batch():
    """2.4e9 elements of q: the last sequence's rows and gradients are those of a call over it alone."""
    Hq, Hk, d, n, window = 64, 1, 128, 200, 64
    T = 2 ** 31 // (Hq * d) + 30000
    q, do = (torch.empty(T, Hq, d, dtype=BF, device="cuda").normal_() for _ in range(2))
    k, v = (torch.empty(T, Hk, d, dtype=BF, device="cuda").normal_() for _ in range(2))
    cu = [0, T - n, T]
    cache = cache_of(q, k, v, cu)
    o = gdn.gdn_attn_fwd(q, k, v, cu, window=window, bwd_cache=cache)
    g = gdn.gdn_attn_bwd(q, k, v, cu, o, grad_o=do, fwd_cache=cache, window=window)
    last = [t[T - n:].clone() for t in (q, k, v, do)]
    c1 = cache_of(*last[:3], [0, n])
    o1 = gdn.gdn_attn_fwd(*last[:3], [0, n], window=window, bwd_cache=c1)
    assert torch.equal(o[T - n:], o1)
    want, bound, grads, bounds = ref.packed(*last[:3], [0, n], d ** -0.5, window, last[3])
    ref.within(o1, want, bound, "o")
    for name, x, y in zip(("dq", "dk", "dv"), grads, bounds):
        ref.within(g[name][T - n:], x, y, name)
    pos = torch.arange(T, dtype=torch.int32, device="cuda")
    freq = torch.rand(32, device="cuda")
    w = rnd(d)
    y, _ = gdn.gdn_qk_norm_rope_fwd(q, None, pos, freq, q_norm_w=w)
    y1, _ = gdn.gdn_qk_norm_rope_fwd(last[0], None, pos[T - n:].clone(), freq, q_norm_w=w)
    assert torch.equal(y[T - n:], y1)
    gx = gdn.gdn_qk_norm_rope_bwd(q, None, pos, freq, grad_q=do, q_norm_w=w)
    g1 = gdn.gdn_qk_norm_rope_bwd(last[0], None, pos[T - n:].clone(), freq, grad_q=last[3], q_norm_w=w)
    assert torch.equal(gx["dq"][T - n:], g1["dq"])


def test_offsets_past_32_bits_in_a_cache():
    """Pages behind the first 2^31 elements: appended, read back, attended."""
    Hq, Hk, d, page = 4, 2, 128, 64
    pages = 2 ** 31 // (page * Hk * d) + 8
    kc, vc = (torch.empty(pages, page, Hk, d, dtype=BF, device="cuda") for _ in range(2))
    ids = [pages - 1, 3, pages - 5, 0]
    small = rnd(4, page, Hk, d, seed=1), rnd(4, page, Hk, d, seed=2)
    for big, s in zip((kc, vc), small):
        big[ids] = s
    table = torch.tensor([[pages - 1, 3, pages - 5, 0]], dtype=torch.int32, device="cuda")
    near = torch.tensor([[0, 1, 2, 3]], dtype=torch.int32, device="cuda")
    ctx = torch.tensor([150], dtype=torch.int32, device="cuda")
    q, k, v = (rnd(1, h, d, seed=s) for s, h in ((3, Hq), (4, Hk), (5, Hk)))
    got, _ = gdn.gdn_kv_append(k, v, kc, vc, table, ctx, q=q)
    want, _ = gdn.gdn_kv_append(k, v, *small, near, ctx, q=q)
    assert torch.equal(got, want)
    for big, s in zip((kc, vc), small):
        assert torch.equal(big[ids], s)
    ctx += 1
    assert torch.equal(gdn.gdn_attn_decode(got, kc, vc, table, ctx), gdn.gdn_attn_decode(want, *small, near, ctx))

"""The paged cache on the GPU: append (norm and rotation on the way) and single-token attention, each
against the plain fp64 form, and both as a serving loop against attention over the whole sequence."""
import pytest
import torch

import attn_ref as ref
from gated_delta_rule_76_b200 import gdn

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


def rnd(*s, seed=0):
    return torch.randn(*s, generator=torch.Generator().manual_seed(seed)).to(BF).cuda()


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def freqs(rot):
    return (10000.0 ** (-torch.arange(0, rot, 2).double() / rot)).float().cuda()


DECODE = [
    # N, Hq, Hk, d, page, contexts, window
    (1, 1, 1, 128, 16, [1], 0),
    (3, 4, 2, 64, 8, [1, 0, 17], 0),
    (2, 8, 1, 128, 16, [63, 64], 0),
    (2, 16, 1, 128, 1, [65, 200], 0),
    (2, 17, 1, 64, 24, [100, 129], 0),
    (1, 33, 1, 128, 7, [300], 0),
    (4, 6, 2, 128, 64, [1000, 5, 513, 700], 0),
    (2, 4, 4, 64, 128, [2100, 1025], 0),
    (3, 4, 2, 128, 16, [900, 40, 3], 64),
    (3, 4, 2, 128, 24, [900, 1500, 3], 700),
    (2, 2, 1, 64, 16, [77, 300], 1),
]


def cache_for(N, Hk, d, page, ctx, seed=0, spare=3):
    need = [max(1, -(-c // page)) for c in ctx]
    most, total = max(need) + 1, sum(need) + spare
    g = torch.Generator().manual_seed(seed)
    ids = torch.randperm(total, generator=g).tolist()
    table = torch.full((N, most), -1, dtype=torch.int32)
    for n in range(N):
        for j in range(need[n]):
            table[n, j] = ids.pop()
    return rnd(total, page, Hk, d, seed=seed + 1), rnd(total, page, Hk, d, seed=seed + 2), table.cuda()


@pytest.mark.parametrize("N,Hq,Hk,d,page,ctx,window", DECODE)
def test_decode(N, Hq, Hk, d, page, ctx, window):
    kc, vc, table = cache_for(N, Hk, d, page, ctx)
    q = rnd(N, Hq, d, seed=9)
    o, bound = ref.decode(q, kc, vc, table.cpu(), ctx, d ** -0.5, window)
    ref.within(gdn.gdn_attn_decode(q, kc, vc, table, i32(ctx), window=window), o, bound, "o")
    got = gdn.gdn_attn_decode(q, kc, vc, table, i32(ctx), window=window, max_context=max(ctx) + 1)
    ref.within(got, o, bound, "o with max_context")


def test_decode_reads_nothing_behind_the_context():
    """NaN in every slot that no context reaches, and in the pages of nobody."""
    N, Hq, Hk, d, page, ctx = 3, 4, 2, 128, 16, [37, 0, 600]
    kc, vc, table = cache_for(N, Hk, d, page, ctx)
    q = rnd(N, Hq, d, seed=9)
    want = gdn.gdn_attn_decode(q, kc, vc, table, i32(ctx))
    used = torch.zeros(kc.shape[0], page, dtype=torch.bool)
    for n in range(N):
        for p in range(ctx[n]):
            used[int(table[n, p // page]), p % page] = True
    kc[~used.cuda()] = float("nan")
    vc[~used.cuda()] = float("nan")
    o = gdn.gdn_attn_decode(q, kc, vc, table, i32(ctx))
    assert torch.equal(o, want) and not o[1].any()


def test_decode_bad_pages_and_lengths():
    N, Hq, Hk, d, page, ctx = 4, 2, 1, 64, 8, [100, 100, 100, 100]
    kc, vc, table = cache_for(N, Hk, d, page, ctx)
    table[1, 3] = -1
    table[2, 5] = kc.shape[0]
    table[3, :] = 2 ** 31 - 1
    q = rnd(N, Hq, d, seed=9)
    lens = [100, 100, 100, 100]
    o, bound = ref.decode(q, kc, vc, table.cpu(), lens, d ** -0.5, 0)
    ref.within(gdn.gdn_attn_decode(q, kc, vc, table, i32(lens)), o, bound, "o")
    # lengths below 0 read as 0, lengths past the table as the table's reach (whose last page is -1 here)
    lens = [-7, 2 ** 31 - 1, 100, 5]
    o, bound = ref.decode(q, kc, vc, table.cpu(), lens, d ** -0.5, 0)
    ref.within(gdn.gdn_attn_decode(q, kc, vc, table, i32(lens)), o, bound, "o")


def test_decode_strided_q_stream_and_graph():
    kc, vc, table = cache_for(3, 2, 64, 16, [700, 64, 1300])
    buf = rnd(3, 5 * 64 + 7, seed=4)
    for a in (0, 2, 1):
        q = buf[:, a:a + 4 * 64].view(3, 4, 64)
        want = gdn.gdn_attn_decode(q.contiguous(), kc, vc, table, i32([700, 64, 1300]))
        assert torch.equal(gdn.gdn_attn_decode(q, kc, vc, table, i32([700, 64, 1300])), want)
    ctx = i32([700, 64, 1300])
    q = q.contiguous()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    other = gdn.gdn_attn_decode(q, kc, vc, table, ctx, stream=side)
    side.synchronize()
    assert torch.equal(want, other)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = gdn.gdn_attn_decode(q, kc, vc, table, ctx)
    ctx.copy_(i32([64, 700, 1]))
    graph.replay()
    o, bound = ref.decode(q, kc, vc, table.cpu(), [64, 700, 1], 64 ** -0.5, 0)
    ref.within(held, o, bound, "o replayed")


APPEND = [
    # lens (None: one token each), contexts, Hq, Hk, d, page, rot, interleaved, norm
    (None, [0], 1, 1, 64, 16, 64, False, True),
    (None, [5, 0, 31, 16], 4, 2, 128, 16, 64, True, True),
    (None, [3] * 40, 0, 1, 64, 8, 32, False, True),
    ([3, 0, 40, 1], [0, 9, 7, 100], 4, 1, 128, 16, 128, False, True),
    ([130], [0], 3, 3, 64, 24, 48, False, False),
    ([17, 20], [1, 2], 2, 1, 128, 1, 0, False, False),
]


@pytest.mark.parametrize("lens,ctx,Hq,Hk,d,page,rot,il,norm", APPEND)
def test_append(lens, ctx, Hq, Hk, d, page, rot, il, norm):
    N = len(ctx)
    new = lens or [1] * N
    T = sum(new)
    kc, vc, table = cache_for(N, Hk, d, page, [c + n for c, n in zip(ctx, new)])
    q = rnd(T, Hq, d, seed=5) if Hq else None
    k, v = rnd(T, Hk, d, seed=6), rnd(T, Hk, d, seed=7)
    w = (1 + 0.2 * torch.randn(d, generator=torch.Generator().manual_seed(8))).to(BF).cuda()
    cu = None if lens is None else [sum(lens[:i]) for i in range(N + 1)]
    kc0, vc0 = kc.clone(), vc.clone()
    q_out, k_out = gdn.gdn_kv_append(k, v, kc, vc, table, i32(ctx), cu_seqlens=cu, q=q, inv_freq=freqs(rot) if rot else None,
                                     q_norm_w=w if norm and Hq else None, k_norm_w=w if norm else None, interleaved=il,
                                     want_k=True)
    pos = torch.tensor([c + i for c, n in zip(ctx, new) for i in range(n)])
    f = ref.f64(freqs(rot)) if rot else None
    y = ref.norm_rope(ref.f64(k), ref.f64(w) if norm else None, pos, f, interleaved=il)
    bound = lambda y: 3e-6 * 2 ** 0.5 * y.abs().amax(-1, keepdim=True) + ref.U * y.abs()  # as for the rotation's own call
    ref.within(k_out, y, bound(y), "k_out")
    if Hq:
        yq = ref.norm_rope(ref.f64(q), ref.f64(w) if norm else None, pos, f, interleaved=il)
        ref.within(q_out, yq, bound(yq), "q_out")
    # the cache holds k_out and v bit for bit in the tokens' slots, and elsewhere what it held
    at = 0
    for n in range(N):
        for i in range(new[n]):
            p = ctx[n] + i
            page_no = int(table[n, p // page])
            kc0[page_no, p % page], vc0[page_no, p % page] = k_out[at], v[at]
            at += 1
    assert torch.equal(kc, kc0) and torch.equal(vc, vc0)


def test_append_leaves_out_what_has_no_place():
    Hk, d, page = 1, 64, 4
    kc, vc = rnd(5, page, Hk, d), rnd(5, page, Hk, d, seed=1)
    kc0, vc0 = kc.clone(), vc.clone()
    table = i32([[-1, 1], [5, 2], [3, 2 ** 31 - 1]])
    k, v, q = rnd(10, Hk, d, seed=2), rnd(10, Hk, d, seed=3), rnd(10, 2, d, seed=4)
    q_out, k_out = torch.full_like(q, 9.0), torch.full_like(k, 9.0)
    # tokens 0-1 go nowhere (page -1), token 2 is past the second sequence's table, 3-4 fill the third's page 3
    # from slot 2 on, the others belong to no sequence
    gdn.gdn_kv_append(k, v, kc, vc, table, i32([0, 8, 2]), cu_seqlens=i32([0, 2, 3, 5]), q=q, q_out=q_out, k_out=k_out)
    kc0[3, 2:4], vc0[3, 2:4] = k[3:5], v[3:5]
    assert torch.equal(kc, kc0) and torch.equal(vc, vc0)
    assert torch.equal(q_out[:5], q[:5]) and torch.equal(k_out[:5], k[:5])
    assert (q_out[5:] == 9.0).all() and (k_out[5:] == 9.0).all()
    # negative lengths, and cu_seqlens out of order or range
    gdn.gdn_kv_append(k, v, kc, vc, table, i32([-3, -2 ** 31, 2 ** 31 - 1]), cu_seqlens=i32([-9, 100, 3, 5]), q=q, q_out=q_out)
    torch.cuda.synchronize()


def test_append_strided_inputs():
    T, Hq, Hk, d, page = 40, 4, 2, 64, 16
    for shift in (0, 8, 3):
        buf = rnd(T, (Hq + 2 * Hk) * d + 16, seed=2)
        at = [shift, shift + Hq * d, shift + (Hq + Hk) * d]
        q, k, v = (buf[:, a:a + h * d].view(T, h, d) for a, h in zip(at, (Hq, Hk, Hk)))
        runs = []
        for f in (lambda t: t, lambda t: t.contiguous()):
            kc, vc, table = cache_for(1, Hk, d, page, [T])
            out = gdn.gdn_kv_append(f(k), f(v), kc, vc, table, i32([0]), cu_seqlens=[0, T], q=f(q), inv_freq=freqs(32), want_k=True)
            runs.append([kc, vc, *out])
        for a, b in zip(*runs):
            assert torch.equal(a, b)


@pytest.mark.parametrize("window", [0, 50])
def test_serving_loop_matches_attention_over_the_whole_sequence(window):
    """Prompts appended and attended, then tokens one by one: every step's output is the row that
    attention over the whole sequences gives."""
    lens, steps, Hq, Hk, d, page, rot = [37, 1, 130], 4, 4, 2, 128, 16, 64
    N = len(lens)
    whole = [n + steps for n in lens]
    g = torch.Generator().manual_seed(0)
    mk = lambda n, h: torch.randn(n, h, d, generator=g).to(BF).cuda()
    q, k, v = ([mk(n, h) for n in whole] for h in (Hq, Hk, Hk))
    w = (1 + 0.1 * torch.randn(d, generator=g)).to(BF).cuda()
    kw = dict(inv_freq=freqs(rot), q_norm_w=w, k_norm_w=w)
    kc, vc, table = cache_for(N, Hk, d, page, whole)
    ctx = i32([0] * N)
    cu = [sum(lens[:i]) for i in range(N + 1)]
    cat = lambda t, m: torch.cat([x[:n] for x, n in zip(t, m)])
    q0, k0 = gdn.gdn_kv_append(cat(k, lens), cat(v, lens), kc, vc, table, ctx, cu_seqlens=cu, q=cat(q, lens), want_k=True, **kw)
    pos = i32([i for n in lens for i in range(n)])
    q1, k1 = gdn.gdn_qk_norm_rope_fwd(cat(q, lens), cat(k, lens), pos, freqs(rot), q_norm_w=w, k_norm_w=w)
    assert torch.equal(q0, q1) and torch.equal(k0, k1)
    o = gdn.gdn_attn_fwd(q0, k0, cat(v, lens), cu, window=window)
    # the whole sequences at once
    cu2 = [sum(whole[:i]) for i in range(N + 1)]
    pos = i32([i for n in whole for i in range(n)])
    qa, ka = gdn.gdn_qk_norm_rope_fwd(cat(q, whole), cat(k, whole), pos, freqs(rot), q_norm_w=w, k_norm_w=w)
    want, bound = ref.packed(qa, ka, cat(v, whole), cu2, d ** -0.5, window)
    for n in range(N):
        ref.within(o[cu[n]:cu[n + 1]], want[cu2[n]:cu2[n] + lens[n]], bound[cu2[n]:cu2[n] + lens[n]], f"prompt {n}")
    ctx += i32(lens)
    for s in range(steps):
        at = [n + s for n in lens]
        one = lambda t: torch.stack([x[a] for x, a in zip(t, at)])
        qs, _ = gdn.gdn_kv_append(one(k), one(v), kc, vc, table, ctx, q=one(q), **kw)
        ctx += 1
        o = gdn.gdn_attn_decode(qs, kc, vc, table, ctx, window=window)
        rows = [cu2[n] + at[n] for n in range(N)]
        ref.within(o, want[rows], bound[rows], f"step {s}")

"""Per-head norm and rotation of q and k on the GPU, forward and backward, against the plain fp64 form.

Bounds.  fp32: the mean of squares (8 terms in a lane, 4 butterfly steps), the square root, the division,
the weights and the rotation's three operations are each off by at most 2^-24 of their size, the
angle by pi 2^-25 and its cosine and sine by 2 ulp: below 24 * 2^-24 < 2e-6 of the row's largest
entry times sqrt(2); 3e-6 is taken.  bf16 results: that and half a step.  The backward has two such
chains in a row (r twice, the mean of gw x): 6e-6 of r (|g| + |x| r mean |g x| r).  The weights' gradient
adds n terms in fp32: at most sqrt(n) * 2^-24 * 8 of the terms' root sum of squares on average; F
of the sum of magnitudes is taken."""
import pytest
import torch

import attn_ref as ref
from gated_delta_rule_76_b200 import gdn

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
CASES = [
    # T, Hq, Hk, d, rot, interleaved, dtype, norm, first position
    (1, 1, 1, 64, 64, False, "f32", True, 0),
    (1, 1, 1, 128, 16, True, "bf16", True, 0),
    (3, 5, 2, 128, 128, False, "bf16", True, 7),
    (7, 3, 3, 64, 48, False, "bf16", True, 0),
    (33, 4, 1, 128, 96, False, "f32", True, 100),
    (33, 4, 1, 128, 96, True, "f32", True, 100),
    (130, 16, 2, 64, 32, True, "bf16", True, 0),
    (65, 2, 2, 128, 64, False, "f32", False, 0),
    (65, 2, 2, 128, 0, False, "bf16", True, 0),
    (2500, 3, 1, 128, 128, True, "f32", True, 2 ** 31 - 2501),
    (10000, 2, 1, 64, 64, False, "bf16", True, 1000000),
]


def make(T, Hq, Hk, d, rot, dtype, norm, first, seed=0):
    g = torch.Generator().manual_seed(seed)
    mk = lambda *s: torch.randn(*s, generator=g).to(DT[dtype]).cuda()
    x = dict(q=mk(T, Hq, d), k=mk(T, Hk, d), gq=mk(T, Hq, d), gk=mk(T, Hk, d))
    x["qw"] = (1 + 0.2 * torch.randn(d, generator=g)).to(DT[dtype]).cuda() if norm else None
    x["kw"] = (1 + 0.2 * torch.randn(d, generator=g)).to(DT[dtype]).cuda() if norm else None
    x["pos"] = (torch.arange(T) + first).to(torch.int32).cuda() if rot else None
    x["freq"] = (10000.0 ** (-torch.arange(0, rot, 2).double() / rot)).float().cuda() if rot else None
    return x


def host(t):
    return None if t is None else ref.f64(t) if t.is_floating_point() else t.cpu()


def forward_bound(y, dtype, scale=1.0):
    row = y.abs().amax(-1, keepdim=True) * 2 ** 0.5
    return 3e-6 * row + (ref.U * y.abs() if dtype == "bf16" else 0)


@pytest.mark.parametrize("T,Hq,Hk,d,rot,il,dtype,norm,first", CASES)
def test_forward_and_backward(T, Hq, Hk, d, rot, il, dtype, norm, first):
    x = make(T, Hq, Hk, d, rot, dtype, norm, first)
    kw = dict(q_norm_w=x["qw"], k_norm_w=x["kw"], interleaved=il, rot_scale=1.25)
    q, k = gdn.gdn_qk_norm_rope_fwd(x["q"], x["k"], x["pos"], x["freq"], **kw)
    grads = gdn.gdn_qk_norm_rope_bwd(x["q"], x["k"], x["pos"], x["freq"], grad_q=x["gq"], grad_k=x["gk"], **kw)
    for got, t, w, g, name in ((q, "q", "qw", "gq", "q"), (k, "k", "kw", "gk", "k")):
        a = [host(x[n]) for n in (t, w, "pos", "freq")]
        rk = dict(interleaved=il, rot_scale=1.25)
        y = ref.norm_rope(*a, **rk)
        ref.within(got, y, forward_bound(y, dtype), name)
        dx, dw = ref.norm_rope_grad(*a, host(x[g]), **rk)
        gx, xx = host(x[g]).abs() * 1.25 * 2 ** 0.5, a[0].abs()
        if norm:
            r = 1 / torch.sqrt((a[0] ** 2).mean(-1, keepdim=True) + 1e-6)
            wmax = a[1].abs().max()
            mag = r * wmax * (gx.amax(-1, keepdim=True) + xx * r * r * (gx.amax(-1, keepdim=True) * xx).mean(-1, keepdim=True))
        else:
            mag = gx.amax(-1, keepdim=True).expand_as(dx)
        ref.within(grads["d" + name], dx, 6e-6 * mag + (ref.U * dx.abs() if dtype == "bf16" else 0), "d" + name)
        if norm:
            terms = (gx.amax(-1, keepdim=True) * xx * r).sum((0, 1))
            ref.within(grads[f"d{name}_norm_w"], dw, ref.F * terms, f"d{name}_norm_w")
        else:
            assert f"d{name}_norm_w" not in grads


@pytest.mark.parametrize("shift", [0, 8, 3])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_strided_inputs_are_the_dense_ones(shift, dtype):
    T, Hq, Hk, d = 50, 3, 2, 64
    buf = torch.randn(T, (Hq + Hk) * d + 16, generator=torch.Generator().manual_seed(1)).to(DT[dtype]).cuda()
    q = buf[:, shift:shift + Hq * d].view(T, Hq, d)
    k = buf[:, shift + Hq * d:shift + (Hq + Hk) * d].view(T, Hk, d)
    x = make(T, Hq, Hk, d, 32, dtype, True, 5)
    kw = dict(q_norm_w=x["qw"], k_norm_w=x["kw"])
    a = gdn.gdn_qk_norm_rope_fwd(q, k, x["pos"], x["freq"], **kw)
    b = gdn.gdn_qk_norm_rope_fwd(q.contiguous(), k.contiguous(), x["pos"], x["freq"], **kw)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    ga = gdn.gdn_qk_norm_rope_bwd(q, k, x["pos"], x["freq"], grad_q=x["gq"], grad_k=x["gk"], **kw)
    gb = gdn.gdn_qk_norm_rope_bwd(q.contiguous(), k.contiguous(), x["pos"], x["freq"], grad_q=x["gq"], grad_k=x["gk"], **kw)
    for n in ga:
        assert torch.equal(ga[n], gb[n]), n


def test_q_alone_one_norm_and_no_tokens():
    x = make(20, 4, 1, 64, 32, "bf16", True, 0)
    both = gdn.gdn_qk_norm_rope_fwd(x["q"], x["k"], x["pos"], x["freq"], q_norm_w=x["qw"])
    alone, none = gdn.gdn_qk_norm_rope_fwd(x["q"], None, x["pos"], x["freq"], q_norm_w=x["qw"])
    assert none is None and torch.equal(both[0], alone)
    y = ref.norm_rope(host(x["k"]), None, host(x["pos"]), host(x["freq"]))
    ref.within(both[1], y, forward_bound(y, "bf16"), "k without a norm")
    g = gdn.gdn_qk_norm_rope_bwd(x["q"], None, x["pos"], x["freq"], grad_q=x["gq"], q_norm_w=x["qw"])
    assert set(g) == {"dq", "dq_norm_w"}
    e = {n: (t[:0].contiguous() if n in ("q", "k", "gq", "gk", "pos") else t) for n, t in x.items()}
    q, k = gdn.gdn_qk_norm_rope_fwd(e["q"], e["k"], e["pos"], e["freq"], q_norm_w=x["qw"], k_norm_w=x["kw"])
    assert q.shape == (0, 4, 64) and k.shape == (0, 1, 64)
    g = gdn.gdn_qk_norm_rope_bwd(e["q"], e["k"], e["pos"], e["freq"], grad_q=e["gq"], grad_k=e["gk"], q_norm_w=x["qw"],
                                 k_norm_w=x["kw"])
    assert not g["dq_norm_w"].any() and not g["dk_norm_w"].any()


def test_special_values_stay_in_their_row():
    x = make(9, 2, 1, 64, 32, "f32", True, 0)
    want = gdn.gdn_qk_norm_rope_fwd(x["q"], x["k"], x["pos"], x["freq"], q_norm_w=x["qw"], k_norm_w=x["kw"])
    x["q"][4, 1, 7] = float("nan")
    x["q"][5, 0] = 0
    got = gdn.gdn_qk_norm_rope_fwd(x["q"], x["k"], x["pos"], x["freq"], q_norm_w=x["qw"], k_norm_w=x["kw"])
    keep = torch.ones(9, 2, dtype=torch.bool)
    keep[4, 1] = keep[5, 0] = False
    assert torch.equal(got[0][keep], want[0][keep]) and torch.equal(got[1], want[1])
    assert torch.isnan(got[0][4, 1]).all() and not got[0][5, 0].any()


def test_same_bits_again_and_in_a_graph():
    x = make(777, 6, 2, 128, 64, "bf16", True, 3)
    kw = dict(q_norm_w=x["qw"], k_norm_w=x["kw"])

    def step():
        return list(gdn.gdn_qk_norm_rope_fwd(x["q"], x["k"], x["pos"], x["freq"], **kw)) + list(
            gdn.gdn_qk_norm_rope_bwd(x["q"], x["k"], x["pos"], x["freq"], grad_q=x["gq"], grad_k=x["gk"], **kw).values())

    want = step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    graph.replay()
    for a, b, c in zip(want, held, step()):
        assert torch.equal(a, b) and torch.equal(a, c)

"""A row's result depends on its own query and the keys it sees alone, bit for bit: not on the rows that share its
warp, whether they are padding, the next sequence's, later tokens of its own or other heads of its group.

The running reference of a row's softmax is what could carry such a dependence: p is rounded to bf16 against it.  The
inputs below make the other rows' maximum jump in a key tile after their first, while the row's own does not."""
import pytest
import torch

from gated_delta_rule_76_b200 import gdn

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


def rnd(*s, seed=0):
    return torch.randn(*s, generator=torch.Generator().manual_seed(seed)).to(BF).cuda()


def jump(q, k, rows, heads):
    """q with `rows` of the heads along one early key: their scores there outgrow all the others."""
    q = q.clone()
    q[rows, heads] = (60 * k[10, 0].float()).to(BF)
    return q


# tokens of the sequence that is looked at, tokens behind it, Hq, Hk, d, window
FORWARD = [
    (300, 40, 2, 1, 128, 0),     # two heads a unit
    (300, 40, 3, 1, 64, 0),      # two tiles of one head
    (300, 40, 2, 1, 64, 295),
    (1790, 30, 2, 1, 128, 0),    # a unit's keys in parts
    (1790, 30, 3, 3, 64, 0),
]


@pytest.mark.parametrize("n,behind,Hq,Hk,d,window", FORWARD)
@pytest.mark.parametrize("sequence", [False, True])
def test_forward_and_backward_rows_do_not_see_what_lies_behind(n, behind, Hq, Hk, d, window, sequence):
    T = n + behind
    q, k, v, do = (rnd(T, h, d, seed=s) for s, h in enumerate((Hq, Hk, Hk, Hq)))
    cu = torch.tensor([0, n, T] if sequence else [0, n, n], dtype=torch.int32, device="cuda")

    def step(q):
        cache = torch.empty(gdn.gdn_attn_fwd_cache_size(q, k, v, cu), dtype=torch.uint8, device="cuda")
        o = torch.zeros_like(q)
        gdn.gdn_attn_fwd(q, k, v, cu, window=window, o=o, bwd_cache=cache)
        plain = torch.zeros_like(q)
        gdn.gdn_attn_fwd(q, k, v, cu, window=window, o=plain)
        g = gdn.gdn_attn_bwd(q, k, v, cu, o, grad_o=do, fwd_cache=cache, window=window)
        return [o[:n], plain[:n], *(g[x][:n] for x in ("dq", "dk", "dv"))]

    for a, b in zip(step(q), step(jump(q, k, slice(n, T), slice(None)))):
        assert torch.equal(a, b)


@pytest.mark.parametrize("n,behind,Hq,Hk,d,window", FORWARD)
def test_forward_rows_do_not_see_later_queries(n, behind, Hq, Hk, d, window):
    q, k, v = (rnd(n, h, d, seed=s) for s, h in enumerate((Hq, Hk, Hk)))
    at = n - 8
    a = gdn.gdn_attn_fwd(q, k, v, [0, n], window=window)
    b = gdn.gdn_attn_fwd(jump(q, k, slice(at, n), slice(None)), k, v, [0, n], window=window)
    assert torch.equal(a[:at], b[:at])
    assert not torch.equal(a[at:], b[at:])


@pytest.mark.parametrize("Hq,Hk,d,page", [(4, 1, 64, 16), (8, 2, 128, 16), (16, 1, 128, 64), (4, 1, 128, 24)])
def test_decode_heads_do_not_see_one_another(Hq, Hk, d, page):
    """Eight sequences of 1500 tokens: chunks of 128, two tiles a warp."""
    N, ctx, G = 8, 1500, Hq // Hk
    pages = -(-ctx // page)
    kc, vc = rnd(N * pages, page, Hk, d, seed=1), rnd(N * pages, page, Hk, d, seed=2)
    table = torch.arange(N * pages, dtype=torch.int32, device="cuda").view(N, pages)
    lens = torch.full((N,), ctx, dtype=torch.int32, device="cuda")
    q = rnd(N, Hq, d, seed=3)
    other = q.clone()
    other.view(N, Hk, G, d)[:, :, 1:] *= 30
    a, b = (gdn.gdn_attn_decode(x, kc, vc, table, lens).view(N, Hk, G, d) for x in (q, other))
    assert torch.equal(a[:, :, 0], b[:, :, 0])
    assert not torch.equal(a[:, :, 1:], b[:, :, 1:])

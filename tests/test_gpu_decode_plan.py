"""Decode attention where its plan leaves the usual chunk lengths: the cap of 512 tokens a chunk, chunks stretched because
the partial results are bounded at 64 MB, and block tables far wider than the contexts.  A sample of rows is compared
with the fp64 form."""
import ctypes

import pytest
import torch

import attn_ref as ref
from gated_delta_rule_76_b200 import gdn

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def part_bytes(N, Hq, Hk, d, page, max_pages, window):
    a = gdn.AttnDecodeArgs(N=N, Hq=Hq, Hk=Hk, d=d, num_pages=8, page_size=page, max_pages=max_pages, window=window, scale=0.1)
    return gdn.load().gdn_attn_decode_workspace_size(ctypes.byref(a))


# N, Hq, Hk, d, page, the table's reach, the long contexts (the others: 1 to 90 tokens), window, splits the plan is to make
PLANS = [
    (256, 8, 2, 64, 16, 5000, {0: 5000, 100: 4097, 255: 512}, 0, 10),            # chunks of 512, the cap
    (64, 64, 8, 64, 16, 20000, {3: 20000, 40: 9999, 63: 1}, 0, 29),             # stretched to 704 tokens
    (64, 64, 8, 64, 16, 20000, {3: 20000, 40: 9999, 63: 1}, 3000, 6),           # a window: its reach is what counts
    (2, 16, 2, 128, 16, 131072, {0: 8191, 1: 600}, 0, None),                    # a wide table
    (2, 16, 2, 128, 24, 131072, {0: 8191, 1: 600}, 100, None),
]


@pytest.mark.parametrize("N,Hq,Hk,d,page,reach,long,window,splits", PLANS)
def test_unusual_plans(N, Hq, Hk, d, page, reach, long, window, splits):
    g = torch.Generator().manual_seed(0)
    max_pages = -(-reach // page)
    ctx = torch.randint(1, 91, (N,), generator=g).tolist()
    for n, c in long.items():
        ctx[n] = c
    need = [-(-c // page) for c in ctx]
    ids = torch.randperm(sum(need), generator=g).tolist()
    table = torch.full((N, max_pages), -1, dtype=torch.int32)
    for n in range(N):
        for j in range(need[n]):
            table[n, j] = ids.pop()
    kc, vc = (torch.randn(sum(need), page, Hk, d, generator=g).to(BF).cuda() for _ in range(2))
    q = torch.randn(N, Hq, d, generator=g).to(BF).cuda()
    if splits is not None:
        assert part_bytes(N, Hq, Hk, d, page, max_pages, window) == -(-splits * N * Hq * (d + 2) * 4 // 256) * 256
    o = gdn.gdn_attn_decode(q, kc, vc, table.cuda(), i32(ctx), window=window)
    assert torch.isfinite(o.float()).all()
    rows = sorted({*long, 1, N // 2})
    rows = [r for r in rows if r < N]
    heads = sorted({0, 1, Hq // Hk, Hq - 1})
    for n in rows:
        for h in heads:
            hk = h // (Hq // Hk)
            want, bound = ref.decode(q[n:n + 1, h:h + 1], kc[:, :, hk:hk + 1], vc[:, :, hk:hk + 1], table[n:n + 1], [ctx[n]],
                                     d ** -0.5, window)
            ref.within(o[n:n + 1, h:h + 1], want, bound, f"sequence {n}, head {h}")
    # a bound on the contexts makes another plan over the same rows
    p = gdn.gdn_attn_decode(q, kc, vc, table.cuda(), i32(ctx), window=window, max_context=max(ctx))
    lim = (2 * ref.U + 1e-3) * vc.float().abs().max()  # two bf16 results of sums whose weights add up to 1
    assert ((o.float() - p.float()).abs() <= lim).all()

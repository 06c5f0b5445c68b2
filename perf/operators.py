"""The softmax-attention operators of hybrid gated-delta-rule stacks, as cases to be measured.

Four operators, each with its plain form (elementary torch operations in fp32, rounded once) and the
calls a user makes of this library:

  qk      per-head RMS norm of q and k with the rotation by position (forward; training: its backward)
  attn    causal attention over packed sequences, grouped heads, optional window (forward; training)
  append  keys and values of new tokens into a paged cache, normalised and rotated on the way
  decode  one query token per sequence over that cache

Head counts, widths and lengths are those of this library's own workloads (16 heads of 128 over
8 x 4096 tokens, 128 value heads over 16 key heads and 16384 tokens, 256 sequences of decode, heads of
64) and odd sizes between them.
"""
import math

import torch

own = False

BF16, F32 = "bf16", "f32"
EPS = 1e-6


# ---------------------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------------------
def listed():
    return [
        # the smallest call: q and k of two tokens of a small fp32 model, half of each head rotated
        dict(name="qk_two_tokens_f32", op="qk", train=False, T=2, Hq=2, Hk=2, d=64, rot=32, interleaved=False, dtype=F32, far=0,
             fused=False),
        # a training step's q and k: 8 sequences of 4096 tokens, 16 query heads over 4 key heads, half of each head rotated
        dict(name="qk_train_32k", op="qk", train=True, T=32768, Hq=16, Hk=4, d=128, rot=64, interleaved=False, dtype=BF16, far=0,
             fused=False),
        # a long prompt of the wide layer, far positions, whole heads in interleaved pairs, read as slices of the fused projection
        dict(name="qk_prompt_far_fused", op="qk", train=False, T=4099, Hq=128, Hk=16, d=128, rot=128, interleaved=True, dtype=BF16,
             far=1000000, fused=True),
        # a few short prompts: latency
        dict(name="attn_short_prompts", op="attn", train=False, lens="1,5,77,64,130", Hq=16, Hk=16, d=64, window=0),
        # ordinary prompts of different lengths, 8 query heads a key head
        dict(name="attn_ragged_prompts", op="attn", train=False, lens="1777,33,2500,129,640,1021,1,2091", Hq=16, Hk=2, d=128,
             window=0),
        # the longest context of the library's workloads
        dict(name="attn_prompt_16k", op="attn", train=False, lens="16384", Hq=8, Hk=1, d=128, window=0),
        # training: forward and gradients over four sequences
        dict(name="attn_train_4x2048", op="attn", train=True, lens="2048,2048,2048,2048", Hq=16, Hk=4, d=128, window=0),
        # training of a windowed layer on packed documents, heads of 64
        dict(name="attn_train_window", op="attn", train=True, lens="3001,511,64,2500,1,999", Hq=8, Hk=4, d=64, window=512),
        # a serving step's new tokens: 256 sequences
        dict(name="append_step_256", op="append", lens="", N=256, Hq=16, Hk=4, d=128, rot=64, interleaved=False, page=16, ctx=500),
        # prompts entering the cache
        dict(name="append_prompts", op="append", lens="4000,13,2047,1,1500", N=5, Hq=16, Hk=4, d=128, rot=128, interleaved=False,
             page=64, ctx=700),
        # one sequence answered alone: latency
        dict(name="decode_one_8k", op="decode", N=1, Hq=16, Hk=2, d=128, page=64, lo=8191, hi=8191, window=0),
        # a full batch of different lengths
        dict(name="decode_batch_256", op="decode", N=256, Hq=16, Hk=2, d=128, page=16, lo=64, hi=4500, window=0),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["qk", "attn", "attn", "append", "decode"])
    d = rng.choice([64, 128])
    Hk = rng.choice([1, 2, 3, 4, 8])
    G = rng.choice([1, 2, 4, 5, 8])
    Hq = Hk * G
    rot = 16 * rng.randint(1, d // 16)
    if op == "qk":
        T = min(_log(rng, 1, 32768), 32768 * 20 * 128 // ((Hq + Hk) * d))
        return dict(op=op, train=rng.random() < 0.5, T=T, Hq=Hq, Hk=Hk, d=d, rot=rot, interleaved=rng.random() < 0.5,
                    dtype=rng.choice([BF16, BF16, F32]), far=rng.choice([0, 100000]), fused=rng.random() < 0.5)
    if op == "attn":
        lens = [_log(rng, 1, 2600) for _ in range(rng.randint(1, 5))]
        while sum(lens) > 6000:  # the plain form looks at every pair of the batch
            lens.pop()
        return dict(op=op, train=rng.random() < 0.5, lens=",".join(map(str, lens)), Hq=min(Hq, 16) // Hk * Hk, Hk=Hk, d=d,
                    window=rng.choice([0, 0, _log(rng, 1, 2000)]))
    if op == "append":
        N = _log(rng, 1, 300)
        lens = "" if rng.random() < 0.5 else ",".join(str(_log(rng, 1, 900)) for _ in range(min(N, 8)))
        return dict(op=op, lens=lens, N=len(lens.split(",")) if lens else N, Hq=Hq, Hk=Hk, d=d, rot=rot,
                    interleaved=rng.random() < 0.5, page=rng.choice([8, 16, 24, 64, 128]), ctx=_log(rng, 1, 600))
    hi = _log(rng, 1, 9000)
    N = _log(rng, 1, max(1, min(256, 256 * 4500 * 2 // (hi * Hk))))
    return dict(op=op, N=N, Hq=Hq, Hk=Hk, d=d, page=rng.choice([8, 16, 24, 64, 128]), lo=rng.randint(1, hi), hi=hi,
                window=rng.choice([0, 0, _log(rng, 1, 3000)]))


# ---------------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------------
def _lens(case):
    return [int(x) for x in case["lens"].split(",")] if case.get("lens") else []


def _cu(lens):
    return [sum(lens[:i]) for i in range(len(lens) + 1)]


def _contexts(case, seed):
    """Lengths of the decoded sequences: spread evenly over the logarithm from `lo` to `hi`, in an order that the seed gives."""
    lo, hi, n = case["lo"], case["hi"], case["N"]
    lens = [int(round(hi * (lo / hi) ** (i / max(1, n - 1)))) for i in range(n)]
    order = torch.randperm(n, generator=torch.Generator().manual_seed(seed)).tolist()
    return [lens[i] for i in order]


def prepare(case, seed):
    dev = "cuda"
    g = torch.Generator(device=dev).manual_seed(seed)
    dt = torch.float32 if case.get("dtype") == F32 else torch.bfloat16

    def randn(*shape, dtype=dt):
        return torch.randn(*shape, generator=g, device=dev).to(dtype)

    def freqs(rot):
        # rotary base 10000, as every second channel of the rotated part
        return (10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)).float().to(dev)

    def norm_w(d):
        return (1 + 0.1 * torch.randn(d, generator=g, device=dev)).to(dt)

    op, Hq, Hk, d = case["op"], case["Hq"], case["Hk"], case["d"]
    s = dict(case=case)
    if op == "qk":
        T = case["T"]
        if case["fused"]:  # slices of one projection buffer
            qkv = randn(T, (Hq + 2 * Hk) * d)
            s["q"] = qkv[:, :Hq * d].view(T, Hq, d)
            s["k"] = qkv[:, Hq * d:(Hq + Hk) * d].view(T, Hk, d)
        else:
            s["q"], s["k"] = randn(T, Hq, d), randn(T, Hk, d)
        s["positions"] = (torch.arange(T, device=dev) % 4096 + case["far"]).to(torch.int32)
        s["inv_freq"], s["q_w"], s["k_w"] = freqs(case["rot"]), norm_w(d), norm_w(d)
        if case["train"]:
            s["gq"], s["gk"] = randn(T, Hq, d), randn(T, Hk, d)
    elif op == "attn":
        lens = _lens(case)
        T = sum(lens)
        s["q"], s["k"], s["v"] = randn(T, Hq, d), randn(T, Hk, d), randn(T, Hk, d)
        s["cu"] = torch.tensor(_cu(lens), dtype=torch.int32, device=dev)
        if case["train"]:
            s["do"] = randn(T, Hq, d)
    elif op == "append":
        lens, N, page = _lens(case), case["N"], case["page"]
        T = sum(lens) if lens else N
        s["q"], s["k"], s["v"] = randn(T, Hq, d), randn(T, Hk, d), randn(T, Hk, d)
        s["ctx"] = torch.randint(0, case["ctx"] + 1, (N,), generator=g, device=dev).to(torch.int32)
        most = -(-(case["ctx"] + (max(lens) if lens else 1)) // page)
        s["table"] = torch.randperm(N * most, generator=g, device=dev).to(torch.int32).view(N, most)
        s["kc"], s["vc"] = (torch.zeros(N * most, page, Hk, d, dtype=dt, device=dev) for _ in range(2))
        s["cu"] = torch.tensor(_cu(lens), dtype=torch.int32, device=dev) if lens else None
        s["inv_freq"], s["q_w"], s["k_w"] = freqs(case["rot"]), norm_w(d), norm_w(d)
    else:
        N, page = case["N"], case["page"]
        lens = _contexts(case, seed)
        need = [-(-n // page) for n in lens]
        most = max(need)
        total = sum(need)
        ids = torch.randperm(total, generator=g, device=dev).to(torch.int32)
        at = torch.tensor(_cu(need), device=dev)
        col = torch.arange(most, device=dev)
        have = col[None, :] < (at[1:] - at[:-1])[:, None]
        s["table"] = torch.where(have, ids[(at[:-1, None] + col[None, :]).clamp(max=total - 1)], 0).contiguous()
        s["ctx"] = torch.tensor(lens, dtype=torch.int32, device=dev)
        s["q"] = randn(N, Hq, d)
        s["kc"], s["vc"] = randn(total, page, Hk, d), randn(total, page, Hk, d)
    return s


# ---------------------------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------------------------
def run(state):
    case = state["case"]
    if own:
        return _OWN[case["op"]](state, case)
    return _PLAIN[case["op"]](state, case)


# ---- the library's calls ------------------------------------------------------------------------
def _own_qk(s, case):
    from gated_delta_rule_76_b200 import gdn
    kw = dict(q_norm_w=s["q_w"], k_norm_w=s["k_w"], norm_eps=EPS, interleaved=case["interleaved"])
    q, k = gdn.gdn_qk_norm_rope_fwd(s["q"], s["k"], s["positions"], s["inv_freq"], **kw)
    if not case["train"]:
        return [q, k]
    r = gdn.gdn_qk_norm_rope_bwd(s["q"], s["k"], s["positions"], s["inv_freq"], grad_q=s["gq"], grad_k=s["gk"], **kw)
    return [q, k, r["dq"], r["dk"], r["dq_norm_w"], r["dk_norm_w"]]


def _own_attn(s, case):
    from gated_delta_rule_76_b200 import gdn
    q, k, v, cu, w = s["q"], s["k"], s["v"], s["cu"], case["window"]
    if not case["train"]:
        return [gdn.gdn_attn_fwd(q, k, v, cu, window=w)]
    cache = torch.empty(gdn.gdn_attn_fwd_cache_size(q, k, v, cu), dtype=torch.uint8, device=q.device)
    o = gdn.gdn_attn_fwd(q, k, v, cu, window=w, bwd_cache=cache)
    r = gdn.gdn_attn_bwd(q, k, v, cu, o, grad_o=s["do"], fwd_cache=cache, window=w)
    return [o, r["dq"], r["dk"], r["dv"]]


def _own_append(s, case):
    from gated_delta_rule_76_b200 import gdn
    q, k = gdn.gdn_kv_append(s["k"], s["v"], s["kc"], s["vc"], s["table"], s["ctx"], cu_seqlens=s["cu"], q=s["q"],
                             inv_freq=s["inv_freq"], q_norm_w=s["q_w"], k_norm_w=s["k_w"], norm_eps=EPS,
                             interleaved=case["interleaved"], want_k=bool(case["lens"]))
    return [q, s["kc"], s["vc"]] + ([k] if case["lens"] else [])


def _own_decode(s, case):
    from gated_delta_rule_76_b200 import gdn
    return [gdn.gdn_attn_decode(s["q"], s["kc"], s["vc"], s["table"], s["ctx"], window=case["window"])]


_OWN = {"qk": _own_qk, "attn": _own_attn, "append": _own_append, "decode": _own_decode}


# ---- the plain forms ------------------------------------------------------------------------------
def _angles(positions, inv_freq):
    """cos and sin [T, 1, rot/2]: far positions need the product in 64 bits."""
    a = positions.double()[:, None, None] * inv_freq.double()
    return a.cos().float(), a.sin().float()


def _rotate(x, c, s, interleaved):
    """The first 2 * c.shape[-1] channels of x rotated."""
    h = c.shape[-1]
    if interleaved:
        a, b = x[..., 0:2 * h:2], x[..., 1:2 * h:2]
        y = torch.stack((a * c - b * s, b * c + a * s), -1).flatten(-2)
    else:
        a, b = x[..., :h], x[..., h:2 * h]
        y = torch.cat((a * c - b * s, b * c + a * s), -1)
    return torch.cat((y, x[..., 2 * h:]), -1)


def _norm_rope(x, w, c, s, interleaved):
    xf = x.float()
    n = xf * torch.rsqrt((xf * xf).mean(-1, keepdim=True) + EPS) * w.float()
    return _rotate(n, c, s, interleaved).to(x.dtype)


def _norm_rope_grad(x, w, g, c, s, interleaved):
    xf = x.float()
    r = torch.rsqrt((xf * xf).mean(-1, keepdim=True) + EPS)
    gn = _rotate(g.float(), c, -s, interleaved)  # the rotation's transpose
    dw = (gn * xf * r).sum((0, 1), dtype=torch.float64).float()
    gw = gn * w.float()
    return (r * (gw - xf * r * r * (gw * xf).mean(-1, keepdim=True))).to(x.dtype), dw


def _plain_qk(s, case):
    c, sn = _angles(s["positions"], s["inv_freq"])
    il = case["interleaved"]
    out = [_norm_rope(s["q"], s["q_w"], c, sn, il), _norm_rope(s["k"], s["k_w"], c, sn, il)]
    if not case["train"]:
        return out
    dq, dqw = _norm_rope_grad(s["q"], s["q_w"], s["gq"], c, sn, il)
    dk, dkw = _norm_rope_grad(s["k"], s["k_w"], s["gk"], c, sn, il)
    return out + [dq, dk, dqw, dkw]


def _grouped(x, Hk):
    """[T, Hk * G, d] -> fp32 [Hk, G * T, d]"""
    T, H, d = x.shape
    return x.float().view(T, Hk, H // Hk, d).permute(1, 2, 0, 3).reshape(Hk, -1, d)


def _ungrouped(x, T, dtype):
    Hk, GT, d = x.shape
    return x.view(Hk, GT // T, T, d).permute(2, 0, 1, 3).reshape(T, -1, d).to(dtype)


def _plain_attn(s, case):
    q, k, v = s["q"], s["k"], s["v"]
    T, Hk, d = k.shape
    G, scale = q.shape[1] // Hk, d ** -0.5
    t = torch.arange(T, device=q.device)
    seq = torch.bucketize(t, s["cu"][1:].long(), right=True)
    hide = (seq[:, None] != seq[None, :]) | (t[None, :] > t[:, None])
    if case["window"]:
        hide |= t[None, :] <= t[:, None] - case["window"]
    qg, kf, vf = _grouped(q, Hk), k.float().transpose(0, 1), v.float().transpose(0, 1)
    p = (qg @ kf.transpose(1, 2)).mul_(scale).view(Hk, G, T, T).masked_fill_(hide, float("-inf"))
    p = p.sub_(p.amax(-1, keepdim=True)).exp_()
    p = p.div_(p.sum(-1, keepdim=True)).view(Hk, G * T, T)
    o = _ungrouped(p @ vf, T, q.dtype)
    if not case["train"]:
        return [o]
    dog = _grouped(s["do"], Hk)
    dv = p.transpose(1, 2) @ dog
    ds = dog @ vf.transpose(1, 2)
    ds = ds.sub_((ds * p).sum(-1, keepdim=True)).mul_(p).mul_(scale)
    dq, dk = ds @ kf, ds.transpose(1, 2) @ qg
    return [o, _ungrouped(dq, T, q.dtype)] + [x.transpose(0, 1).to(k.dtype).contiguous() for x in (dk, dv)]


def _plain_append(s, case):
    T, (N, most), page, dev = s["k"].shape[0], s["table"].shape, case["page"], s["k"].device
    t = torch.arange(T, device=dev)
    if s["cu"] is None:
        seq, i = t, torch.zeros_like(t)
    else:
        seq = torch.bucketize(t, s["cu"][1:].long(), right=True)
        i = t - s["cu"].long()[seq]
    pos = s["ctx"].long()[seq] + i
    c, sn = _angles(pos, s["inv_freq"])
    q = _norm_rope(s["q"], s["q_w"], c, sn, case["interleaved"])
    k = _norm_rope(s["k"], s["k_w"], c, sn, case["interleaved"])
    slot = s["table"].long()[seq, pos // page] * page + pos % page
    s["kc"].view(-1, *k.shape[1:])[slot] = k
    s["vc"].view(-1, *k.shape[1:])[slot] = s["v"]
    return [q, s["kc"], s["vc"]] + ([k] if case["lens"] else [])


def _plain_decode(s, case):
    q, ctx, page = s["q"], s["ctx"].long(), case["page"]
    N, Hq, d = q.shape
    Hk = s["kc"].shape[2]
    j = torch.arange(s["table"].shape[1] * page, device=q.device)
    slot = s["table"].long()[:, j // page] * page + j % page
    hide = j[None, :] >= ctx[:, None]
    if case["window"]:
        hide |= j[None, :] < ctx[:, None] - case["window"]
    k = s["kc"].view(-1, Hk, d)[slot].float().transpose(1, 2)  # [N, Hk, L, d]
    v = s["vc"].view(-1, Hk, d)[slot].float().transpose(1, 2)
    x = (q.float().view(N, Hk, Hq // Hk, d) @ k.transpose(2, 3)) * d ** -0.5
    x = x.masked_fill(hide[:, None, None, :], float("-inf"))
    p = (x - x.amax(-1, keepdim=True)).exp()
    p = p / p.sum(-1, keepdim=True)
    return [(p @ v).view(N, Hq, d).to(q.dtype)]


_PLAIN = {"qk": _plain_qk, "attn": _plain_attn, "append": _plain_append, "decode": _plain_decode}


# ---------------------------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------------------------
def _pairs(n, w):
    """(query, key) pairs of a causal sequence of n tokens, window w (0: none)."""
    if not w or w >= n:
        return n * (n + 1) // 2
    return w * (w + 1) // 2 + (n - w) * w


def work(case):
    op, Hq, Hk, d = case["op"], case["Hq"], case["Hk"], case["d"]
    if op == "qk":
        es, n = (4 if case["dtype"] == F32 else 2), case["T"] * (Hq + Hk) * d
        once = n * es * 2 + case["T"] * 4
        return {"bytes": once + (n * es * 3 + case["T"] * 4 + 8 * d if case["train"] else 0), "flops": n * (25 if case["train"] else 10)}
    if op == "attn":
        lens = _lens(case)
        T, pairs = sum(lens), sum(_pairs(n, case["window"]) for n in lens)
        qb, kb = T * Hq * d * 2, T * Hk * d * 2
        fwd = {"bytes": 2 * qb + 2 * kb, "flops": 4 * d * Hq * pairs}
        if not case["train"]:
            return fwd
        # forward, then q, k, v, o, do read and dq, dk, dv written: five products of the forward's two
        return {"bytes": fwd["bytes"] + 4 * qb + 4 * kb, "flops": 14 * d * Hq * pairs}
    if op == "append":
        T = sum(_lens(case)) or case["N"]
        n = T * (2 * Hq + 4 * Hk + (Hk if case["lens"] else 0)) * d
        return {"bytes": 2 * n, "flops": 10 * T * (Hq + Hk) * d}
    seen = [min(n, case["window"] or n) for n in _contexts(case, 1)]
    return {"bytes": sum(seen) * Hk * d * 4 + case["N"] * Hq * d * 4, "flops": 4 * d * Hq * sum(seen)}


# ---------------------------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------------------------
def _exact_rope(x, w, pos, f, interleaved, rot):
    """RMS norm and rotation of [T, H, d] by complex multiplication."""
    x = x.double()
    n = x / ((x ** 2).sum(-1, keepdim=True) / x.shape[-1] + EPS).sqrt() * w.double()
    turn = torch.polar(torch.ones_like(pos.double())[:, None].expand(-1, rot // 2).contiguous(), pos.double()[:, None] * f.double())[:, None, :]
    first = slice(0, rot, 2) if interleaved else slice(0, rot // 2)
    second = slice(1, rot, 2) if interleaved else slice(rot // 2, rot)
    z = torch.complex(n[..., first].contiguous(), n[..., second].contiguous()) * turn
    y = n.clone()
    y[..., first], y[..., second] = z.real, z.imag
    return y


def _exact_rows(q, k, v, scale, window, do=None):
    """One head of one sequence, [n, d] each: o, and with `do` the gradients."""
    n = q.shape[0]
    i = torch.arange(n, device=q.device)
    see = i[:, None] >= i[None, :]
    if window:
        see &= i[:, None] - i[None, :] < window
    x = torch.where(see, scale * (q @ k.T), -math.inf)
    p = torch.exp(x - torch.logsumexp(x, 1, keepdim=True))
    o = p @ v
    if do is None:
        return o, None, None, None
    ds = p * (do @ v.T - (do * o).sum(1, keepdim=True))
    return o, scale * ds @ k, scale * ds.T @ q, p.T @ do


def exact(case, seed):
    s = prepare(case, seed)
    op, Hq, Hk, d = case["op"], case["Hq"], case["Hk"], case["d"]
    G = Hq // Hk
    if op == "qk":
        pos, f, args = s["positions"], s["inv_freq"], (case["interleaved"], case["rot"])
        if not case["train"]:
            return [_exact_rope(s["q"], s["q_w"], pos, f, *args), _exact_rope(s["k"], s["k_w"], pos, f, *args)]
        out, dx, dw = [], [], []
        for x, w, g in ((s["q"], s["q_w"], s["gq"]), (s["k"], s["k_w"], s["gk"])):
            x, w = x.double().requires_grad_(), w.double().requires_grad_()
            y = _exact_rope(x, w, pos, f, *args)
            gx, gw = torch.autograd.grad(y, (x, w), g.double())
            out.append(y.detach())
            dx.append(gx)
            dw.append(gw)
        return out + dx + dw
    if op == "attn":
        q, k, v = s["q"].double(), s["k"].double(), s["v"].double()
        do = s["do"].double() if case["train"] else None
        o, dq, dk, dv = torch.zeros_like(q), torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
        a = 0
        for n in _lens(case):
            r = slice(a, a + n)
            for h in range(Hq):
                y = _exact_rows(q[r, h], k[r, h // G], v[r, h // G], d ** -0.5, case["window"], None if do is None else do[r, h])
                o[r, h] = y[0]
                if do is not None:
                    dq[r, h] = y[1]
                    dk[r, h // G] += y[2]
                    dv[r, h // G] += y[3]
            a += n
        return [o, dq, dk, dv] if do is not None else [o]
    if op == "append":
        lens = _lens(case) or [1] * case["N"]
        ctx, table, page = s["ctx"].tolist(), s["table"].tolist(), case["page"]
        pos = [ctx[n] + i for n, m in enumerate(lens) for i in range(m)]
        slot = [table[n][(ctx[n] + i) // page] * page + (ctx[n] + i) % page for n, m in enumerate(lens) for i in range(m)]
        p, at = torch.tensor(pos, device="cuda"), torch.tensor(slot, device="cuda")
        q = _exact_rope(s["q"], s["q_w"], p, s["inv_freq"], case["interleaved"], case["rot"])
        k = _exact_rope(s["k"], s["k_w"], p, s["inv_freq"], case["interleaved"], case["rot"])
        kc, vc = s["kc"].double(), s["vc"].double()
        kc.view(-1, Hk, d).index_copy_(0, at, k)
        vc.view(-1, Hk, d).index_copy_(0, at, s["v"].double())
        return [q, kc, vc] + ([k] if case["lens"] else [])
    o = torch.zeros(case["N"], Hq, d, dtype=torch.float64, device="cuda")
    for n, m in enumerate(_contexts(case, seed)):
        pages = s["table"][n, :-(-m // case["page"])].long()
        first = max(0, m - case["window"]) if case["window"] else 0
        k = s["kc"][pages].flatten(0, 1)[first:m].double()
        v = s["vc"][pages].flatten(0, 1)[first:m].double()
        x = torch.einsum("hgd,lhd->hgl", s["q"][n].double().view(Hk, G, d), k) * d ** -0.5
        o[n] = torch.einsum("hgl,lhd->hgd", torch.softmax(x, -1), v).reshape(Hq, d)
    return [o]

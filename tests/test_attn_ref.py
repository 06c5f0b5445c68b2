"""The tests' plain fp64 forms of the softmax-attention layer, pinned to mathematics: gradients
against central differences, rotations against complex multiplication, closed forms.  CPU only."""
import math

import pytest
import torch

import attn_ref as ref


def _rand(*s, seed=0):
    return torch.randn(*s, generator=torch.Generator().manual_seed(seed), dtype=torch.float64)


def differences(f, x, g, h=1e-6):
    """Central differences of sum(f(x) * g) in every element of x."""
    d = torch.zeros_like(x)
    flat, out = x.view(-1), d.view(-1)
    for i in range(x.numel()):
        keep = flat[i].item()
        flat[i] = keep + h
        up = (f() * g).sum()
        flat[i] = keep - h
        down = (f() * g).sum()
        flat[i] = keep
        out[i] = (up - down) / (2 * h)
    return d


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("rot", [0, 4, 8])
@pytest.mark.parametrize("norm", [False, True])
def test_norm_rope_gradients_against_differences(interleaved, rot, norm):
    x, g = _rand(3, 2, 8), _rand(3, 2, 8, seed=1)
    w = 1 + 0.3 * _rand(8, seed=2) if norm else None
    pos, freq = torch.tensor([0, 5, 1000]), (10.0 ** -torch.arange(rot // 2).double() if rot else None)
    kw = dict(interleaved=interleaved, rot_scale=1.3)
    f = lambda: ref.norm_rope(x, w, pos, freq, **kw)
    dx, dw = ref.norm_rope_grad(x, w, pos, freq, g, **kw)
    assert torch.allclose(dx, differences(f, x, g), atol=1e-7)
    if norm:
        assert torch.allclose(dw, differences(f, w, g), atol=1e-7)
    else:
        assert dw is None


def test_rotation_is_complex_multiplication_and_keeps_products_of_equal_distance():
    q, k = _rand(1, 1, 8), _rand(1, 1, 8, seed=3)
    freq = torch.tensor([1.0, 0.1, 0.01, 0.001], dtype=torch.float64)
    for il in (False, True):
        y = ref.norm_rope(q, None, torch.tensor([7]), freq, interleaved=il)
        a, b = (q[..., 0::2], q[..., 1::2]) if il else (q[..., :4], q[..., 4:])
        z = torch.complex(a, b) * torch.polar(torch.ones(4, dtype=torch.float64), 7 * freq)
        got = torch.complex(*((y[..., 0::2].contiguous(), y[..., 1::2].contiguous()) if il
                              else (y[..., :4].contiguous(), y[..., 4:].contiguous())))
        assert torch.allclose(got, z)
        dot = lambda i, j: (ref.norm_rope(q, None, torch.tensor([i]), freq, interleaved=il)
                            * ref.norm_rope(k, None, torch.tensor([j]), freq, interleaved=il)).sum()
        assert math.isclose(dot(9, 4), dot(105, 100), rel_tol=1e-9)


@pytest.mark.parametrize("window", [0, 1, 3])
def test_attention_gradients_against_differences(window):
    n, d, scale = 5, 4, 0.7
    q, k, v, do = _rand(n, d), _rand(n, d, seed=1), _rand(n, d, seed=2), _rand(n, d, seed=3)
    see = ref.visible(n, window)
    (dq, dk, dv), _ = ref.attend_grad(q, k, v, see, scale, do)
    f = lambda: ref.attend(q, k, v, see, scale)[0]
    for x, g in ((q, dq), (k, dk), (v, dv)):
        assert torch.allclose(g, differences(f, x, do), atol=1e-7)


def test_attention_closed_forms():
    v = _rand(6, 3)
    zeros = torch.zeros(6, 3, dtype=torch.float64)
    o, _, _ = ref.attend(zeros, zeros, v, ref.visible(6, 0), 1.0)  # equal scores: running means
    assert torch.allclose(o, v.cumsum(0) / torch.arange(1, 7).double()[:, None])
    o, _, _ = ref.attend(_rand(6, 3, seed=5), _rand(6, 3, seed=6), v, ref.visible(6, 1), 1.0)  # a window of one token
    assert torch.allclose(o, v)
    o, b, p = ref.attend(v, v, v, torch.zeros(6, 6, dtype=torch.bool), 1.0)  # rows that see nothing
    assert not o.any() and not b.any() and not p.any()


def test_packed_shares_heads_and_separates_sequences():
    q, k, v, do = _rand(7, 4, 3), _rand(7, 2, 3, seed=1), _rand(7, 2, 3, seed=2), _rand(7, 4, 3, seed=3)
    cu = [0, 3, 3, 7]
    o, _, (dq, dk, dv), _ = ref.packed(q, k, v, cu, 0.5, 0, do)
    kk, vv = k.repeat_interleave(2, 1), v.repeat_interleave(2, 1)
    o2, _, (dq2, dk2, dv2), _ = ref.packed(q, kk, vv, cu, 0.5, 0, do)
    assert torch.allclose(o, o2) and torch.allclose(dq, dq2)
    assert torch.allclose(dk, dk2.view(7, 2, 2, 3).sum(2)) and torch.allclose(dv, dv2.view(7, 2, 2, 3).sum(2))
    alone, _ = ref.packed(q[3:], k[3:], v[3:], [0, 4], 0.5, 0)
    assert torch.allclose(o[3:], alone)


def test_decode_is_the_last_row_of_the_packed_form():
    q, k, v = _rand(9, 4, 3), _rand(9, 2, 3, seed=1), _rand(9, 2, 3, seed=2)
    kc, vc = torch.zeros(4, 4, 2, 3, dtype=torch.float64), torch.zeros(4, 4, 2, 3, dtype=torch.float64)
    table = torch.tensor([[2, 0, 3, 9]])
    for t in range(9):
        kc[table[0, t // 4], t % 4], vc[table[0, t // 4], t % 4] = k[t], v[t]
    for window in (0, 5):
        full, _ = ref.packed(q, k, v, [0, 9], 0.5, window)
        one, _ = ref.decode(q[-1:], kc, vc, table, [9], 0.5, window)
        assert torch.allclose(one[0], full[-1])
    # a page out of range holds nothing; a context of 0 gives 0
    assert torch.equal(ref.decode(q[-1:], kc, vc, table, [16], 0.5, 0)[0], ref.decode(q[-1:], kc, vc, table, [12], 0.5, 0)[0])
    assert not ref.decode(q[-1:], kc, vc, table, [0], 0.5, 0)[0].any()

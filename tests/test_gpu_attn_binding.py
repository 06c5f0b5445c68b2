"""Arguments of the attention layer's calls that Python itself has to judge say the same through the native marshalling
and the general one; and tokens that share a slot of the cache."""
import pytest
import torch

from gated_delta_rule_76_b200 import gdn

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


def rnd(*s, seed=0):
    return torch.randn(*s, generator=torch.Generator().manual_seed(seed)).to(BF).cuda()


class Undecided:
    def __bool__(self):
        raise ValueError("neither true nor false")


class NoNumber:
    def __float__(self):
        raise ZeroDivisionError("no value")

    __index__ = __int__ = __float__


@pytest.mark.parametrize("native", [True, False])
def test_errors_of_an_argument_reach_the_caller(native, monkeypatch):
    if not native:
        monkeypatch.setattr(gdn, "_native", None)
    k, kc, vc = rnd(2, 2, 64), rnd(4, 16, 2, 64), rnd(4, 16, 2, 64)
    table, ctx = torch.zeros(2, 2, dtype=torch.int32, device="cuda"), torch.zeros(2, dtype=torch.int32, device="cuda")
    cu = torch.tensor([0, 2], dtype=torch.int32, device="cuda")
    before = gdn.kernel_launches()
    with pytest.raises(ValueError, match="neither true nor false"):
        gdn.gdn_kv_append(k, k, kc, vc, table, ctx, want_k=Undecided())
    with pytest.raises(TypeError):
        gdn.gdn_attn_fwd(k, k, k, cu, scale="large")
    with pytest.raises(TypeError):
        gdn.gdn_attn_fwd(k, k, k, cu, window="wide")
    with pytest.raises(ZeroDivisionError):
        gdn.gdn_attn_fwd(k, k, k, cu, scale=NoNumber())
    with pytest.raises(TypeError):
        gdn.gdn_qk_norm_rope_fwd(k, None, norm_eps=None)
    with pytest.raises(TypeError):
        gdn.gdn_attn_decode(k, kc, vc, table, ctx, max_context=1.5)
    assert gdn.kernel_launches() == before


def test_tokens_in_one_slot_leave_values_of_either():
    """Two sequences whose tables name the same page: every value there is one of the two tokens', nothing else changes."""
    N, Hk, d, page = 64, 2, 128, 16
    kc, vc = rnd(4, page, Hk, d, seed=1), rnd(4, page, Hk, d, seed=2)
    kc0, vc0 = kc.clone(), vc.clone()
    k, v = rnd(N, Hk, d, seed=3), rnd(N, Hk, d, seed=4)
    table = torch.full((N, 1), 2, dtype=torch.int32, device="cuda")
    ctx = torch.full((N,), 5, dtype=torch.int32, device="cuda")
    gdn.gdn_kv_append(k, v, kc, vc, table, ctx)
    for cache, held, new in ((kc, kc0, k), (vc, vc0, v)):
        assert (cache[2, 5] == new).any(0).all()
        held[2, 5] = cache[2, 5]
        assert torch.equal(cache, held)

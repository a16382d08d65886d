"""Infinities and NaN in V under dak_attn, dak_attn_acc and dak_attn_prefix: the elements that a counted row has them in
are infinite or none (P enters P.V in parts, one of which may be zero), and every other element has the bits that it has
without them."""
import math

import pytest

import synth
from gpu_util import bits_of, to_dev
from test_cache_ops_gpu import _i32, _ok, dak  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("kind,fp32", [("attn", False), ("acc", False), ("acc", True), ("prefix", False), ("prefix", True)])
def test_infinities_in_v(dak, kind, fp32, D):
    import torch
    B, Hq, Hkv, L, Lp = 3, 8, 2, 1500, 700
    q, k, v = synth.attn_inputs(B, Hq, Hkv, D, L, seed=D)
    _, pk, pv = synth.attn_inputs(2, Hq, Hkv, D, Lp, seed=3)
    lens, of = _i32([L, 900, 64]), _i32([0, 1, 0])
    odd = torch.zeros(B, Hkv, L, D, device="cuda")
    odd[0, 0, 1200, 5], odd[0, 0, 3, 6], odd[0, 0, 77, 7] = math.inf, -math.inf, math.nan
    odd[1, 1, 899, 40], odd[1, 1, 900, 41] = math.inf, math.inf  # row 900 lies behind the cache
    odd_p = torch.zeros(2, Hkv, Lp, D, device="cuda")
    odd_p[0, 0, 600, 9], odd_p[1, 1, 0, 10] = -math.inf, math.inf
    hit = torch.zeros(B, Hq, D, dtype=torch.bool, device="cuda")
    hit[0, :4, 5:8] = hit[1, 4:, 40] = True
    if kind == "prefix":
        hit[0, :4, 9] = hit[2, :4, 9] = hit[1, 4:, 10] = True
    out = []
    for bad in (True, False):
        def mixed(x, o):
            return torch.where(o != 0, o if bad else torch.zeros_like(o), to_dev(x).float()).to(torch.bfloat16)
        kv = dak.dak_place_kv_heads(to_dev(k), mixed(v, odd), 1)
        if kind == "attn":
            o = dak.dak_attn(to_dev(q), kv, lens)
        elif kind == "acc":
            o = dak.dak_attn_acc(to_dev(q), kv, seq_lens=lens, o_fp32=fp32)[0]
        else:
            pre = dak.dak_place_kv_heads(to_dev(pk), mixed(pv, odd_p), 1)
            o = dak.dak_attn_prefix(to_dev(q), kv, pre, prefix_of=of, seq_lens=lens, o_fp32=fp32)
        _ok(dak)
        out.append(o)
    got, clean = out
    assert torch.isfinite(clean).all()
    assert not torch.isfinite(got[hit]).any() and torch.isfinite(got[~hit]).all()
    same = bits_of(got) == bits_of(clean)
    assert same[~hit.cpu().numpy()].all()


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Hq,Hkv", [(4, 4), (8, 2), (16, 1)])
@pytest.mark.parametrize("fp32", [False, True])
def test_rows_behind_the_length_reach_nothing(dak, fp32, Hq, Hkv, D):
    """Rows behind a request's length may hold anything: the bits of a cache with zeros there."""
    import torch
    lens = [1, 15, 16, 17, 31, 63, 64, 65, 127, 128, 190]
    B, L = len(lens), 200
    q, k, v = synth.attn_inputs(B, Hq, Hkv, D, L, seed=1)
    behind = (torch.arange(L, device="cuda") >= _i32(lens)[:, None])[:, None, :, None]
    f = dak.dak_attn_f32 if fp32 else dak.dak_attn
    out = []
    for kb, vb in ((0.0, 0.0), (math.nan, math.inf), (-math.inf, math.nan)):
        kv = dak.dak_place_kv_heads(to_dev(k).masked_fill(behind, kb), to_dev(v).masked_fill(behind, vb), 5)
        out.append(f(to_dev(q), kv, _i32(lens)))
        _ok(dak)
    assert torch.isfinite(out[0]).all()
    for o in out[1:]:
        assert torch.equal(out[0], o)


def test_a_draft_that_was_not_kept(dak):
    """A drafted row of infinities that is not accepted lies behind the cache for the decode steps after it."""
    import torch
    B, T, Hq, Hkv, D, L, n = 2, 5, 8, 2, 128, 300, 100
    q, k, v = synth.attn_inputs(B, Hq, Hkv, D, L, seed=2)
    K, V = to_dev(k).clone(), to_dev(v).clone()
    V[:, :, n + 2:n + T] = math.inf
    kv = dak.dak_place_kv_heads(K, V, 1)
    lens = dak.dak_kv_commit(kv, _i32([n] * B), _i32([[0, 1]] * B), _i32([2, 1]), T)
    o = dak.dak_attn(to_dev(q), kv, lens)
    acc = dak.dak_attn_acc(to_dev(q), kv, seq_lens=lens)[0]
    _ok(dak)
    assert torch.isfinite(o).all() and torch.isfinite(acc).all()

"""Infinities and NaN in rows behind a request's length under dak_attn and the cache operators."""
import math

import pytest

import synth
from gpu_util import to_dev
from test_cache_ops_gpu import _i32, _ok, dak  # noqa: F401

pytestmark = pytest.mark.gpu


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

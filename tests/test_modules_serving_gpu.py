"""SplitK_FlashAttn over a tracked cache and over shared prefixes: the same bits as the library calls
that it makes, over a chat that is evicted twice."""
import numpy as np
import pytest

import synth
from gpu_util import to_dev

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dak(cuda_ok):
    import __graft_entry__
    __graft_entry__.build()
    import direct_host_memory_gb300 as m
    return m


def _i32(x):
    import torch
    return torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("fp32,n_split,use_prefix", [(False, 0, False), (True, 3, False), (False, 2, True), (True, 0, True)])
def test_tracked_cache(dak, fp32, n_split, use_prefix):
    import torch
    B, Hq, Hkv, D, L, keep, recent = 3, 8, 2, 64, 80, 48, 8
    _, k, v = synth.attn_inputs(B, Hq, Hkv, D, L, seed=5)
    kw = dict(prefix=None)
    if use_prefix:
        _, pk, pv = synth.attn_inputs(2, Hq, Hkv, D, 150, seed=6)
        kw = dict(prefix=dak.dak_place_kv_heads(pk, pv, 1), prefix_of=_i32([1, -1, 0]), prefix_lens=_i32([150, 77]))
    attn = dak.SplitK_FlashAttn(to_dev(k), to_dev(v), n_host_heads=2, n_split=n_split, fp32_out=fp32)
    other = dak.dak_place_kv_heads(k, v, 2)
    attn.track()
    acc = torch.zeros(B, Hkv, L, device="cuda")
    sp = torch.arange(L, dtype=torch.int32, device="cuda").repeat(B, Hkv, 1)
    assert torch.equal(attn.weights, acc) and torch.equal(attn.slot_pos, sp)
    rope = dak.dak_rope_make(D, theta=10000.0)
    lens, pos = _i32([40, 50, 60]), _i32([40, 50, 60])
    tun = dict(n_split=n_split) if n_split else None
    rng = np.random.default_rng(1)
    evictions = 0
    for step in range(70):
        x = torch.from_numpy(rng.standard_normal((B, Hq + 2 * Hkv, D)).astype(np.float32)).cuda()
        new = (x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:])
        q = attn.append_rope(rope, *new, lens, positions=pos)
        q2 = dak.dak_kv_append_rope(other, rope, *new, lens, positions=pos, slot_pos=sp)
        lens, pos = lens + 1, pos + 1
        o = attn(q.view(B, Hq, 1, D), seq_lens=lens, **kw)
        if use_prefix:
            o2 = dak.dak_attn_prefix(q2, other, seq_lens=lens, acc_in=acc, acc_out=acc, o_fp32=fp32, tuning=tun, **kw)
        else:
            o2, _ = dak.dak_attn_acc(q2, other, acc_in=acc, acc_out=acc, seq_lens=lens, o_fp32=fp32, tuning=tun)
        assert tuple(o.shape) == (B, Hq, 1, D) and o.dtype == (torch.float32 if fp32 else torch.bfloat16)
        assert torch.equal(q, q2) and torch.equal(o.view(B, Hq, D), o2)
        assert torch.equal(attn.weights, acc) and torch.equal(attn.slot_pos, sp)
        if lens.max().item() == L:
            new_lens, _ = dak.dak_kv_evict(other, lens, keep, recent, acc, sp)
            lens = attn.evict(lens, keep, recent)
            assert torch.equal(lens, new_lens)
            evictions += 1
    torch.cuda.synchronize()
    assert evictions >= 2 and dak.dak_last_error()[0] == 0
    assert torch.equal(attn.weights, acc) and torch.equal(attn.slot_pos, sp)
    with pytest.raises(ValueError):
        attn.append(x[:, :Hkv], x[:, :Hkv], lens)


def test_untracked_cache(dak):
    """Rows appended as they are equal append's, a prefix is attended over, and nothing is tracked."""
    import torch
    B, Hq, Hkv, D, L = 2, 4, 2, 128, 70
    q, k, v = synth.attn_inputs(B, Hq, Hkv, D, L, seed=8)
    _, pk, pv = synth.attn_inputs(1, Hq, Hkv, D, 90, seed=9)
    a, b = (dak.SplitK_FlashAttn(to_dev(k), to_dev(v), offload_ratio=0.5) for _ in range(2))
    kn, vn = (to_dev(synth.normal_bf16(10, j, B * Hkv * D).reshape(B, Hkv, D)) for j in (1, 2))
    a.append(kn, vn, _i32([3, 64]))
    assert b.append_rope(None, None, kn, vn, _i32([3, 64])) is None
    lens = _i32([4, 70])
    assert torch.equal(a(to_dev(q), seq_lens=lens), b(to_dev(q), seq_lens=lens))
    pre = dak.dak_place_kv_heads(pk, pv, 0)
    o = a(to_dev(q), seq_lens=lens, prefix=pre)
    assert torch.equal(o, dak.dak_attn_prefix(to_dev(q), b.placement, pre, seq_lens=lens))
    assert a.weights is None and dak.dak_last_error()[0] == 0
    with pytest.raises(ValueError):
        a.evict(lens, 8)
    with pytest.raises(ValueError):
        a(to_dev(q), seq_lens=lens, prefix_lens=_i32([3]))

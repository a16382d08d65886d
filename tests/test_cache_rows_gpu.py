"""Rows of a placed cache that are written again: what the operators keep of the token before."""
import numpy as np
import pytest

import synth
from gpu_util import bits_of, to_dev
from oracle import cache as oc

pytestmark = pytest.mark.gpu

U32 = 2.0 ** -24


@pytest.fixture(scope="module")
def dak(cuda_ok):
    import __graft_entry__
    __graft_entry__.build()
    import direct_host_memory_gb300 as m
    return m


def _i32(x):
    import torch
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def _cache(kv):
    import torch
    torch.cuda.synchronize()
    parts = [bits_of(t) for t in kv.slabs() if t is not None]
    return oc.slab_rows(np.concatenate(parts), kv.meta["H_kv"], kv.meta["L"])


@pytest.mark.parametrize("D,T,fp32,inter,rot", [(128, 1, False, False, 128), (64, 5, True, True, 64), (64, 70, False, False, 32),
                                                (128, 2, True, False, 120)])
def test_append_rope_clears_the_weights_of_the_rows_it_writes(dak, D, T, fp32, inter, rot):
    import torch
    B, Hq, Hkv, L = 3, 4, 2, T + 40
    z = np.zeros((B, Hkv, L, D), np.uint16)
    kv = dak.dak_place_kv_heads(z, z, 2)
    rope = dak.dak_rope_make(D, rot_dim=rot, interleaved=inter)
    x = torch.randn(B, T, Hq + 2 * Hkv, D, device="cuda").to(torch.float32 if fp32 else torch.bfloat16)
    slots, n_new = [7, 0, 40], [T, 0, max(1, T - 1)]
    acc = torch.rand(B, Hkv, L, device="cuda") + 1.0
    want = acc.cpu().numpy().copy()
    for b in range(B):
        want[b, :, slots[b]:slots[b] + n_new[b]] = 0.0
    for with_pos in (False, True):
        a, sp = acc.clone(), torch.full((B, Hkv, L), -5, dtype=torch.int32, device="cuda")
        dak.dak_kv_append_rope(kv, rope, x[:, :, :Hq], x[:, :, Hq:Hq + Hkv], x[:, :, Hq + Hkv:], _i32(slots),
                               n_new=_i32(n_new), slot_pos=sp if with_pos else None, acc=a)
        assert dak.dak_last_error()[0] == 0
        assert np.array_equal(a.cpu().numpy(), want)
    # a row outside the cache is skipped, in its table too
    a = acc.clone()
    dak.dak_kv_append_rope(kv, rope, None, x[:, :, Hq:Hq + Hkv], x[:, :, Hq + Hkv:], _i32([L, L, -T]), acc=a)
    assert dak.dak_last_error()[0] == 8 and torch.equal(a, acc)
    with pytest.raises(ValueError):
        dak.dak_kv_append_rope(kv, rope, None, x[:, :, Hq:Hq + Hkv], x[:, :, Hq + Hkv:], _i32(slots), acc=a[:, :1])
    kv.free()


def test_a_tracked_row_starts_without_its_last_tokens_weight(dak):
    """Tokens are attended to, taken back and written again, and one request begins a new chat at row 0:
    the weights are those of the tokens that the rows now hold, and the eviction goes by them."""
    import torch
    B, Hq, Hkv, D, L, keep = 2, 4, 2, 64, 96, 40
    G, rng = Hq // Hkv, np.random.default_rng(4)
    z = torch.zeros(B, Hkv, L, D, dtype=torch.bfloat16)
    attn = dak.SplitK_FlashAttn(z, z, n_host_heads=1)
    attn.track()
    rope = dak.dak_rope_make(D, theta=10000.0)
    want = np.zeros((B, Hkv, L))  # accumulated weights of the tokens that the rows hold
    spent = np.zeros((B, Hkv, L))

    def append(T, slots, positions):
        x = torch.from_numpy(rng.standard_normal((B, T, Hq + 2 * Hkv, D)).astype(np.float32)).cuda()
        q = attn.append_rope(rope, x[:, :, :Hq], x[:, :, Hq:Hq + Hkv], x[:, :, Hq + Hkv:], _i32(slots),
                             positions=_i32(positions))
        for b in range(B):
            want[b, :, slots[b]:slots[b] + T] = 0.0
        return q[:, -1].contiguous()

    def attend(q, lens):
        attn(q, seq_lens=_i32(lens))
        w = oc.attention(bits_of(q), *_cache(attn.placement), lens)[1]
        np.add(want, w, out=want)
        np.add(spent, w, out=spent)

    q = append(50, [0, 0], [0, 0])
    for n in (50, 49, 50):
        attend(q, [n, n])
    q = append(20, [40, 0], [40, 0])  # ten tokens taken back and twenty written; a new chat of twenty
    for _ in range(3):
        attend(q, [60, 20])
    q = append(30, [60, 20], [60, 20])
    attend(q, [90, 50])
    # a weight is off by the scores' rounding, 2 (D + 2) reach and 16 u with reach below 16 here, and its
    # sums: seven calls of G weights and one addition each
    got = attn.weights.cpu().numpy()
    tol = (2 * ((D + 2) * 16 + 16) + L + 8 * (G + 2)) * U32
    for b, n in enumerate((90, 50)):
        assert (np.abs(got[b, :, :n] - want[b, :, :n]) <= tol * (spent[b, :, :n] + 1e-3)).all()
    assert np.array_equal(attn.slot_pos.cpu().numpy()[:, :, :50], np.broadcast_to(np.arange(50), (B, Hkv, 50)))
    a0, p0 = got.copy(), attn.slot_pos.cpu().numpy()
    lens = attn.evict(_i32([90, 50]), keep, 8)
    wl, _, wa, wp = oc.evict([90, 50], keep, 8, a0, p0)
    assert lens.tolist() == wl.tolist()
    for b, n in enumerate((90, 50)):
        assert np.array_equal(attn.weights.cpu().numpy()[b, :, :n], wa[b, :, :n])
        assert np.array_equal(attn.slot_pos.cpu().numpy()[b, :, :n], wp[b, :, :n])
    assert dak.dak_last_error()[0] == 0

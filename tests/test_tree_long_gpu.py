"""Drafted trees over caches whose offsets pass 32 bits, and calls on two streams at once."""
import math

import numpy as np
import pytest

from test_cache_ops_gpu import _check_attn, _i32, _ok, dak  # noqa: F401

pytestmark = pytest.mark.gpu


def _rows(kv, slab, lo, hi):
    """Rows lo .. hi - 1 of a slab's K and V, [2][hi - lo][D]: piece c of row t lies at c ^ (t % 8)."""
    import torch
    x = kv.slabs()[1][slab, lo // 64:-(-hi // 64)]
    D = x.shape[-1]
    x = x.transpose(0, 1).reshape(2, -1, D // 8, 8)
    t = torch.arange(x.shape[1], device=x.device)
    x = torch.gather(x, 2, (torch.arange(D // 8, device=x.device) ^ (t[:, None] & 7))[None, :, :, None].expand_as(x))
    return x.reshape(2, -1, D)[:, lo % 64:lo % 64 + hi - lo]


@pytest.fixture
def long_cache(dak):
    """Two requests of eight heads over 1.1 million rows: 2^31 elements lie before the second request."""
    import torch
    B, Hkv, L, D = 2, 8, 1100000, 128
    g = torch.Generator(device="cuda").manual_seed(3)
    k, v = (torch.randn(B, Hkv, L, D, generator=g, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    kv = dak.dak_place_kv_heads(k, v, 0)
    yield kv, k, v
    kv.free()


@pytest.mark.parametrize("T,Hq,fp32", [(2, 32, False), (12, 32, False), (12, 32, True), (66, 32, False)])
def test_attn_tree_long(dak, long_cache, T, Hq, fp32):
    import torch
    kv, k, v = long_cache
    B, Hkv, L, D = k.shape
    G, n = Hq // Hkv, L - T
    g = torch.Generator(device="cuda").manual_seed(T)
    q = torch.randn(B, T, Hq, D, generator=g, device="cuda", dtype=torch.bfloat16)
    # scores of a standard deviation of 11: a token's weight lies on a few rows, which may be any
    o = dak.dak_attn_tree(q, kv, _i32([5, n]), scale=1.0, o_fp32=fp32)
    _ok(dak)
    seen = torch.ones(T, G, L, dtype=torch.bool, device="cuda")
    seen[:, :, n:] = torch.ones(T, T, dtype=torch.bool, device="cuda").tril()[:, None]
    seen = seen.view(T * G, L)
    ref, spread, reach = (torch.empty(T, Hq, *s, dtype=torch.float64, device="cuda") for s in ((D,), (D,), ()))
    for h in (0, Hkv - 1):
        kk, vv = k[1, h].double(), v[1, h].double()
        hs = slice(h * G, (h + 1) * G)
        x = q[1, :, hs].double().reshape(T * G, D)
        for at in range(0, T * G, 8):
            p = (x[at:at + 8] @ kk.T).masked_fill(~seen[at:at + 8], -math.inf).softmax(1)
            rows = torch.arange(at, min(at + 8, T * G), device="cuda")
            to = rows // G, h * G + rows % G
            ref[to], spread[to], reach[to] = p @ vv, p @ vv.abs(), (x[rows].abs() @ kk.abs().T).amax(1)
        _check_attn(o[1, :, hs], ref[:, hs].cpu().numpy(), spread[:, hs].cpu().numpy(), reach[:, hs].cpu().numpy(), D, L, fp32)


def test_append_commit_and_fork_long(dak, long_cache):
    """Drafts appended at the end of the last slab, the accepted ones kept, and the whole request taken over."""
    import torch
    kv, k, _ = long_cache
    B, Hkv, L, D = k.shape
    T, last = 12, B * Hkv - 1
    n = L - T - 3
    g = torch.Generator(device="cuda").manual_seed(9)
    new = torch.randn(2, B, T, Hkv, D, generator=g, device="cuda", dtype=torch.bfloat16)
    before = _rows(kv, last, n - 70, L).clone()
    rope = dak.dak_rope_axes_make(dak.dak_rope_make(D))
    # at positions of zero the rotation leaves the keys as they are
    dak.dak_kv_append_rope_axes(kv, rope, None, new[0], new[1], _i32([0, n]), torch.zeros(B, T, 1, dtype=torch.int32, device="cuda"))
    _ok(dak)
    want = before.clone()
    want[:, 70:70 + T] = new[:, 1, :, Hkv - 1]
    assert torch.equal(_rows(kv, last, n - 70, L), want)
    path = [0, 3, 4, 11]
    lens = dak.dak_kv_commit(kv, _i32([0, n]), _i32([path, path]), _i32([0, 4]), T)
    _ok(dak)
    assert lens.tolist() == [0, n + 4]
    want[:, 70:74] = new[:, 1, path, Hkv - 1]
    assert torch.equal(_rows(kv, last, n - 70, L), want)
    first = 1000
    keep = [_rows(kv, s, 0, first + 100).clone() for s in (0, Hkv - 1)]
    lens = dak.dak_kv_fork(kv, _i32([1, -1]), lens, first=_i32([first, 0]))
    _ok(dak)
    assert lens.tolist() == [n + 4, n + 4]
    for s, kept in zip((0, Hkv - 1), keep):
        assert torch.equal(_rows(kv, s, 0, first), kept[:, :first])
        for lo in (first, L // 2, n + 4 - 100):
            assert torch.equal(_rows(kv, s, lo, lo + 100), _rows(kv, s + Hkv, lo, lo + 100))
    whole, end = kv.slabs()[1].view(B, Hkv, -1, 2, 64, D), (n + 4) // 64
    assert torch.equal(whole[0, :, 16:end], whole[1, :, 16:end])
    assert not torch.equal(_rows(kv, 0, n + 4, L), _rows(kv, Hkv, n + 4, L))


@pytest.mark.parametrize("T,Hq", [(3, 8), (20, 32)])
def test_attn_tree_on_two_streams(dak, T, Hq):
    """Two calls at once, each with a workspace of its own, give what each gives alone."""
    import torch
    B, Hkv, L, D = 9, 4, 3000, 128
    g = torch.Generator(device="cuda").manual_seed(T)
    k, v = (torch.randn(B, Hkv, L, D, generator=g, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    kv = dak.dak_place_kv_heads(k, v, 5)
    q = torch.randn(2, B, T, Hq, D, generator=g, device="cuda", dtype=torch.bfloat16)
    lens = [_i32([L - T - 300 * b for b in range(B)]), _i32([310 * b for b in range(B)])]
    alone = [dak.dak_attn_tree(q[i], kv, lens[i]) for i in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [[torch.zeros_like(q[0]) for _ in range(8)] for _ in range(2)]
    torch.cuda.synchronize()
    for j in range(8):
        for i, s in enumerate(streams):
            dak.dak_attn_tree(q[i], kv, lens[i], O=outs[i][j], stream=s)
    torch.cuda.synchronize()
    _ok(dak)
    assert np.all([torch.equal(o, alone[i]) for i in range(2) for o in outs[i]])
    kv.free()

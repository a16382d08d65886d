"""Drafted trees, rotations by axes, commits and forks at sizes where the kernels change their plan: short tiles that
are not cut, many tokens of few heads, long paths of many slabs, few sources of many takers."""
import numpy as np
import pytest

import test_tree_ops_gpu as ops
from test_cache_ops_gpu import _i32, _ok, dak  # noqa: F401
from test_tree_ops_gpu import _inputs

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("case", [
    # B, T, Hq, Hkv, D, L, lens, n_new, mask, fp32, host slabs
    # a cache in which tiles might be cut, of lengths at which they are not
    (40, 8, 32, 8, 128, 1500, [310 + 2 * b for b in range(40)], None, "one", False, 0),
    (24, 70, 16, 4, 64, 1200, [200 + 9 * b for b in range(24)], None, "chain", False, 50),
    (30, 40, 24, 4, 128, 900, [150 + 3 * b for b in range(30)], [40 - b for b in range(30)], "chain", True, 7),
    (90, 3, 16, 4, 128, 1000, [5 * b for b in range(90)], None, "one", False, 41),
    # one long request among short ones
    (40, 5, 16, 4, 64, 4000, [3990] + [60 + b for b in range(39)], None, "chain", False, 3),
    (33, 12, 16, 2, 128, 3000, [40 + b for b in range(32)] + [2980], None, "one", False, 60),
    # caches of up to a few chunks, more tiles than CTAs
    (80, 7, 16, 8, 64, 9, [b % 3 for b in range(80)], None, "chain", False, 100),
    (70, 2, 24, 8, 128, 30, [b % 29 for b in range(70)], [b % 3 for b in range(70)], "one", True, 9),
    (1, 4, 32, 8, 128, 250, [246], None, "tree", False, 2),
    (2, 169, 2, 1, 128, 203, [6, 34], None, "chain", False, 0),
], ids=lambda c: str(c[:6]))
def test_attn_tree_sizes(dak, case):
    ops.test_attn_tree(dak, case)


@pytest.mark.parametrize("lens", [[5 + 3 * b for b in range(50)], [700 + b for b in range(50)], [0] * 49 + [2000]])
@pytest.mark.parametrize("T,Hq,fp32", [(2, 8, False), (20, 32, False), (50, 16, True)])
def test_attn_tree_does_not_depend_on_the_tiers(dak, T, Hq, fp32, lens):
    """Also where more ranges of whole tiles touch the host than CTAs may."""
    import torch
    from gpu_util import to_dev
    B, Hkv, D, L = 50, 4, 64, 2100
    q, k, v = _inputs(T, B, T, Hq, Hkv, D, L)
    outs = []
    for host in (0, 77, 200):
        kv = dak.dak_place_kv_heads(k, v, host)
        for tuning in (None, dict(host_ctas=3, window=1)):
            outs.append(dak.dak_attn_tree(to_dev(q), kv, _i32(lens), o_fp32=fp32, tuning=tuning))
        _ok(dak)
        torch.cuda.synchronize()
        kv.free()
    assert all(torch.equal(o, outs[0]) for o in outs)


@pytest.mark.parametrize("case", [
    (320, 40, 2, 64, 64, 40, True, 100),
    (90, 100, 8, 128, 120, 77, False, 13),
], ids=lambda c: str(c[:6]))
@pytest.mark.parametrize("tracked", [False, True])
def test_commit_sizes(dak, case, tracked):
    ops.test_commit(dak, case, tracked)


@pytest.mark.parametrize("B,src_B,Hkv,D,L,src_L", [(60, 1, 1, 128, 400, 380), (7, 2, 2, 64, 90, 100), (2, 1, 1, 64, 65, 65)])
def test_fork_from_few_sources(dak, B, src_B, Hkv, D, L, src_L):
    rng = np.random.default_rng(B)
    of, lens = rng.integers(0, src_B, B), [min(L, src_L) - 3 * i for i in range(src_B)]
    for first in (None, rng.integers(0, 70, B)):
        assert ops._fork_case(dak, B, src_B, Hkv, D, L, src_L, of, lens, first, B // 3, 1, True) == 0


def test_fork_of_one_request_in_place(dak):
    assert ops._fork_case(dak, 40, None, 2, 128, 150, 150, [17] * 40, [150] * 40, [3 * b for b in range(40)], 11, 0, True) == 0


@pytest.mark.parametrize("case", [
    # B, T, Hq, Hkv, D, rot, inter, axes, fp32, host slabs
    (2, 700, 4, 1, 128, 128, False, 3, False, 1),
    (2, 650, 2, 2, 64, 48, False, 4, True, 0),
    (3, 450, 5, 1, 128, 12, False, 2, True, 2),
    (2, 700, 3, 1, 64, 64, True, 3, False, 0),
    (1, 1300, 10, 1, 128, 96, False, 2, False, 0),
    (2, 620, 16, 4, 128, 64, False, 1, False, 3),
], ids=lambda c: str(c[:6]))
def test_append_rope_axes_many_tokens(dak, case):
    ops.test_append_rope_axes(dak, case, 0)


@pytest.mark.parametrize("case", [
    (2, 50, 5, 1, 128, 42, False, 2, True, 0),
    (1, 3, 4, 2, 64, 22, False, 1, False, 1),
    (2, 9, 3, 3, 128, 126, False, 3, False, 2),
], ids=str)
@pytest.mark.parametrize("far", [0, 1000000000])
def test_append_rope_axes_odd_halves(dak, case, far):
    ops.test_append_rope_axes(dak, case, far)


@pytest.mark.parametrize("fp32", [False, True])
@pytest.mark.parametrize("rot", [128, 120, 112, 64, 42, 16, 12, 2])
@pytest.mark.parametrize("B,T,Hq,Hkv", [(3, 7, 8, 2), (2, 700, 4, 1)])
def test_axes_of_a_run_are_append_rope(dak, B, T, Hq, Hkv, rot, fp32):
    """Positions one after the other on every axis: the same bits as one position a request, in blocks of either size."""
    import torch
    D, L = 128, T + 9
    g = torch.Generator(device="cuda").manual_seed(rot)
    x = torch.randn(B, T, Hq + 2 * Hkv, D, generator=g, device="cuda", dtype=torch.float32 if fp32 else torch.bfloat16)
    parts = x[:, :, :Hq], x[:, :, Hq:Hq + Hkv], x[:, :, Hq + Hkv:]
    rope = dak.dak_rope_make(D, rot_dim=rot, theta=10000.0)
    start, slots = _i32([4000 + b for b in range(B)]), _i32([b for b in range(B)])
    zero = torch.zeros(B, Hkv, L, D, dtype=torch.bfloat16, device="cuda")
    one, many = dak.dak_place_kv_heads(zero, zero, 1), dak.dak_place_kv_heads(zero, zero, 0)
    q = dak.dak_kv_append_rope(one, rope, *parts, slots, positions=start)
    at = (start[:, None] + torch.arange(T, device="cuda", dtype=torch.int32))[:, :, None].expand(B, T, 3).contiguous()
    axes = dak.dak_rope_axes_make(rope, [i % 3 for i in range(rot // 2)], n_axes=3)
    assert torch.equal(dak.dak_kv_append_rope_axes(many, axes, *parts, slots, at), q)
    _ok(dak)
    host, hbm = one.slabs()
    torch.cuda.synchronize()
    assert torch.equal(torch.cat([host.cuda(), hbm]), many.slabs()[1])

"""Infinities and NaN in V under the attention of drafted trees: an element is what the rows that its token sees
hold there (an infinity, NaN with infinities of both signs or a NaN), whatever their weights and wherever the work
is cut, in cached rows as in drafted ones; every other element has the bits that it has without them."""
import math

import numpy as np
import pytest

from gpu_util import to_dev
from oracle import tree as ot
from test_cache_ops_gpu import _i32, _ok, dak  # noqa: F401
from test_tree_ops_gpu import _bits, _inputs, _mask_dev

pytestmark = pytest.mark.gpu

CASES = [
    # B, T, Hq, Hkv, D, L, lens, host slabs
    (1, 2, 8, 2, 128, 3000, [2800], 0),            # 8 rows a kv head, a tile in many ranges
    (2, 3, 10, 2, 64, 2500, [2490, 700], 1),       # 15
    (1, 20, 8, 2, 128, 3000, [2900], 0),           # 80
    (2, 40, 3, 1, 64, 2500, [2400, 70], 1),        # 120
    (1, 80, 8, 2, 128, 3000, [2800], 2),           # 320: tiles of two halves and of one
    (2, 256, 2, 2, 64, 1500, [1200, 1244], 0),
    (9, 4, 4, 4, 128, 200, [190, 0, 64, 63, 5, 128, 130, 1, 100], 17),  # short: tiles whole
    (9, 30, 8, 2, 64, 200, [160, 0, 64, 63, 5, 128, 130, 1, 100], 3),
    # several tiles a CTA, one after the other
    (80, 32, 64, 8, 128, 200, [(37 * i) % 168 for i in range(80)], 100),
    (60, 32, 32, 4, 64, 150, [(29 * i) % 118 for i in range(60)], 0),
    (300, 3, 4, 2, 64, 100, [(13 * i) % 94 for i in range(300)], 0),
]


@pytest.mark.parametrize("scale", [0.0, 8.0])  # weights of one size, and weights that mostly are below the least fp32
@pytest.mark.parametrize("fp32", [False, True])
@pytest.mark.parametrize("case", CASES, ids=str)
def test_infinities_in_v(dak, case, fp32, scale):
    import torch
    B, T, Hq, Hkv, D, L, lens, host = case
    rng = np.random.default_rng(B * 1000 + T)
    q, k, v = _inputs(B + T, B, T, Hq, Hkv, D, L)
    mask = _mask_dev(_bits(rng, "any", B, T))
    bits = ot.bits(mask.cpu().numpy(), T)
    seen = np.zeros((B, T, L), np.float32)
    odd = np.zeros((B, Hkv, L, D), np.float32)
    for b in range(B):
        seen[b, :, :lens[b]] = 1
        seen[b, :, lens[b]:lens[b] + T] = bits[b]
        if b % 5 == 4:
            continue  # none here: the tile before had some
        for g in range(Hkv):
            rows = np.concatenate([rng.integers(0, max(lens[b], 1), 6), lens[b] + rng.integers(0, T, 6)])
            odd[b, g, rows, rng.integers(0, D, 12)] = rng.choice([math.inf, -math.inf, math.nan], 12, p=[0.45, 0.45, 0.1])
            odd[b, g, rows[0], 3], odd[b, g, rows[1], 3] = math.inf, math.inf
            odd[b, g, rows[2], 4], odd[b, g, rows[7], 4] = math.inf, -math.inf
    O, V = torch.from_numpy(odd).cuda(), to_dev(v).float()
    is_odd = (O != 0)  # NaN too
    out = []
    for vx in (torch.where(is_odd, O, V), V.masked_fill(is_odd, 0.0)):
        kv = dak.dak_place_kv_heads(to_dev(k), vx.to(torch.bfloat16), host)
        out.append(dak.dak_attn_tree(to_dev(q), kv, _i32(lens), mask=mask, scale=scale, o_fp32=fp32).float())
        _ok(dak)
    got, clean = out
    assert torch.isfinite(clean).all()
    s = torch.from_numpy(seen).cuda()[:, None]  # [B][1][T][L]
    up, down, none = (torch.matmul(s, x.float()) > 0 for x in (O == math.inf, O == -math.inf, O.isnan()))
    want = clean.clone().view(B, T, Hkv, Hq // Hkv, D).permute(0, 2, 3, 1, 4)  # [B][Hkv][G][T][D]
    up, down, none = up[:, :, None], down[:, :, None], none[:, :, None]
    want = torch.where(up & ~down, torch.full_like(want, math.inf), want)
    want = torch.where(down & ~up, torch.full_like(want, -math.inf), want)
    want = torch.where(none | (up & down), torch.full_like(want, math.nan), want)
    want = want.permute(0, 3, 1, 2, 4).reshape(B, T, Hq, D)
    assert want.isinf().any() and want.isnan().any() and want.isfinite().any()
    assert torch.equal(got.isnan(), want.isnan())
    assert torch.equal(got.nan_to_num(5.0, math.inf, -math.inf), want.nan_to_num(5.0, math.inf, -math.inf))


@pytest.mark.parametrize("T,Hq,Hkv,D", [(2, 8, 2, 128), (20, 8, 2, 128), (20, 8, 2, 64), (80, 8, 2, 128)])
@pytest.mark.parametrize("where", [0, 30, 2000])
def test_an_infinity_of_next_to_no_weight(dak, T, Hq, Hkv, D, where):
    """A draft with infinities in V whose score lies hundreds below one that comes in another warp's rows, another
    stream's or another range's."""
    import torch
    L, n = 3000, 2800
    q, k, v = _inputs(1, 1, T, Hq, Hkv, D, L)
    Q, K, V = to_dev(q).abs(), to_dev(k).clone(), to_dev(v).clone()
    K[0, 0, n], K[0, 0, where] = -20.0, 20.0
    V[0, 0, n, 5] = math.inf
    kv = dak.dak_place_kv_heads(K, V, 0)
    for fp32 in (False, True):
        o = dak.dak_attn_tree(Q, kv, _i32([n]), o_fp32=fp32)
        _ok(dak)
        assert (o[0, :, :Hq // Hkv, 5] == math.inf).all()
        o[0, :, :Hq // Hkv, 5] = 0.0
        assert torch.isfinite(o).all()


@pytest.mark.parametrize("T,Hq", [(3, 8), (16, 8), (70, 8)])
def test_a_kept_draft_counts_as_it_did(dak, T, Hq):
    """The same row as a draft that every token sees, and after dak_kv_commit."""
    import torch
    B, Hkv, D, L, n = 1, 2, 128, 700, 500
    q, k, v = _inputs(T, B, T, Hq, Hkv, D, L)
    V = to_dev(v).clone()
    V[0, :, n, ::3] = math.inf
    V[0, 1, n, 1::3] = -math.inf
    kv = dak.dak_place_kv_heads(to_dev(k), V, 1)
    as_draft = dak.dak_attn_tree(to_dev(q), kv, _i32([n]))
    lens = dak.dak_kv_commit(kv, _i32([n]), _i32([[0]]), _i32([1]), T)
    kept = dak.dak_attn_tree(to_dev(q), kv, lens)
    _ok(dak)
    for o in (as_draft, kept):
        assert (o[..., ::3] == math.inf).all() and (o[..., Hq // 2:, 1::3] == -math.inf).all()
        assert o[:, :, :Hq // 2, 1::3].isfinite().all() and o[..., 2::3].isfinite().all()

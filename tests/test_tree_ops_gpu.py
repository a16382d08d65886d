"""Drafted trees over a placed cache, tokens with positions of their own, accepted paths and forked caches
on the GPU against the fp64 oracle."""
import math

import numpy as np
import pytest

import synth
from gpu_util import bits_of, to_dev, to_np
from oracle import cache as oc
from oracle import tree as ot
from test_cache_ops_gpu import BOUNDS, U32, _cache, _check_attn, _i32, _ok, dak  # noqa: F401

pytestmark = pytest.mark.gpu


def _mask_dev(bits):
    """bool [B][T][T] -> int64 CUDA [B][T][words]."""
    import torch
    B, T, _ = bits.shape
    w = np.zeros((B, T, -(-T // 64) * 64), np.uint8)
    w[..., :T] = bits
    return torch.from_numpy(np.packbits(w, axis=-1, bitorder="little").view(np.int64).copy()).cuda()


def _bits(rng, kind, B, T):
    """Masks: 'tree' (ancestors and itself), 'any' (any bits, some rows without one), 'none', 'one' (a tree for
    all) or 'chain'."""
    if kind == "chain":
        return np.broadcast_to(np.tril(np.ones((T, T), bool)), (B, T, T))
    if kind == "none":
        return np.zeros((B, T, T), bool)
    if kind == "any":
        m = rng.random((B, T, T)) < rng.choice([0.05, 0.5, 0.95], (B, T, 1))
        m[:, ::3] &= rng.random((B, len(range(0, T, 3)), 1)) < 0.5
        return m
    m = np.zeros((1 if kind == "one" else B, T, T), bool)
    for x in m:
        for t in range(T):
            parent = rng.integers(-1, t) if t else -1
            if parent >= 0:
                x[t] = x[parent]
            x[t, t] = True
    return m


def _inputs(seed, B, T, Hq, Hkv, D, L):
    q = synth.normal_bf16(seed, 1, B * T * Hq * D).reshape(B, T, Hq, D)
    k, v = (synth.normal_bf16(seed, i, B * Hkv * L * D).reshape(B, Hkv, L, D) for i in (2, 3))
    return q, k, v


TREE_CASES = [
    # B, T, Hq, Hkv, D, L, lens, n_new, mask, fp32, host slabs
    (1, 1, 8, 2, 128, 1, [0], None, "tree", False, 0),
    (1, 1, 1, 1, 64, 700, [699], None, "chain", True, 0),
    (2, 3, 4, 4, 64, 70, [0, 64], [3, 1], "tree", False, 3),
    (3, 8, 32, 8, 128, 520, [500, 0, 63], None, "tree", False, 0),
    (4, 5, 6, 2, 128, 140, [64, 65, 127, 128], [5, 0, 2, 5], "any", True, 5),
    (2, 16, 8, 2, 64, 1300, [1283, 1000], [16, 9], "one", False, 1),
    (1, 64, 4, 2, 128, 400, [300], None, "tree", False, 0),
    (2, 64, 8, 1, 128, 200, [1, 136], [64, 50], "any", True, 1),
    (2, 65, 3, 3, 64, 193, [128, 100], [65, 65], "tree", True, 2),
    (1, 33, 16, 1, 128, 333, [290], None, "chain", False, 0),
    (2, 24, 32, 2, 64, 90, [50, 0], [24, 24], "any", False, 4),
    (1, 130, 5, 1, 128, 200, [61], None, "tree", False, 0),
    (1, 256, 2, 2, 64, 1000, [700], [255], "any", True, 1),
    (1, 256, 16, 1, 128, 330, [70], None, "tree", False, 0),
    (3, 7, 4, 2, 128, 50, [0, 0, 0], [7, 3, 0], "none", False, 2),
    (40, 2, 4, 2, 64, 130, [3 * i for i in range(40)], None, "chain", False, 11),
    (1, 4, 8, 2, 128, 20000, [19990], None, "tree", False, 0),
    (5, 12, 9, 1, 128, 900, [888, 0, 300, 64, 711], [12, 12, 1, 0, 6], "any", False, 2),
    # several tiles of two halves, of one and of both kinds one after the other in a CTA
    (80, 32, 64, 8, 128, 200, [(37 * i) % 168 for i in range(80)], None, "one", False, 100),
    (40, 48, 32, 8, 64, 300, [(61 * i) % 252 for i in range(40)], [48 - i for i in range(40)], "chain", False, 0),
    (60, 32, 32, 4, 64, 150, [(29 * i) % 118 for i in range(60)], [(i % 3) * 16 for i in range(60)], "one", True, 7),
    (300, 6, 8, 2, 64, 100, [(13 * i) % 94 for i in range(300)], None, "one", False, 0),
]


@pytest.mark.parametrize("case", TREE_CASES, ids=str)
def test_attn_tree(dak, case):
    import torch
    B, T, Hq, Hkv, D, L, lens, n_new, kind, fp32, host = case
    rng = np.random.default_rng(B * 1000 + T)
    q, k, v = _inputs(B + T, B, T, Hq, Hkv, D, L)
    bits = _bits(rng, kind, B, T)
    kv = dak.dak_place_kv_heads(k, v, host)
    before = torch.full((B, T, Hq, D), 7.0, dtype=torch.float32 if fp32 else torch.bfloat16, device="cuda")
    o = dak.dak_attn_tree(to_dev(q), kv, _i32(lens), mask=None if kind == "chain" else _mask_dev(bits),
                          n_new=None if n_new is None else _i32(n_new), O=before.clone(), o_fp32=fp32)
    _ok(dak)
    mask = None if kind == "chain" else _mask_dev(bits).cpu().numpy()
    ref, spread, reach = ot.attention(q, k, v, lens, mask, n_new)
    for b in range(B):
        m = T if n_new is None else n_new[b]
        assert torch.equal(o[b, m:], before[b, m:])
        if m:
            _check_attn(o[b, :m], ref[b, :m], spread[b, :m], reach[b, :m], D, lens[b] + m, fp32)


@pytest.mark.parametrize("fp32", [False, True])
@pytest.mark.parametrize("D", [64, 128])
def test_attn_tree_large_scores_and_scale(dak, D, fp32):
    """Scores that spread over hundreds, whose maximum moves on from chunk to chunk and lies in the drafts."""
    B, T, Hq, Hkv, L = 2, 9, 8, 2, 500
    rng = np.random.default_rng(D)
    q, k, v = _inputs(3, B, T, Hq, Hkv, D, L)
    grow = np.linspace(0.1, 4.0, L)[None, None, :, None]
    k = bits_of(to_dev(k) * to_dev(synth.normal_bf16(1, 1, 1)).new_tensor(grow))
    bits = _bits(rng, "any", B, T)
    mask, lens = _mask_dev(bits), [480, 123]
    kv = dak.dak_place_kv_heads(k, v, 0)
    o = dak.dak_attn_tree(to_dev(q), kv, _i32(lens), mask=mask, scale=0.9, o_fp32=fp32)
    _ok(dak)
    ref, spread, reach = ot.attention(q, k, v, lens, mask.cpu().numpy(), scale=0.9)
    _check_attn(o, ref, spread, reach, D, L, fp32)


@pytest.mark.parametrize("fp32", [False, True])
@pytest.mark.parametrize("T,Hq,Hkv,lens", [(7, 4, 2, 100), (40, 16, 2, 61), (90, 4, 1, 30), (70, 1, 1, 0)])
def test_attn_tree_hidden_rows_reach_nothing(dak, fp32, T, Hq, Hkv, lens):
    """Drafted rows that hold infinities and NaN, in K, V or both, seen by no token but a few: the others'
    outputs are what they are with clean rows, and rows behind the drafts may hold anything."""
    import torch
    B, D, L = 2, 128, lens + T + 70
    rng = np.random.default_rng(T)
    q, k, v = _inputs(T, B, T, Hq, Hkv, D, L)
    bits = _bits(rng, "any", B, T)
    bad = rng.choice(T, 5, replace=False)
    bits[:, :, bad] = False
    bits[1, 2, bad[0]] = bits[1, 5, bad[1]] = True  # these see one
    kb, vb = (to_dev(x).float() for x in (k, v))
    for i, s in enumerate(bad):
        if i != 0:
            kb[:, :, lens + s, ::7] = [math.inf, -math.inf, math.nan][i % 3]
        vb[:, :, lens + s, ::(i + 1)] = [math.inf, math.nan, -math.inf][i % 3]
    kb[:, :, lens + T:], vb[:, :, lens + T:] = math.nan, math.inf
    mask = _mask_dev(bits)

    def run(kx, vx):
        kv = dak.dak_place_kv_heads(kx.to(torch.bfloat16), vx.to(torch.bfloat16), 1)
        o = dak.dak_attn_tree(to_dev(q), kv, _i32([lens] * B), mask=mask, o_fp32=fp32)
        _ok(dak)
        return o

    got, clean = run(kb, vb), run(to_dev(k).float(), to_dev(v).float())
    sees = torch.from_numpy(bits[:, :, bad].any(-1)).cuda()
    assert torch.isfinite(got[~sees]).all()
    ref, spread, reach = ot.attention(q, k, v, [lens] * B, mask.cpu().numpy())
    ok = ~sees.cpu().numpy()
    for b in range(B):
        _check_attn(got[b][~sees[b]], ref[b][ok[b]], spread[b][ok[b]], reach[b][ok[b]], D, lens + T, fp32)
    assert torch.equal(got[~sees], clean[~sees])
    # token 2 of request 1 sees infinities in V of a row whose scores are sound: all its elements there
    assert (got[1, 2] == math.inf).all()
    assert not torch.isfinite(got[1, 5]).any()  # token 5 of request 1 sees a score that is none


def test_attn_tree_nan_in_the_cache_is_kept(dak):
    """A score of NaN or infinity gives NaN, whatever range of the cache it lies in."""
    import torch
    B, T, Hq, Hkv, D, L = 1, 3, 4, 2, 64, 9000
    q, k, v = _inputs(5, B, T, Hq, Hkv, D, L)
    for at in (0, 4444, 8990):
        for bad in (math.nan, math.inf):
            kx = to_dev(k).clone()
            kx[0, 0, at] = bad
            if bad == math.inf:
                kx[0, 0, at, 1:] = 0.0
                qx = to_dev(q).clone().abs()
            else:
                qx = to_dev(q)
            kv = dak.dak_place_kv_heads(kx, to_dev(v), 0)
            o = dak.dak_attn_tree(qx, kv, _i32([8991]))
            _ok(dak)
            assert torch.isnan(o[:, :, :2]).all() and torch.isfinite(o[:, :, 2:]).all()


@pytest.mark.parametrize("T,fp32", [(11, False), (11, True), (3, False), (8, True), (140, False)])
def test_attn_tree_does_not_depend_on_the_tiers(dak, T, fp32):
    import torch
    B, Hq, Hkv, D, L = 6, 8, 4, 128, 1500
    q, k, v = _inputs(9, B, T, Hq, Hkv, D, L)
    lens = _i32([L - T, 3, 800, 0, 64, 1111])
    mask = _mask_dev(_bits(np.random.default_rng(2), "tree", B, T))
    want = None
    for host in (0, 1, 7, 13, 24):
        for tun in (None, dict(host_ctas=3, window=2, hbm_window=1), dict(host_ctas=1)):
            kv = dak.dak_place_kv_heads(k, v, host)
            o = dak.dak_attn_tree(to_dev(q), kv, lens, mask=mask, tuning=tun, o_fp32=fp32)
            _ok(dak)
            want = o if want is None else want
            assert torch.equal(o, want), (host, tun)


def test_attn_tree_drafts_past_the_cache(dak):
    """Drafted rows at L and behind do not exist: reported, and the rest is attended."""
    B, T, Hq, Hkv, D, L = 3, 6, 4, 2, 64, 100
    q, k, v = _inputs(4, B, T, Hq, Hkv, D, L)
    lens = [97, 100, 40]
    kv = dak.dak_place_kv_heads(k, v, 0)
    o = dak.dak_attn_tree(to_dev(q), kv, _i32([97, 1000, 40]))
    st, info = dak.dak_last_error()
    assert st == BOUNDS
    ref, spread, reach = ot.attention(q, k, v, lens)
    _check_attn(o, ref, spread, reach, D, L, False)
    o = dak.dak_attn_tree(to_dev(q), kv, _i32([-5, 3, 40]), n_new=_i32([99, 1, -1]))
    _ok(dak)
    ref, spread, reach = ot.attention(q, k, v, [0, 3, 40], n_new=[6, 1, 0])
    _check_attn(o[0], ref[0], spread[0], reach[0], D, L, False)
    _check_attn(o[1, :1], ref[1, :1], spread[1, :1], reach[1, :1], D, L, False)


def test_attn_tree_captured_on_another_stream(dak):
    """A captured call follows lengths, masks and drafts that change between replays; two graphs."""
    import torch
    B, T, Hq, Hkv, D, L = 3, 10, 8, 2, 128, 700
    q, k, v = _inputs(8, B, T, Hq, Hkv, D, L)
    Q, lens, n_new = to_dev(q), _i32([10, 20, 30]), _i32([10, 10, 10])
    rng = np.random.default_rng(0)
    mask = _mask_dev(_bits(rng, "any", B, T))
    kv = dak.dak_place_kv_heads(k, v, 2)
    outs = [torch.zeros(B, T, Hq, D, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    dak.dak_attn_tree(Q, kv, lens, mask=mask, n_new=n_new, O=outs[0], stream=s)
    s.synchronize()
    graphs = []
    for o in outs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            dak.dak_attn_tree(Q, kv, lens, mask=mask, n_new=n_new, O=o)
        graphs.append(g)
    for new in ([680, 0, 300], [1, 690, 64]):
        bits = _bits(rng, "any", B, T)
        mask.copy_(_mask_dev(bits))
        lens.copy_(_i32(new))
        torch.cuda.synchronize()
        for g in graphs:
            g.replay()
        _ok(dak)
        ref, spread, reach = ot.attention(q, k, v, new, mask.cpu().numpy())
        for o in outs:
            _check_attn(o, ref, spread, reach, D, L, False)


def test_attn_tree_alignment_and_unused_rows(dak):
    """An O that is 16-byte aligned but not 32, and a workspace likewise; nothing around them is written."""
    import torch
    for T, Hq, Hkv, fp32 in ((20, 8, 2, False), (20, 8, 2, True), (3, 4, 2, False), (40, 16, 2, False)):
        B, D, L = 3, 64, 1700
        q, k, v = _inputs(T, B, T, Hq, Hkv, D, L)
        lens, n_new = _i32([L - T, 900, 0]), _i32([T, T - 2, 1])
        kv = dak.dak_place_kv_heads(k, v, 2)
        dtype, item = (torch.float32, 4) if fp32 else (torch.bfloat16, 2)
        need = dak.dak_attn_tree_workspace_bytes(kv, T, Hq)
        n = B * T * Hq * D
        got = []
        for shift in (0, 16):
            buf = torch.full((n + 64,), 7.0, dtype=dtype, device="cuda")
            ws = torch.full((need + 64,), 3, dtype=torch.uint8, device="cuda")
            o = buf[shift // item:shift // item + n].view(B, T, Hq, D)
            dak.dak_attn_tree(to_dev(q), kv, lens, n_new=n_new, O=o, o_fp32=fp32, workspace=ws[shift:shift + need])
            _ok(dak)
            assert (buf[:shift // item] == 7).all() and (buf[shift // item + n:] == 7).all()
            assert (ws[:shift] == 3).all() and (ws[shift + need:] == 3).all()
            assert (o[1, T - 2:] == 7).all() and (o[2, 1:] == 7).all()
            got.append(o.clone())
        assert torch.equal(got[0], got[1])


def test_attn_tree_without_a_tensor_map(dak):
    """A tensor map that cannot be encoded is an error, and nothing is written."""
    import torch
    kv = dak.dak_place_kv_heads(*_inputs(1, 2, 9, 4, 2, 64, 50)[1:], 0)
    q, lens = torch.ones(2, 9, 4, 64, dtype=torch.bfloat16, device="cuda"), _i32([1, 2])
    o = torch.full_like(q, 7.0)
    for skip in (0, 1):
        dak.dak_inject_fault(dak.FAULT_TENSOR_MAP, 1, skip)
        with pytest.raises(dak.DakError) as e:
            dak.dak_attn_tree(q, kv, lens, O=o)
        assert e.value.status == 5 and dak.dak_fault_pending(dak.FAULT_TENSOR_MAP) == 0
    torch.cuda.synchronize()
    assert (o == 7).all()
    dak.dak_attn_tree(q, kv, lens, O=o)
    _ok(dak)
    assert not (o == 7).any()


def test_attn_tree_arguments(dak):
    import torch
    kv = dak.dak_place_kv_heads(*_inputs(1, 2, 1, 4, 2, 64, 50)[1:], 0)
    q = torch.zeros(2, 3, 4, 64, dtype=torch.bfloat16, device="cuda")
    lens, mask = _i32([1, 2]), torch.zeros(2, 3, 1, dtype=torch.int64, device="cuda")
    for a, kw in (((q[:, 0], lens), {}), ((q[:1], lens), {}), ((q.float(), lens), {}), ((q, lens.long()), {}), ((q, lens[:1]), {}),
                  ((q, None), {}), ((q, lens), dict(mask=mask[:, :2])), ((q, lens), dict(mask=mask.int())),
                  ((q, lens), dict(mask=mask.cpu())), ((q, lens), dict(n_new=_i32([1]))), ((q, lens), dict(O=q.float())),
                  ((q.transpose(1, 2), lens), {}), ((q, lens), dict(workspace=torch.zeros(4, device="cuda")))):
        with pytest.raises((ValueError, dak.DakError)):
            dak.dak_attn_tree(a[0], kv, a[1], **kw)
    with pytest.raises(dak.DakError):
        dak.dak_attn_tree(q, kv, lens, O=q)
    ws = torch.empty(dak.dak_attn_tree_workspace_bytes(kv, 3, 4), dtype=torch.uint8, device="cuda")
    o = dak.dak_attn_tree(q, kv, lens, mask=mask[:1], workspace=ws)
    assert o.shape == q.shape
    _ok(dak)


# ---------------------------------------------------------------- rotation by axes

AXES_CASES = [
    # B, T, Hq, Hkv, D, rot, inter, axes, fp32, host slabs
    (1, 1, 32, 8, 128, 128, False, 1, False, 0),
    (2, 9, 4, 2, 64, 64, False, 3, True, 1),
    (3, 33, 5, 1, 128, 120, True, 4, False, 2),
    (2, 70, 6, 2, 64, 56, False, 2, False, 3),
    (1, 130, 3, 3, 128, 2, True, 1, True, 0),
    (2, 3, 0, 2, 128, 128, False, 3, False, 0),
    (70, 2, 4, 2, 64, 32, True, 3, True, 20),
]


@pytest.mark.parametrize("case", AXES_CASES, ids=str)
@pytest.mark.parametrize("far", [0, 1000000000])
def test_append_rope_axes(dak, case, far):
    import torch
    B, T, Hq, Hkv, D, rot, inter, A, fp32, host = case
    L, H, scale = T + 67, Hq + 2 * Hkv, 1.25
    rng = np.random.default_rng(B * 1000 + T)
    x = rng.standard_normal((B, T, H, D)).astype(np.float32)
    X = torch.from_numpy(x).cuda()
    if not fp32:
        X = X.to(torch.bfloat16)
        x = to_np(X)
    k0, v0 = synth.normal_bf16(7, 1, B * Hkv * L * D), synth.normal_bf16(7, 2, B * Hkv * L * D)
    kv = dak.dak_place_kv_heads(k0.reshape(B, Hkv, L, D), v0.reshape(B, Hkv, L, D), host)
    slots, n_new = rng.integers(0, L - T + 1, B), rng.integers(0, T + 1, B)
    n_new[0] = T
    pos = rng.integers(-3000, 3000, (B, T, A)) + far
    axis = rng.integers(0, A, rot // 2)
    rope = dak.dak_rope_axes_make(dak.dak_rope_make(D, rot_dim=rot, theta=10000.0, interleaved=inter, attn_scale=scale), axis,
                                  n_axes=A)
    q_out = torch.full((B, T, Hq, D), 7.0, dtype=torch.bfloat16, device="cuda")
    slot_pos = torch.full((B, Hkv, L), -5, dtype=torch.int32, device="cuda")
    acc = torch.full((B, Hkv, L), 3.0, device="cuda")
    dak.dak_kv_append_rope_axes(kv, rope, X[:, :, :Hq] if Hq else None, X[:, :, Hq:Hq + Hkv], X[:, :, Hq + Hkv:], _i32(slots),
                                _i32(pos), n_new=_i32(n_new), q_out=q_out if Hq else None, slot_pos=slot_pos, acc=acc)
    _ok(dak)
    freqs = oc.inv_freq(rot, 10000.0)
    y = ot.rotate_axes(np.asarray(x, np.float64).reshape(B * T, H, D), pos.reshape(B * T, A), axis, freqs, inter, scale)
    y = y.reshape(B, T, H, D)
    y[:, :, Hq + Hkv:] = x[:, :, Hq + Hkv:]
    # as for one position a request: angles of 2^-24 turns, sincos one unit, times |x1| + |x2|
    slack = (2 * math.pi * 2.0 ** -24 + 2.0 ** -23 + 4 * U32 + np.abs(pos).max() * 2.0 ** -51) * 2 * np.abs(x).max() * scale
    K, V = _cache(kv)
    wk, wv = oc._f64(k0).reshape(B, Hkv, L, D).copy(), oc._f64(v0).reshape(B, Hkv, L, D).copy()
    want_pos, want_acc = np.full((B, Hkv, L), -5), np.full((B, Hkv, L), 3.0)
    q = to_np(q_out)
    for b in range(B):
        n, r = n_new[b], slots[b]
        assert (q[b, n:] == 7.0).all()
        err = np.abs(q[b, :n] - y[b, :n, :Hq])
        assert (err <= slack + 2.0 ** -8 * np.abs(y[b, :n, :Hq])).all()
        wk[b, :, r:r + n] = y[b, :n, Hq:Hq + Hkv].transpose(1, 0, 2)
        wv[b, :, r:r + n] = y[b, :n, Hq + Hkv:].transpose(1, 0, 2)
        want_pos[b, :, r:r + n], want_acc[b, :, r:r + n] = pos[b, :n, 0], 0.0
    assert (np.abs(oc._f64(K) - wk) <= slack + 2.0 ** -8 * np.abs(wk)).all()
    assert (np.abs(oc._f64(V) - wv) <= 2.0 ** -8 * np.abs(wv)).all()
    assert np.array_equal(slot_pos.cpu().numpy(), want_pos) and np.array_equal(acc.cpu().numpy(), want_acc)


def test_axes_with_equal_positions_are_append_rope(dak):
    """One position per request and t on every axis: the bits of dak_kv_append_rope."""
    import torch
    B, T, Hq, Hkv, D, L = 2, 20, 8, 2, 128, 90
    X = to_dev(synth.normal_bf16(4, 1, B * T * 12 * D)).view(B, T, 12, D)
    rope = dak.dak_rope_make(D, scaling="by_parts", factor=8.0, orig_len=4096.0)
    axes = dak.dak_rope_axes_make(rope, [i % 3 for i in range(64)])
    start, slots = _i32([100000, 7]), _i32([0, 50])
    pos = (start[:, None, None] + torch.arange(T, device="cuda", dtype=torch.int32)[:, None]).expand(B, T, 3).contiguous()
    zero = np.zeros((B, Hkv, L, D), np.uint16)
    one, two = dak.dak_place_kv_heads(zero, zero, 1), dak.dak_place_kv_heads(zero, zero, 3)
    args = (X[:, :, :8], X[:, :, 8:10], X[:, :, 10:], slots)
    q1 = dak.dak_kv_append_rope(one, rope, *args, positions=start)
    q2 = dak.dak_kv_append_rope_axes(two, axes, *args, pos)
    _ok(dak)
    assert torch.equal(q1, q2)
    for a, b in zip(_cache(one), _cache(two)):
        assert np.array_equal(a, b)


def test_axes_rows_outside_and_arguments(dak):
    import torch
    B, T, D, L = 2, 4, 64, 20
    zero = np.zeros((B, 1, L, D), np.uint16)
    kv = dak.dak_place_kv_heads(zero, zero, 0)
    X = torch.ones(B, T, 3, D, dtype=torch.bfloat16, device="cuda")
    rope = dak.dak_rope_axes_make(dak.dak_rope_make(D), [0, 1] * 16)
    pos = torch.zeros(B, T, 2, dtype=torch.int32, device="cuda")
    q = dak.dak_kv_append_rope_axes(kv, rope, X[:, :, :1], X[:, :, 1:2], X[:, :, 2:], _i32([18, -1]), pos)
    assert dak.dak_last_error()[0] == BOUNDS
    assert (q == 1).all()
    K, _ = _cache(kv)
    rows = (K[:, 0] != 0).any(-1)
    assert np.flatnonzero(rows[0]).tolist() == [18, 19] and np.flatnonzero(rows[1]).tolist() == [0, 1, 2]
    for bad in (None, pos[:, :, :1].contiguous(), pos.long(), pos[:1], pos.cpu()):
        with pytest.raises(ValueError):
            dak.dak_kv_append_rope_axes(kv, rope, None, X[:, :, 1:2], X[:, :, 2:], _i32([0, 0]), bad)


# ---------------------------------------------------------------- commit

COMMIT_CASES = [
    # B, T, Hkv, D, L, most, ragged, host slabs
    (1, 1, 1, 64, 1, 1, False, 0),
    (3, 16, 2, 128, 200, 5, False, 4),
    (4, 64, 1, 64, 130, 64, True, 2),
    (2, 256, 3, 128, 400, 200, True, 0),
    (2, 256, 1, 64, 256, 256, False, 1),
    (50, 7, 2, 128, 64, 7, True, 33),
]


@pytest.mark.parametrize("tracked", [False, True])
@pytest.mark.parametrize("case", COMMIT_CASES, ids=str)
def test_commit(dak, case, tracked):
    import torch
    B, T, Hkv, D, L, most, ragged, host = case
    rng = np.random.default_rng(T + B)
    k, v = (synth.normal_bf16(T, i, B * Hkv * L * D).reshape(B, Hkv, L, D) for i in (1, 2))
    lens = rng.integers(0, L - T + 1, B)
    n_new = rng.integers(1, T + 1, B) if ragged else np.full(B, T)
    n_path = np.minimum(rng.integers(0, most + 1, B), n_new)
    n_path[0] = min(most, n_new[0])
    path = np.full((B, most), 10 ** 6)  # behind n_path it may hold anything
    for b in range(B):
        path[b, :n_path[b]] = np.sort(rng.choice(n_new[b], n_path[b], replace=False))
    pos, acc = rng.integers(0, 10 ** 6, (B, Hkv, L)).astype(np.int32), rng.random((B, Hkv, L)).astype(np.float32)
    kv = dak.dak_place_kv_heads(k, v, host)
    P, A = (torch.from_numpy(pos).cuda(), torch.from_numpy(acc).cuda()) if tracked else (None, None)
    out = dak.dak_kv_commit(kv, _i32(lens), _i32(path), _i32(n_path), T, n_new=_i32(n_new) if ragged else None, slot_pos=P, acc=A)
    _ok(dak)
    (wk, wv), wl, wp, wa = ot.commit([k, v], lens, path, n_path, n_new, pos, acc)
    K, V = _cache(kv)
    assert np.array_equal(K, wk) and np.array_equal(V, wv) and out.cpu().tolist() == wl.tolist()
    if tracked:
        assert np.array_equal(P.cpu().numpy(), wp) and np.array_equal(A.cpu().numpy(), wa)


def test_commit_bad_paths(dak):
    """Paths out of order, with a draft twice, of drafts that are none or lie past the cache: reported, the rows
    stay, nothing counts as accepted; other requests are served. Lengths and counts are clamped."""
    import torch
    T, Hkv, D, L = 8, 2, 64, 40
    paths = [[3, 1, 5], [2, 2, 3], [-1, 0, 1], [0, 1, 8], [0, 1, 6], [1, 4, 5], [0, 6, 7], [1, 2, 3]]
    n_path = [3, 3, 3, 3, 3, 3, 3, 9]
    n_new = [8, 8, 8, 9, 6, 8, 8, 8]
    lens = [4, 4, 4, 4, 4, 4, 33, -3]
    B = len(paths)
    k, v = (synth.normal_bf16(2, i, B * Hkv * L * D).reshape(B, Hkv, L, D) for i in (1, 2))
    kv = dak.dak_place_kv_heads(k, v, 3)
    P, A = torch.ones(B, Hkv, L, dtype=torch.int32, device="cuda"), torch.ones(B, Hkv, L, device="cuda")
    out = dak.dak_kv_commit(kv, _i32(lens), _i32(paths), _i32(n_path), T, n_new=_i32(n_new), slot_pos=P, acc=A)
    assert dak.dak_last_error()[0] == BOUNDS
    (wk, wv), wl, wp, wa = ot.commit([k, v], lens, paths, [3] * 8, np.minimum(n_new, T), np.ones((B, Hkv, L), int), np.ones((B, Hkv, L)))
    assert wl.tolist() == [4, 4, 4, 4, 4, 7, 33, 3]
    K, V = _cache(kv)
    assert np.array_equal(K, wk) and np.array_equal(V, wv) and out.cpu().tolist() == wl.tolist()
    assert np.array_equal(P.cpu().numpy(), wp) and np.array_equal(A.cpu().numpy(), wa)


# ---------------------------------------------------------------- fork

def _fork_case(dak, B, src_B, Hkv, D, L, src_L, of, lens, first, host, src_host, tracked, seed=1):
    import torch
    same = src_B is None
    rng = np.random.default_rng(seed)

    def make(n, l, s):
        k, v = (synth.normal_bf16(s, i, n * Hkv * l * D).reshape(n, Hkv, l, D) for i in (1, 2))
        return [k, v, rng.integers(0, 10 ** 6, (n, Hkv, l)).astype(np.int32), rng.random((n, Hkv, l)).astype(np.float32)]

    to = make(B, L, seed)
    src = to if same else make(src_B, src_L, seed + 50)
    kv = dak.dak_place_kv_heads(to[0], to[1], host)
    kw = {}
    tables = [torch.from_numpy(x).cuda() for x in to[2:]] if tracked else [None, None]
    before = rng.integers(0, 9, B)
    if not same:
        kw = dict(source=dak.dak_place_kv_heads(src[0], src[1], src_host), lens_out=_i32(before))
        if tracked:
            kw.update(source_slot_pos=torch.from_numpy(src[2]).cuda(), source_acc=torch.from_numpy(src[3]).cuda())
    out = dak.dak_kv_fork(kv, _i32(of), _i32(lens), first=None if first is None else _i32(first), slot_pos=tables[0],
                          acc=tables[1], **kw)
    status = dak.dak_last_error()[0]
    want, wl = ot.fork(to, src, of, lens, first, same, before)
    K, V = _cache(kv)
    assert np.array_equal(K, want[0]) and np.array_equal(V, want[1]) and out.cpu().tolist() == wl.tolist()
    if tracked:
        assert np.array_equal(tables[0].cpu().numpy(), want[2]) and np.array_equal(tables[1].cpu().numpy(), want[3])
    if not same:
        for a, b in zip(_cache(kw["source"]), src):
            assert np.array_equal(a, b)
    return status


@pytest.mark.parametrize("tracked", [False, True])
@pytest.mark.parametrize("B,Hkv,D,L,host", [(1, 1, 64, 5, 0), (2, 2, 128, 64, 0), (4, 2, 128, 300, 3), (16, 1, 64, 131, 16),
                                            (61, 2, 64, 200, 50), (300, 1, 64, 70, 100)])
def test_fork_in_place(dak, B, Hkv, D, L, host, tracked):
    """Any map: swaps, cycles, chains and several takers of one, each with its own first row."""
    rng = np.random.default_rng(B)
    for kind in range(3):
        of = [rng.permutation(B), rng.integers(-1, B, B), np.full(B, B - 1)][kind]
        lens = rng.integers(0, L + 1, B)
        lens[-1] = L
        first = None if kind == 0 else rng.integers(0, L + 1, B)
        assert _fork_case(dak, B, None, Hkv, D, L, L, of, lens, first, host, 0, tracked, seed=kind + 1) == 0


@pytest.mark.parametrize("tracked", [False, True])
@pytest.mark.parametrize("B,src_B,Hkv,D,L,src_L,host,src_host", [(8, 1, 2, 128, 200, 300, 0, 0), (5, 3, 1, 64, 400, 100, 2, 1),
                                                                (33, 40, 2, 64, 150, 150, 9, 60), (2, 2000, 1, 64, 20, 20, 0, 0)])
def test_fork_from_another_placement(dak, B, src_B, Hkv, D, L, src_L, host, src_host, tracked):
    rng = np.random.default_rng(B)
    of = rng.integers(-1, src_B, B)
    lens = rng.integers(0, min(L, src_L) + 1, src_B)
    lens[of[0]] = min(L, src_L)
    first = rng.integers(0, 30, B)
    assert _fork_case(dak, B, src_B, Hkv, D, L, src_L, of, lens, first, host, src_host, tracked) == 0
    assert _fork_case(dak, B, src_B, Hkv, D, L, src_L, of, lens, None, host, src_host, tracked, seed=2) == 0


def test_fork_bounds(dak):
    """Requests that are none, lengths out of range, and a cache too small for its source."""
    assert _fork_case(dak, 4, None, 2, 64, 70, 70, [9, 0, -7, 4], [500, -3, 7, 9], [-5, 2, 3, 99], 1, 0, True) == BOUNDS
    assert _fork_case(dak, 3, 2, 1, 128, 70, 200, [0, 1, 0], [200, 66], [0, 80, 60], 1, 1, True) == BOUNDS
    assert _fork_case(dak, 2, None, 1, 64, 70, 70, [0, 1], [5, 7], None, 0, 0, True) == 0  # nobody takes over


def test_fork_many_requests(dak):
    """As many requests as a call takes: the staged stretch is then a few bytes of a row."""
    B = 2048
    of = np.random.default_rng(3).permutation(B)
    assert _fork_case(dak, B, None, 1, 64, 3, 3, of, np.full(B, 3), None, 700, 0, True) == 0


def test_commit_and_fork_arguments(dak):
    import torch
    zero = np.zeros((2, 1, 64, 64), np.uint16)
    kv, other = dak.dak_place_kv_heads(zero, zero, 0), dak.dak_place_kv_heads(zero, zero, 0)
    two, path = _i32([1, 1]), _i32([[0], [0]])
    for a in ((two, path[0], two, 4), (two[:1], path, two, 4), (two, path, two.long(), 4), (two, path.cpu(), two, 4)):
        with pytest.raises(ValueError):
            dak.dak_kv_commit(kv, *a)
    with pytest.raises(dak.DakError):
        dak.dak_kv_commit(kv, two, path, two, 0)
    with pytest.raises(dak.DakError):
        dak.dak_kv_commit(kv, two, path, _i32([0, 0]), 4, lens_out=two)
    t = torch.zeros(2, 1, 64, dtype=torch.int32, device="cuda")
    for a, kw in (((two[:1], two), {}), ((two, two.cpu()), {}), ((two, two), dict(first=path)), ((two, two), dict(source=other)),
                  ((two, two), dict(source_slot_pos=t)), ((two, two), dict(slot_pos=t[:1]))):
        with pytest.raises(ValueError):
            dak.dak_kv_fork(kv, *a, **kw)
    with pytest.raises(dak.DakError):
        dak.dak_kv_fork(kv, two, _i32([1, 1]), lens_out=two)
    with pytest.raises(dak.DakError):
        dak.dak_kv_fork(kv, two, two, source=other, lens_out=_i32([0, 0]), slot_pos=t)
    _ok(dak)

"""Drafted trees and forked caches without a GPU: the oracle's own pins, masks from parents, plans of
several axes, and every refusal that is decided before a CUDA call."""
import ctypes

import numpy as np
import pytest

import synth
from oracle import cache as oc
from oracle import tree as ot
from test_cache_ops import ALIGN, CUDA, INVALID, UNSUPPORTED, _kv, dak, no_gpu  # noqa: F401

pytestmark = pytest.mark.cpu


# ---------------------------------------------------------------- the oracle

def test_oracle_chain_is_single_tokens():
    """A chain's tokens are decode steps, each over one row more than the one before."""
    B, T, Hq, Hkv, D, L = 2, 3, 4, 2, 64, 20
    rng = np.random.default_rng(1)
    q, k, v = rng.standard_normal((B, T, Hq, D)), rng.standard_normal((B, Hkv, L, D)), rng.standard_normal((B, Hkv, L, D))
    o, spread, reach = ot.attention(q, k, v, [10, 0])
    for t in range(T):
        want, _, s, r = oc.attention(q[:, t], k, v, [10 + t + 1, t + 1])
        np.testing.assert_allclose(o[:, t], want, atol=1e-14)
        np.testing.assert_allclose(spread[:, t], s, atol=1e-14)
        np.testing.assert_allclose(reach[:, t], r, atol=1e-14)


def test_oracle_commit_and_fork():
    k = np.arange(2 * 1 * 8).reshape(2, 1, 8)
    (k2,), lens, pos, acc = ot.commit([k], [2, 3], [[1, 3], [0, 9]], [2, 2], [4, 4], slot_pos=k + 100, acc=k * 1.0)
    assert k2[0, 0].tolist() == [0, 1, 3, 5, 4, 5, 6, 7] and k2[1].tolist() == k[1].tolist()  # draft 9 is none
    assert lens.tolist() == [4, 3] and pos[0, 0].tolist() == [100, 101, 103, 105, -1, -1, 106, 107]
    assert acc[1, 0].tolist() == [8, 9, 10, 0, 0, 0, 0, 15]
    (k3,), lens = ot.fork([k], [k], [1, 0], [5, 7], [2, 0])
    assert k3[0, 0].tolist() == [0, 1, 10, 11, 12, 13, 14, 7] and k3[1, 0, :6].tolist() == [0, 1, 2, 3, 4, 13]
    assert lens.tolist() == [7, 5]


def test_oracle_axes_with_equal_positions_are_one():
    f = oc.inv_freq(32)
    x = synth.normal_bf16(3, 1, 4 * 2 * 64).reshape(4, 2, 64)
    p = np.array([0, 5, 900, 77])
    for inter in (False, True):
        y = ot.rotate_axes(x, np.stack([p, p, p], 1), [i % 3 for i in range(16)], f, inter)
        np.testing.assert_allclose(y, oc.rotate(x, p, f, inter), atol=1e-14)


# ---------------------------------------------------------------- masks and plans

def test_tree_mask(dak):
    m, d = dak.dak_tree_mask([-1, 0, 0, 1, -1, 3], device="cpu")
    assert m.shape == (1, 6, 1) and m[0, :, 0].tolist() == [1, 3, 5, 11, 16, 43]
    assert d.tolist() == [[0, 1, 1, 2, 0, 3]]
    T = 130
    m, d = dak.dak_tree_mask([list(range(-1, T - 1)), [-1] * T], device="cpu")  # a chain, and all siblings
    seen = ot.bits(m.numpy(), T)
    assert m.shape == (2, T, 3) and (seen[0] == np.tril(np.ones((T, T), bool))).all() and (seen[1] == np.eye(T, dtype=bool)).all()
    assert d[0].tolist() == list(range(T)) and not d[1].any()
    for bad in ([0], [-2], [-1, 1], [[-1], [0]], [], [[[-1]]]):
        with pytest.raises(ValueError):
            dak.dak_tree_mask(bad, device="cpu")


def test_rope_axes_make(dak):
    r = dak.dak_rope_make(128, rot_dim=96)
    p = dak.dak_rope_axes_make(r, [i % 3 for i in range(48)])
    assert p.n_axes == 3 and list(p.axis)[:48] == [i % 3 for i in range(48)] and not any(list(p.axis)[48:])
    assert list(p.rope.turns) == list(r.turns) and p.rope.rot_dim == 96
    assert dak.dak_rope_axes_make(r).n_axes == 1 and dak.dak_rope_axes_make(r, [0] * 48, n_axes=4).n_axes == 4
    with pytest.raises(ValueError):
        dak.dak_rope_axes_make(r, [0] * 47)
    for kw in (dict(axis=[4] * 48), dict(axis=[2] * 48, n_axes=2), dict(axis=[-1] * 48, n_axes=1), dict(n_axes=0), dict(n_axes=5)):
        with pytest.raises(dak.DakError) as e:
            dak.dak_rope_axes_make(r, **kw)
        assert e.value.status == INVALID
    out, byref = dak.dak_rope_axes_plan(), ctypes.byref
    assert dak.lib.dak_rope_axes_make(None, 1, None, byref(out)) == INVALID
    assert dak.lib.dak_rope_axes_make(byref(r), 1, None, None) == INVALID
    for bad in (dict(head_dim=96, rot_dim=64), dict(head_dim=128, rot_dim=130), dict(head_dim=64, rot_dim=7), dict(head_dim=64)):
        assert dak.lib.dak_rope_axes_make(byref(dak.dak_rope_plan(**bad)), 1, None, byref(out)) == INVALID


# ---------------------------------------------------------------- refusals before any CUDA call

def test_append_rope_axes_refusals(dak, no_gpu):
    kv, rope = _kv(), dak.dak_rope_axes_make(dak.dak_rope_make(128), [0, 1] * 32)
    row, q_row = 4 * 128, 8 * 128
    good = dict(KV=ctypes.byref(kv), rope=ctypes.byref(rope), q=0x100000, k=0x200000, v=0x300000, fp32=0, T=3, Hq=8,
                qp=q_row, kp=row, vp=row, slots=0x4000, pos=0x5000, n_new=0x6000, q_out=0x400000, slot_pos=0x7000,
                acc=0x8000, stream=None)

    def call(**kw):
        a = dict(good, **kw)
        return dak.lib.dak_kv_append_rope_axes(*[a[k] for k in good])

    assert call() == CUDA and call(n_new=None, slot_pos=None, acc=None) == CUDA
    broken = dak.dak_rope_axes_plan.from_buffer_copy(rope)
    broken.axis[63] = 2
    none = dak.dak_rope_axes_plan.from_buffer_copy(rope)
    none.n_axes = 0
    for kw in (dict(KV=None), dict(KV=ctypes.byref(_kv(kind=0))), dict(KV=ctypes.byref(_kv(D=64))), dict(rope=None),
               dict(rope=ctypes.byref(broken)), dict(rope=ctypes.byref(none)), dict(pos=None), dict(slots=None),
               dict(q_out=None), dict(T=0), dict(kp=row - 8), dict(q_out=0x100000)):
        assert call(**kw) == INVALID, kw
    for kw in (dict(q=0x100008), dict(pos=0x5002), dict(acc=0x8001), dict(kp=row + 2)):
        assert call(**kw) == ALIGN, kw


def test_attn_tree_refusals(dak, no_gpu):
    kv, r = _kv(), ctypes.byref
    size = dak.lib.dak_attn_tree_workspace_bytes
    n = size(r(kv), 70, 8)
    assert n > 0
    for p, T, hq in ((None, 1, 8), (r(_kv(kind=0)), 1, 8), (r(kv), 0, 8), (r(kv), 257, 8), (r(kv), 1, 0), (r(kv), 1, 6),
                     (r(kv), 1, 68)):
        assert size(p, T, hq) == 0
    good = dict(Q=0x1000000, KV=r(kv), lens=0x1000, T=70, mask=0x3000, pitch=140, n_new=0x5000, Hq=8, scale=0.0, O=0x2000000,
                f32=0, ws=0x4000000, n=n, tun=None, stream=None)

    def call(**kw):
        a = dict(good, **kw)
        return dak.lib.dak_attn_tree(*[a[k] for k in good])

    assert call() == CUDA and call(pitch=0) == CUDA and call(mask=None, pitch=1, n_new=None) == CUDA and call(pitch=1000) == CUDA
    q_bytes = 2 * 70 * 8 * 128 * 2
    for kw in (dict(Q=None), dict(KV=None), dict(KV=r(_kv(kind=0))), dict(lens=None), dict(O=None), dict(ws=None), dict(T=0),
               dict(Hq=0), dict(Hq=6), dict(n=n - 1), dict(pitch=139), dict(pitch=-1), dict(O=0x1000000),
               dict(O=0x1000000 + q_bytes - 16), dict(O=0x1000000 - 16), dict(f32=1, O=0x1000000 - 2 * q_bytes + 16)):
        assert call(**kw) == INVALID, kw
    assert call(O=0x1000000 + q_bytes) == CUDA and call(f32=1, O=0x1000000 - 2 * q_bytes) == CUDA
    assert call(T=257, n=1 << 40, pitch=257 * 5) == UNSUPPORTED and call(Hq=68, n=1 << 40) == UNSUPPORTED
    for kw in (dict(Q=0x1000008), dict(O=0x2000008), dict(ws=0x4000008), dict(lens=0x1002), dict(mask=0x3004),
               dict(n_new=0x5001)):
        assert call(**kw) == ALIGN, kw


def test_commit_refusals(dak, no_gpu):
    good = dict(KV=ctypes.byref(_kv()), lens=0x1000, T=10, n_new=0x1100, path=0x2000, P=4, n_path=0x1200, out=0x1300,
                pos=0x4000, acc=0x5000, stream=None)

    def call(**kw):
        a = dict(good, **kw)
        return dak.lib.dak_kv_commit(*[a[k] for k in good])

    assert call() == CUDA and call(n_new=None, pos=None, acc=None, P=10) == CUDA
    for kw in (dict(KV=None), dict(KV=ctypes.byref(_kv(kind=0))), dict(lens=None), dict(path=None), dict(n_path=None),
               dict(out=None), dict(T=0), dict(P=0), dict(P=11), dict(out=0x1000), dict(out=0x1104), dict(out=0x1200 - 4),
               dict(out=0x2000 + 28)):
        assert call(**kw) == INVALID, kw
    assert call(T=257) == UNSUPPORTED and call(T=256, P=256) == CUDA
    for name in ("lens", "n_new", "path", "n_path", "out", "pos", "acc"):
        assert call(**{name: good[name] + 2}) == ALIGN, name


def test_fork_refusals(dak, no_gpu):
    kv, other, r = _kv(), _kv(B=5, L=300), ctypes.byref
    kp = ctypes.pointer(kv)
    good = dict(KV=kp, src=kp, of=0x1000, lens=0x1100, first=0x1200, out=0x1300, spos=0x100000, pos=0x100000, sacc=0x200000,
                acc=0x200000, stream=None)

    def call(**kw):
        a = dict(good, **kw)
        return dak.lib.dak_kv_fork(*[a[k] for k in good])

    two = dict(src=r(other), spos=0x300000, sacc=0x400000)
    assert call() == CUDA and call(**two) == CUDA and call(first=None, spos=None, pos=None, sacc=None, acc=None) == CUDA
    table = 2 * 4 * 100 * 4
    for kw in (dict(KV=None), dict(src=None), dict(src=r(_kv(kind=0))), dict(of=None), dict(lens=None), dict(out=None),
               dict(src=r(_kv(H=2))), dict(src=r(_kv(D=64))), dict(src=r(_kv(device=1))), dict(spos=None), dict(pos=None),
               dict(sacc=None), dict(acc=None), dict(spos=0x300000), dict(acc=0x300000), dict(out=0x1000), dict(out=0x1104),
               dict(out=0x1200 + 4), dict(two, spos=0x100000 + table - 4), dict(two, out=0x1100 + 16)):
        assert call(**kw) == INVALID, kw
    assert call(**dict(two, spos=0x100000 + table)) == CUDA and call(**dict(two, out=0x1100 + 20)) == CUDA
    assert call(KV=r(_kv(B=2049)), **two) == UNSUPPORTED and call(**dict(two, src=r(_kv(B=2049)))) == UNSUPPORTED
    for name in ("of", "lens", "first", "out"):
        assert call(**{name: good[name] + 2}) == ALIGN, name
    assert call(spos=0x100002, pos=0x100002) == ALIGN and call(sacc=0x200001, acc=0x200001) == ALIGN

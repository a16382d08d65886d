"""The cache operators without a GPU: the oracle's own pins, the rotation's frequencies and their
fixed-point form, and every refusal that is decided before a CUDA call."""
import ctypes
import math

import numpy as np
import pytest

import synth
from oracle import attention as oa
from oracle import cache as oc

pytestmark = pytest.mark.cpu

INVALID, ALIGN, CUDA, UNSUPPORTED = 1, 2, 5, 7


@pytest.fixture(scope="module")
def dak():
    import __graft_entry__
    __graft_entry__.build()
    import direct_host_memory_gb300 as m
    return m


# ---------------------------------------------------------------- the oracle

def test_oracle_rotation_is_a_rotation():
    f = oc.inv_freq(64)
    x = synth.normal_bf16(3, 1, 5 * 2 * 128).reshape(5, 2, 128)
    pos = [0, 1, 77, 4096, 1000000]
    for inter in (False, True):
        y = oc.rotate(x, pos, f, inter)
        x64 = oc._f64(x)
        assert np.array_equal(y[0], x64[0])  # position 0 turns nothing
        assert np.array_equal(y[..., 64:], x64[..., 64:])  # past rot_dim nothing turns
        np.testing.assert_allclose((y ** 2).sum(-1), (x64 ** 2).sum(-1), rtol=1e-12)
        back = oc.rotate(y, [-p for p in pos], f, inter)
        np.testing.assert_allclose(back, x64, atol=1e-12)
        # the scores of rotated q and k depend on the distance alone
        q = oc.rotate(np.repeat(x64[:1], 2, 0), [100, 5100], f, inter)
        k = oc.rotate(np.repeat(x64[1:2], 2, 0), [40, 5040], f, inter)
        s = (q * k).sum(-1)
        np.testing.assert_allclose(s[0], s[1], rtol=1e-9)


def test_oracle_attention_matches_the_plain_one():
    q, k, v = synth.attn_inputs(3, 8, 2, 64, 50, seed=4)
    lens = [50, 7, 1]
    o, w, _, _ = oc.attention(q, k, v, lens)
    np.testing.assert_allclose(o, oa.decode_attention_ref(q, k, v, seq_lens=lens), atol=1e-13)
    np.testing.assert_allclose(w.sum(-1), 4.0)  # four query heads a kv head
    # a prefix is nothing but rows in front
    o2, w2, _, _ = oc.attention(q, k[:, :, 30:], v[:, :, 30:], [20] * 3, (k[1:2, :, :30], v[1:2, :, :30]),
                                [-1, 0, -1])
    np.testing.assert_allclose(o2[1], oa.decode_attention_ref(q, k, v)[1], atol=1e-13)
    assert (w2[1].sum(-1) < 4.0).all()
    o3, w3, _, _ = oc.attention(q, k, v, [0, 0, 0])
    assert not o3.any() and not w3.any()


def test_oracle_eviction():
    acc = np.array([[[5, 1, np.nan, 3, -0.0, 0.0, 9, 2, 77]]], np.float32)
    pos = np.arange(9, dtype=np.int64)[None, None]
    lens, src, a, p = oc.evict([8], 4, 1, acc, pos)
    # slot 7 is newest; then 9 (6), 5 (0), 3 (3); freed slots 1, 2 take 6, 7
    assert lens.tolist() == [4] and src[0, 0].tolist() == [0, 6, 7, 3]
    assert a[0, 0].tolist() == [5, 9, 2, 3, 0, 0, 0, 0, 77] and p[0, 0].tolist() == [0, 6, 7, 3, -1, -1, -1, -1, 8]
    # the zeros are equal, the lower slot stays; NaN goes first
    _, src, _, _ = oc.evict([8], 7, 0, acc, pos)
    assert src[0, 0].tolist() == [0, 1, 7, 3, 4, 5, 6]
    _, src, _, _ = oc.evict([3], 4, 0, acc, pos)
    assert src[0, 0].tolist() == [0, 1, 2, -1]


# ---------------------------------------------------------------- frequencies

@pytest.mark.parametrize("scaling", ["none", "linear", "ntk", "by_parts"])
@pytest.mark.parametrize("D,rot", [(128, 128), (128, 64), (64, 2), (64, 56), (128, 120)])
def test_rope_make_matches_the_formulas(dak, scaling, D, rot):
    for factor, orig in ((8.0, 8192.0), (1.0, 4096.0), (40.0, 100.0)):
        r = dak.dak_rope_make(D, rot_dim=rot, theta=10000.0, scaling=scaling, factor=factor, orig_len=orig,
                              low_turns=1.0, high_turns=4.0, attn_scale=1.25, interleaved=True)
        assert (r.head_dim, r.rot_dim, r.interleaved, r.scale) == (D, rot, 1, 1.25)
        f = oc.inv_freq(rot, 10000.0, scaling, factor, orig, 1.0, 4.0)
        got = np.array([r.turns[i] for i in range(rot // 2)], np.float64) * 2.0 ** -64 * 2 * math.pi
        # pow and the division by 2 pi are good to a few units of 2^-53, the fraction to 2^-65 turns
        np.testing.assert_allclose(got, f, rtol=2e-15, atol=2.0 ** -64 * 2 * math.pi)
        assert not any(r.turns[i] for i in range(rot // 2, 64))


def test_rope_turns_are_exact_far_out(dak):
    """position * turns mod 2^64 against exact rational arithmetic on the double frequencies."""
    from fractions import Fraction
    f = [1.0, 0.123456789, 3.3e-6, 1e-12, 25.0, -0.5, 0.0]
    r = dak.dak_rope_from_freqs(64, f)
    assert r.rot_dim == 14 and r.scale == 1.0
    two_pi = Fraction(6.283185307179586) + Fraction(2.4492935982947064e-16)  # 2 pi to 2^-105
    for i, x in enumerate(f):
        for pos in (1, 4095, 1000003, 2 ** 31 - 1, -7):
            turn = ((pos * r.turns[i]) % 2 ** 64) / 2 ** 64
            want = float((Fraction(x) * pos / two_pi) % 1)
            gap = abs(turn - want)
            # the double division leaves 2^-52 relative of the turns, the fraction 2^-65 * pos
            assert min(gap, 1 - gap) <= abs(pos) * (2.0 ** -65 + abs(x) / 6.28 * 2.0 ** -51) + 1e-15


def test_rope_refusals(dak):
    for kw, status in (
            (dict(rot_dim=3), INVALID), (dict(rot_dim=130), INVALID), (dict(theta=float("nan")), INVALID),
            (dict(theta=float("inf")), INVALID), (dict(factor=float("inf")), INVALID),
            (dict(scaling="by_parts"), INVALID), (dict(scaling="by_parts", orig_len=-1.0), INVALID),
            (dict(scaling="by_parts", orig_len=4096.0, low_turns=4.0, high_turns=4.0), INVALID),
            (dict(scaling="by_parts", orig_len=4096.0, low_turns=-1.0, high_turns=4.0), INVALID),
            (dict(attn_scale=float("inf")), INVALID), (dict(attn_scale=float("nan")), INVALID)):
        with pytest.raises(dak.DakError) as e:
            dak.dak_rope_make(128, **kw)
        assert e.value.status == status, kw
    with pytest.raises(dak.DakError) as e:
        dak.dak_rope_make(96)
    assert e.value.status == UNSUPPORTED
    with pytest.raises(ValueError):
        dak.dak_rope_make(128, scaling="spiral")
    for f in ([], [0.1] * 65, [float("inf")], [float("nan")]):
        with pytest.raises(dak.DakError) as e:
            dak.dak_rope_from_freqs(128, f)
        assert e.value.status == INVALID
    c = dak.dak_rope_config(scaling=9)
    assert dak.lib.dak_rope_make(128, ctypes.byref(c), ctypes.byref(dak.dak_rope_plan())) == INVALID
    assert dak.lib.dak_rope_make(128, None, ctypes.byref(dak.dak_rope_plan())) == INVALID
    assert dak.lib.dak_rope_make(128, ctypes.byref(c), None) == INVALID


# ---------------------------------------------------------------- refusals before any CUDA call

class _Kv(ctypes.Structure):
    """The library's placement of a KV cache, written by hand so that argument checks run where no
    cache can be allocated. Its fields are checked through dak_placement_info below."""
    _fields_ = [("kind", ctypes.c_int), ("device", ctypes.c_int), ("glu", ctypes.c_int), ("host_ptr", ctypes.c_void_p),
                ("host_dev", ctypes.c_void_p), ("hbm_ptr", ctypes.c_void_p), ("host_bytes", ctypes.c_int64),
                ("hbm_bytes", ctypes.c_int64), ("M", ctypes.c_int64), ("K", ctypes.c_int64), ("K_pad", ctypes.c_int64),
                ("tile_m", ctypes.c_int), ("T", ctypes.c_int), ("h", ctypes.c_int), ("tile_bytes", ctypes.c_int64),
                ("B", ctypes.c_int), ("H_kv", ctypes.c_int), ("L", ctypes.c_int), ("D", ctypes.c_int),
                ("h_s", ctypes.c_int), ("head_bytes", ctypes.c_int64)]


def _kv(B=2, H=4, L=100, D=128, kind=1, device=0):
    hb = -(-L // 64) * 2 * 64 * D * 2
    return _Kv(kind=kind, device=device, host_ptr=0x7000, hbm_ptr=0x9000, host_bytes=3 * hb, hbm_bytes=(B * H - 3) * hb,
               B=B, H_kv=H, L=L, D=D, h_s=3, head_bytes=hb)


@pytest.fixture(scope="module")
def no_gpu():
    import torch
    if torch.cuda.is_available():
        pytest.skip("made-up addresses: only where no kernel can launch")


def test_handmade_placement_is_the_librarys(dak, no_gpu):
    p = _kv()
    hb, gb, u, hu = (ctypes.c_int64() for _ in range(4))
    r = ctypes.byref
    assert dak.lib.dak_placement_info(r(p), r(hb), r(gb), r(u), r(hu)) == 0
    assert (hb.value, gb.value, u.value, hu.value) == (p.host_bytes, p.hbm_bytes, 8, 3)
    h, g = ctypes.c_void_p(), ctypes.c_void_p()
    assert dak.lib.dak_placement_data(r(p), r(h), r(g)) == 0 and (h.value, g.value) == (0x7000, 0x9000)
    assert dak.lib.dak_placement_data(r(p), None, None) == 0
    assert dak.lib.dak_placement_data(None, r(h), r(g)) == INVALID
    assert dak.lib.dak_kv_evict_workspace_bytes(r(p)) >= 8 * (1 + 100) * 4
    assert dak.lib.dak_kv_evict_workspace_bytes(r(_kv(kind=0))) == 0
    assert dak.lib.dak_kv_evict_workspace_bytes(None) == 0


def test_append_rope_refusals(dak, no_gpu):
    kv, rope = _kv(), dak.dak_rope_make(128)
    row, q_row = 4 * 128, 8 * 128
    good = dict(KV=ctypes.byref(kv), rope=ctypes.byref(rope), q=0x100000, k=0x200000, v=0x300000, fp32=0, T=3, Hq=8,
                qp=q_row, kp=row, vp=row, slots=0x4000, pos=0x5000, n_new=0x6000, q_out=0x400000, slot_pos=0x7000,
                stream=None)

    def call(**kw):
        a = dict(good, **kw)
        return dak.lib.dak_kv_append_rope(*[a[k] for k in good])

    assert call() == CUDA  # every argument passed, and there is no device
    for kw in (dict(KV=None), dict(KV=ctypes.byref(_kv(kind=0))), dict(rope=None), dict(q=None), dict(k=None),
               dict(v=None), dict(slots=None), dict(q_out=None), dict(T=0), dict(T=-1), dict(Hq=-1), dict(qp=q_row - 8),
               dict(kp=row - 8), dict(vp=0), dict(rope=ctypes.byref(dak.dak_rope_make(64))), dict(T=1 << 30),
               dict(rope=ctypes.byref(dak.dak_rope_plan(head_dim=128, rot_dim=130))),
               dict(rope=ctypes.byref(dak.dak_rope_plan(head_dim=128, rot_dim=0))),
               # q_out over one of the inputs
               dict(q_out=0x100000), dict(q_out=0x200000 + 16), dict(q_out=0x300000 - 16),
               dict(q_out=0x100000 + (5 * q_row + q_row) * 2 - 16)):
        assert call(**kw) == INVALID, kw
    for kw in (dict(q=0x100008), dict(k=0x200002), dict(v=0x300004), dict(q_out=0x400008), dict(qp=q_row + 4),
               dict(kp=row + 2), dict(vp=row + 1), dict(slots=0x4002), dict(pos=0x5001), dict(n_new=0x6002),
               dict(slot_pos=0x7003)):
        assert call(**kw) == ALIGN, kw
    assert call(fp32=1, qp=q_row + 4, q_out=0x800000) == CUDA  # 16 bytes are four fp32 elements
    assert call(q=None, Hq=0, qp=0, q_out=None, pos=None, n_new=None, slot_pos=None) == CUDA


def test_evict_refusals(dak, no_gpu):
    kv = _kv()
    good = dict(KV=ctypes.byref(kv), lens=0x1000, keep=50, recent=10, acc=0x100000, acc_out=0x100000, pos=0x200000,
                pos_out=0x300000, lens_out=0x2000, src=0x400000, ws=0x500000,
                n=dak.lib.dak_kv_evict_workspace_bytes(ctypes.byref(kv)), stream=None)

    def call(**kw):
        a = dict(good, **kw)
        return dak.lib.dak_kv_evict(*[a[k] for k in good])

    assert call() == CUDA
    assert call(keep=100, recent=100, src=None) == CUDA
    for kw in (dict(KV=None), dict(KV=ctypes.byref(_kv(kind=0))), dict(lens=None), dict(acc=None), dict(acc_out=None),
               dict(pos=None), dict(pos_out=None), dict(lens_out=None), dict(ws=None), dict(keep=0), dict(keep=101),
               dict(keep=-1), dict(recent=-1), dict(recent=51), dict(n=good["n"] - 1), dict(acc_out=0x100004),
               dict(pos_out=0x200000 + 8 * 100 * 4 - 4), dict(lens_out=0x1000), dict(lens_out=0x1004)):
        assert call(**kw) == INVALID, kw
    for kw in (dict(lens=0x1002), dict(acc=0x100001, acc_out=0x900000), dict(acc_out=0x900002), dict(pos=0x600001),
               dict(pos_out=0x300002), dict(lens_out=0x2001), dict(src=0x400002), dict(ws=0x500008)):
        assert call(**kw) == ALIGN, kw


def test_serving_attention_refusals(dak, no_gpu):
    kv, pre = _kv(), _kv(B=3, L=1000)
    r = ctypes.byref
    ws_acc = dak.lib.dak_attn_acc_workspace_bytes(r(kv), 8, 0)
    assert ws_acc >= 2 * 8 * (100 + 130) * 4
    for bad in (dict(p=None), dict(p=r(_kv(kind=0))), dict(hq=0), dict(hq=6), dict(split=2000)):
        a = dict(dict(p=r(kv), hq=8, split=0), **bad)
        assert dak.lib.dak_attn_acc_workspace_bytes(a["p"], a["hq"], a["split"]) == 0
        assert dak.lib.dak_attn_prefix_workspace_bytes(a["p"], r(pre), a["hq"], a["split"], 1) == 0
    assert dak.lib.dak_attn_prefix_workspace_bytes(r(kv), None, 8, 0, 0) == 0
    good = dict(Q=0x100000, KV=r(kv), lens=0x1000, Hq=8, scale=0.0, O=0x200000, f32=0, acc_in=0x300000,
                acc_out=0x300000, ws=0x400000, n=ws_acc, tun=None, stream=None)

    def acc(**kw):
        a = dict(good, **kw)
        return dak.lib.dak_attn_acc(*[a[k] for k in good])

    assert acc() == CUDA
    for kw in (dict(Q=None), dict(KV=None), dict(KV=r(_kv(kind=0))), dict(O=None), dict(acc_out=None), dict(ws=None),
               dict(Hq=0), dict(Hq=6), dict(n=ws_acc - 1), dict(acc_in=0x300004),
               dict(tun=r(dak.dak_tuning(n_split=1025)))):
        assert acc(**kw) == INVALID, kw
    assert acc(Hq=68, n=1 << 40) == UNSUPPORTED  # 17 query heads a kv head
    assert acc(KV=r(_kv(L=34_000_000)), n=1 << 50, acc_in=None, acc_out=1 << 40) == UNSUPPORTED
    assert acc(KV=r(_kv(L=33_000_000)), n=1 << 50, acc_in=None, acc_out=1 << 40) == CUDA
    for kw in (dict(Q=0x100008), dict(O=0x200008), dict(ws=0x400008), dict(acc_in=0x500002), dict(acc_out=0x500001)):
        assert acc(**kw) == ALIGN, kw

    ws_pre = dak.lib.dak_attn_prefix_workspace_bytes(r(kv), r(pre), 8, 0, 0)
    good2 = dict(Q=0x100000, KV=r(kv), lens=0x1000, P=r(pre), plens=0x2000, of=0x3000, Hq=8, scale=0.0, O=0x200000,
                 f32=0, acc_in=None, acc_out=None, ws=0x400000, n=ws_pre, tun=None, stream=None)

    def prefix(**kw):
        a = dict(good2, **kw)
        return dak.lib.dak_attn_prefix(*[a[k] for k in good2])

    assert prefix() == CUDA
    assert prefix(lens=None, plens=None, of=None) == CUDA
    for kw in (dict(P=None), dict(P=r(_kv(kind=0))), dict(P=r(_kv(H=2))), dict(P=r(_kv(D=64))),
               dict(P=r(_kv(device=1))), dict(n=ws_pre - 1), dict(Q=None), dict(Hq=7),
               dict(acc_out=0x300000)):  # the scores need more workspace
        assert prefix(**kw) == INVALID, kw
    assert prefix(acc_out=0x300000, n=dak.lib.dak_attn_prefix_workspace_bytes(r(kv), r(pre), 8, 0, 1)) == CUDA
    assert prefix(P=r(_kv(B=1025, L=64)), n=1 << 40) == UNSUPPORTED
    assert prefix(P=r(_kv(B=1024, L=64)), n=1 << 40) == CUDA

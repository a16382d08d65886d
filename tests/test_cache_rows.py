"""What the cache operators' calls refuse or promise beyond tests/test_cache_ops.py, without a GPU."""
import ctypes

import pytest

from test_cache_ops import ALIGN, CUDA, INVALID, _kv, dak, no_gpu  # noqa: F401 (fixtures)

pytestmark = pytest.mark.cpu


def test_append_rope_acc_refusals(dak, no_gpu):  # noqa: F811
    kv, rope = _kv(), dak.dak_rope_make(128)
    good = dict(KV=ctypes.byref(kv), rope=ctypes.byref(rope), q=0x100000, k=0x200000, v=0x300000, fp32=0, T=3, Hq=8,
                qp=8 * 128, kp=4 * 128, vp=4 * 128, slots=0x4000, pos=0x5000, n_new=0x6000, q_out=0x400000,
                slot_pos=0x7000, acc=0x8000, stream=None)

    def call(**kw):
        a = dict(good, **kw)
        return dak.lib.dak_kv_append_rope_acc(*[a[k] for k in good])

    assert call() == CUDA and call(acc=None) == CUDA and call(slot_pos=None) == CUDA
    assert call(acc=0x8002) == ALIGN
    assert call(KV=None) == INVALID and call(slots=None) == INVALID and call(T=0) == INVALID


class _Placement:
    host_bytes = 0


def test_forward_after_several_new_tokens_is_launched_without_pdl(dak, monkeypatch):  # noqa: F811
    """Programmatic launch lets attention read all rows but the newest before the kernel in front of it has
    ended: after append_rope of more than one token the next forward, and only that one, is launched
    without it."""
    import torch
    from direct_host_memory_gb300 import _lib
    seen = []

    def attn(q, KV, **kw):
        seen.append(kw["tuning"].get("pdl", 0))
        return q

    for name, fake in (("dak_place_kv_heads", lambda *a: _Placement()), ("dak_attn_default_split", lambda p: 1),
                       ("dak_attn_workspace_bytes", lambda *a: 0), ("dak_attn", attn),
                       ("dak_attn_prefix", lambda q, *a, **kw: q), ("dak_kv_append", lambda *a: None),
                       ("dak_kv_append_rope", lambda *a, **kw: None)):
        monkeypatch.setattr(_lib, name, fake)
    B, Hkv, D = 2, 2, 64
    z = torch.zeros(B, Hkv, 96, D, dtype=torch.bfloat16)
    q, one, many = torch.zeros(B, 4, D), torch.zeros(B, Hkv, D), torch.zeros(B, 3, Hkv, D)
    at = torch.zeros(B, dtype=torch.int32)
    m = dak.SplitK_FlashAttn(z, z, tuning=dict(pdl=2, hbm_window=3))
    m(q)
    m.append(one, one, at)
    m(q)
    m.append_rope(None, None, one, one, at)
    m.append_rope(None, None, one[:, None], one[:, None], at)
    m(q)
    assert seen == [2, 2, 2]
    m.append_rope(None, None, many, many, at)
    m.append_rope(None, None, one, one, at)
    m(q)
    m(q)
    assert seen[3:] == [0, 2]
    m.append_rope(None, None, many, many, at)
    m(q, prefix=_Placement())  # waits for the rows itself
    m(q)
    assert seen[5:] == [2] and m.tuning == dict(pdl=2, hbm_window=3)


@pytest.mark.parametrize("theta", [500000.0, 10000.0])
def test_rope_turns_are_as_good_as_the_header_says(dak, theta):  # noqa: F811
    """position * turns mod 2^64 within |position| (|f| 2^-55 + 2^-65) turns of the double frequency's angle, by
    rational arithmetic; and no bound that does not grow with the position holds."""
    from fractions import Fraction
    two_pi = Fraction(6.283185307179586) + Fraction(2.4492935982947064e-16)  # 2 pi to 2^-105
    f = [theta ** (-2.0 * i / 128) for i in range(64)] + [-0.75, 3.5]
    worst = 0.0
    for r, part in ((dak.dak_rope_from_freqs(128, f[:64]), f[:64]), (dak.dak_rope_from_freqs(128, f[64:]), f[64:])):
        for i, x in enumerate(part):
            for pos in (1, 4095, 1000000, 2 ** 31 - 1, -2 ** 31):
                want = (Fraction(x) * pos / two_pi) % 1
                gap = abs(Fraction((pos * r.turns[i]) % 2 ** 64, 2 ** 64) - want)
                gap = min(gap, 1 - gap)
                assert gap <= abs(pos) * (abs(Fraction(x)) / 2 ** 55 + Fraction(1, 2 ** 65)) + Fraction(1, 2 ** 80)
                worst = max(worst, float(gap))
    assert worst > 2.0 ** -33

"""NaN and infinities in rows that count: a softmax over such scores is NaN, and the attention of the cache
operators says so instead of answering zero; what the rows of others hold stays theirs."""
import numpy as np
import pytest

import synth
from gpu_util import bits_of, to_dev, to_np
from oracle import cache as oc

pytestmark = [pytest.mark.gpu, pytest.mark.filterwarnings("ignore::RuntimeWarning")]

NAN, INF, NINF = 0x7FC0, 0x7F80, 0xFF80


@pytest.fixture(scope="module")
def dak(cuda_ok):
    import __graft_entry__
    __graft_entry__.build()
    import direct_host_memory_gb300 as m
    return m


def _i32(x):
    import torch
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def _same_nans(dak, got, want, clean):
    """NaN exactly where the definition has NaN, and elsewhere the bits of the call without the odd values."""
    assert dak.dak_last_error()[0] == 0
    nan = np.isnan(want)
    assert nan.any() and not nan.all()
    assert np.array_equal(np.isnan(to_np(got)), nan)
    same = bits_of(got) == bits_of(clean)
    return same | nan


CASES = [
    # B, Hq, Hkv, D, L, prefix rows (0: none), fp32
    (4, 8, 2, 128, 200, 0, False),
    (4, 8, 2, 64, 200, 0, True),
    (4, 16, 1, 128, 70, 0, False),
    (200, 16, 4, 64, 20, 0, False),   # the merge by warps
    (4, 8, 2, 128, 70, 150, False),
    (4, 8, 2, 64, 70, 150, True),
    (70, 8, 2, 128, 20, 150, False),  # two row tiles
    (160, 16, 4, 64, 9, 40, True),    # the merge by warps
]


@pytest.mark.parametrize("case", CASES, ids=str)
def test_nan_and_infinite_scores(dak, case):
    import torch
    B, Hq, Hkv, D, L, Lp, fp32 = case
    G = Hq // Hkv
    q, k, v = synth.attn_inputs(B, Hq, Hkv, D, L, seed=L + D)
    lens = [L] * B
    lens[-1] = 0
    prefix = pre = None
    if Lp:
        prefix = synth.attn_inputs(2, Hq, Hkv, D, Lp, seed=3)[1:]
        pre = dak.dak_place_kv_heads(*prefix, 0)
    of = [b % 2 - (b == B - 1) * 2 for b in range(B)]  # the last request has no rows at all
    of[-1] = -1
    clean = None
    for odd in (None, "q", "k", "+inf", "-inf"):
        q2, k2 = q.copy(), k.copy()
        if odd == "q":
            q2[1, G - 1, 5] = NAN   # one head
        elif odd == "k":
            k2[0, 1 % Hkv, 7, 3] = NAN  # one row: its kv head's query heads
        elif odd == "+inf":
            k2[1, 0, L - 1, 0] = INF
        elif odd == "-inf":         # every own score of kv head 0 of a request
            q2[2, :G, 0], k2[2, 0, :, 0] = 0x3F80, NINF
        kv = dak.dak_place_kv_heads(k2, v, 0)
        acc = torch.zeros(B, Hkv, L, device="cuda")
        if Lp:
            O = dak.dak_attn_prefix(to_dev(q2), kv, pre, prefix_of=_i32(of), seq_lens=_i32(lens), acc_out=acc, o_fp32=fp32)
        else:
            O, _ = dak.dak_attn_acc(to_dev(q2), kv, acc_out=acc, seq_lens=_i32(lens), o_fp32=fp32)
        assert not to_np(O)[-1].any() and not acc[-1].any()
        kv.free()
        if odd is None:
            clean, clean_acc = O, acc
            assert torch.isfinite(O).all() and torch.isfinite(acc).all()
            continue
        o, w, _, _ = oc.attention(q2, k2, v, lens, prefix, of if Lp else None)
        if odd == "-inf" and Lp:  # the prefix's rows carry all the weight
            assert np.isfinite(to_np(O)).all() and not acc[2, 0].any()
            assert np.abs(to_np(O) - o).max() < 0.05
            continue
        touched = np.zeros((B, Hq, 1), bool)
        touched[{"q": 1, "k": 0, "+inf": 1, "-inf": 2}[odd]] = True  # heads whose inputs changed
        assert (_same_nans(dak, O, o, clean) | touched).all()
        wn = np.isnan(w)
        got = acc.cpu().numpy()
        assert np.array_equal(np.isnan(got), wn)
        assert ((got == clean_acc.cpu().numpy()) | wn | touched[:, :Hkv]).all()
    if pre:
        pre.free()

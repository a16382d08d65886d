"""What the attention of the cache operators keeps of a weight: outputs near zero, that cancel to far
below the values' magnitude, show each rounding of the weights on the way that the output's own
rounding hides elsewhere."""
import math

import numpy as np
import pytest

from gpu_util import to_np

pytestmark = pytest.mark.gpu

U32, U16 = 2.0 ** -24, 2.0 ** -8  # half a step of fp32 and of bf16


@pytest.fixture(scope="module")
def dak(cuda_ok):
    import __graft_entry__
    __graft_entry__.build()
    import direct_host_memory_gb300 as m
    return m


def _two_rows(B, Hq, Hkv, D):
    """Inputs of two rows a kv head: keys 0 and -e0, so that query h weighs them 1 to c = exp(-q_h0 / sqrt(D)),
    c in [1/2, 1); values -(1/2 + d / 256) and 1, of which for every c some column's sum nearly cancels.
    Returns q, k, v (torch, bf16), c [B][Hq][1] and the outputs in 64 bits."""
    import torch
    rng = np.random.default_rng(B + Hq + D)
    x = rng.uniform(0.01, math.log(2.0) - 0.01, (B, Hq)) * math.sqrt(D)
    q = torch.zeros(B, Hq, D, dtype=torch.bfloat16)
    q[..., 0] = torch.from_numpy(x).to(torch.bfloat16)
    k = torch.zeros(1, Hkv, 2, D, dtype=torch.bfloat16)
    k[:, :, 1, 0] = -1.0
    v = torch.ones(1, Hkv, 2, D, dtype=torch.bfloat16)
    v[:, :, 0] = -(0.5 + torch.arange(D) * (0.5 / D))
    c = np.exp(-q[..., 0].double().numpy() / math.sqrt(D))[..., None]
    return q.cuda(), k.cuda(), v.cuda(), c, (v[0, 0, 0].double().numpy() + c) / (1 + c)


def _check(o, c, ref, fp32):
    """The numerator v0 + c: c's score is one exact product below 1 / log2 e times scale log2 e (a rounded
    constant, a rounded product: 2 ln 2 units of c), exp2 is good to 4, the weight's parts to half a
    step each, and the sums of three products of parts cut off at most 2 units of 1 each. The
    denominator (8 units), merge and division (8) count relative to the output, as its own rounding."""
    parts = U16 ** 3 if fp32 else U16 ** 2
    tol = ((6 * U32 + parts) * c + 6 * U32) / (1 + c) + (16 * U32 + (U32 if fp32 else U16)) * np.abs(ref)
    err = np.abs(to_np(o) - ref)
    assert (err <= tol).all(), f"max err/tol {np.max(err / tol):.2f}"


@pytest.mark.parametrize("fp32", [False, True])
@pytest.mark.parametrize("B,Hq,Hkv,D", [(3, 8, 2, 128), (32, 8, 2, 128), (33, 8, 2, 128), (100, 8, 2, 128),
                                        (9, 16, 1, 64), (70, 6, 2, 64), (200, 2, 2, 64)])
def test_attn_prefix_weights_at_any_number_of_rows(dak, B, Hq, Hkv, D, fp32):
    """A request's weights keep as many bits behind a prefix of many requests as behind its own."""
    import torch
    q, k, v, c, ref = _two_rows(B, Hq, Hkv, D)
    own = torch.zeros(B, Hkv, 1, D, dtype=torch.bfloat16, device="cuda")
    kv, pre = dak.dak_place_kv_heads(own, own, 0), dak.dak_place_kv_heads(k, v, 0)
    O = dak.dak_attn_prefix(q, kv, pre, seq_lens=torch.zeros(B, dtype=torch.int32, device="cuda"), o_fp32=fp32)
    assert dak.dak_last_error()[0] == 0
    _check(O, c, ref, fp32)
    kv.free()
    pre.free()


@pytest.mark.parametrize("fp32", [False, True])
@pytest.mark.parametrize("B,Hq,Hkv,D", [(3, 8, 2, 128), (40, 6, 2, 64), (5, 16, 1, 64), (4, 24, 2, 128)])
def test_attn_acc_weights(dak, B, Hq, Hkv, D, fp32):
    """The same over the own caches, and the accumulated weights beside it."""
    import torch
    q, k, v, c, ref = _two_rows(B, Hq, Hkv, D)
    kv = dak.dak_place_kv_heads(k.expand(B, -1, -1, -1).contiguous(), v.expand(B, -1, -1, -1).contiguous(), 1)
    O, acc = dak.dak_attn_acc(q, kv, o_fp32=fp32)
    assert dak.dak_last_error()[0] == 0
    _check(O, c, ref, fp32)
    # fp32 weights: c's 6 units, the denominator's 8, the product with its reciprocal 2, G of them added
    w = np.concatenate([1 / (1 + c), c / (1 + c)], -1).reshape(B, Hkv, Hq // Hkv, 2).sum(2)
    assert (np.abs(to_np(acc) - w) <= (16 + Hq // Hkv) * U32 * w).all()
    kv.free()


def test_attn_acc_fp32_sums_have_no_bias(dak):
    """Equal scores over positive values: the weights are one and their sum the row count, both exact, so
    that an output's error is that of its numerator's sum. Rounded to nearest, each of a warp's 1024
    additions of a chunk's product is off by at most half a unit in the last place either way: the mean over
    1024 outputs stays below 2 units of 2^-24 (6 standard deviations of 0.29 units in the last place, at most
    2 of 2^-24, a third of them weighing in by the growing sum: sqrt(1024 / 3) * 0.58 / sqrt(1024) * 6).
    A chunk's product itself may lose 16 (its sixteen terms cut off below the largest's 2^-24), the merge
    and the division 4. Summed in the tensor cores, which cut off towards zero each time, the mean is below
    by dozens of units."""
    import torch
    B, Hkv, D, L = 8, 2, 64, 65536
    gen = torch.Generator(device="cuda").manual_seed(3)
    v = torch.rand(B, Hkv, L, D, device="cuda", generator=gen) + 1.0
    v = (v * torch.exp2(-12.0 * torch.rand(B, Hkv, L, D, device="cuda", generator=gen))).to(torch.bfloat16)
    kv = dak.dak_place_kv_heads(torch.zeros_like(v), v, 0)
    q = torch.randn(B, Hkv, D, device="cuda", generator=gen).to(torch.bfloat16)
    O, _ = dak.dak_attn_acc(q, kv, o_fp32=True, tuning=dict(n_split=1))
    assert dak.dak_last_error()[0] == 0
    ref = v.double().mean(2)
    rel = ((O.double() - ref) / ref).flatten() / U32
    assert abs(rel.mean().item()) <= 2 + 16 + 4, f"mean error {rel.mean().item():.1f} units of 2^-24"
    assert rel.abs().max().item() <= 1024 + 16 + 4
    kv.free()

"""Forms of the cache operators' kernels that the sizes of tests/test_cache_ops_gpu.py do not reach: many query
heads a kv head, the eviction's other cluster and register splits, and attention launched while the
append in front of it runs."""
import numpy as np
import pytest

import synth
from gpu_util import to_dev
from oracle import cache as oc
from test_cache_ops_gpu import _cache, _check_attn, _check_weights, _evict_inputs, _i32, _ok, dak  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("case", [
    # B, Hq, Hkv, D, L, lens, fp32, host slabs, n_split
    (3, 16, 1, 128, 300, [300, 0, 65], False, 1, 0),
    (2, 18, 2, 128, 130, [130, 1], False, 0, 2),     # 9 query heads a kv head
    (3, 24, 2, 64, 200, [200, 64, 199], False, 3, 3),
    (2, 32, 2, 64, 257, [257, 256], True, 0, 0),
    (2, 11, 1, 64, 90, None, True, 2, 2),
    (2, 30, 2, 128, 100, None, True, 4, 1),
], ids=str)
def test_attn_acc_of_many_query_heads(dak, case):  # noqa: F811
    import torch
    B, Hq, Hkv, D, L, lens, fp32, host, n_split = case
    q, k, v = synth.attn_inputs(B, Hq, Hkv, D, L, seed=Hq + D)
    if lens is not None:
        for b, n in enumerate(lens):
            k[b, :, n:], v[b, :, n:] = 0x7FC0, 0x7F80
    o, w, spread, reach = oc.attention(q, k, v, lens)
    kv = dak.dak_place_kv_heads(k, v, host)
    acc_in = np.random.default_rng(5).random((B, Hkv, L)).astype(np.float32)
    acc = torch.from_numpy(acc_in).cuda()
    O, _ = dak.dak_attn_acc(to_dev(q), kv, acc_in=acc, acc_out=acc, seq_lens=None if lens is None else _i32(lens),
                            o_fp32=fp32, tuning=dict(n_split=n_split) if n_split else None)
    _ok(dak)
    _check_attn(O, o, spread, reach, D, L, fp32)
    _check_weights(acc, acc_in, w, acc_in, lens, reach, Hq // Hkv, D, L)
    kv.free()


@pytest.mark.parametrize("case", [
    # B, Hq, Hkv, D, L, lens, prefix lens, prefix of, fp32, host slabs of cache and prefix
    (3, 18, 2, 128, 70, [70, 0, 65], [257], None, False, 1, 1),
    (50, 16, 1, 128, 9, None, [200, 90], [b % 2 for b in range(50)], False, 0, 0),  # 400 rows a prefix
    (30, 30, 2, 64, 9, None, [140], None, False, 0, 1),                              # 450 rows
    (20, 13, 1, 64, 70, None, [1, 300], [b % 3 - 1 for b in range(20)], True, 3, 0),
    (40, 22, 2, 128, 5, None, [129], None, True, 0, 0),
], ids=lambda c: "-".join(str(x) for x in c[:5]) + f"-{c[6]}-{c[8]}")
@pytest.mark.parametrize("with_acc", [False, True])
def test_attn_prefix_of_many_query_heads(dak, case, with_acc):  # noqa: F811
    import torch
    B, Hq, Hkv, D, L, lens, plens, of, fp32, host, phost = case
    Lp = max(plens) + 30
    q, k, v = synth.attn_inputs(B, Hq, Hkv, D, L, seed=Hq + D)
    _, pk, pv = synth.attn_inputs(len(plens), Hq, Hkv, D, Lp, seed=Hq + D + 1)
    for f, n in enumerate(plens):
        pk[f, :, n:], pv[f, :, n:] = 0x7F80, 0x7FC0
    o, w, spread, reach = oc.attention(q, k, v, lens, (pk, pv), of, plens)
    kv, pre = dak.dak_place_kv_heads(k, v, host), dak.dak_place_kv_heads(pk, pv, phost)
    zeros = np.zeros((B, Hkv, L), np.float32)
    acc = torch.zeros(B, Hkv, L, device="cuda") if with_acc else None
    O = dak.dak_attn_prefix(to_dev(q), kv, pre, prefix_of=None if of is None else _i32(of), prefix_lens=_i32(plens),
                            seq_lens=None if lens is None else _i32(lens), acc_out=acc, o_fp32=fp32)
    _ok(dak)
    _check_attn(O, o, spread, reach, D, L + Lp, fp32)
    if with_acc:
        _check_weights(acc, None, w, zeros, lens, reach, Hq // Hkv, D, L + Lp)
    kv.free()
    pre.free()


@pytest.mark.parametrize("B,H,L,D,lens,keep,recent,kind", [
    (5, 8, 16384, 64, [16384, 4000, 0, 16001, 8200], 8000, 300, "ties"),     # two CTAs a slab, 8 slots a thread
    (10, 8, 16384, 64, [16384] + [9] * 8 + [12000], 6000, 6000, "odd"),     # a CTA a slab, 16 slots a thread
    (10, 8, 8193, 128, [8193, 8192] + [0] * 8, 4096, 0, "ties"),
    (2, 8, 40000, 64, [40000, 39999], 39000, 20, "plain"),                   # eight CTAs, and four of 16 slots
    (9, 8, 40000, 64, [40000] + [100] * 8, 20000, 20, "odd"),
    (1, 1, 131072, 64, [131072], 70000, 0, "ties"),                          # all that a cluster holds
])
def test_evict_by_other_splits(dak, B, H, L, D, lens, keep, recent, kind):  # noqa: F811
    import torch
    acc, pos = _evict_inputs(B, H, L, kind, L + keep)
    gen = torch.Generator(device="cuda").manual_seed(L)
    k, v = (torch.randn(B, H, L, D, device="cuda", generator=gen).to(torch.bfloat16) for _ in range(2))
    want_lens, src, want_acc, want_pos = oc.evict(lens, keep, recent, acc, pos)
    kv = dak.dak_place_kv_heads(k, v, 1)
    a, p = torch.from_numpy(acc).cuda(), torch.from_numpy(pos).cuda()
    got_lens, got_src = dak.dak_kv_evict(kv, _i32(lens), keep, recent, a, p)
    _ok(dak)
    assert np.array_equal(got_lens.cpu().numpy(), want_lens) and np.array_equal(got_src.cpu().numpy(), src)
    np.testing.assert_array_equal(a.cpu().numpy(), want_acc)
    np.testing.assert_array_equal(p.cpu().numpy(), want_pos)
    K, V = _cache(kv)
    k, v = (t.view(torch.int16).cpu().numpy().view(np.uint16) for t in (k, v))
    for b in range(B):
        m = want_lens[b]
        for g in range(H):
            s = src[b, g, :m]
            assert np.array_equal(K[b, g, :m], k[b, g, s]) and np.array_equal(V[b, g, :m], v[b, g, s])
            assert np.array_equal(K[b, g, m:], k[b, g, m:]) and np.array_equal(V[b, g, m:], v[b, g, m:])
    kv.free()


@pytest.mark.parametrize("host", [0, 3, 8])
@pytest.mark.parametrize("n_split", [1, 4, 9])
def test_attn_acc_launched_while_the_append_runs(dak, host, n_split):  # noqa: F811
    """A captured chain of appends of one token and attention with pdl 2, replayed, against the same launched
    one after the other: every length's newest row lies elsewhere in its chunk."""
    import torch
    B, Hq, Hkv, D, L, steps = 4, 8, 2, 128, 560, 4
    _, k, v = synth.attn_inputs(B, Hq, Hkv, D, L, seed=3)
    start = np.array([0, 61, 63, L - steps])
    slots, lens = [_i32(start + i) for i in range(steps)], [_i32(start + i + 1) for i in range(steps)]
    gen = torch.Generator(device="cuda").manual_seed(n_split)
    X = [torch.randn(B, Hq + 2 * Hkv, D, device="cuda", generator=gen).to(torch.bfloat16) for _ in range(steps)]
    rope = dak.dak_rope_make(D)

    def chain(kv, pdl, acc):
        outs = []
        for x, at, n in zip(X, slots, lens):
            q = dak.dak_kv_append_rope(kv, rope, x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:], at)
            outs.append(dak.dak_attn_acc(q, kv, acc_in=acc, acc_out=acc, seq_lens=n,
                                         tuning=dict(n_split=n_split, pdl=pdl))[0])
        return outs

    ref, kv = dak.dak_place_kv_heads(k, v, host), dak.dak_place_kv_heads(k, v, host)
    acc0, acc = torch.zeros(B, Hkv, L, device="cuda"), torch.zeros(B, Hkv, L, device="cuda")
    chain(kv, 2, acc)
    torch.cuda.synchronize()
    acc.zero_()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        outs = chain(kv, 2, acc)
    for rep in range(3):  # new tokens over the rows of the last replay's
        for x in X:
            x.copy_(torch.randn(x.shape, device="cuda", generator=gen))
        want = chain(ref, 0, acc0)
        g.replay()
        torch.cuda.synchronize()
        for a, b in zip(outs, want):
            assert torch.equal(a, b)
        assert torch.equal(acc, acc0)
    _ok(dak)
    ref.free()
    kv.free()


@pytest.mark.parametrize("B,Hq,H,D,P,Lp", [(512, 16, 1, 128, 1, 16384), (128, 64, 8, 128, 3, 16384), (1, 32, 8, 128, 1, 9000),
                                           (1000, 8, 8, 64, 900, 500), (4, 32, 8, 128, 1, 257)])
def test_prefix_workspace_is_in_proportion(dak, B, Hq, H, D, P, Lp):  # noqa: F811
    """A wide batch's partials over a prefix do not take a place for every row in as many ranges as there are
    SMs (545 MB for the first case)."""
    import torch
    kv, pre = (dak.dak_place_kv_heads(z, z, 0) for z in (
        torch.zeros(n, H, rows, D, dtype=torch.bfloat16, device="cuda") for n, rows in ((B, 64), (P, Lp))))
    got = dak.dak_attn_prefix_workspace_bytes(kv, pre, Hq, 1)
    sms, rows, place = dak.dak_sm_count(), B * Hq, (D + 2) * 4
    # a place a row is D + 2 floats; the own pass takes one, as it is in one split; the prefix one for each
    # range, but no more than 64 MiB where one range takes less
    most = max(rows * place, min(rows * place * max(1, sms // H), 64 << 20))
    assert rows * 2 * place <= got <= rows * place + most + B * 4 + 5 * 256
    kv.free()
    pre.free()


@pytest.mark.parametrize("P,B,Hq,Hkv,D", [(3, 128, 64, 8, 128), (1, 300, 16, 1, 64), (90, 400, 8, 8, 64), (33, 60, 32, 4, 128),
                                          (1, 97, 20, 2, 128), (200, 50, 4, 2, 64)])
def test_prefix_call_stays_inside_its_workspace(dak, P, B, Hq, Hkv, D):  # noqa: F811
    """What lies right behind the workspace is left as it was, for prefixes of every length and tile kind,
    and the result does not depend on where it lies."""
    import torch
    rng = np.random.default_rng(P + B)
    gen = torch.Generator(device="cuda").manual_seed(P)
    L, Lp = 3, 2500

    def rand(*s):
        return torch.randn(*s, device="cuda", generator=gen).to(torch.bfloat16)

    kv = dak.dak_place_kv_heads(rand(B, Hkv, L, D), rand(B, Hkv, L, D), 0)
    pre = dak.dak_place_kv_heads(rand(P, Hkv, Lp, D), rand(P, Hkv, Lp, D), 0)
    n = dak.dak_attn_prefix_workspace_bytes(kv, pre, Hq)
    q = rand(B, Hq, D)
    for rep in range(6):
        plens = np.exp(rng.uniform(0, np.log(Lp + 1), P)).astype(int).clip(0, Lp)
        of = rng.integers(-1, P, B) if rep % 2 else np.where(rng.random(B) < 0.7, 0, rng.integers(-1, P, B))
        ws = torch.full((n + (1 << 20),), 0x5A, dtype=torch.uint8, device="cuda")
        O = dak.dak_attn_prefix(q, kv, pre, prefix_of=_i32(of), prefix_lens=_i32(plens), workspace=ws[:n])
        one = dak.dak_attn_prefix(q, kv, pre, prefix_of=_i32(of), prefix_lens=_i32(plens))
        _ok(dak)
        assert (ws[n:] == 0x5A).all() and torch.equal(O, one)
    kv.free()
    pre.free()

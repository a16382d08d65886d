"""The cache operators on the GPU against the fp64 oracle: rotate and append, attention over a
shared prefix, attention that accumulates weights, eviction, and a run of them together."""
import math

import numpy as np
import pytest

import synth
from gpu_util import bits_of, to_dev, to_np
from oracle import cache as oc

pytestmark = pytest.mark.gpu

BOUNDS = 8
U32, U16 = 2.0 ** -24, 2.0 ** -8  # half a step of fp32 and of bf16


@pytest.fixture(scope="module")
def dak(cuda_ok):
    import __graft_entry__
    __graft_entry__.build()
    import direct_host_memory_gb300 as m
    return m


def _i32(x):
    import torch
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def _ok(dak):
    st, info = dak.dak_last_error()
    assert st == 0, f"device status {st} info {info:#x}"


def _cache(kv):
    """The rows K, V [B][H_kv][L][D] of a placed cache as bf16 bits, from both tiers."""
    import torch
    torch.cuda.synchronize()
    parts = [bits_of(t) for t in kv.slabs() if t is not None]
    return oc.slab_rows(np.concatenate(parts), kv.meta["H_kv"], kv.meta["L"])


def _weight_tol(D, n, reach):
    """Relative error of a softmax weight over n rows: a score of D products summed in fp32 is off
    by at most (D + 2) u times the products' magnitudes (reach), and so is the maximum it is
    taken against; exp2 and the rescalings add a few u; the denominator is a sum of n terms."""
    return 2 * ((D + 2) * reach + 16) * U32 + n * U32


def _attn_tol(D, n, ref, spread, reach, fp32, parts=None):
    """Bound of |o - ref|: every weight's relative error, the rounding of the weights to bf16 parts
    (half a step each: one part 2^-8, two 2^-16, three 2^-24; two unless given, three with fp32),
    the fp32 sum of n products, and the output's own. sum_j p_j |v_j| (spread) carries the weights'
    relative errors into the output."""
    parts = (3 if fp32 else 2) if parts is None else parts
    rel = _weight_tol(D, n, reach)[..., None] + U16 ** parts + n * U32
    return rel * spread * 1.01 + (U32 if fp32 else U16) * np.abs(ref) + 1e-30


def _check_attn(o, ref, spread, reach, D, n, fp32, parts=None):
    err = np.abs(to_np(o) - ref)
    tol = _attn_tol(D, n, ref, spread, reach, fp32, parts)
    assert np.isfinite(err).all()
    assert (err <= tol).all(), f"max err/tol {np.max(err / tol):.3f} at {np.unravel_index(np.argmax(err / tol), err.shape)}"


def _check_weights(acc_out, acc_in, w, before, seq_lens, reach, G, D, n):
    """Accumulated weights: G weights of relative error as above, summed and added in fp32; entries
    behind each length as they were."""
    got = acc_out.detach().cpu().numpy()
    B, H, L = got.shape
    rel = _weight_tol(D, n, reach.reshape(B, H, G).max(2))[..., None] + (G + 2) * U32
    start = np.zeros_like(w) if acc_in is None else acc_in
    want = start + w
    for b in range(B):
        m = L if seq_lens is None else seq_lens[b]
        err = np.abs(got[b, :, :m] - want[b, :, :m])
        assert (err <= rel[b] * w[b, :, :m] + U32 * np.abs(want[b, :, :m]) + 1e-30).all()
        assert np.array_equal(got[b, :, m:], before[b, :, m:])


# ---------------------------------------------------------------- rotate and append

ROPE_CASES = [
    # B, T, Hq, Hkv, D, rot, inter, scaling, fp32, host slabs
    (1, 1, 32, 8, 128, 128, False, "none", False, 0),
    (3, 1, 8, 2, 128, 64, True, "linear", True, 2),
    (2, 5, 4, 4, 64, 64, False, "ntk", False, 8),
    (2, 70, 6, 2, 64, 56, False, "by_parts", True, 3),
    (2, 33, 5, 1, 128, 120, True, "by_parts", False, 1),
    (1, 130, 3, 3, 128, 2, False, "none", True, 0),
    (1, 64, 16, 1, 64, 2, True, "none", False, 0),
    (257, 1, 4, 2, 64, 32, False, "none", False, 100),
    (2, 3, 0, 2, 128, 128, False, "none", False, 0),
]


@pytest.mark.parametrize("case", ROPE_CASES, ids=str)
@pytest.mark.parametrize("far", [0, 1000000000])
def test_append_rope(dak, case, far):
    import torch
    B, T, Hq, Hkv, D, rot, inter, scaling, fp32, host = case
    L = T + 67
    scale = 1.25
    H = Hq + 2 * Hkv
    rng = np.random.default_rng(B * 1000 + T)
    x = rng.standard_normal((B, T, H, D)).astype(np.float32)
    X = torch.from_numpy(x).cuda()
    if not fp32:
        X = X.to(torch.bfloat16)
        x = to_np(X)
    k0, v0 = synth.normal_bf16(7, 1, B * Hkv * L * D), synth.normal_bf16(7, 2, B * Hkv * L * D)
    kv = dak.dak_place_kv_heads(k0.reshape(B, Hkv, L, D), v0.reshape(B, Hkv, L, D), host)
    slots = rng.integers(0, L - T + 1, B)
    pos = rng.integers(0, 5000, B) + far
    n_new = rng.integers(0, T + 1, B)
    n_new[0] = T
    rope = dak.dak_rope_make(D, rot_dim=rot, theta=10000.0, interleaved=inter, scaling=scaling, factor=4.0,
                             orig_len=1000.0, attn_scale=scale)
    q_out = torch.full((B, T, Hq, D), 7.0, dtype=torch.bfloat16, device="cuda")
    slot_pos = torch.full((B, Hkv, L), -5, dtype=torch.int32, device="cuda")
    dak.dak_kv_append_rope(kv, rope, X[:, :, :Hq] if Hq else None, X[:, :, Hq:Hq + Hkv], X[:, :, Hq + Hkv:],
                           _i32(slots), positions=_i32(pos), n_new=_i32(n_new), q_out=q_out if Hq else None,
                           slot_pos=slot_pos)
    _ok(dak)
    freqs = oc.inv_freq(rot, 10000.0, scaling, 4.0, 1000.0)
    at = (pos[:, None] + np.arange(T)).reshape(-1)
    y = oc.rotate(np.asarray(x, np.float64).reshape(B * T, H, D), at, freqs, inter, scale).reshape(B, T, H, D)
    y[:, :, Hq + Hkv:] = x[:, :, Hq + Hkv:]
    # fp64 angles of the oracle: pos * f to 2^-52; the kernel's: 2^-25 turns from the fp32 fraction,
    # 2^-25 turns from its 32 bits, sincos one unit (2^-23), all times |x1| + |x2| <= 2 max |x|
    slack = (2 * math.pi * 2.0 ** -24 + 2.0 ** -23 + 4 * U32 + at.max() * 2.0 ** -51) * 2 * np.abs(x).max() * scale
    K, V = _cache(kv)
    wk, wv = oc._f64(k0).reshape(B, Hkv, L, D).copy(), oc._f64(v0).reshape(B, Hkv, L, D).copy()
    touched = np.zeros((B, L), bool)
    q = to_np(q_out)
    sp = slot_pos.cpu().numpy()
    for b in range(B):
        n, r = n_new[b], slots[b]
        touched[b, r:r + n] = True
        wk[b, :, r:r + n] = y[b, :n, Hq:Hq + Hkv].transpose(1, 0, 2)
        wv[b, :, r:r + n] = y[b, :n, Hq + Hkv:].transpose(1, 0, 2)
        assert (np.abs(q[b, :n] - y[b, :n, :Hq]) <= U16 * np.abs(y[b, :n, :Hq]) + slack).all()
        assert (q[b, n:] == 7.0).all()  # rows behind the last token
        assert (sp[b, :, r:r + n] == pos[b] + np.arange(n)).all()
    k64, v64 = oc._f64(K), oc._f64(V)
    t = np.broadcast_to(touched[:, None, :, None], wk.shape)
    assert np.array_equal(k64[~t], wk[~t]) and np.array_equal(v64[~t], wv[~t])
    assert (np.abs(k64 - wk)[t] <= (U16 * np.abs(wk) + slack)[t]).all()
    assert (np.abs(v64 - wv)[t] <= U16 * np.abs(wv)[t]).all()
    assert (sp.transpose(0, 2, 1)[~touched] == -5).all()
    kv.free()


def test_append_rope_defaults_and_bounds(dak):
    """positions default to the slots; a row past the cache is reported and skipped, its query is not."""
    import torch
    B, Hkv, L, D = 3, 2, 10, 64
    z = np.zeros((B, Hkv, L, D), np.uint16)
    kv = dak.dak_place_kv_heads(z, z, 0)
    rope = dak.dak_rope_make(D, theta=10000.0)
    x = torch.ones(B, 4, D, dtype=torch.bfloat16, device="cuda")
    q = dak.dak_kv_append_rope(kv, rope, x[:, :2].contiguous(), x[:, 2:], x[:, 2:], _i32([9, 10, -1]))
    st, _ = dak.dak_last_error()
    assert st == BOUNDS
    K, V = _cache(kv)
    want = oc.rotate(np.ones((3, 2, D)), [9, 10, -1], oc.inv_freq(D, 10000.0))
    assert np.abs(to_np(q) - want).max() <= 2 * U16
    assert np.abs(oc._f64(K)[0, :, 9] - want[0]).max() <= 2 * U16
    assert not K[1:].any() and not V[1:].any() and not K[0, :, :9].any()
    with pytest.raises(ValueError):
        dak.dak_kv_append_rope(kv, rope, None, x[:, 2:, ::2], x[:, 2:], _i32([0, 0, 0]))
    with pytest.raises(ValueError):
        dak.dak_kv_append_rope(kv, rope, None, x[:, 2:], x[:, 2:], _i32([0, 0]))
    kv.free()


# ---------------------------------------------------------------- accumulated weights

ACC_CASES = [
    # B, Hq, Hkv, D, L, lens, fp32, host slabs, n_split
    (3, 8, 2, 128, 300, [300, 0, 1], False, 0, 0),
    (3, 8, 2, 128, 300, [299, 64, 65], True, 3, 4),
    (2, 5, 1, 64, 130, [63, 130], False, 1, 1),
    (2, 16, 1, 128, 1000, [1000, 511], True, 0, 3),
    (4, 4, 4, 64, 77, None, False, 16, 2),
    (1, 32, 8, 128, 2049, [2049], False, 0, 0),
    (1, 1, 1, 128, 1, [1], True, 0, 0),
    (1, 7, 7, 64, 64, [64], False, 2, 64),
    (170, 15, 3, 128, 70, [(7 * b) % 71 for b in range(170)], False, 3, 2),  # many heads, few splits each
    (340, 16, 4, 64, 20, None, True, 0, 0),
]


@pytest.mark.parametrize("case", ACC_CASES, ids=lambda c: str(c) if c[0] < 100 else f"{c[:5]}")
def test_attn_acc(dak, case):
    import torch
    B, Hq, Hkv, D, L, lens, fp32, host, n_split = case
    q, k, v = synth.attn_inputs(B, Hq, Hkv, D, L, seed=L + D)
    if lens is not None:  # what lies behind a request's tokens is never used
        for b, n in enumerate(lens):
            k[b, :, n:] = 0x7FC0  # NaN
            v[b, :, n:] = 0x7F80  # infinity
    o, w, spread, reach = oc.attention(q, k, v, lens)
    kv = dak.dak_place_kv_heads(k, v, host)
    rng = np.random.default_rng(5)
    acc_in = rng.random((B, Hkv, L)).astype(np.float32)
    acc_out = torch.full((B, Hkv, L), -3.0, device="cuda")
    before = acc_out.cpu().numpy()
    tun = dict(n_split=n_split) if n_split else None
    sl = None if lens is None else _i32(lens)
    O, got = dak.dak_attn_acc(to_dev(q), kv, acc_in=torch.from_numpy(acc_in).cuda(), acc_out=acc_out, seq_lens=sl,
                              o_fp32=fp32, tuning=tun)
    _ok(dak)
    assert got is acc_out and O.dtype == (torch.float32 if fp32 else torch.bfloat16)
    _check_attn(O, o, spread, reach, D, L, fp32)
    _check_weights(got, acc_in, w, before, lens, reach, Hq // Hkv, D, L)
    # in place and from zeros, the same bits as apart
    same = torch.from_numpy(acc_in).cuda()
    O2, _ = dak.dak_attn_acc(to_dev(q), kv, acc_in=same, acc_out=same, seq_lens=sl, o_fp32=fp32, tuning=tun)
    O3, fresh = dak.dak_attn_acc(to_dev(q), kv, seq_lens=sl, o_fp32=fp32, tuning=tun)
    _ok(dak)
    assert np.array_equal(bits_of(O2), bits_of(O)) and np.array_equal(bits_of(O3), bits_of(O))
    for b in range(B):
        m = L if lens is None else lens[b]
        assert torch.equal(same[b, :, :m], got[b, :, :m])
        assert np.array_equal(same[b, :, m:].cpu().numpy(), acc_in[b, :, m:])
    _check_weights(fresh, None, w, np.zeros_like(acc_in), lens, reach, Hq // Hkv, D, L)
    kv.free()


def test_attn_acc_is_the_same_at_every_split_between_the_tiers(dak):
    import torch
    q, k, v = synth.attn_inputs(3, 8, 2, 128, 500, seed=9)
    lens = _i32([500, 77, 333])
    base = None
    for host in (0, 1, 3, 6):
        kv = dak.dak_place_kv_heads(k, v, host)
        O, acc = dak.dak_attn_acc(to_dev(q), kv, seq_lens=lens)
        _ok(dak)
        if base is None:
            base = (O, acc)
        assert torch.equal(O, base[0]) and torch.equal(acc, base[1])
        kv.free()


def test_attn_acc_lengths_out_of_range_are_clamped(dak):
    import torch
    q, k, v = synth.attn_inputs(2, 4, 2, 64, 90, seed=2)
    kv = dak.dak_place_kv_heads(k, v, 0)
    a = dak.dak_attn_acc(to_dev(q), kv, seq_lens=_i32([1000, -4]))
    b = dak.dak_attn_acc(to_dev(q), kv, seq_lens=_i32([90, 0]))
    _ok(dak)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    assert not b[0][1].any() and not b[1][1].any()
    kv.free()


# ---------------------------------------------------------------- shared prefixes

PREFIX_CASES = [
    # B, Hq, Hkv, D, L, lens, prefix lens, prefix of, fp32, host slabs of cache and prefix
    (4, 8, 2, 128, 70, [0, 1, 64, 70], [257], None, False, 0, 0),
    (4, 8, 2, 128, 70, [0, 0, 3, 65], [130, 0, 64], [0, 1, -1, 2], True, 3, 2),
    (3, 5, 1, 64, 10, [10, 0, 1], [1, 700], [1, 0, 1], False, 1, 1),
    (5, 16, 1, 128, 33, [33, 32, 0, 0, 5], [1000], None, True, 0, 1),
    (2, 4, 4, 64, 64, None, [128, 129], [1, 1], False, 8, 0),
    (40, 8, 2, 128, 16, None, [300], None, False, 0, 0),      # 160 rows a kv head
    (70, 16, 4, 64, 9, None, [200, 333], [b % 2 for b in range(70)], False, 0, 0),
    (70, 12, 2, 128, 9, None, [333, 5], [0 if b % 7 else -1 for b in range(70)], True, 0, 4),  # 360 rows
    (130, 8, 8, 128, 4, None, [150], None, False, 0, 0),      # no sharing of heads
    (100, 5, 1, 64, 3, None, [140], None, True, 0, 0),        # 500 rows
    (1, 1, 1, 64, 1, [0], [1], None, False, 0, 0),
    (1, 32, 8, 128, 5, [5], [2050], None, False, 0, 8),
]


@pytest.mark.parametrize("case", PREFIX_CASES, ids=lambda c: "-".join(str(x) for x in c[:5]) + f"-{c[6]}-{c[8]}")
@pytest.mark.parametrize("with_acc", [False, True])
def test_attn_prefix(dak, case, with_acc):
    import torch
    B, Hq, Hkv, D, L, lens, plens, of, fp32, host, phost = case
    P, Lp = len(plens), max(max(plens), 1) + 30
    q, k, v = synth.attn_inputs(B, Hq, Hkv, D, L, seed=L + D)
    _, pk, pv = synth.attn_inputs(P, Hq, Hkv, D, Lp, seed=L + D + 1)
    if lens is not None:
        for b, n in enumerate(lens):
            k[b, :, n:], v[b, :, n:] = 0x7FC0, 0x7F80
    for f, n in enumerate(plens):
        pk[f, :, n:], pv[f, :, n:] = 0x7F80, 0x7FC0
    o, w, spread, reach = oc.attention(q, k, v, lens, (pk, pv), of, plens)
    kv, pre = dak.dak_place_kv_heads(k, v, host), dak.dak_place_kv_heads(pk, pv, phost)
    acc_in = np.random.default_rng(5).random((B, Hkv, L)).astype(np.float32)
    acc = torch.from_numpy(acc_in).cuda() if with_acc else None
    sl = None if lens is None else _i32(lens)
    O = dak.dak_attn_prefix(to_dev(q), kv, pre, prefix_of=None if of is None else _i32(of), prefix_lens=_i32(plens),
                            seq_lens=sl, acc_in=acc, acc_out=acc, o_fp32=fp32)
    _ok(dak)
    # prefixes of more query rows than a 128-row tile holds take the weights as one bf16 part
    counts = [sum(1 for b in range(B) if (0 if of is None else of[b]) == f) for f in range(P)]
    wide = max(counts) > 128 // (Hq // Hkv)
    _check_attn(O, o, spread, reach, D, L + Lp, fp32, parts=1 if wide and not fp32 else None)
    if with_acc:
        _check_weights(acc, acc_in, w, acc_in, lens, reach, Hq // Hkv, D, L + Lp)
    kv.free()
    pre.free()


def test_attn_prefix_tiers_streams_and_repeats(dak):
    """The same bits wherever prefix and cache lie, on a stream of the caller's, again and in a graph
    that is replayed on changed inputs."""
    import torch
    B, Hq, Hkv, D, L, Lp = 6, 8, 2, 128, 40, 500
    q, k, v = synth.attn_inputs(B, Hq, Hkv, D, L, seed=1)
    _, pk, pv = synth.attn_inputs(2, Hq, Hkv, D, Lp, seed=2)
    of, lens, plens = _i32([0, 1, 0, -1, 1, 1]), _i32([1, 40, 0, 7, 0, 39]), _i32([500, 123])
    Q = to_dev(q)
    base = None
    for host, phost in ((0, 0), (5, 1), (12, 4), (0, 3)):
        kv, pre = dak.dak_place_kv_heads(k, v, host), dak.dak_place_kv_heads(pk, pv, phost)
        O = dak.dak_attn_prefix(Q, kv, pre, prefix_of=of, prefix_lens=plens, seq_lens=lens)
        _ok(dak)
        base = O if base is None else base
        assert torch.equal(O, base)
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        out = torch.empty_like(O)
        ws = torch.empty(dak.dak_attn_prefix_workspace_bytes(kv, pre, Hq), dtype=torch.uint8, device="cuda")
        torch.cuda.synchronize()
        dak.dak_attn_prefix(Q, kv, pre, prefix_of=of, prefix_lens=plens, seq_lens=lens, O=out, workspace=ws, stream=s)
        s.synchronize()
        assert torch.equal(out, base)
        g = torch.cuda.CUDAGraph()
        Qg, of_g, lens_g = Q.clone(), of.clone(), lens.clone()
        with torch.cuda.graph(g):
            dak.dak_attn_prefix(Qg, kv, pre, prefix_of=of_g, prefix_lens=plens, seq_lens=lens_g, O=out, workspace=ws)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, base)
        Qg.copy_(Q.flip(0))
        of_g.copy_(of.flip(0))
        lens_g.copy_(lens.flip(0))
        g.replay()
        want = dak.dak_attn_prefix(Qg, kv, pre, prefix_of=of_g, prefix_lens=plens, seq_lens=lens_g)
        torch.cuda.synchronize()
        assert torch.equal(out, want)
        _ok(dak)
        kv.free()
        pre.free()


def test_attn_prefix_out_of_range_prefix_is_reported(dak):
    import torch
    q, k, v = synth.attn_inputs(3, 4, 2, 64, 20, seed=3)
    _, pk, pv = synth.attn_inputs(2, 4, 2, 64, 70, seed=4)
    kv, pre = dak.dak_place_kv_heads(k, v, 0), dak.dak_place_kv_heads(pk, pv, 0)
    a = dak.dak_attn_prefix(to_dev(q), kv, pre, prefix_of=_i32([0, 2, 1]))
    assert dak.dak_last_error()[0] == BOUNDS
    b = dak.dak_attn_prefix(to_dev(q), kv, pre, prefix_of=_i32([0, -1, 1]))
    _ok(dak)
    assert torch.equal(a, b)
    kv.free()
    pre.free()


# ---------------------------------------------------------------- eviction

def _evict_inputs(B, H, L, kind, seed):
    rng = np.random.default_rng(seed)
    acc = np.exp(2 * rng.standard_normal((B, H, L))).astype(np.float32)
    if kind == "ties":
        acc = rng.integers(0, 3, (B, H, L)).astype(np.float32) * np.float32(-1.0)  # -0, -1, -2
        acc[rng.random((B, H, L)) < 0.3] = 0.0
    elif kind == "odd":
        acc[rng.random((B, H, L)) < 0.2] = np.nan
        acc[rng.random((B, H, L)) < 0.1] = np.inf
        acc[rng.random((B, H, L)) < 0.1] = -np.inf
        acc[rng.random((B, H, L)) < 0.1] = 1e-42
    elif kind == "equal":
        acc[:] = 1.0
    pos = np.stack([rng.permutation(2 * L)[:L] for _ in range(B * H)]).reshape(B, H, L).astype(np.int32)
    if kind == "equal":
        pos[:] = 4  # a table that was never filled in: all are newest, and the lower slots stay
    return acc, pos


EVICT_CASES = [
    # B, H, L, D, lens, keep, recent, kind, host slabs
    (3, 2, 300, 128, [300, 100, 101], 100, 10, "plain", 0),
    (3, 2, 300, 64, [299, 0, 1], 1, 0, "plain", 3),
    (2, 3, 1000, 128, [1000, 777], 776, 776, "odd", 6),
    (2, 3, 1500, 64, [1500, 1025], 600, 0, "ties", 2),
    (2, 2, 513, 128, [513, 512], 512, 100, "odd", 0),
    (1, 2, 700, 64, [700], 33, 33, "equal", 0),
    (2, 1, 64, 128, [64, 64], 64, 5, "plain", 0),
    (1, 1, 2, 64, [2], 1, 1, "plain", 0),
    (1, 2, 5000, 64, [4999], 2500, 77, "ties", 0),
    (1, 3, 9001, 64, [9001], 5000, 100, "plain", 1),        # a cluster a slab
    (1, 1, 100000, 64, [99999], 60001, 5000, "ties", 0),    # the largest cluster
    (2, 80, 4500, 64, [4500, 4400], 2200, 64, "plain", 7),  # a CTA a slab
    (1, 1, 140000, 64, [139999], 70001, 5, "odd", 0),       # longer than a cluster holds
]


@pytest.mark.parametrize("case", EVICT_CASES, ids=str)
@pytest.mark.parametrize("in_place", [True, False])
def test_evict(dak, case, in_place):
    import torch
    B, H, L, D, lens, keep, recent, kind, host = case
    acc, pos = _evict_inputs(B, H, L, kind, L + keep)
    k, v = (synth.normal_bf16(11, j, B * H * L * D).reshape(B, H, L, D) for j in (1, 2))
    want_lens, src, want_acc, want_pos = oc.evict(lens, keep, recent, acc, pos)
    kv = dak.dak_place_kv_heads(k, v, host)
    a, p = torch.from_numpy(acc).cuda(), torch.from_numpy(pos).cuda()
    kw = {} if in_place else dict(acc_out=torch.full_like(a, 9.0), slot_pos_out=torch.full_like(p, 99))
    got_lens, got_src = dak.dak_kv_evict(kv, _i32(lens), keep, recent, a, p, **kw)
    _ok(dak)
    assert np.array_equal(got_lens.cpu().numpy(), want_lens)
    assert np.array_equal(got_src.cpu().numpy(), src)
    ga, gp = (a, p) if in_place else (kw["acc_out"], kw["slot_pos_out"])
    for b in range(B):
        n = lens[b]
        np.testing.assert_array_equal(ga[b, :, :n].cpu().numpy(), want_acc[b, :, :n])
        np.testing.assert_array_equal(gp[b, :, :n].cpu().numpy(), want_pos[b, :, :n])
        if in_place:
            np.testing.assert_array_equal(ga[b, :, n:].cpu().numpy(), acc[b, :, n:])
        else:
            assert (ga[b, :, n:] == 9.0).all() and (gp[b, :, n:] == 99).all()
    K, V = _cache(kv)
    for b in range(B):
        m = want_lens[b]
        for g in range(H):
            s = src[b, g, :m]
            assert np.array_equal(K[b, g, :m], k[b, g, s]) and np.array_equal(V[b, g, :m], v[b, g, s])
            assert np.array_equal(K[b, g, m:], k[b, g, m:]) and np.array_equal(V[b, g, m:], v[b, g, m:])
    kv.free()


def test_evict_repeats_and_refuses(dak):
    import torch
    B, H, L, D, keep = 2, 4, 900, 64, 300
    acc, pos = _evict_inputs(B, H, L, "plain", 1)
    k, v = (synth.normal_bf16(12, j, B * H * L * D).reshape(B, H, L, D) for j in (1, 2))
    kv = dak.dak_place_kv_heads(k, v, 2)
    a, p, lens = torch.from_numpy(acc).cuda(), torch.from_numpy(pos).cuda(), _i32([900, 450])
    outs = []
    for _ in range(2):  # apart from its inputs an eviction can be run again
        ao, po = torch.zeros_like(a), torch.zeros_like(p)
        l1, s1 = dak.dak_kv_evict(kv, lens, keep, 50, a, p, acc_out=ao, slot_pos_out=po)
        outs.append((l1, s1, ao, po) + tuple(torch.from_numpy(x.astype(np.int32)) for x in _cache(kv)))
    _ok(dak)
    assert all(torch.equal(x, y) for x, y in zip(*outs))
    for bad in (dict(n_keep=0), dict(n_keep=L + 1), dict(n_recent=keep + 1), dict(lens_out=lens)):
        kw = dict(dict(n_keep=keep, n_recent=0), **bad)
        with pytest.raises(dak.DakError) as e:
            dak.dak_kv_evict(kv, lens, acc=a, slot_pos=p, **kw)
        assert e.value.status == 1
    kv.free()


# ---------------------------------------------------------------- sizes, streams and graphs

def _prefix_run(dak, B, Hq, Hkv, D, L, lens, plens, of, fp32):
    import torch
    q, k, v = synth.attn_inputs(B, Hq, Hkv, D, L, seed=B + D)
    _, pk, pv = synth.attn_inputs(len(plens), Hq, Hkv, D, max(plens), seed=B + D + 1)
    o, w, spread, reach = oc.attention(q, k, v, lens, (pk, pv), of, plens)
    kv, pre = dak.dak_place_kv_heads(k, v, 3), dak.dak_place_kv_heads(pk, pv, min(5, len(plens) * Hkv - 1))
    acc = torch.zeros(B, Hkv, L, device="cuda")
    O = dak.dak_attn_prefix(to_dev(q), kv, pre, prefix_of=_i32(of), prefix_lens=_i32(plens), seq_lens=_i32(lens),
                            acc_out=acc, o_fp32=fp32)
    _ok(dak)
    n = L + max(plens)
    _check_attn(O, o, spread, reach, D, n, fp32, parts=None if fp32 else 1)
    _check_weights(acc, None, w, np.zeros(w.shape, np.float32), lens, reach, Hq // Hkv, D, n)
    kv.free()
    pre.free()


@pytest.mark.parametrize("P,B,Hq,Hkv,D,fp32", [
    (60, 170, 8, 4, 64, False),    # more tiles than the GPU has SMs, more than 128 requests
    (45, 300, 32, 4, 128, False),  # of one and of two 128-row halves, some prefixes with no request
    (70, 140, 6, 3, 128, True),
    (200, 210, 1, 1, 64, False),   # more prefixes than tiles
    (3, 180, 16, 2, 64, True),     # the merge by warps
])
def test_attn_prefix_of_many(dak, P, B, Hq, Hkv, D, fp32):
    rng = np.random.default_rng(P)
    plens = rng.integers(0, 200, P)
    plens[:3] = [0, 1, 200]
    of = np.where(rng.random(B) < 0.25, min(4, P - 1), rng.integers(-1, P, B))  # one prefix with many requests
    lens = rng.integers(0, 6, B)
    _prefix_run(dak, B, Hq, Hkv, D, 5, lens.tolist(), plens.tolist(), of.tolist(), fp32)


def test_attn_prefix_long_in_many_ranges(dak):
    """One kv head: a prefix is cut into as many ranges as the GPU has SMs."""
    _prefix_run(dak, 3, 4, 1, 64, 700, [700, 0, 3], [30001, 20], [0, 0, 1], False)
    _prefix_run(dak, 40, 4, 1, 128, 9, [k % 9 for k in range(40)], [20000, 9000], [k % 3 - 1 for k in range(40)], True)


def test_attn_prefix_fp32_sums_do_not_drift(dak):
    """Over values of one the output is one: the weights' sum by the products against their sum by the
    softmax, for so many rows that every CTA sums a whole prefix of 512 steps."""
    import torch
    B, Hq, Hkv, D, Lp = 640, 64, 8, 64, 32768
    gen = torch.Generator(device="cuda").manual_seed(2)
    k = torch.randn(1, Hkv, Lp, D, device="cuda", generator=gen).to(torch.bfloat16)
    q = torch.randn(B, Hq, D, device="cuda", generator=gen).to(torch.bfloat16)
    own = torch.zeros(B, Hkv, 1, D, dtype=torch.bfloat16, device="cuda")
    kv, pre = dak.dak_place_kv_heads(own, own, 0), dak.dak_place_kv_heads(k, torch.ones_like(k), 0)
    O = dak.dak_attn_prefix(q, kv, pre, seq_lens=torch.zeros(B, dtype=torch.int32, device="cuda"), o_fp32=True)
    _ok(dak)
    # the three parts of a weight 1; a step's 12 instructions cut off at most 2 each; 512 steps' products
    # added; the softmax's sum of a step's weights 18 and of the steps 512; rescales, merge, division 10
    assert (O - 1.0).abs().max().item() <= (1 + 24 + 512 + 18 + 512 + 10) * U32
    kv.free()
    pre.free()


def test_attn_acc_in_many_splits(dak):
    import torch
    B, Hq, Hkv, D, L = 2, 3, 1, 64, 66001
    q, k, v = synth.attn_inputs(B, Hq, Hkv, D, L, seed=4)
    lens = [L, 40000]
    o, w, spread, reach = oc.attention(q, k, v, lens)
    kv = dak.dak_place_kv_heads(k, v, 0)
    for split in (1024, 300, 0):
        O, acc = dak.dak_attn_acc(to_dev(q), kv, seq_lens=_i32(lens), tuning=dict(n_split=split))
        _ok(dak)
        _check_attn(O, o, spread, reach, D, L, False)
        _check_weights(acc, None, w, np.zeros(w.shape, np.float32), lens, reach, Hq // Hkv, D, L)
    kv.free()


def test_a_cache_past_32_bit_offsets(dak):
    """The last request of a cache of more than 4 GiB a tier against the same request alone."""
    import torch
    B, Hq, Hkv, D, L = 34, 4, 4, 128, 65600
    gen = torch.Generator(device="cuda").manual_seed(1)
    k, v = (torch.zeros(B, Hkv, L, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    for t in (k, v):
        t[-1].normal_(generator=gen)
    big, one = dak.dak_place_kv_heads(k, v, 0), dak.dak_place_kv_heads(k[-1:].contiguous(), v[-1:].contiguous(), 0)
    del k, v
    assert big.hbm_bytes > 1 << 32
    rope = dak.dak_rope_make(D)
    x = torch.randn(B, Hq + 2 * Hkv, D, device="cuda", generator=gen)
    slots = torch.full((B,), L - 1, dtype=torch.int32, device="cuda")
    acc = torch.rand(B, Hkv, L, device="cuda", generator=gen)
    sp = torch.arange(L, dtype=torch.int32, device="cuda").repeat(B, Hkv, 1)
    out = []
    for kv, sel in ((big, slice(None)), (one, slice(-1, None))):
        xx, a, p = x[sel].contiguous(), acc[sel].clone(), sp[sel].clone()
        q = dak.dak_kv_append_rope(kv, rope, xx[:, :Hq], xx[:, Hq:2 * Hq], xx[:, 2 * Hq:], slots[sel], slot_pos=p)
        lens = slots[sel] + 1
        O, a = dak.dak_attn_acc(q, kv, acc_in=a, acc_out=a, seq_lens=lens, tuning=dict(n_split=8))
        lens, src = dak.dak_kv_evict(kv, lens, 30000, 100, a, p)
        O2 = dak.dak_attn_prefix(q, kv, kv, prefix_of=slots[sel] * 0 + kv.shape[0] - 1, seq_lens=lens,
                                 prefix_lens=torch.full((kv.shape[0],), 30000, dtype=torch.int32, device="cuda"),
                                 tuning=dict(n_split=8))
        _ok(dak)
        out.append([t[-1].clone() for t in (q, O, a, p, src)] + [lens[-1:], kv.slabs()[1][-Hkv:].clone()])
        # the prefix of 34 requests is cut elsewhere than that of one: another order of the sums
        out[-1].append(O2[-1].float())
    for a, b in zip(out[0][:-1], out[1][:-1]):
        assert torch.equal(a, b)
    # |o| <= max |v| < 8 and each side is off by at most 2^-8 of the weighted |v| (one bf16 part) and
    # 2^-9 of the output; both outputs lie far below 1
    assert (out[0][-1] - out[1][-1]).abs().max().item() <= 2 * (U16 + U16) * 1.0
    big.free()
    one.free()


def test_graphs_and_streams_with_memory_of_their_own(dak):
    """Two graphs that were captured without a workspace replay in turn and beside eager calls; calls
    on another stream take their memory with them."""
    import torch
    B, Hq, Hkv, D, L = 4, 8, 2, 64, 1500
    q, k, v = synth.attn_inputs(B, Hq, Hkv, D, L, seed=21)
    _, pk, pv = synth.attn_inputs(1, Hq, Hkv, D, 900, seed=22)
    kv, pre = dak.dak_place_kv_heads(k, v, 2), dak.dak_place_kv_heads(pk, pv, 1)
    Q = to_dev(q)
    lens = [_i32([1500, 700, 0, 3]), _i32([9, 1400, 64, 65])]
    calls = [lambda: dak.dak_attn_acc(Q, kv, seq_lens=lens[0], tuning=dict(n_split=20)),
             lambda: (dak.dak_attn_prefix(Q, kv, pre, seq_lens=lens[1]),)]
    want = [c() for c in calls]
    torch.cuda.synchronize()
    graphs, outs = [], []
    for c in calls:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(c())
        graphs.append(g)
    for _ in range(3):
        for g, o in zip(graphs, outs):
            for t in o:
                t.fill_(-1.0)
            if len(o) == 2:
                o[1].zero_()
            g.replay()
        eager = [c() for c in calls]
        torch.cuda.synchronize()
        for o, e, w in zip(outs, eager, want):
            assert torch.equal(o[0], w[0]) and torch.equal(e[0], w[0])
            if len(o) == 2:
                assert torch.equal(o[1], w[1]) and torch.equal(e[1], w[1])
    s = torch.cuda.Stream()
    for stream in (s, s.cuda_stream):
        s.wait_stream(torch.cuda.current_stream())
        O, acc = torch.empty_like(want[0][0]), torch.zeros_like(want[0][1])
        O2 = torch.empty_like(want[1][0])
        torch.cuda.synchronize()
        dak.dak_attn_acc(Q, kv, acc_out=acc, seq_lens=lens[0], O=O, tuning=dict(n_split=20), stream=stream)
        junk = [torch.full((1 << 22,), 1e30, device="cuda") for _ in range(4)]  # on the current stream
        dak.dak_attn_prefix(Q, kv, pre, seq_lens=lens[1], O=O2, stream=stream)
        junk += [torch.full((1 << 22,), 1e30, device="cuda") for _ in range(4)]
        torch.cuda.synchronize()
        assert torch.equal(O, want[0][0]) and torch.equal(acc, want[0][1]) and torch.equal(O2, want[1][0])
        # results that a call makes itself are made for its stream
        junk += [torch.full((1 << 22,), 1e30, device="cuda") for _ in range(4)]
        got = dak.dak_attn_acc(Q, kv, seq_lens=lens[0], tuning=dict(n_split=20), stream=stream)
        got2 = dak.dak_attn_prefix(Q, kv, pre, seq_lens=lens[1], stream=stream)
        assert torch.cuda.current_stream() != s
        s.synchronize()
        assert torch.equal(got[0], want[0][0]) and torch.equal(got[1], want[0][1]) and torch.equal(got2, want[1][0])
    with torch.cuda.stream(s):
        tab = torch.arange(L, dtype=torch.int32, device="cuda").repeat(B, Hkv, 1)
        keep, src = dak.dak_kv_evict(kv, lens[0], 600, 10, want[0][1].clone(), tab.clone())
        apart = (want[0][1].clone(), torch.empty_like(tab), torch.empty_like(want[0][1]))
    again, src2 = dak.dak_kv_evict(kv, lens[0], 600, 10, apart[0], tab, slot_pos_out=apart[1], acc_out=apart[2], stream=s)
    s.synchronize()
    assert torch.equal(keep, again) and torch.equal(src, src2) and keep.tolist() == [600, 600, 0, 3]
    _ok(dak)
    kv.free()
    pre.free()


def test_attn_acc_in_a_handoff_sequence(dak):
    """Launches of a host-link handoff sequence give the bits of launches by themselves."""
    import torch
    B, Hq, Hkv, D, L = 4, 8, 2, 128, 700
    q, k, v = synth.attn_inputs(B, Hq, Hkv, D, L, seed=31)
    Q, lens = to_dev(q), _i32([700, 64, 0, 333])
    kvs = [dak.dak_place_kv_heads(k, v, h) for h in (3, 8, 0)]
    want = dak.dak_attn_acc(Q, kvs[0], seq_lens=lens)
    dak.dak_link_timeouts()
    for slot in (0, 2, 2):
        if slot:
            dak.dak_link_begin(slot)
        acc = [torch.zeros(B, Hkv, L, device="cuda") for _ in kvs]
        out = [dak.dak_attn_acc(Q, kv, acc_out=a, seq_lens=lens, tuning=dict(pdl=1, link=slot))[0]
               for kv, a in zip(kvs, acc)]
        torch.cuda.synchronize()
        _ok(dak)
        assert all(torch.equal(o, want[0]) for o in out) and all(torch.equal(a, want[1]) for a in acc)
    assert dak.dak_link_timeouts() == 0
    for kv in kvs:
        kv.free()


def test_calls_refused_before_a_launch(dak):
    import torch
    q, k, v = synth.attn_inputs(2, 4, 2, 64, 64, seed=1)
    kv, Q = dak.dak_place_kv_heads(k, v, 0), to_dev(q)
    W = dak.dak_place_matrix(synth.normal_bf16(1, 1, 64 * 64).reshape(64, 64), 0)
    lens = _i32([3, 4])
    acc, sp = torch.zeros(2, 2, 64, device="cuda"), torch.zeros(2, 2, 64, dtype=torch.int32, device="cuda")
    host = torch.empty(1 << 22, dtype=torch.uint8)
    for call in (lambda: dak.dak_attn_acc(Q, W), lambda: dak.dak_attn_prefix(Q, W, kv), lambda: dak.dak_attn_prefix(Q, kv, W),
                 lambda: dak.dak_kv_evict(W, lens, 2, 0, acc, sp), lambda: dak.dak_attn_acc(Q, kv, workspace=host),
                 lambda: dak.dak_attn_prefix(Q, kv, kv, workspace=host),
                 lambda: dak.dak_kv_evict(kv, lens, 2, 0, acc, sp, workspace=host),
                 lambda: dak.dak_kv_append_rope(W, dak.dak_rope_make(64), None, Q, Q, lens),
                 lambda: dak.dak_attn_acc(Q, kv, seq_lens=lens.cpu()), lambda: dak.dak_attn_acc(Q.cpu(), kv),
                 lambda: dak.dak_attn_acc(Q, kv, acc_out=acc[:, :1]), lambda: dak.dak_attn_acc(Q, kv, seq_lens=lens.long())):
        with pytest.raises(ValueError):
            call()
    for heads, status in ((3, 1), (34, 7)):  # not a multiple of the kv heads; 17 query heads a kv head
        with pytest.raises(dak.DakError) as e:
            dak.dak_attn_acc(torch.zeros(2, heads, 64, dtype=torch.bfloat16, device="cuda"), kv)
        assert e.value.status == status
        with pytest.raises(dak.DakError) as e:
            dak.dak_attn_prefix(torch.zeros(2, heads, 64, dtype=torch.bfloat16, device="cuda"), kv, kv)
        assert e.value.status == status
    _ok(dak)
    kv.free()


# ---------------------------------------------------------------- together

@pytest.mark.parametrize("use_prefix", [False, True])
def test_a_chat_over_its_budget(dak, use_prefix):
    """Prompt, then steps of rotate-and-append, attention with weights, and eviction whenever a
    cache is full, against the same in fp64 that keeps every surviving row by its position."""
    import torch
    B, Hq, Hkv, D, L, T, keep, recent, steps = 2, 8, 2, 64, 96, 60, 64, 16, 90
    G, freqs = Hq // Hkv, oc.inv_freq(64, 10000.0)
    rope = dak.dak_rope_make(D, theta=10000.0)
    z = np.zeros((B, Hkv, L, D), np.uint16)
    kv = dak.dak_place_kv_heads(z, z, 1)
    prefix = pre = None
    if use_prefix:
        prefix = synth.attn_inputs(1, Hq, Hkv, D, 200, seed=77)[1:]
        pre = dak.dak_place_kv_heads(*prefix, 1)
    acc = torch.zeros(B, Hkv, L, device="cuda")
    sp = torch.full((B, Hkv, L), -1, dtype=torch.int32, device="cuda")
    rng = np.random.default_rng(3)
    n_new = [T, T - 9]
    x = torch.from_numpy(rng.standard_normal((B, T, Hq + 2 * Hkv, D)).astype(np.float32)).cuda().to(torch.bfloat16)
    start = _i32([0, 0])
    dak.dak_kv_append_rope(kv, rope, x[:, :, :Hq], x[:, :, Hq:Hq + Hkv], x[:, :, Hq + Hkv:], start, n_new=_i32(n_new),
                           slot_pos=sp)
    lens, pos = _i32(n_new), _i32(n_new)
    evictions = 0
    for step in range(steps):
        x = torch.from_numpy(rng.standard_normal((B, Hq + 2 * Hkv, D)).astype(np.float32)).cuda()
        q = dak.dak_kv_append_rope(kv, rope, x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:], lens, positions=pos,
                                   slot_pos=sp)
        lens, pos = lens + 1, pos + 1
        before, hl = acc.cpu().numpy(), lens.tolist()
        if use_prefix:
            O = dak.dak_attn_prefix(q, kv, pre, seq_lens=lens, acc_in=acc, acc_out=acc)
        else:
            O, _ = dak.dak_attn_acc(q, kv, acc_in=acc, acc_out=acc, seq_lens=lens)
        _ok(dak)
        if step % 15 == 0 or step == steps - 1:
            K, V = _cache(kv)
            o, w, spread, reach = oc.attention(bits_of(q), K, V, hl, prefix)
            _check_attn(O, o, spread, reach, D, L + 200, False)
            _check_weights(acc, before, w, before, hl, reach, G, D, L + 200)
            tab = sp.cpu().numpy()
            for b in range(B):
                for g in range(Hkv):
                    live = tab[b, g, :hl[b]]
                    assert len(set(live.tolist())) == hl[b] and live.max() == pos[b].item() - 1
                    # the newest tokens are all there
                    assert set(range(pos[b].item() - recent, pos[b].item())) <= set(live.tolist())
        if max(hl) == L:
            a0, p0 = acc.cpu().numpy(), sp.cpu().numpy()
            k0, v0 = _cache(kv)
            lens, src = dak.dak_kv_evict(kv, lens, keep, recent, acc, sp)
            wl, ws, wa, wp = oc.evict(hl, keep, recent, a0, p0)
            assert lens.tolist() == wl.tolist() and np.array_equal(src.cpu().numpy(), ws)
            assert np.array_equal(acc.cpu().numpy(), wa) and np.array_equal(sp.cpu().numpy(), wp)
            evictions += 1
    assert evictions >= 2
    kv.free()
    if pre:
        pre.free()

"""SplitK_FlashAttn with drafted trees: a run of drafting, attending, accepting and forking leaves the
rows that decoding the accepted tokens one by one leaves, and attends as it does."""
import numpy as np
import pytest

from gpu_util import to_np
from oracle import cache as oc
from test_cache_ops_gpu import _attn_tol, _cache, _i32, _ok, dak  # noqa: F401

pytestmark = pytest.mark.gpu


def _zeros(B, H, L, D):
    import torch
    return torch.zeros(B, H, L, D, dtype=torch.bfloat16, device="cuda")


@pytest.mark.parametrize("tracked,fp32,host", [(False, False, 3), (True, True, 0)])
def test_drafting_run(dak, tracked, fp32, host):
    """Six steps of seven drafts each, of which a random path is accepted, against the same tokens decoded one by
    one; then requests swap and go on."""
    import torch
    B, T, Hq, Hkv, D, L, prompt = 3, 7, 8, 2, 64, 200, 70
    rng = np.random.default_rng(11)
    attn = dak.SplitK_FlashAttn(_zeros(B, Hkv, L, D), _zeros(B, Hkv, L, D), n_host_heads=host, fp32_out=fp32,
                                tuning=dict(pdl=2))
    one = dak.SplitK_FlashAttn(_zeros(B, Hkv, L, D), _zeros(B, Hkv, L, D), n_host_heads=1, fp32_out=fp32)
    if tracked:
        attn.track(), one.track()
    rope = dak.dak_rope_make(D, theta=10000.0)
    axes = dak.dak_rope_axes_make(rope)
    H = Hq + 2 * Hkv

    def tokens(n):
        return torch.from_numpy(rng.standard_normal((B, n, H, D)).astype(np.float32)).cuda().to(torch.bfloat16)

    x = tokens(prompt)
    lens = _i32([prompt, prompt - 20, 3])
    for m in (attn, one):
        m.append_rope(rope, None, x[:, :, Hq:Hq + Hkv], x[:, :, Hq + Hkv:], _i32([0] * B), n_new=lens)
    lens1 = lens.clone()
    for step in range(6):
        parents = np.array([[rng.integers(-1, t) if t else -1 for t in range(T)] for _ in range(B)])
        mask, depth = dak.dak_tree_mask(parents)
        x = tokens(T)
        at = (lens[:, None] + depth)[:, :, None].contiguous()
        q = attn.append_rope(axes, x[:, :, :Hq], x[:, :, Hq:Hq + Hkv], x[:, :, Hq + Hkv:], lens, positions=at)
        o = attn.forward_tree(q, lens, mask=mask)
        assert o.dtype == (torch.float32 if fp32 else torch.bfloat16) and o.shape == q.shape
        # accepted: a random node's ancestors and itself, or none
        path, n_path = np.zeros((B, T), int), np.zeros(B, int)
        for b in range(B):
            node, nodes = rng.integers(-1, T), []
            while node >= 0:
                nodes.append(node)
                node = parents[b, node]
            path[b, :len(nodes)], n_path[b] = nodes[::-1], len(nodes)
        lens = attn.commit(lens, _i32(path), _i32(n_path), T)
        # the same tokens one by one
        for i in range(n_path.max()):
            new = _i32((n_path > i).astype(int))
            sel = torch.from_numpy(path[:, i]).cuda()
            y = x[torch.arange(B, device="cuda"), sel][:, None]
            q1 = one.append_rope(rope, y[:, :, :Hq], y[:, :, Hq:Hq + Hkv], y[:, :, Hq + Hkv:], lens1, n_new=new)
            lens1 = lens1 + new
            o1 = one(q1[:, 0], seq_lens=lens1)
            K, V = (oc._f64(c) for c in _cache(one.placement))
            for b in np.flatnonzero(n_path > i):
                n = int(lens1[b])
                assert torch.equal(q1[b, 0], q[b, path[b, i]])
                # both within the attention's own bound of the exact result
                ref, _, spread, reach = oc.attention(to_np(q1[b:b + 1, 0]), K[b:b + 1, :, :n], V[b:b + 1, :, :n], [n])
                tol = _attn_tol(D, n, ref, spread, reach, fp32, parts=None if fp32 or tracked else 1)
                assert (np.abs(to_np(o[b:b + 1, path[b, i]]) - ref) <= tol).all()
                assert (np.abs(to_np(o1[b:b + 1]) - ref) <= tol).all()
        assert torch.equal(lens, lens1)
        _ok(dak)
        a, c = _cache(attn.placement), _cache(one.placement)
        for b in range(B):
            n = int(lens[b])
            for u, v in zip(a, c):
                assert np.array_equal(u[b, :, :n], v[b, :, :n])
            if tracked:
                assert torch.equal(attn.slot_pos[b, :, :n], one.slot_pos[b, :, :n])
                assert not attn.weights[b, :, n:n + 1].any()
    # beams: 0 and 2 swap, 1 goes on from 2's rows
    before, tables = _cache(attn.placement), attn.slot_pos.clone() if tracked else None
    old = lens.tolist()
    lens = attn.fork(_i32([2, 2, 0]), lens)
    assert lens.tolist() == [old[2], old[2], old[0]]
    for u, v in zip(_cache(attn.placement), before):
        for b, f in enumerate((2, 2, 0)):
            assert np.array_equal(u[b, :, :old[f]], v[f, :, :old[f]])
    if tracked:
        assert torch.equal(attn.slot_pos[2, :, :old[0]], tables[0, :, :old[0]])
    # the other module takes one of them over
    lens1 = one.fork(_i32([-1, 2, -1]), lens, source=attn, lens=lens1)
    assert lens1.tolist() == [old[0], old[0], old[2]]
    for u, v in zip(_cache(one.placement), _cache(attn.placement)):
        assert np.array_equal(u[1, :, :old[0]], v[2, :, :old[0]])
    q = tokens(1)[:, 0, :Hq].contiguous()
    o = attn(q, seq_lens=lens)
    # requests 0 and 1 hold the same rows now
    two = attn(q[:1].expand(B, Hq, D).contiguous(), seq_lens=lens)
    assert torch.equal(two[0], two[1]) and torch.equal(o[0], two[0])
    _ok(dak)


def test_module_refusals(dak):
    import torch
    a, b = (dak.SplitK_FlashAttn(_zeros(2, 1, 64, 64), _zeros(2, 1, 64, 64)) for _ in range(2))
    lens = _i32([3, 4])
    with pytest.raises(ValueError):
        a.fork(lens, lens, lens=lens)
    with pytest.raises(ValueError):
        a.fork(_i32([0, 1]), lens, source=b)
    a.track()
    with pytest.raises(ValueError):
        a.fork(_i32([0, 1]), lens, source=b, lens=lens)
    rope = dak.dak_rope_axes_make(dak.dak_rope_make(64))
    x = torch.zeros(2, 3, 1, 64, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ValueError):
        a.append_rope(rope, None, x, x, lens)  # positions are each token's own
    _ok(dak)

"""The merge of dak_attn_tree's partial results over many pieces: one request whose tiles are cut into as many
ranges as there are, against the fp64 oracle. A warp of the merge takes pieces two at a time for heads of 64 and
one at a time for heads of 128, in rounds of 32."""
import numpy as np
import pytest

import synth
from gpu_util import to_dev
from oracle import tree as ot
from test_cache_ops_gpu import _check_attn, _i32, _ok, dak  # noqa: F401

pytestmark = pytest.mark.gpu

# A range is at least 8 (up to 16 rows a kv head) or 9 units long, a chunk of 64 keys 2 of them, a tile by itself 4 or 6,
# so that a tile of c chunks is cut into about (4 + 2 c) / 8 or (6 + 2 c) / 9 pieces where CTAs are enough.
CASES = [(T, Hq, D, c * 64 - 7) for D in (64, 128) for T, Hq in ((3, 2), (16, 1)) for c in (126, 128, 130, 134, 250, 254, 258, 262)]
CASES += [(T, Hq, D, c * 64 - 7) for D in (64, 128) for T, Hq in ((20, 2),) for c in (141, 144, 146, 150, 280, 284, 290, 294)]
CASES += [(3, 2, 64, 100 * 64), (3, 2, 64, 20000), (150, 1, 64, 12001), (20, 3, 64, 19999)]


@pytest.mark.parametrize("fp32", [False, True])
@pytest.mark.parametrize("T,Hq,D,rows", CASES)
def test_many_pieces(dak, T, Hq, D, rows, fp32):
    q = synth.normal_bf16(T, 1, T * Hq * D).reshape(1, T, Hq, D)
    k, v = (synth.normal_bf16(rows, i, rows * D).reshape(1, 1, rows, D) for i in (2, 3))
    kv = dak.dak_place_kv_heads(k, v, 0)
    o = dak.dak_attn_tree(to_dev(q), kv, _i32([rows - T]), o_fp32=fp32)
    _ok(dak)
    ref, spread, reach = ot.attention(q, k, v, [rows - T])
    _check_attn(o, ref, spread, reach, D, rows, fp32)


@pytest.mark.parametrize("T,Hq", [(3, 2), (20, 2)])
@pytest.mark.parametrize("D", [64, 128])
def test_every_piece_counts_once(dak, T, Hq, D):
    """V is one in 64 keys and zero elsewhere, scores are all zero: the result is those keys' share, for every
    chunk, so that a piece that is left out, taken twice or weighed by another's factor shows."""
    import torch
    chunks = 290
    rows = chunks * 64
    q = torch.zeros(1, T, Hq, D, dtype=torch.bfloat16, device="cuda")
    k = torch.zeros(1, 1, rows, D, dtype=torch.bfloat16, device="cuda")
    lens = _i32([rows - T])
    for first in range(0, chunks, D):  # a column a chunk
        v = torch.zeros(1, 1, rows, D, dtype=torch.bfloat16, device="cuda")
        n = min(D, chunks - first)
        for c in range(n):
            v[0, 0, (first + c) * 64:(first + c + 1) * 64, c] = 1.0
        kv = dak.dak_place_kv_heads(k, v, 0)
        o = dak.dak_attn_tree(q, kv, lens, o_fp32=True)
        _ok(dak)
        for t in range(T):
            seen = rows - T + t + 1
            have = np.clip(seen - (first + np.arange(n)) * 64, 0, 64)
            # sums of at most 2^15 ones are exact; a quotient and the merge's products round a few times
            np.testing.assert_allclose(o[0, t, :, :n].cpu().numpy(), np.broadcast_to(have / seen, (Hq, n)), rtol=2.0 ** -21)
            assert (o[0, t, :, n:] == 0).all()

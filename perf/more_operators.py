"""What a serving program that drafts tokens does with a placed KV cache, as timed cases: rotate
and append tokens whose positions have several axes (or one, of siblings in a tree), attend with
a tree of drafted tokens over a cache, keep the accepted path of the tree, and let requests take
over the rows of others (beams, samples of one prompt).

`run` computes each operator in its plain form (elementary torch operations in 32 bits, angles
in 64) or, where `own` is true, with the package's entry points; both take what `prepare`
makes. A cache is returned as its slabs lie in memory: [slabs][chunks of 64 tokens][K, V][64][D],
where the 8-element piece c of token t's row is stored at piece c ^ (t % 8).
"""
import math
import random

import torch

own = False

CHUNK = 64


def listed():
    return [
        # ---- attention of a tree of drafted tokens over each request's cache
        # one chat of the 8B shape over 4K context, a small tree: latency
        dict(name="tree_one", op="tree", B=1, T=8, Hq=32, Hkv=8, D=128, L=4109, lo=4001, hi=4001, ragged=False,
             blank=False, fp32=False),
        # 32 chats of that shape over up to 8K, 16 drafted tokens each
        dict(name="tree_batch", op="tree", B=32, T=16, Hq=32, Hkv=8, D=128, L=8192, lo=7000, hi=8170, ragged=True,
             blank=False, fp32=False),
        # wide trees of the 70B shape, 512 query rows a kv head, over contexts of up to 2K
        dict(name="tree_wide", op="tree", B=48, T=64, Hq=64, Hkv=8, D=128, L=2112, lo=1500, hi=2047, ragged=True,
             blank=False, fp32=False),
        # 64-wide heads without sharing, ragged from empty on, tokens that see no draft, fp32 output
        dict(name="tree_mha_fp32", op="tree", B=12, T=5, Hq=16, Hkv=16, D=64, L=2507, lo=0, hi=2500, ragged=True,
             blank=True, fp32=True),
        # ---- rotation by per-token positions and append
        # the drafted tokens of 32 chats from the projection's fp32 output: siblings share a position
        dict(name="axes_tree", op="axes", B=32, T=16, Hq=32, Hkv=8, D=128, rot=128, inter=False, axes=1, cycled=False,
             L=130, far=100000, fp32=True, tracked=True),
        # prompts of text and pictures: time, height and width, each its block of the pairs
        dict(name="axes_prompt", op="axes", B=2, T=4096, Hq=32, Hkv=8, D=128, rot=128, inter=False, axes=3,
             cycled=False, L=4200, far=60000, fp32=False, tracked=False),
        # ---- the accepted path of the tree becomes part of the cache
        # 32 chats, up to five of 16 drafts accepted: latency
        dict(name="commit_step", op="commit", B=32, T=16, Hkv=8, D=128, L=1000, lo=100, hi=984, most=5, tracked=False),
        # a wide batch in a tracked cache, long paths
        dict(name="commit_wide", op="commit", B=256, T=64, Hkv=8, D=128, L=300, lo=0, hi=236, most=48, tracked=True),
        # ---- requests take over the rows of others
        # four beams each of four requests go on from others of their group, in place, behind their prompts
        dict(name="fork_beams", op="fork", B=16, group=4, source=0, Hkv=8, D=128, L=1100, lo=300, hi=1100, first=256,
             tracked=False),
        # 16 samples of two prompts from a placement of their own
        dict(name="fork_samples", op="fork", B=16, group=8, source=2, Hkv=8, D=128, L=8192, lo=6001, hi=8000, first=0,
             tracked=False),
        # a tracked cache of 64-wide heads in which every request goes on from any other, in place
        dict(name="fork_any", op="fork", B=61, group=61, source=0, Hkv=4, D=64, L=3001, lo=0, hi=3001, first=0,
             tracked=True),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["tree", "tree", "axes", "commit", "fork"])
    D = rng.choice([64, 128, 128])
    Hkv = rng.choice([1, 2, 4, 8, 8])
    G = rng.choice([1, 2, 4, 4, 5, 8])
    if op == "tree":
        T = _log_int(rng, 1, 256 if rng.random() < 0.2 else 64)
        B = _log_int(rng, 1, 64)
        L = T + _log_int(rng, 1, min(8192, 1_900_000 // (B * Hkv), 8_000_000 // (B * max(T, 8) * G)))
        hi = L - T - rng.choice([0, 0, (L - T) // 9])
        return dict(op=op, B=B, T=T, Hq=Hkv * G, Hkv=Hkv, D=D, L=L, lo=rng.randint(0, hi), hi=hi,
                    ragged=rng.random() < 0.5, blank=rng.random() < 0.3, fp32=rng.random() < 0.25)
    if op == "axes":
        T = _log_int(rng, 1, 4096)
        B = _log_int(rng, 1, max(1, min(256, 262144 // (T * Hkv * max(G, 4)))))
        rot = rng.choice([D, D, D // 2, D - 8, 12])
        return dict(op=op, B=B, T=T, Hq=Hkv * G, Hkv=Hkv, D=D, rot=rot, inter=rng.random() < 0.3,
                    axes=rng.choice([1, 2, 3, 3, 4]), cycled=rng.random() < 0.5, L=T + rng.randint(0, 200),
                    far=_log_int(rng, T, 1000000), fp32=rng.random() < 0.3, tracked=rng.random() < 0.5)
    if op == "commit":
        T = _log_int(rng, 1, 256)
        B = _log_int(rng, 1, max(1, min(256, 16384 // T)))
        L = T + _log_int(rng, 1, 1000)
        return dict(op=op, B=B, T=T, Hkv=Hkv, D=D, L=L, lo=rng.randint(0, L - T), hi=L - T, most=rng.randint(1, T),
                    tracked=rng.random() < 0.5)
    B = _log_int(rng, 2, 64)
    source = rng.choice([0, 0, 1, 3])
    L = _log_int(rng, 4, min(8192, 800000 // (B * Hkv)))
    lo = rng.randint(0, L)
    return dict(op=op, B=B, group=rng.randint(1, B), source=source, Hkv=Hkv, D=D, L=L, lo=lo, hi=rng.randint(lo, L),
                first=rng.choice([0, 0, lo // 2]), tracked=rng.random() < 0.3)


# ------------------------------------------------------------------ what a case fixes besides its numbers

def _lens(case, n=None):
    """Ragged lengths of a case, spread over lo..hi out of order (the last request's is hi)."""
    B, lo, hi = n or case["B"], case["lo"], case["hi"]
    return [hi if b == B - 1 else lo + (hi - lo) * ((b * 37 + 11) % B) // B for b in range(B)]


def _n_new(case):
    """Drafted tokens of each request: all T, or in ragged batches up to a quarter fewer."""
    B, T = case["B"], case["T"]
    if not case.get("ragged"):
        return [T] * B
    return [T - ((b * 5 + 3) % B) * T // (4 * B) for b in range(B)]


def _n_path(case):
    """Accepted drafts of each request, from none to `most`."""
    return [(b * 7 + case["most"]) % (case["most"] + 1) for b in range(case["B"])]


def _source_of(case):
    """Whose rows each request takes over: any of its group's, or (a source placement) its group's prompt. In
    groups of three and more the last request stays as it is."""
    B, group, rng = case["B"], case["group"], random.Random(case["B"] * 1000 + case["group"])
    of = []
    for b in range(B):
        g0 = b // group * group
        size = min(group, B - g0)
        if case["source"]:
            of.append(b // group % case["source"])
        elif size >= 3 and b == g0 + size - 1:
            of.append(-1)
        else:
            of.append(g0 + rng.randrange(size))
    return of


def work(case):
    op, B, D, Hkv = case["op"], case["B"], case["D"], case["Hkv"]
    if op == "axes":
        n, size = B * case["T"], 4 if case["fp32"] else 2
        row = (case["Hq"] + 2 * Hkv) * D
        return {"bytes": n * (row * (size + 2) + 4 * case["axes"] + Hkv * (8 if case["tracked"] else 4)),
                "flops": 3 * n * (case["Hq"] + Hkv) * case["rot"]}
    if op == "tree":
        Hq, n_new, lens = case["Hq"], _n_new(case), _lens(case)
        out = 4 if case["fp32"] else 2
        nbytes = sum(m * Hq * D * (2 + out) + m * 8 * (-(-case["T"] // 64)) for m in n_new)
        nbytes += sum((n + m) * Hkv * D * 4 for n, m in zip(lens, n_new))
        return {"bytes": nbytes, "flops": sum(4 * m * (n + m) * Hq * D for n, m in zip(lens, n_new))}
    if op == "commit":
        # a path of n of T drafts, ascending: about n / (T + 1) of its rows lie where they belong already
        T, moved = case["T"], 0.0
        for n in _n_path(case):
            moved += n * (1 - n / (T + 1))
        return {"bytes": int(Hkv * moved * D * 8 + B * 4 * (case["most"] + 3)
                             + (8 * B * Hkv * T if case["tracked"] else 0)), "flops": 0}
    of, lens = _source_of(case), _lens(case, case["source"])
    row = D * 4 + (8 if case["tracked"] else 0)
    take = [(b, f) for b, f in enumerate(of) if f >= 0 and (case["source"] or f != b)]
    rows = sum(max(0, lens[f] - case["first"]) for _, f in take)
    rows += sum(max(0, lens[f] - case["first"]) for f in {f for _, f in take})
    return {"bytes": rows * Hkv * row + 12 * B, "flops": 0}


# ------------------------------------------------------------------ rotation

THETA = 500000.0


def _inv_freq(case):
    """Inverse frequencies, radians per position, in 64 bits."""
    return THETA ** (-torch.arange(0, case["rot"], 2, dtype=torch.float64) / case["rot"])


def _axis(case):
    """The axis of each pair: blocks of the pairs, or the axes in turn."""
    n, A = case["rot"] // 2, case["axes"]
    return [i % A if case["cycled"] else min(A - 1, i * A // n) for i in range(n)]


def _slab_index(L, D, device):
    """Where element (token, d) of a K or V slab lies: (chunk, token in chunk, stored d), each [L][D]."""
    t = torch.arange(L, device=device)[:, None]
    d = torch.arange(D, device=device)[None, :]
    return (t // CHUNK).expand(L, D), (t % CHUNK).expand(L, D), ((d // 8) ^ (t % 8)) * 8 + d % 8


def _to_slabs(k, v):
    """K, V [B][H][L][D] as the placed cache lies: [B*H][chunks][2][64][D], zero behind L."""
    B, H, L, D = k.shape
    out = torch.zeros(B * H, -(-L // CHUNK), 2, CHUNK, D, dtype=k.dtype, device=k.device)
    c, t, d = _slab_index(L, D, k.device)
    out[:, c, 0, t, d] = k.reshape(B * H, L, D)
    out[:, c, 1, t, d] = v.reshape(B * H, L, D)
    return out


# ------------------------------------------------------------------ inputs

def _trees(case, seed):
    """Masks int64 [B][T][words of 64] of random trees (bit s: the token sees draft s) and depths [B][T]."""
    B, T, rng = case["B"], case["T"], random.Random(seed)
    masks, depths = [], []
    for _ in range(B):
        seen, depth = [], []
        for t in range(T):
            parent = rng.randrange(max(0, t - 8), t) if t and rng.random() > 0.05 else -1
            seen.append((seen[parent] if parent >= 0 else 0) | 1 << t)
            depth.append(depth[parent] + 1 if parent >= 0 else 0)
        if case.get("blank"):
            seen[::7] = [0] * len(seen[::7])
        masks.append([[(m >> 64 * w) & (1 << 64) - 1 for w in range(-(-T // 64))] for m in seen])
        depths.append(depth)
    signed = [[[w - (1 << 64) if w >> 63 else w for w in row] for row in m] for m in masks]
    return torch.tensor(signed, dtype=torch.int64), torch.tensor(depths, dtype=torch.int32)


def _positions(case, seed, start):
    """Per-token positions int32 [B][T][axes]: a tree's depths, or text and then pictures of 24 x 32 patches."""
    B, T, A = case["B"], case["T"], case["axes"]
    if A == 1:
        return start[:, None, None] + _trees(case, seed)[1][:, :, None]
    i = torch.arange(T)
    text = T // 4
    j = (i - text).clamp_min(0)
    axes = [text + j // 768, text + j // 32 % 24, text + j % 32, j % 7][:A]
    grid = torch.stack([torch.where(i < text, i, a) for a in axes], -1).int()
    return start[:, None, None] + grid


def _inputs(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def normal(*shape, dtype=torch.bfloat16):
        return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32).to(dtype)

    def ints(x):
        return torch.tensor(x, dtype=torch.int32, device="cuda")

    def table(n, L):
        acc = torch.rand(n, Hkv, L, generator=g, device="cuda")
        pos = (torch.rand(n, Hkv, L, generator=g, device="cuda") * 100000).int()
        return pos, acc

    op, B, Hkv, D, L = case["op"], case["B"], case["Hkv"], case["D"], case["L"]
    s = {"case": case}
    if op == "axes":
        T, H = case["T"], case["Hq"] + 2 * Hkv
        # the projection's output: query, key and value rows of each token side by side
        s["qkv"] = normal(B, T, H * D, dtype=torch.float32 if case["fp32"] else torch.bfloat16)
        s["slots"] = (torch.rand(B, generator=g, device="cuda") * (L - T + 1)).int()
        start = (torch.rand(B, generator=g, device="cuda") * (case["far"] - T + 1)).int()
        s["positions"] = _positions(case, seed, start.cpu()).to("cuda").int().contiguous()
        s["k"], s["v"] = normal(B, Hkv, L, D), normal(B, Hkv, L, D)
        s["pos"], acc = table(B, L)
        s["acc"] = acc if case["tracked"] else None
        s["q_out"] = torch.zeros(B, T, case["Hq"], D, dtype=torch.bfloat16, device="cuda")
        return s
    n = case["source"] if op == "fork" and case["source"] else B
    s["lens"] = ints(_lens(case, n))
    s["k"], s["v"] = normal(B, Hkv, L, D), normal(B, Hkv, L, D)
    if op == "tree":
        T = case["T"]
        s["q"] = normal(B, T, case["Hq"], D)
        s["mask"] = _trees(case, seed)[0].to("cuda")
        s["n_new"] = ints(_n_new(case))
        s["o"] = torch.zeros(B, T, case["Hq"], D, dtype=torch.float32 if case["fp32"] else torch.bfloat16, device="cuda")
        return s
    s["pos"], s["acc"] = table(B, L) if case["tracked"] else (None, None)
    if op == "commit":
        # ascending paths: the first of a random order of the drafts, sorted
        order = torch.rand(B, case["T"], generator=g, device="cuda").argsort(-1)
        behind = torch.arange(case["most"], device="cuda") >= ints(_n_path(case))[:, None]
        path = order[:, :case["most"]].masked_fill(behind, case["T"]).sort(-1).values
        s["path"], s["n_path"] = path.masked_fill(behind, 0).int().contiguous(), ints(_n_path(case))
        return s
    s["of"] = ints(_source_of(case))
    s["first"] = ints([case["first"]] * B)
    if case["source"]:
        s["k2"], s["v2"] = normal(n, Hkv, L, D), normal(n, Hkv, L, D)
        s["pos2"], s["acc2"] = table(n, L) if case["tracked"] else (None, None)
        s["own_lens"] = ints([0] * B)
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    op, D = case["op"], case["D"]
    if op != "tree" and not own:
        s["slabs"] = _to_slabs(s.pop("k"), s.pop("v"))
        if "k2" in s:
            s["slabs2"] = _to_slabs(s.pop("k2"), s.pop("v2"))
    if op == "axes":
        s["inv_freq"], s["axis"] = _inv_freq(case).cuda(), torch.tensor(_axis(case), device="cuda")
    if own:
        import direct_host_memory_gb300 as dak
        s["kv"] = dak.dak_place_kv_heads(s.pop("k"), s.pop("v"), 0)
        if "k2" in s:
            s["kv2"] = dak.dak_place_kv_heads(s.pop("k2"), s.pop("v2"), 0)
        if op == "axes":
            rope = dak.dak_rope_make(D, rot_dim=case["rot"], theta=THETA, interleaved=case["inter"])
            s["rope"] = dak.dak_rope_axes_make(rope, _axis(case), n_axes=case["axes"])
            B, T, Hq, Hkv = case["B"], case["T"], case["Hq"], case["Hkv"]
            x = s["qkv"].view(B, T, Hq + 2 * Hkv, D)
            s["q"], s["kn"], s["vn"] = x[:, :, :Hq], x[:, :, Hq:Hq + Hkv], x[:, :, Hq + Hkv:]
        if op != "tree":
            s["slabs"] = s["kv"].slabs()[1]
    return s


# ------------------------------------------------------------------ the operators

def run(state):
    return {"tree": _tree, "axes": _axes, "commit": _commit, "fork": _fork}[state["case"]["op"]](state)


def _seen(s):
    """Which rows each drafted token sees, [B][T][L]: those in the cache before, and its mask's drafts."""
    c = s["case"]
    B, T, L = c["B"], c["T"], c["L"]
    dev = s["q"].device
    bits = (s["mask"][..., None] >> torch.arange(64, device=dev)) & 1
    bits = bits.flatten(-2)[..., :T].bool() & (torch.arange(T, device=dev) < s["n_new"][:, None])[:, None]
    draft = torch.arange(L, device=dev) - s["lens"][:, None]  # [B][L]
    at = draft.clamp(0, T - 1)[:, None].expand(B, T, L)
    return (draft < 0)[:, None] | ((draft >= 0) & (draft < T))[:, None] & bits.gather(-1, at)


def _tree(s):
    """o[b, t] = softmax(q[b, t] . K^T / sqrt(D)) V over the rows that the token sees; none: zeros."""
    c = s["case"]
    if own:
        import direct_host_memory_gb300 as dak
        return dak.dak_attn_tree(s["q"], s["kv"], s["lens"], mask=s["mask"], n_new=s["n_new"], O=s["o"],
                                 o_fp32=c["fp32"])
    B, T, Hq, Hkv, D, L = c["B"], c["T"], c["Hq"], c["Hkv"], c["D"], c["L"]
    G = Hq // Hkv
    q = s["q"].float().view(B, T, Hkv, G, D).permute(0, 2, 1, 3, 4).reshape(B, Hkv, T * G, D) / math.sqrt(D)
    x = (q @ s["k"].float().transpose(-1, -2)).view(B, Hkv, T, G, L)
    x = x.masked_fill(~_seen(s)[:, None, :, None], -math.inf)
    m = x.amax(-1, keepdim=True)
    e = torch.exp(x - torch.where(m == -math.inf, torch.zeros_like(m), m))
    z = e.sum(-1, keepdim=True)
    p = torch.where(z > 0, e / z, torch.zeros_like(e))
    # rows behind a request's drafts may hold anything
    behind = torch.arange(L, device=x.device) >= (s["lens"] + s["n_new"])[:, None]
    v = s["v"].float().masked_fill(behind[:, None, :, None], 0.0)
    o = (p.view(B, Hkv, T * G, L) @ v).view(B, Hkv, T, G, D).permute(0, 2, 1, 3, 4).reshape(B, T, Hq, D)
    new = torch.arange(T, device=x.device) < s["n_new"][:, None]
    s["o"][new] = o.to(s["o"].dtype)[new]
    return s["o"]


def _axes(s):
    """Rotate each token's query into q_out and its key into the cache row it is appended to, with its value:
    pair i turns by the token's position on the pair's axis times f_i."""
    c = s["case"]
    if own:
        import direct_host_memory_gb300 as dak
        dak.dak_kv_append_rope_axes(s["kv"], s["rope"], s["q"], s["kn"], s["vn"], s["slots"], s["positions"],
                                    q_out=s["q_out"], slot_pos=s["pos"], acc=s["acc"])
        return {"q": s["q_out"], "slabs": s["slabs"], "pos": s["pos"], "acc": s["acc"]}
    B, T, Hq, Hkv, D, R = c["B"], c["T"], c["Hq"], c["Hkv"], c["D"], c["rot"]
    dev = s["qkv"].device
    x = s["qkv"].view(B, T, Hq + 2 * Hkv, D)
    angle = s["positions"].double()[:, :, s["axis"]] * s["inv_freq"]  # [B][T][R/2]
    cos, sin = torch.cos(angle).float()[:, :, None], torch.sin(angle).float()[:, :, None]
    qk = x[:, :, :Hq + Hkv].float()
    if c["inter"]:
        a, b = qk[..., 0:R:2], qk[..., 1:R:2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = qk[..., :R // 2], qk[..., R // 2:R]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    qk = torch.cat([turned, qk[..., R:]], -1).to(torch.bfloat16)
    s["q_out"].copy_(qk[:, :, :Hq])
    b = torch.arange(B, device=dev)[:, None].expand(B, T).reshape(-1)
    row = (s["slots"].long()[:, None] + torch.arange(T, device=dev)).reshape(-1)
    rows = s["slabs"].view(B, Hkv, -1, 2, CHUNK, D // 8, 8)
    piece = torch.arange(D // 8, device=dev)
    kv = torch.stack([qk[:, :, Hq:], x[:, :, Hq + Hkv:].to(torch.bfloat16)], 3).view(B * T, Hkv, 2, D // 8, 8)
    rows[b[:, None], :, (row // CHUNK)[:, None], :, (row % CHUNK)[:, None], piece ^ (row % 8)[:, None]] = \
        kv.permute(0, 3, 1, 2, 4)
    s["pos"][b, :, row] = s["positions"][:, :, 0].reshape(-1, 1).expand(-1, Hkv)
    if s["acc"] is not None:
        s["acc"][b, :, row] = 0.0
    return {"q": s["q_out"], "slabs": s["slabs"], "pos": s["pos"], "acc": s["acc"]}


def _commit(s):
    """Row lens + path[i] of every kv head becomes row lens + i, for i below n_path; the table entries of the
    drafts that are not kept become -1 and 0. Returns the new lengths too."""
    c = s["case"]
    if own:
        import direct_host_memory_gb300 as dak
        lens = dak.dak_kv_commit(s["kv"], s["lens"], s["path"], s["n_path"], c["T"], slot_pos=s["pos"], acc=s["acc"])
        return {"slabs": s["slabs"], "lens": lens, "pos": s["pos"], "acc": s["acc"]}
    B, T, Hkv, D, L = c["B"], c["T"], c["Hkv"], c["D"], c["L"]
    dev = s["lens"].device
    i = torch.arange(c["most"], device=dev)
    b, i = (i < s["n_path"][:, None]).nonzero(as_tuple=True)
    base = s["lens"].long()[b]
    fr, to = base + s["path"].long()[b, i], base + i
    rows = s["slabs"].view(B, Hkv, -1, 2, CHUNK, D // 8, 8)
    piece = torch.arange(D // 8, device=dev)
    moved = rows[b[:, None], :, (fr // CHUNK)[:, None], :, (fr % CHUNK)[:, None], piece ^ (fr % 8)[:, None]]
    rows[b[:, None], :, (to // CHUNK)[:, None], :, (to % CHUNK)[:, None], piece ^ (to % 8)[:, None]] = moved
    lens = s["lens"] + s["n_path"]
    if s["pos"] is not None:
        slot = torch.arange(L, device=dev)
        gone = ((slot >= lens[:, None]) & (slot < s["lens"][:, None] + T))[:, None].expand(B, Hkv, L)
        for t, empty in ((s["pos"], -1), (s["acc"], 0)):
            t[b, :, to] = t[b, :, fr]
            t.masked_fill_(gone, empty)
    return {"slabs": s["slabs"], "lens": lens, "pos": s["pos"], "acc": s["acc"]}


def _fork(s):
    """Request b's rows from first[b] on become those of request of[b] (negative: b stays), all at once."""
    c = s["case"]
    B, Hkv, L = c["B"], c["Hkv"], c["L"]
    if own:
        import direct_host_memory_gb300 as dak
        kw = {}
        if c["source"]:
            kw = dict(source=s["kv2"], lens_out=s["own_lens"], source_slot_pos=s["pos2"], source_acc=s["acc2"])
        lens = dak.dak_kv_fork(s["kv"], s["of"], s["lens"], first=s["first"], slot_pos=s["pos"], acc=s["acc"], **kw)
        return {"slabs": s["slabs"], "lens": lens, "pos": s["pos"], "acc": s["acc"]}
    dev = s["of"].device
    of = s["of"].long()
    takes, at = of >= 0, of.clamp_min(0)
    n = s["lens"][at]
    slot = torch.arange(L, device=dev)
    new = (takes[:, None] & (slot >= s["first"][:, None]) & (slot < n[:, None]))[:, None].expand(B, Hkv, L)
    own_lens = s["own_lens"] if c["source"] else s["lens"]
    dst = s["slabs"].view(B, Hkv, -1, 2, CHUNK, c["D"])
    src = s["slabs2"].view(c["source"], Hkv, -1, 2, CHUNK, c["D"]) if c["source"] else dst
    rows = torch.zeros(B, Hkv, dst.shape[2] * CHUNK, dtype=torch.bool, device=dev)
    rows[..., :L] = new
    rows = rows.view(B, Hkv, -1, 1, CHUNK, 1)
    dst.copy_(torch.where(rows, src[at], dst))
    lens = torch.where(takes, n, own_lens)
    if s["pos"] is not None:
        tables = ((s["pos"], s["pos2"] if c["source"] else s["pos"]), (s["acc"], s["acc2"] if c["source"] else s["acc"]))
        for t, u in tables:
            t.copy_(torch.where(new, u[at], t))
    return {"slabs": s["slabs"], "lens": lens, "pos": s["pos"], "acc": s["acc"]}


# ------------------------------------------------------------------ 64 bits

def exact(case, seed):
    op, B, Hkv, D, L = case["op"], case["B"], case["Hkv"], case["D"], case["L"]
    if op in ("commit", "fork"):
        return None  # copies: nothing in them is computed in floating point
    s = _inputs(case, seed)
    T, Hq = case["T"], case["Hq"]
    if op == "axes":
        R = case["rot"]
        f = THETA ** (-2 * torch.arange(R // 2, device="cuda", dtype=torch.float64) / R)
        pos = s["positions"].double()
        x = s["qkv"].double().view(B, T, Hq + 2 * Hkv, D)
        y = x.clone()
        for i, axis in enumerate(_axis(case)):
            first, second = (2 * i, 2 * i + 1) if case["inter"] else (i, i + R // 2)
            a = (pos[:, :, axis] * f[i])[:, :, None]
            h = slice(0, Hq + Hkv)
            y[:, :, h, first] = x[:, :, h, first] * a.cos() - x[:, :, h, second] * a.sin()
            y[:, :, h, second] = x[:, :, h, second] * a.cos() + x[:, :, h, first] * a.sin()
        k, v, sp = s["k"].double(), s["v"].double(), s["pos"].clone()
        acc = None if s["acc"] is None else s["acc"].double()
        for b in range(B):
            r = slice(int(s["slots"][b]), int(s["slots"][b]) + T)
            k[b, :, r] = y[b, :, Hq:Hq + Hkv].transpose(0, 1)
            v[b, :, r] = y[b, :, Hq + Hkv:].transpose(0, 1)
            sp[b, :, r] = s["positions"][b, :, 0]
            if acc is not None:
                acc[b, :, r] = 0.0
        return {"q": y[:, :, :Hq].contiguous(), "slabs": _to_slabs(k, v), "pos": sp, "acc": acc}
    G = Hq // Hkv
    o = torch.zeros(B, T, Hq, D, dtype=torch.float64, device="cuda")
    words = s["mask"].cpu().tolist()
    for b, (n, m) in enumerate(zip(_lens(case), _n_new(case))):
        k, v = s["k"][b, :, :n + m].double(), s["v"][b, :, :n + m].double()
        sees = torch.ones(m, n + m, dtype=torch.bool)
        for t in range(m):
            sees[t, n:] = torch.tensor([words[b][t][j // 64] >> j % 64 & 1 for j in range(m)], dtype=torch.bool)
        sees = sees.cuda()
        q = s["q"][b, :m].double().view(m, Hkv, G, D)
        x = torch.einsum("thgd,hld->hgtl", q, k) / math.sqrt(D)
        p = torch.softmax(x.masked_fill(~sees, -math.inf), -1)
        p = torch.where(sees.any(-1)[:, None], p, torch.zeros_like(p))
        o[b, :m] = torch.einsum("hgtl,hld->thgd", p, v).reshape(m, Hq, D)
    return o

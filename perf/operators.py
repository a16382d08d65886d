"""What a serving program does with a placed KV cache, as timed cases: rotate and append new
tokens, attend with a shared prefix, attend while accumulating each position's weight, and
evict by that weight.

`run` computes each operator in its plain form (elementary torch operations in 32 bits, angles
in 64) or, where `own` is true, with the package's entry points; both take what `prepare`
makes. A cache is returned as its slabs lie in memory: [slabs][chunks of 64 tokens][K, V][64][D],
where the 8-element piece c of token t's row is stored at piece c ^ (t % 8).
"""
import math

import torch

own = False

CHUNK = 64


def listed():
    return [
        # ---- attention over a shared prefix and each request's own cache
        # a few chats that have just begun behind a short system prompt: latency
        dict(name="prefix_few", op="prefix", B=4, Hq=32, Hkv=8, D=128, Lp="257", L=64, lo=0, hi=40, none=0,
             fp32=False),
        # 32 requests of the 8B-shaped layer behind one 8K prompt
        dict(name="prefix_batch", op="prefix", B=32, Hq=32, Hkv=8, D=128, Lp="8192", L=1024, lo=1, hi=1024, none=0,
             fp32=False),
        # a wide batch of the 70B-shaped layer behind three prompts of uneven length, some requests without one
        dict(name="prefix_wide", op="prefix", B=128, Hq=64, Hkv=8, D=128, Lp="16384/9001/130", L=256, lo=0, hi=256,
             none=9, fp32=False),
        # ---- attention that accumulates each position's weight
        # one request of the 8B shape over 4K context, one token: latency
        dict(name="acc_one", op="acc", B=1, Hq=32, Hkv=8, D=128, L=4096, lo=4001, hi=4001, fp32=False),
        # 32 requests over an 8K cache
        dict(name="acc_batch", op="acc", B=32, Hq=32, Hkv=8, D=128, L=8192, lo=7000, hi=8192, fp32=False),
        # 64-wide heads without sharing, ragged from empty on, the parity mode's fp32 output
        dict(name="acc_mha_fp32", op="acc", B=12, Hq=16, Hkv=16, D=64, L=2500, lo=0, hi=2500, fp32=True),
        # ---- eviction
        # every step a few tokens over the budget, slots in no order of position after earlier evictions: latency
        dict(name="evict_step", op="evict", B=16, Hkv=8, D=128, L=4096, lo=2049, hi=2064, keep=2048, recent=256,
             mixed=True),
        # after 8K-token prompts half of each cache goes
        dict(name="evict_half", op="evict", B=16, Hkv=8, D=128, L=8192, lo=6000, hi=8192, keep=4096, recent=1024,
             mixed=False),
        # one request with a very long context
        dict(name="evict_long", op="evict", B=1, Hkv=8, D=128, L=131072, lo=131001, hi=131001, keep=65536,
             recent=4096, mixed=False),
        # ---- rotation and append
        # one request, one token, the 8B shape: latency
        dict(name="rope_one", op="rope", B=1, T=1, Hq=32, Hkv=8, D=128, rot=128, inter=False, scaling="none", L=4096,
             far=100000, fp32=False),
        # a wide batch's step from the projection's fp32 output, half of each head rotated in adjacent pairs
        dict(name="rope_step", op="rope", B=256, T=1, Hq=32, Hkv=8, D=128, rot=64, inter=True, scaling="linear",
             L=130, far=30000, fp32=True),
        # ragged prompt chunks far into a context scaled by parts
        dict(name="rope_prompt", op="rope", B=4, T=2048, Hq=32, Hkv=8, D=128, rot=128, inter=False, scaling="by_parts",
             L=4096, far=500000, fp32=False),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["prefix", "acc", "evict", "rope"])
    D = rng.choice([64, 128, 128])
    Hkv = rng.choice([1, 2, 4, 8, 8])
    G = rng.choice([1, 2, 4, 4, 5, 8])
    if op == "prefix":
        B = _log_int(rng, 1, 128)
        P = rng.choice([1, 1, 2, 3])
        L = _log_int(rng, 1, 1024 if B <= 32 else 256)
        Lp = "/".join(str(_log_int(rng, 1, min(16384, 900000 // B) // P)) for _ in range(P))
        return dict(op=op, B=B, Hq=Hkv * G, Hkv=Hkv, D=D, Lp=Lp, L=L, lo=rng.randint(0, L), hi=L,
                    none=rng.choice([0, 0, 5]), fp32=rng.random() < 0.25)
    if op == "acc":
        B = _log_int(rng, 1, 32)
        L = _log_int(rng, 1, 7000)
        return dict(op=op, B=B, Hq=Hkv * G, Hkv=Hkv, D=D, L=L, lo=rng.randint(0, L), hi=L, fp32=rng.random() < 0.25)
    if op == "evict":
        B = _log_int(rng, 1, 16)
        L = _log_int(rng, 16, 131072 // B)
        keep = rng.randint(1, L - 1)
        return dict(op=op, B=B, Hkv=Hkv, D=D, L=L, lo=rng.randint(min(L, keep + 1), L), hi=L, keep=keep,
                    recent=rng.randint(0, keep), mixed=rng.random() < 0.5)
    T = _log_int(rng, 1, 2048)
    B = _log_int(rng, 1, max(1, min(256, 262144 // (T * Hkv * max(G, 4)))))
    return dict(op=op, B=B, T=T, Hq=Hkv * G, Hkv=Hkv, D=D, rot=rng.choice([D, D, D // 2, D - 8, 2]),
                inter=rng.random() < 0.5, scaling=rng.choice(["none", "linear", "ntk", "by_parts"]),
                L=T + rng.randint(0, 200), far=_log_int(rng, T, 1000000), fp32=rng.random() < 0.3)


# ------------------------------------------------------------------ what a case fixes besides its numbers

def _lens(case):
    """Ragged lengths of a case, spread over lo..hi out of order (the last request's is hi)."""
    B, lo, hi = case["B"], case["lo"], case["hi"]
    return [hi if b == B - 1 else lo + (hi - lo) * ((b * 37 + 11) % B) // B for b in range(B)]


def _prefix_lens(case):
    return [int(x) for x in case["Lp"].split("/")]


def _prefix_of(case):
    """Prefix of each request: round the prefixes; every `none`-th request has none (-1)."""
    P = len(_prefix_lens(case))
    return [-1 if case["none"] and b % case["none"] == case["none"] - 1 else b % P for b in range(case["B"])]


def _n_new(case):
    """New tokens of each request: all T, except that later requests of a prompt chunk end early."""
    return [case["T"] - (b * case["T"]) // (4 * case["B"]) for b in range(case["B"])]


THETA = 500000.0
FACTOR, ORIG_LEN, LOW_TURNS, HIGH_TURNS = 8.0, 8192.0, 1.0, 32.0


def work(case):
    op, B, D = case["op"], case["B"], case["D"]
    if op == "rope":
        n = sum(_n_new(case))
        size = 4 if case["fp32"] else 2
        row = (case["Hq"] + 2 * case["Hkv"]) * D
        return {"bytes": n * row * (size + 2) + 4 * n * case["Hkv"],
                "flops": 3 * n * (case["Hq"] + case["Hkv"]) * case["rot"]}
    Hkv, lens = case["Hkv"], _lens(case)
    if op == "evict":
        total = 0.0
        for n in lens:
            if n <= case["keep"]:
                continue
            recent, keep = min(case["recent"], n), case["keep"]
            share = (keep - recent) / max(1, n - recent)
            if case["mixed"]:
                moved = (n - keep) * keep / n
            else:
                tail_recent = min(recent, n - keep)
                moved = tail_recent + share * (n - keep - tail_recent)
            total += Hkv * (moved * 4 * D * 2 + n * 16 + keep * 4)
        return {"bytes": int(total), "flops": 0}
    Hq = case["Hq"]
    nbytes = B * Hq * D * (2 + (4 if case["fp32"] else 2)) + sum(lens) * Hkv * D * 4
    flops = 4 * sum(lens) * Hq * D
    if op == "acc":
        return {"bytes": nbytes + sum(lens) * Hkv * 8, "flops": flops}
    plens, of = _prefix_lens(case), _prefix_of(case)
    for g, n in enumerate(plens):
        members = of.count(g)
        if members:
            nbytes += n * Hkv * D * 4
            flops += 4 * n * members * Hq * D
    return {"bytes": nbytes, "flops": flops}


# ------------------------------------------------------------------ the rotation's frequencies

def _inv_freq(case):
    """Inverse frequencies (radians per position, 64 bits) and the factor on cos and sin."""
    R = case["rot"]
    i = torch.arange(0, R, 2, dtype=torch.float64)
    inv = THETA ** (-i / R)
    if case["scaling"] == "linear":
        return inv / FACTOR, 1.0
    if case["scaling"] == "ntk":
        base = THETA * FACTOR ** (R / (R - 2)) if R > 2 else THETA
        return base ** (-i / R), 1.0
    if case["scaling"] == "by_parts":
        turns = ORIG_LEN * inv / (2 * math.pi)
        ramp = ((turns - LOW_TURNS) / (HIGH_TURNS - LOW_TURNS)).clamp(0, 1)
        return inv / FACTOR * (1 - ramp) + inv * ramp, 0.1 * math.log(FACTOR) + 1
    return inv, 1.0


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

def _inputs(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def normal(*shape, dtype=torch.bfloat16):
        return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32).to(dtype)

    def ints(x):
        return torch.tensor(x, dtype=torch.int32, device="cuda")

    op, B, Hkv, D = case["op"], case["B"], case["Hkv"], case["D"]
    s = {"case": case}
    if op == "rope":
        T, L = case["T"], case["L"]
        H = case["Hq"] + 2 * Hkv
        # the projection's output: query, key and value rows of each token side by side
        s["qkv"] = normal(B, T, H * D, dtype=torch.float32 if case["fp32"] else torch.bfloat16)
        s["n_new"] = ints(_n_new(case))
        s["slots"] = (torch.rand(B, generator=g, device="cuda") * (L - T + 1)).int()
        s["positions"] = (torch.rand(B, generator=g, device="cuda") * (case["far"] - T + 1)).int()
        s["k"], s["v"] = normal(B, Hkv, L, D), normal(B, Hkv, L, D)
        s["slot_pos"] = torch.full((B, Hkv, L), -1, dtype=torch.int32, device="cuda")
        s["q_out"] = torch.zeros(B, T, case["Hq"], D, dtype=torch.bfloat16, device="cuda")
        return s
    L = case["L"]
    s["lens"] = ints(_lens(case))
    s["k"], s["v"] = normal(B, Hkv, L, D), normal(B, Hkv, L, D)
    if op == "evict":
        # accumulated weights spread over orders of magnitude; some tokens were never attended
        acc = torch.exp(2.0 * normal(B, Hkv, L, dtype=torch.float32))
        s["acc"] = torch.where(torch.rand(B, Hkv, L, generator=g, device="cuda") < 0.03, torch.zeros_like(acc), acc)
        if case["mixed"]:
            # earlier evictions left the slots below each length in any order of position, with gaps
            r = torch.rand(B, Hkv, L, generator=g, device="cuda")
            beyond = torch.arange(L, device="cuda") >= s["lens"][:, None, None]
            order = r.masked_fill(beyond, 2.0).argsort(-1).argsort(-1)
            s["slot_pos"] = (order * 3 // 2 + (order >= L // 2).int()).int()
        else:
            s["slot_pos"] = torch.arange(L, dtype=torch.int32, device="cuda").expand(B, Hkv, L).contiguous()
        s["acc_out"] = torch.zeros_like(s["acc"])
        s["pos_out"] = torch.full_like(s["slot_pos"], -1)
        return s
    s["q"] = normal(B, case["Hq"], D)
    if op == "acc":
        s["acc"] = torch.rand(B, Hkv, L, generator=g, device="cuda") * 2.0
        s["acc_out"] = torch.zeros_like(s["acc"])
        return s
    plens = _prefix_lens(case)
    s["plens"], s["of"] = ints(plens), ints(_prefix_of(case))
    s["pk"], s["pv"] = normal(len(plens), Hkv, max(plens), D), normal(len(plens), Hkv, max(plens), D)
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    op, D = case["op"], case["D"]
    if op in ("rope", "evict") and not own:
        s["slabs"] = _to_slabs(s.pop("k"), s.pop("v"))
    if op == "rope":
        s["inv_freq"], s["factor"] = _inv_freq(case)
        s["inv_freq"] = s["inv_freq"].cuda()
    if own:
        import direct_host_memory_gb300 as dak
        s["kv"] = dak.dak_place_kv_heads(s.pop("k"), s.pop("v"), 0)
        if op == "prefix":
            s["pkv"] = dak.dak_place_kv_heads(s.pop("pk"), s.pop("pv"), 0)
        if op == "rope":
            s["rope"] = dak.dak_rope_make(D, rot_dim=case["rot"], theta=THETA, interleaved=case["inter"],
                                          scaling=case["scaling"], factor=FACTOR, orig_len=ORIG_LEN,
                                          low_turns=LOW_TURNS, high_turns=HIGH_TURNS, attn_scale=s["factor"])
            B, T, Hq, Hkv = case["B"], case["T"], case["Hq"], case["Hkv"]
            x = s["qkv"].view(B, T, Hq + 2 * Hkv, D)
            s["q"], s["kn"], s["vn"] = x[:, :, :Hq], x[:, :, Hq:Hq + Hkv], x[:, :, Hq + Hkv:]
        if op in ("rope", "evict"):
            s["slabs"] = s["kv"].slabs()[1]
    return s


# ------------------------------------------------------------------ the operators

def run(state):
    return {"prefix": _prefix, "acc": _acc, "evict": _evict, "rope": _rope}[state["case"]["op"]](state)


def _softmax(s):
    """Softmax over the last axis; a row of minus infinities gives zeros."""
    m = s.amax(-1, keepdim=True)
    e = torch.exp(s - torch.where(m == -math.inf, torch.zeros_like(m), m))
    z = e.sum(-1, keepdim=True)
    return torch.where(z > 0, e / z, torch.zeros_like(e))


def _prefix(s):
    """o[b] = softmax(q[b] . [K_prefix(b), K_own(b)] / sqrt(D)) [V_prefix(b), V_own(b)]."""
    c = s["case"]
    if own:
        import direct_host_memory_gb300 as dak
        return dak.dak_attn_prefix(s["q"], s["kv"], s["pkv"], prefix_of=s["of"], prefix_lens=s["plens"],
                                   seq_lens=s["lens"], o_fp32=c["fp32"])
    B, Hq, Hkv, D, L = c["B"], c["Hq"], c["Hkv"], c["D"], c["L"]
    P, Lp, G = s["pk"].shape[0], s["pk"].shape[2], c["Hq"] // c["Hkv"]
    dev = s["q"].device
    q = s["q"].float().view(B, Hkv, G, D) / math.sqrt(D)
    own_s = q @ s["k"].float().transpose(-1, -2)  # [B][Hkv][G][L]
    own_s = own_s.masked_fill(torch.arange(L, device=dev) >= s["lens"].view(B, 1, 1, 1), -math.inf)
    # the products with every prefix, [P][Hkv][B*G][Lp], of which each request takes its own's
    rows = q.permute(1, 0, 2, 3).reshape(1, Hkv, B * G, D)
    all_s = (rows @ s["pk"].float().transpose(-1, -2)).view(P, Hkv, B, G, Lp)
    of = s["of"].long()
    at, b = of.clamp_min(0), torch.arange(B, device=dev)
    pre_s = all_s[at, :, b]  # [B][Hkv][G][Lp]
    hidden = (torch.arange(Lp, device=dev) >= s["plens"].long()[at][:, None]) | (of < 0)[:, None]
    pre_s = pre_s.masked_fill(hidden.view(B, 1, 1, Lp), -math.inf)
    p = _softmax(torch.cat([pre_s, own_s], -1))
    placed = torch.zeros_like(all_s)
    placed[at, :, b] = p[..., :Lp]
    o = (placed.view(P, Hkv, B * G, Lp) @ s["pv"].float()).sum(0).view(Hkv, B, G, D).permute(1, 0, 2, 3)
    o = (o + p[..., Lp:] @ s["v"].float()).reshape(B, Hq, D)
    return o if c["fp32"] else o.to(torch.bfloat16)


def _acc(s):
    """Single-query attention, and acc + the probabilities summed over the query heads of a kv head."""
    c = s["case"]
    if own:
        import direct_host_memory_gb300 as dak
        o, acc = dak.dak_attn_acc(s["q"], s["kv"], acc_in=s["acc"], acc_out=s["acc_out"], seq_lens=s["lens"],
                                  o_fp32=c["fp32"])
        return {"o": o, "acc": acc}
    B, Hq, Hkv, D, L = c["B"], c["Hq"], c["Hkv"], c["D"], c["L"]
    q = s["q"].float().view(B, Hkv, Hq // Hkv, D) / math.sqrt(D)
    beyond = torch.arange(L, device=q.device) >= s["lens"].view(B, 1, 1, 1)
    p = _softmax((q @ s["k"].float().transpose(-1, -2)).masked_fill(beyond, -math.inf))
    o = (p @ s["v"].float()).view(B, Hq, D)
    acc = torch.where(beyond[:, :, 0], s["acc_out"], s["acc"] + p.sum(2))
    return {"o": o if c["fp32"] else o.to(torch.bfloat16), "acc": acc}


def _evict(s):
    """Keep `keep` slots of each (request, kv head): the `recent` newest positions, then the
    largest weights, ties to the lower slot; kept rows from behind `keep` fill the holes
    before it, both in ascending order."""
    c = s["case"]
    keep, recent = c["keep"], c["recent"]
    if own:
        import direct_host_memory_gb300 as dak
        lens, src = dak.dak_kv_evict(s["kv"], s["lens"], keep, recent, s["acc"], s["slot_pos"],
                                     acc_out=s["acc_out"], slot_pos_out=s["pos_out"])
        return {"slabs": s["slabs"], "acc": s["acc_out"], "pos": s["pos_out"], "lens": lens, "src": src}
    B, Hkv, L, D = c["B"], c["Hkv"], c["L"], c["D"]
    acc, pos, slabs = s["acc"], s["slot_pos"], s["slabs"]
    dev = acc.device
    slot = torch.arange(L, device=dev)
    n = s["lens"].view(B, 1, 1)
    valid = (slot < n).expand(B, Hkv, L)
    newest = torch.where(valid, pos, torch.full_like(pos, -2**31)).amax(-1, keepdim=True)
    key = torch.where(valid & (pos.long() > newest.long() - recent), torch.full_like(acc, math.inf), acc)
    key = torch.where(valid, key, torch.full_like(acc, -math.inf))
    rank = torch.sort(key, dim=-1, descending=True, stable=True).indices.argsort(-1)
    kept = valid & ((rank < keep) | (n <= keep))
    hole, mover = valid & ~kept & (slot < keep), kept & (slot >= keep)
    # the r-th mover of each slab goes to its r-th hole
    hr, mr = hole.cumsum(-1) - 1, mover.cumsum(-1) - 1
    at = torch.where(mover, mr, torch.full_like(mr, L))
    table = torch.zeros(B, Hkv, L + 1, dtype=torch.int64, device=dev).scatter_(-1, at, slot.expand(B, Hkv, L))
    src = torch.where(hole, table.gather(-1, hr.clamp_min(0)), slot.expand(B, Hkv, L))
    inside = slot < n.clamp_max(keep)
    acc_out = torch.where(inside, acc.gather(-1, src), torch.where(valid, torch.zeros_like(acc), s["acc_out"]))
    pos_out = torch.where(inside, pos.gather(-1, src), torch.where(valid, torch.full_like(pos, -1), s["pos_out"]))
    # the moved rows, K and V, from their slots into the holes
    bh, to = hole.view(B * Hkv, L).nonzero(as_tuple=True)
    fr = src.view(B * Hkv, L)[bh, to]
    piece = torch.arange(D // 8, device=dev)
    rows = slabs.view(B * Hkv, -1, 2, CHUNK, D // 8, 8)
    moved = rows[bh[:, None], (fr // CHUNK)[:, None], :, (fr % CHUNK)[:, None], piece ^ (fr % 8)[:, None]]
    rows[bh[:, None], (to // CHUNK)[:, None], :, (to % CHUNK)[:, None], piece ^ (to % 8)[:, None]] = moved
    out_src = torch.where(inside, src, torch.full_like(src, -1))[..., :keep].int()
    return {"slabs": slabs, "acc": acc_out, "pos": pos_out, "lens": s["lens"].clamp_max(keep), "src": out_src}


def _rope(s):
    """Rotate each new token's query into q_out and its key into the cache row it is appended to, with its value."""
    c = s["case"]
    if own:
        import direct_host_memory_gb300 as dak
        dak.dak_kv_append_rope(s["kv"], s["rope"], s["q"], s["kn"], s["vn"], s["slots"], positions=s["positions"],
                               n_new=s["n_new"], q_out=s["q_out"], slot_pos=s["slot_pos"])
        return {"q": s["q_out"], "slabs": s["slabs"], "pos": s["slot_pos"]}
    B, T, Hq, Hkv, D, R = c["B"], c["T"], c["Hq"], c["Hkv"], c["D"], c["rot"]
    dev = s["qkv"].device
    x = s["qkv"].view(B, T, Hq + 2 * Hkv, D)
    t = torch.arange(T, device=dev)
    angle = (s["positions"].double()[:, None] + t)[..., None] * s["inv_freq"]  # [B][T][R/2]
    cos = (torch.cos(angle) * s["factor"]).float()[:, :, None]
    sin = (torch.sin(angle) * s["factor"]).float()[:, :, None]
    qk = x[:, :, :Hq + Hkv].float()
    if c["inter"]:
        a, b = qk[..., 0:R:2], qk[..., 1:R:2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = qk[..., :R // 2], qk[..., R // 2:R]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    qk = torch.cat([turned, qk[..., R:]], -1).to(torch.bfloat16)
    new = t < s["n_new"][:, None]  # [B][T]
    s["q_out"][new] = qk[:, :, :Hq][new]
    b, tok = new.nonzero(as_tuple=True)
    row = s["slots"].long()[b] + tok
    rows = s["slabs"].view(B, Hkv, -1, 2, CHUNK, D // 8, 8)
    piece = torch.arange(D // 8, device=dev)
    kv = torch.stack([qk[:, :, Hq:], x[:, :, Hq + Hkv:].to(torch.bfloat16)], 3)[b, tok]  # [new][Hkv][2][D]
    kv = kv.view(-1, Hkv, 2, D // 8, 8).permute(0, 3, 1, 2, 4)
    rows[b[:, None], :, (row // CHUNK)[:, None], :, (row % CHUNK)[:, None], piece ^ (row % 8)[:, None]] = kv
    s["slot_pos"][b, :, row] = (s["positions"][b] + tok.int())[:, None].expand(-1, Hkv)
    return {"q": s["q_out"], "slabs": s["slabs"], "pos": s["slot_pos"]}


# ------------------------------------------------------------------ 64 bits

def exact(case, seed):
    s = _inputs(case, seed)
    op, B, Hkv, D = case["op"], case["B"], case["Hkv"], case["D"]
    if op == "rope":
        T, Hq, R, L = case["T"], case["Hq"], case["rot"], case["L"]
        inv, factor = _inv_freq(case)
        pos = s["positions"].double()[:, None] + torch.arange(T, device="cuda", dtype=torch.float64)
        turn = torch.polar(torch.full((1,), factor, dtype=torch.float64, device="cuda"),
                           pos[:, :, None, None] * inv.cuda())  # [B][T][1][R/2]
        x = s["qkv"].double().view(B, T, Hq + 2 * Hkv, D)
        i = torch.arange(R // 2, device="cuda")
        first, second = (2 * i, 2 * i + 1) if case["inter"] else (i, i + R // 2)
        z = torch.complex(x[..., first], x[..., second]) * turn
        y = x.clone()
        y[..., first], y[..., second] = z.real, z.imag
        y[:, :, Hq + Hkv:] = x[:, :, Hq + Hkv:]
        q_out = torch.zeros(B, T, Hq, D, dtype=torch.float64, device="cuda")
        k, v, sp = s["k"].double(), s["v"].double(), s["slot_pos"].clone()
        for b, n in enumerate(_n_new(case)):
            r = int(s["slots"][b])
            q_out[b, :n] = y[b, :n, :Hq]
            k[b, :, r:r + n] = y[b, :n, Hq:Hq + Hkv].transpose(0, 1)
            v[b, :, r:r + n] = y[b, :n, Hq + Hkv:].transpose(0, 1)
            sp[b, :, r:r + n] = int(s["positions"][b]) + torch.arange(n, dtype=torch.int32, device="cuda")
        return {"q": q_out, "slabs": _to_slabs(k, v), "pos": sp}
    lens = _lens(case)
    L = case["L"]
    if op == "evict":
        return None  # choices and copies: nothing in it is computed in floating point
    Hq = case["Hq"]
    G = Hq // Hkv
    q = s["q"].double().view(B, Hkv, G, D) / math.sqrt(D)
    o = torch.zeros(B, Hkv, G, D, dtype=torch.float64, device="cuda")
    acc = s["acc_out"].double() if op == "acc" else None
    of = _prefix_of(case) if op == "prefix" else [-1] * B
    plens = _prefix_lens(case) if op == "prefix" else []
    for b, n in enumerate(lens):
        k, v = s["k"][b, :, :n].double(), s["v"][b, :, :n].double()
        if of[b] >= 0:
            m = plens[of[b]]
            k = torch.cat([s["pk"][of[b], :, :m].double(), k], 1)
            v = torch.cat([s["pv"][of[b], :, :m].double(), v], 1)
        if k.shape[1] == 0:
            continue
        p = torch.softmax(torch.einsum("hgd,hld->hgl", q[b], k), -1)
        o[b] = torch.einsum("hgl,hld->hgd", p, v)
        if acc is not None:
            acc[b, :, :n] = s["acc"][b, :, :n].double() + p.sum(1)
    o = o.view(B, Hq, D)
    return {"o": o, "acc": acc} if op == "acc" else o

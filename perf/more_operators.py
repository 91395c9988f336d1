"""What the operators for a tree of drafted tokens are measured on: new tokens rotated and written
into the latent cache, latent attention of a tree's nodes over the cache, the KDA recurrence along a
tree's branches, and the log probabilities that a server answers with.

`run` computes a case in its plain form (elementary torch operations) where `own` is false and
through the framework's entry points where it is true.

Case kinds
  rope    rotate the position parts of T new tokens' keys and queries, write the keys into a paged
          cache, and read the same tokens back
  attend  absorbed attention of the K nodes of a tree of drafts a sequence over the paged cache
  state   KDA outputs of the K nodes of a tree a sequence from a pool of states
  score   log probability, rank and entropy of given tokens, and the most likely ones
"""
import math
import random

import torch

own = False

DC, DR = 512, 64                 # latent and position part of a cached token
ROW = {"bf16": 1152, "e4m3": 656}
E4M3_MAX = 448.0


# ---- cases -----------------------------------------------------------------------------------

def listed():
    return [
        # the nodes of 64 sequences' trees entering the cache, far into their prompts
        {"name": "rope_tree_64", "kind": "rope", "cache": "e4m3", "page": 64, "n": 64, "lo": 12, "hi": 12, "h": 32,
         "before": 142000, "inter": False, "q": "absorbed", "lens_seed": 1},
        # a 32768-token chunk of a prompt; queries as the projection writes them
        {"name": "rope_prompt_32768", "kind": "rope", "cache": "bf16", "page": 64, "n": 1, "lo": 32768, "hi": 32768, "h": 32,
         "before": 32768, "inter": False, "q": "expanded", "lens_seed": 2},
        # ragged short prompts on a shard of the heads, neighbouring pairs, pages that no tile divides
        {"name": "rope_ragged", "kind": "rope", "cache": "e4m3", "page": 48, "n": 12, "lo": 1, "hi": 2000, "h": 4,
         "before": 0, "inter": True, "q": "alone", "lens_seed": 3},
        # a few short chats on a head shard: latency
        {"name": "attend_short", "kind": "attend", "cache": "bf16", "page": 16, "n": 3, "lo": 1, "hi": 200, "h": 4, "k": 12,
         "reach": 4, "lens_seed": 4},
        # a serving batch of mixed lengths, trees of up to eight nodes, over the quantised cache
        {"name": "attend_batch16", "kind": "attend", "cache": "e4m3", "page": 64, "n": 16, "lo": 1024, "hi": 65536, "h": 32,
         "k": 8, "reach": 4, "lens_seed": 5},
        # wide trees on a shard of the heads
        {"name": "attend_wide4", "kind": "attend", "cache": "bf16", "page": 48, "n": 4, "lo": 8192, "hi": 32768, "h": 8, "k": 64,
         "reach": 16, "lens_seed": 6},
        # one sequence's tree: latency
        {"name": "state_one", "kind": "state", "n": 1, "h": 32, "d": 128, "k": 8, "reach": 4, "decay": "channel", "out": "bf16",
         "lens_seed": 7},
        # a serving batch, trees of up to sixteen nodes
        {"name": "state_batch256", "kind": "state", "n": 256, "h": 32, "d": 128, "k": 16, "reach": 6, "decay": "channel",
         "out": "bf16", "lens_seed": 8},
        # the scalar-gate layout on a shard of the heads, wide trees
        {"name": "state_shard64", "kind": "state", "n": 64, "h": 8, "d": 64, "k": 48, "reach": 12, "decay": "head",
         "out": "f32", "lens_seed": 9},
        # the tokens of one sequence's step, with the alternatives that a user asks for
        {"name": "score_step", "kind": "score", "r": 4, "v": 131072, "type": "f32", "top": 20, "pad": 0, "scale": 1.0,
         "sharp": 2.0},
        # a serving batch over a vocabulary of odd size in padded rows; the next drafts are among the alternatives
        {"name": "score_batch256", "kind": "score", "r": 256, "v": 100003, "type": "bf16", "top": 8, "pad": 29, "scale": 0.7,
         "sharp": 2.5},
        # scoring a prompt
        {"name": "score_prompt2048", "kind": "score", "r": 2048, "v": 131072, "type": "bf16", "top": 1, "pad": 0, "scale": 1.0,
         "sharp": 2.5},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["rope", "attend", "attend", "state", "state", "score", "score"])
    cache = rng.choice(["bf16", "e4m3"])
    page = rng.choice([16, 32, 48, 64, 128])
    ls = rng.randrange(1 << 30)
    h = rng.choice([1, 2, 3, 4, 8, 16, 20, 32, 64])
    if kind == "rope":
        n = _log_int(rng, 1, 512)
        hi = _log_int(rng, 1, max(1, 32768 * 32 // (n * max(h, 32))))
        return {"kind": kind, "cache": cache, "page": page, "n": n, "lo": max(1, hi // 4), "hi": hi, "h": h,
                "before": rng.choice([0, rng.randrange(1000000)]), "inter": rng.random() < 0.5,
                "q": rng.choice(["alone", "expanded", "absorbed"]), "lens_seed": ls}
    if kind == "attend":
        k = _log_int(rng, 1, min(64, 512 // h))
        n = _log_int(rng, 1, 64)
        hi = _log_int(rng, 1, min(145408, max(1, 580000 // (n * max(1, k * h // 64)))))
        return {"kind": kind, "cache": cache, "page": page, "n": n, "lo": max(1, hi // 32), "hi": hi, "h": h, "k": k,
                "reach": rng.randrange(1, 17), "lens_seed": ls}
    if kind == "state":
        d, k = rng.choice([64, 128]), _log_int(rng, 1, 64)
        n = _log_int(rng, 1, min(512, 8192 // h, 131072 // (h * k)))
        return {"kind": kind, "n": n, "h": h, "d": d, "k": k, "reach": rng.randrange(1, 17),
                "decay": rng.choice(["channel", "channel", "head", "none"]), "out": rng.choice(["bf16", "f32"]), "lens_seed": ls}
    v = _log_int(rng, 1000, 160000)
    r = _log_int(rng, 1, min(2048, 120000000 // v))
    return {"kind": kind, "r": r, "v": v, "type": rng.choice(["bf16", "f32"]), "top": rng.choice([0, 1, 5, 20, 32]),
            "pad": rng.choice([0, 0, 1, 61]), "scale": round(rng.uniform(0.3, 2.0), 2), "sharp": round(rng.uniform(0.5, 4.0), 2)}


def _lens(case):
    r = random.Random(case["lens_seed"])
    return [min(case["hi"], max(case["lo"], _log_int(r, case["lo"], case["hi"]))) for _ in range(case["n"])]


def _parents(case):
    """A tree a sequence: node 0 is the last token, a later one hangs on one of the `reach` nodes before
    it; the places behind a sequence's last node (some have fewer than k) hold -2."""
    r = random.Random(case["lens_seed"] + 1)
    k, rows = case["k"], []
    for _ in range(case["n"]):
        m = r.randrange(max(1, k // 2), k + 1)
        rows.append([-1 if j == 0 else r.randrange(max(0, j - case["reach"]), j) if j < m else -2 for j in range(k)])
    return rows


# ---- inputs ----------------------------------------------------------------------------------

def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _quantise(c):
    """Codes and the scale a token of latents [T, DC]: s = 2^e with the smallest e that keeps the
    row's largest magnitude within the type's 448, rounded to nearest even."""
    x = c.float()
    amax = x.abs().amax(dim=-1)
    m, e = torch.frexp(amax / E4M3_MAX)                    # amax = 448 m 2^e, m in [1/2, 1)
    e = torch.where(m == 0.5, e - 1, e).clamp(-117, 119)
    s = ((torch.where(amax > 0, e, torch.zeros_like(e)) + 127) << 23).to(torch.int32).view(torch.float32)
    codes = (x / s[:, None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
    return codes, s


def _pack(c, r, cache):
    """Cache rows (bytes) of latents [T, DC] and position keys [T, DR]."""
    if cache == "bf16":
        return torch.cat([c, r], dim=1).view(torch.uint8)
    codes, s = _quantise(c)
    pad = torch.zeros(c.shape[0], ROW["e4m3"] - DC - 2 * DR - 4, dtype=torch.uint8, device=c.device)
    return torch.cat([codes.view(torch.uint8), r.contiguous().view(torch.uint8), s[:, None].view(torch.uint8), pad], dim=1)


def _unpack(rows, cache):
    """The values that cache rows [..., ROW] stand for: latents and position keys."""
    if cache == "bf16":
        x = rows.view(torch.bfloat16).float()
        return x[..., :DC], x[..., DC:]
    c = rows[..., :DC].view(torch.float8_e4m3fn).float()
    s = rows[..., DC + 2 * DR:DC + 2 * DR + 4].contiguous().view(torch.float32).float()
    return c * s, rows[..., DC:DC + 2 * DR].contiguous().view(torch.bfloat16).float()


def _pages(total_lens, page, g):
    """A block table over shuffled pages, and how many pages the cache has."""
    need = [-(-x // page) for x in total_lens]
    num = sum(need) + 3
    perm = torch.randperm(num, generator=g, device="cuda").to(torch.int32)
    table = torch.zeros(len(need), max(max(need), 1), dtype=torch.int32, device="cuda")
    at = 0
    for i, x in enumerate(need):
        table[i, :x] = perm[at:at + x]
        at += x
    return table, num


def _latents(g, T):
    """Normalised latents with a few loud channels, and position keys."""
    c = _randn(g, T, DC)
    c[:, 7::101] *= 6.0
    c = c * torch.rsqrt(c.square().mean(dim=-1, keepdim=True))
    return c.to(torch.bfloat16), _randn(g, T, DR).to(torch.bfloat16)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    kind = case["kind"]
    s = dict(case)
    if kind == "score":
        r, v = case["r"], case["v"]
        x = _randn(g, r, v + case["pad"]) * case["sharp"]
        x[:, :v].scatter_add_(1, torch.randint(0, v, (r, 4), generator=g, device="cuda"), 3.0 * case["sharp"] + _randn(g, r, 4))
        x = x.to(torch.bfloat16) if case["type"] == "bf16" else x
        s["x"] = x[:, :v]
        # the given tokens: mostly likely ones, as a sampler draws them, some at random
        best = s["x"].float().topk(8, dim=1).indices
        pick = best.gather(1, torch.randint(0, 8, (r, 1), generator=g, device="cuda"))[:, 0]
        other = torch.randint(0, v, (r,), generator=g, device="cuda")
        s["t"] = torch.where(torch.rand(r, generator=g, device="cuda") < 0.7, pick, other).to(torch.int32)
        return s
    if kind == "state":
        n, h, d, k = case["n"], case["h"], case["d"], case["k"]
        unit = lambda t: t / t.norm(dim=-1, keepdim=True)
        s["q"], s["k_"] = (unit(_randn(g, n, k, h, d)).to(torch.bfloat16) for _ in range(2))
        s["v"] = _randn(g, n, k, h, d).to(torch.bfloat16)
        s["beta"] = torch.sigmoid(_randn(g, n, k, h)).to(torch.bfloat16)
        shape = {"channel": (n, k, h, d), "head": (n, k, h), "none": None}[case["decay"]]
        s["la"] = None if shape is None else -torch.nn.functional.softplus(_randn(g, *shape) - 2.0)
        s["pool"] = _randn(g, n + 3, h, d, d) * 0.05
        s["slots"] = torch.randperm(n + 3, generator=g, device="cuda")[:n].to(torch.int32)
        s["parents"] = torch.tensor(_parents(case), dtype=torch.int32).cuda()
        return s
    lens, page, cache, n, h = _lens(case), case["page"], case["cache"], case["n"], case["h"]
    if kind == "rope":
        s["table"], num = _pages(lens, page, g)
        T = sum(lens)
        c, r = _latents(g, T)
        both = torch.cat([c, r], dim=1)              # slices of one projection's output rows
        s["c"], s["r"] = both[:, :DC], both[:, DC:]
        cu = torch.tensor([0] + lens, dtype=torch.int64).cumsum(0).to(torch.int32)
        s["cu_host"], s["cu"] = cu, cu.cuda()
        seq = torch.repeat_interleave(torch.arange(n, device="cuda"), torch.tensor(lens, device="cuda"))
        at = torch.arange(T, device="cuda") - s["cu"].long()[seq]
        s["slots"] = (s["table"].long()[seq, at // page] * page + at % page).to(torch.int32)
        s["pos"] = (at + case["before"]).to(torch.int32)
        s["freq"] = (10000.0 ** (-torch.arange(0, DR, 2, dtype=torch.float64) / DR)).float().cuda()
        width = {"alone": DR, "expanded": 192, "absorbed": DC + DR}[case["q"]]
        s["q"] = _randn(g, T, h, width if case["q"] == "expanded" else DR).to(torch.bfloat16)[..., -DR:]
        # where the absorbed query's position part goes: the rows that the attention reads
        s["q_out"] = torch.zeros(T, h, width, dtype=torch.bfloat16, device="cuda")[..., -DR:] if case["q"] != "alone" else None
        s["pages"] = torch.zeros(num, page, ROW[cache], dtype=torch.uint8, device="cuda")
        return s
    k = case["k"]
    total = [x + k for x in lens]
    s["table"], num = _pages(total, page, g)
    c, r = _latents(g, num * page)
    s["pages"] = _pack(c, r, cache).view(num, page, ROW[cache])
    s["lens"] = torch.tensor(total, dtype=torch.int32, device="cuda")
    s["q"] = _randn(g, n, k, h, DC + DR).to(torch.bfloat16)
    s["parents"] = torch.tensor(_parents(case), dtype=torch.int32).cuda()
    s["scale"] = (128 + DR) ** -0.5
    return s


# ---- plain forms -----------------------------------------------------------------------------

def _rotate(x, cos, sin, inter):
    """x [..., DR] in pairs of neighbours, or of the two halves."""
    x = x.float()
    a, b = (x[..., 0::2], x[..., 1::2]) if inter else (x[..., :DR // 2], x[..., DR // 2:])
    a, b = a * cos - b * sin, a * sin + b * cos
    return (torch.stack([a, b], dim=-1).flatten(-2) if inter else torch.cat([a, b], dim=-1)).to(torch.bfloat16)


def _plain_rope(s):
    angle = s["pos"].double()[:, None] * s["freq"].double()
    cos, sin = torch.cos(angle).float(), torch.sin(angle).float()
    r = _rotate(s["r"], cos, sin, s["inter"])
    q = _rotate(s["q"], cos[:, None], sin[:, None], s["inter"])
    flat = s["pages"].view(-1, ROW[s["cache"]])
    flat[s["slots"].long()] = _pack(s["c"].contiguous(), r, s["cache"])
    if s["q_out"] is not None:
        s["q_out"].copy_(q)
        q = s["q_out"]
    c, r = _unpack(flat[s["slots"].long()], s["cache"])
    return [c.to(torch.bfloat16), r.to(torch.bfloat16), q]


def _lineage(parents):
    """[N, K, K]: node j has i among its ancestors or is it; a place that holds no node has none."""
    n, k = parents.shape
    up = torch.zeros(n, k, k, dtype=torch.bool, device=parents.device)
    b = torch.arange(n, device=parents.device)
    for j in range(k):
        p = parents[:, j].long()
        up[:, j] = up[b, p.clamp_min(0)] & (p >= 0)[:, None]
        up[:, j, j] = p >= -1
    return up


def _plain_attend(s):
    n, k, h, page = s["n"], s["k"], s["h"], s["page"]
    ctx = s["lens"].long() - k
    t = torch.arange(s["hi"] + k, device="cuda")
    at = torch.clamp_max(t // page, s["table"].shape[1] - 1)
    rows = s["table"].long()[:, at] * page + t % page
    c, r = _unpack(s["pages"].view(-1, ROW[s["cache"]])[rows], s["cache"])
    q = s["q"].float().view(n, k * h, DC + DR)
    x = (torch.matmul(q[..., :DC], c.transpose(1, 2)) + torch.matmul(q[..., DC:], r.transpose(1, 2))) * s["scale"]
    up = _lineage(s["parents"])
    sees = (t < ctx[:, None])[:, None] & up.any(dim=2)[..., None]
    sees = sees.scatter(2, (ctx[:, None] + torch.arange(k, device="cuda"))[:, None].expand(-1, k, -1), up)
    x = x.view(n, k, h, -1).masked_fill_(~sees[:, :, None], -math.inf).view(n, k * h, -1)
    m = x.amax(dim=-1, keepdim=True)
    p = torch.exp(x - torch.where(torch.isinf(m), torch.zeros_like(m), m))
    l = p.sum(dim=-1, keepdim=True)
    o = torch.matmul(p, c) / torch.where(l > 0, l, torch.ones_like(l))
    lse = (m + torch.log(l))[..., 0]
    return [o.view(n, k, h, DC).to(torch.bfloat16), lse.view(n, k, h)]


def _plain_state(s):
    n, k, h, d = s["n"], s["k"], s["h"], s["d"]
    b = torch.arange(n, device="cuda")
    after = torch.empty(k + 1, n, h, d, d, device="cuda")             # the state before the tree, then after each node
    after[0] = s["pool"][s["slots"].long()]
    out = torch.zeros(n, k, h, d, device="cuda")
    alpha = None if s["la"] is None else torch.exp(s["la"])
    for j in range(k):
        p = s["parents"][:, j].long()
        S = after[(p + 1).clamp_min(0), b]
        key, beta = s["k_"][:, j].float(), s["beta"][:, j].float()[..., None]
        if alpha is not None:
            S = S * (alpha[:, j][..., None] if alpha.dim() == 4 else alpha[:, j][..., None, None])
        u = beta * (s["v"][:, j].float() - (S * key[..., None]).sum(dim=2))
        S = S + key[..., None] * u[:, :, None]
        after[j + 1] = S
        o = (S * s["q"][:, j].float()[..., None]).sum(dim=2)
        out[:, j] = torch.where((p >= -1)[:, None, None], o, torch.zeros_like(o))
    return [out.to(torch.bfloat16) if s["out"] == "bf16" else out]


def _plain_score(s):
    raw, t = s["x"].float(), s["t"].long()
    x = raw * s["scale"]
    m = x.amax(dim=1, keepdim=True)
    e = torch.exp(x - m)
    l = e.sum(dim=1, keepdim=True)
    lse = m + torch.log(l)
    xt = raw.gather(1, t[:, None])
    before = torch.arange(raw.shape[1], device="cuda") < t[:, None]
    rank = 1 + ((raw > xt) | ((raw == xt) & before)).sum(dim=1)
    entropy = torch.log(l[:, 0]) - (e * (x - m)).sum(dim=1) / l[:, 0]
    outs = [(xt * s["scale"] - lse)[:, 0], rank.to(torch.int32), entropy]
    if s["top"]:
        v, i = torch.sort(raw, dim=1, descending=True, stable=True)
        outs += [v[:, :s["top"]] * s["scale"] - lse, i[:, :s["top"]].to(torch.int32)]
    return outs


# ---- the framework's calls -------------------------------------------------------------------

def _own(s):
    from kimi_delta_attention_06_gb300 import kda

    kind = s["kind"]
    if kind == "score":
        lp, rank, entropy, top_lp, top_t = kda.token_logprobs(s["x"], s["t"], top=s["top"], scale=s["scale"])
        return [lp, rank, entropy] + ([top_lp, top_t] if s["top"] else [])
    if kind == "state":
        decay = {"channel": kda.KDA_DECAY_CHANNEL, "head": kda.KDA_DECAY_HEAD, "none": kda.KDA_DECAY_NONE}[s["decay"]]
        out = torch.bfloat16 if s["out"] == "bf16" else torch.float32
        return [kda.decode_tree(s["q"], s["k_"], s["v"], s["la"], s["beta"], s["pool"], s["parents"], state_slots=s["slots"],
                                out_dtype=out, decay=decay)]
    dtype = kda.KDA_CACHE_BF16 if s["cache"] == "bf16" else kda.KDA_CACHE_E4M3
    if kind == "attend":
        return list(kda.latent_decode_tree(s["q"], s["pages"], dtype, s["table"], s["lens"], s["parents"], s["scale"],
                                           want_lse=True))
    q = kda.latent_append_rope(s["c"], s["r"], s["pages"], dtype, s["slots"], s["pos"], s["freq"], q=s["q"], q_out=s["q_out"],
                               interleaved=s["inter"])
    return list(kda.latent_gather(s["pages"], dtype, s["table"], s["cu_host"], cu_seqlens=s["cu"])) + [q]


def run(state):
    if own:
        return _own(state)
    return {"rope": _plain_rope, "attend": _plain_attend, "state": _plain_state, "score": _plain_score}[state["kind"]](state)


def work(case):
    kind = case["kind"]
    if kind == "score":
        r, v, size = case["r"], case["v"], 2 if case["type"] == "bf16" else 4
        return {"bytes": r * (v * size + 16 + 8 * case["top"]), "flops": 5 * r * v}
    if kind == "rope":
        T, h, row = sum(_lens(case)), case["h"], ROW[case["cache"]]
        return {"bytes": T * (2 * ROW["bf16"] + row + 8 + 4 * h * DR), "flops": 3 * T * (h + 1) * DR}
    rows = _parents(case)
    nodes, h, k = sum(p >= -1 for row in rows for p in row), case["h"], case["k"]
    if kind == "state":
        d = case["d"]
        decay = {"channel": 4 * d, "head": 4, "none": 0}[case["decay"]]
        return {"bytes": case["n"] * (4 * h * d * d + 4 * k + 4) + nodes * h * (6 * d + decay + 2) +
                case["n"] * k * h * d * (2 if case["out"] == "bf16" else 4), "flops": 4 * nodes * h * d * d}
    lens = _lens(case)
    pairs = 0
    for x, row in zip(lens, rows):
        depth = {-1: 0}
        for j, p in enumerate(row):
            if p >= -1:
                depth[j] = depth[p] + 1
                pairs += x + depth[j]
    T = sum(lens) + case["n"] * k
    return {"bytes": T * ROW[case["cache"]] + nodes * h * 2 * (DC + DR) + case["n"] * k * (h * (2 * DC + 4) + 4),
            "flops": 2 * pairs * h * (2 * DC + DR)}


# ---- in 64 bits, from the definitions --------------------------------------------------------

def _exact_codes(c):
    """The values e4m3 rows hold, by searching each latent's nearest code among all codes."""
    c = c.double()
    codes = torch.tensor(sorted({m / 8 * 2.0 ** -6 for m in range(8)} |
                                {(1 + m / 8) * 2.0 ** e for e in range(-6, 9) for m in range(8)
                                 if (1 + m / 8) * 2.0 ** e <= E4M3_MAX}), dtype=torch.float64, device=c.device)
    amax = c.abs().amax(dim=1, keepdim=True)
    powers = torch.tensor([2.0 ** e for e in range(-117, 120)], dtype=torch.float64, device=c.device)
    least = torch.searchsorted(E4M3_MAX * powers, amax).clamp_max(len(powers) - 1)
    s = torch.where(amax > 0, powers[least], torch.ones_like(amax))
    x = (c.abs() / s).clamp_max(E4M3_MAX)
    hi = torch.searchsorted(codes, x.contiguous()).clamp_max(len(codes) - 1)
    lo = (hi - 1).clamp_min(0)
    up, down = codes[hi] - x, x - codes[lo]
    take_lo = (down < up) | ((down == up) & (lo % 2 == 0))
    return torch.sign(c) * torch.where(take_lo, codes[lo], codes[hi]) * s


def _exact_read(rows, cache):
    """The values of cache rows [T, ROW], each code by the type's own definition."""
    if cache == "bf16":
        x = rows.view(torch.bfloat16).double()
        return x[:, :DC], x[:, DC:]
    b = torch.arange(256, dtype=torch.float64, device=rows.device)
    e, m = torch.floor(b / 8) % 16, b % 8
    powers = torch.tensor([2.0 ** (max(i, 1) - 7) for i in range(16)], dtype=torch.float64, device=rows.device)
    mag = ((e > 0) + m / 8) * powers[e.long()]
    value = torch.where(b >= 128, -mag, mag)
    value[[127, 255]] = math.nan
    s = rows[:, DC + 2 * DR:DC + 2 * DR + 4].contiguous().view(torch.float32).double()
    return value[rows[:, :DC].long()] * s, rows[:, DC:DC + 2 * DR].contiguous().view(torch.bfloat16).double()


def _exact_rope(s):
    turn = torch.polar(torch.ones((), dtype=torch.float64, device="cuda"), s["pos"].double()[:, None] * s["freq"].double())

    def spin(x, w):
        x = x.double()
        x = x.unflatten(-1, (DR // 2, 2)) if s["inter"] else x.unflatten(-1, (2, DR // 2)).transpose(-1, -2)
        y = torch.view_as_real(torch.view_as_complex(x.contiguous()) * w)
        return (y if s["inter"] else y.transpose(-1, -2)).flatten(-2)

    c = s["c"].double() if s["cache"] == "bf16" else _exact_codes(s["c"])
    return [c, spin(s["r"], turn), spin(s["q"], turn[:, None])]


def _path(row, j):
    """The places from the root to place j, or nothing where it holds no node."""
    path = []
    while j >= 0:
        if row[j] < -1:
            return []
        path.append(j)
        j = row[j]
    return path[::-1]


def _exact_attend(s):
    n, k, h = s["n"], s["k"], s["h"]
    flat = s["pages"].view(-1, ROW[s["cache"]])
    o = torch.zeros(n, k, h, DC, dtype=torch.float64, device="cuda")
    lse = torch.full((n, k, h), -math.inf, dtype=torch.float64, device="cuda")
    trees = s["parents"].tolist()
    for i in range(n):
        L = int(s["lens"][i])
        t = torch.arange(L, device="cuda")
        c, r = _exact_read(flat[s["table"][i].long()[t // s["page"]] * s["page"] + t % s["page"]], s["cache"])
        key = torch.cat([c, r], dim=1)
        shared = s["q"][i].double() @ key[:L - k].T * s["scale"]               # [k, h, context]
        for j in range(k):
            path = _path(trees[i], j)
            if path:
                mine = torch.tensor(path, device="cuda") + L - k
                x = torch.cat([shared[j], s["q"][i, j].double() @ key[mine].T * s["scale"]], dim=1)
                p = torch.softmax(x, dim=1)
                o[i, j] = p[:, :L - k] @ c[:L - k] + p[:, L - k:] @ c[mine]
                lse[i, j] = torch.logsumexp(x, dim=1)
    return [o, lse]


def _exact_state(s):
    n, k, h, d = s["n"], s["k"], s["h"], s["d"]
    out = torch.zeros(n, k, h, d, dtype=torch.float64, device="cuda")
    eye = torch.eye(d, dtype=torch.float64, device="cuda")
    trees = s["parents"].tolist()
    for i in range(n):
        start = s["pool"][int(s["slots"][i])].double()
        after = {}
        for j in range(k):
            if trees[i][j] < -1:
                continue
            before = start if trees[i][j] == -1 else after[trees[i][j]]
            key = s["k_"][i, j].double()[..., None]                            # [h, d, 1]
            beta = s["beta"][i, j].double()[:, None, None]
            la = torch.zeros(h, 1, dtype=torch.float64, device="cuda") if s["la"] is None else s["la"][i, j].double().view(h, -1)
            step = (eye - beta * key @ key.transpose(1, 2)) * torch.exp(la)[:, None]   # (I - beta k k^T) Diag(alpha)
            after[j] = step @ before + beta * key @ s["v"][i, j].double()[:, None]
            out[i, j] = (s["q"][i, j].double()[:, None] @ after[j])[:, 0]
    return [out]


def _exact_score(s):
    x = s["x"].double() * s["scale"]
    lp = torch.log_softmax(x, dim=1)
    entropy = -(torch.exp(lp) * lp).sum(dim=1)
    outs = [lp.gather(1, s["t"].long()[:, None])[:, 0], None, entropy]
    if s["top"]:
        outs += [lp.topk(s["top"], dim=1).values, None]
    return outs


def exact(case, seed):
    if case["kind"] == "state" and case["n"] * case["k"] > 20000:
        return None
    s = prepare(case, seed)
    return {"rope": _exact_rope, "attend": _exact_attend, "state": _exact_state, "score": _exact_score}[case["kind"]](s)

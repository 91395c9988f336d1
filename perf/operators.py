"""What the latent-attention serving operators are measured on: a cache of one latent vector a
token (bf16, or e4m3 with a scale a token) as it is written and read back, the absorbed attention
that reads it, the expanded attention of a prompt, and the verification of drafted tokens.

`run` computes a case in its plain form (elementary torch operations) where `own` is false and
through the framework's entry points where it is true.

Case kinds
  append   write T new tokens of N sequences into a paged cache and read the same tokens back
  gather   read whole cached sequences back as dense rows
  decode   absorbed attention of K new tokens a sequence over the paged cache
  prefill  expanded causal attention of packed prompts
  verify   verification of K drafted tokens a sequence
"""
import math
import random

import torch

own = False

DC, DR = 512, 64                 # latent and shared position key of a cached token
DN, DV = 128, 128                # per-head key part and value of the expanded form
ROW = {"bf16": 1152, "e4m3": 656}
E4M3_MAX = 448.0


# ---- cases -----------------------------------------------------------------------------------

def listed():
    return [
        # one decode step's new rows of 512 concurrent sequences
        {"name": "append_step_512", "kind": "append", "cache": "e4m3", "page": 64, "n": 512, "lo": 1, "hi": 1,
         "before": 4000, "fused": True, "lens_seed": 1},
        # the rows of one 145408-token prompt
        {"name": "append_prompt_145408", "kind": "append", "cache": "e4m3", "page": 64, "n": 1, "lo": 145408,
         "hi": 145408, "before": 0, "fused": True, "lens_seed": 2},
        # 16 cached prefixes of 1k to 64k tokens read back to be expanded; a page size that no tile divides
        {"name": "gather_varlen16", "kind": "gather", "cache": "e4m3", "page": 48, "n": 16, "lo": 1024, "hi": 65536,
         "lens_seed": 3},
        # a few short chats on a head shard: latency
        {"name": "decode_short", "kind": "decode", "cache": "bf16", "page": 16, "n": 3, "lo": 1, "hi": 200, "h": 4,
         "k": 2, "lens_seed": 4},
        # one long agentic prompt, one token
        {"name": "decode_one_145408", "kind": "decode", "cache": "bf16", "page": 64, "n": 1, "lo": 145408,
         "hi": 145408, "h": 32, "k": 1, "lens_seed": 5},
        # a serving batch of mixed lengths, one token each
        {"name": "decode_batch64", "kind": "decode", "cache": "bf16", "page": 64, "n": 64, "lo": 1024, "hi": 65536,
         "h": 32, "k": 1, "lens_seed": 6},
        # a speculative step (four query tokens a sequence) over the quantised cache
        {"name": "decode_spec16", "kind": "decode", "cache": "e4m3", "page": 64, "n": 16, "lo": 1024, "hi": 65536,
         "h": 32, "k": 4, "lens_seed": 3},
        # one 8192-token prompt, all heads
        {"name": "prefill_8192", "kind": "prefill", "h": 32, "n": 1, "lo": 8192, "hi": 8192, "prefix": 0,
         "joint": True, "lens_seed": 8},
        # ragged short prompts on a shard of the heads
        {"name": "prefill_ragged", "kind": "prefill", "h": 4, "n": 12, "lo": 1, "hi": 2000, "prefix": 0,
         "joint": False, "lens_seed": 9},
        # a 2048-token chunk of a prompt whose 32768 tokens before it are cached
        {"name": "prefill_chunk", "kind": "prefill", "h": 32, "n": 1, "lo": 2048, "hi": 2048, "prefix": 32768,
         "joint": True, "lens_seed": 10},
        # one sequence's three drafts
        {"name": "verify_one", "kind": "verify", "n": 1, "k": 3, "v": 131072, "sharp": 2.0, "draft": True},
        # a serving batch's drafts over a vocabulary of odd size
        {"name": "verify_batch", "kind": "verify", "n": 256, "k": 4, "v": 100003, "sharp": 2.0, "draft": True},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["append", "gather", "decode", "decode", "prefill", "verify"])
    cache = rng.choice(["bf16", "e4m3"])
    page = rng.choice([16, 32, 48, 64, 128])
    ls = rng.randrange(1 << 30)
    if kind == "append":
        n = _log_int(rng, 1, 512)
        hi = _log_int(rng, 1, 145408 // n)
        return {"kind": kind, "cache": cache, "page": page, "n": n, "lo": max(1, hi // 4), "hi": hi,
                "before": rng.randrange(0, 4000 if n > 8 else 100), "fused": rng.random() < 0.5, "lens_seed": ls}
    if kind == "gather":
        n = _log_int(rng, 1, 32)
        hi = _log_int(rng, 1, 200000 // n)
        return {"kind": kind, "cache": cache, "page": page, "n": n, "lo": max(1, hi // 16), "hi": hi, "lens_seed": ls}
    if kind == "decode":
        h = rng.choice([1, 3, 4, 8, 16, 20, 32, 64])
        k = rng.randrange(1, 9 if h <= 32 else 5)
        n = _log_int(rng, 1, 64)
        hi = _log_int(rng, 1, min(145408, 9000000 // (n * max(1, h * k // 32))))
        return {"kind": kind, "cache": cache, "page": page, "n": n, "lo": max(1, hi // 32), "hi": hi, "h": h, "k": k,
                "lens_seed": ls}
    if kind == "prefill":
        h = rng.choice([1, 3, 4, 8, 16, 32])
        n = _log_int(rng, 1, 12)
        hi = _log_int(rng, 1, 8000 // n)
        prefix = rng.choice([0, 0, _log_int(rng, 1, 24000 // n)])
        if h * n * hi * n * (hi + prefix) > (1 << 31):
            prefix = 0
        return {"kind": kind, "h": h, "n": n, "lo": max(1, hi // 8), "hi": hi, "prefix": prefix,
                "joint": rng.random() < 0.5, "lens_seed": ls}
    v = _log_int(rng, 1000, 160000)
    n = _log_int(rng, 1, max(1, min(256, 100000000 // (4 * v))))
    return {"kind": "verify", "n": n, "k": rng.randrange(1, 8 if n < 64 else 5), "v": v,
            "sharp": round(rng.uniform(0.5, 4.0), 2), "draft": rng.random() < 0.7}


def _lens(case):
    r = random.Random(case["lens_seed"])
    return [min(case["hi"], max(case["lo"], _log_int(r, case["lo"], case["hi"]))) for _ in range(case["n"])]


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
    return torch.cat([codes.view(torch.uint8), r.view(torch.uint8), s[:, None].view(torch.uint8), pad], dim=1)


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


def _cu(lens):
    cu = torch.zeros(len(lens) + 1, dtype=torch.int64)
    cu[1:] = torch.cumsum(torch.tensor(lens, dtype=torch.int64), 0)
    cu = cu.to(torch.int32)
    return cu, cu.cuda()


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
    if kind == "verify":
        n, k, v = case["n"], case["k"], case["v"]
        logits = _randn(g, n, k + 1, v) * case["sharp"]
        s["p"] = torch.softmax(logits, dim=-1)
        if case["draft"]:
            logits = logits[:, :k] + 0.5 * case["sharp"] * _randn(g, n, k, v)
            s["q"] = torch.softmax(logits, dim=-1)
            pick = s["q"]
        else:
            s["q"] = None
            pick = s["p"][:, :k]
        x = pick.cumsum(dim=-1, dtype=torch.float32)
        u = torch.rand(n, k, 1, generator=g, device="cuda") * x[..., -1:]
        s["x"] = torch.searchsorted(x, u, right=True).clamp_max(v - 1)[..., 0].to(torch.int32)
        s["u"] = torch.rand(n, k, generator=g, device="cuda")
        s["us"] = torch.rand(n, generator=g, device="cuda")
        return s
    lens = _lens(case)
    n = case["n"]
    if kind == "prefill":
        h = case["h"]
        lens_k = [x + case["prefix"] for x in lens]
        s["cu_q_host"], s["cu_q"] = _cu(lens)
        s["cu_k_host"], s["cu_k"] = _cu(lens_k)
        tq, tk = sum(lens), sum(lens_k)
        s["q"] = _randn(g, tq, h, DN + DR).to(torch.bfloat16)
        if case["joint"]:            # keys and values as one projection writes them
            kv = _randn(g, tk, h, DN + DV).to(torch.bfloat16)
            s["k"], s["v"] = kv[..., :DN], kv[..., DN:]
        else:
            s["k"], s["v"] = (_randn(g, tk, h, DN).to(torch.bfloat16) for _ in range(2))
        s["r"] = _randn(g, tk, DR).to(torch.bfloat16)
        s["causal"] = 1
        s["scale"] = (DN + DR) ** -0.5
        return s
    page, cache = case["page"], case["cache"]
    before = case.get("before", 0)
    total = [x + before for x in lens]
    s["table"], num = _pages(total, page, g)
    s["cu_host"], s["cu"] = _cu(lens)
    if kind == "append":
        T = sum(lens)
        c, r = _latents(g, T)
        if case["fused"]:            # slices of one projection's output rows
            both = torch.cat([c, r, c[:, :64]], dim=1)
            c, r = both[:, :DC], both[:, DC:DC + DR]
        s["c"], s["r"] = c, r
        s["start"] = torch.full((n,), before, dtype=torch.int32, device="cuda")
        seq = torch.repeat_interleave(torch.arange(n, device="cuda"), torch.tensor(lens, device="cuda"))
        pos = torch.arange(T, device="cuda") - s["cu"].long()[seq] + before
        s["slots"] = (s["table"].long()[seq, pos // page] * page + pos % page).to(torch.int32)
        s["pages"] = torch.zeros(num, page, ROW[cache], dtype=torch.uint8, device="cuda")
        return s
    c, r = _latents(g, num * page)
    s["pages"] = _pack(c, r, cache).view(num, page, ROW[cache])
    if kind == "decode":
        s["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
        s["q"] = _randn(g, n, case["k"], case["h"], DC + DR).to(torch.bfloat16)
        s["scale"] = (DN + DR) ** -0.5
    return s


# ---- plain forms -----------------------------------------------------------------------------

def _rows(s):
    """Cache row of every packed token of the sequences (from `start` on where there is one)."""
    cu, page = s["cu"].long(), s["page"]
    T = int(s["cu_host"][-1])
    t = torch.arange(T, device="cuda")
    seq = torch.searchsorted(cu[1:], t, right=True)
    pos = t - cu[seq] + (s["start"].long()[seq] if "start" in s else 0)
    return s["table"].long()[seq, pos // page] * page + pos % page


def _attend(x, values):
    """Softmax over the last axis of scores with -inf at masked places, the weighted values, and
    the log of the sum; a row with nothing to see gives zeros and -inf."""
    m = x.amax(dim=-1, keepdim=True)
    p = torch.exp(x - torch.where(torch.isinf(m), torch.zeros_like(m), m))
    l = p.sum(dim=-1, keepdim=True)
    o = torch.matmul(p, values) / torch.where(l > 0, l, torch.ones_like(l))
    return o, (m + torch.log(l))[..., 0]


def _plain_append(s):
    flat = s["pages"].view(-1, ROW[s["cache"]])
    flat[s["slots"].long()] = _pack(s["c"].contiguous(), s["r"].contiguous(), s["cache"])
    return _plain_gather(s)


def _plain_gather(s):
    c, r = _unpack(s["pages"].view(-1, ROW[s["cache"]])[_rows(s)], s["cache"])
    return [c.to(torch.bfloat16), r.to(torch.bfloat16)]


def _plain_decode(s):
    n, k, h = s["n"], s["k"], s["h"]
    lens, page = s["lens"].long(), s["page"]
    t = torch.arange(s["hi"], device="cuda")
    at = torch.clamp_max(t // page, s["table"].shape[1] - 1)
    rows = s["table"].long()[:, at] * page + t % page                          # [n, hi]
    c, r = _unpack(s["pages"].view(-1, ROW[s["cache"]])[rows], s["cache"])
    q = s["q"].float().view(n, k * h, DC + DR)
    x = (torch.matmul(q[..., :DC], c.transpose(1, 2)) + torch.matmul(q[..., DC:], r.transpose(1, 2))) * s["scale"]
    sees = lens[:, None] - (k - 1) + torch.arange(k, device="cuda")            # [n, k] tokens that query j sees
    sees = sees.repeat_interleave(h, dim=1)
    x = torch.where(t < sees[..., None], x, torch.full_like(x[:1, :1, :1], -math.inf))
    o, lse = _attend(x, c)
    return [o.view(n, k, h, DC).to(torch.bfloat16), lse.view(n, k, h)]


def _plain_prefill(s):
    tq, tk = int(s["cu_q_host"][-1]), int(s["cu_k_host"][-1])
    cq, ck = s["cu_q"].long(), s["cu_k"].long()
    i, j = torch.arange(tq, device="cuda"), torch.arange(tk, device="cuda")
    sq, sk = torch.searchsorted(cq[1:], i, right=True), torch.searchsorted(ck[1:], j, right=True)
    last = ck[sq + 1] - cq[sq + 1] + i                                         # last key that query i sees
    q = s["q"].float().transpose(0, 1)
    k = torch.cat([s["k"].float(), s["r"].float()[:, None].expand(-1, s["h"], -1)], dim=-1).transpose(0, 1)
    x = torch.matmul(q, k.transpose(1, 2)) * s["scale"]
    x.masked_fill_(((sq[:, None] != sk) | (j > last[:, None]))[None], -math.inf)
    o, lse = _attend(x, s["v"].float().transpose(0, 1))
    return [o.transpose(0, 1).to(torch.bfloat16).contiguous(), lse.transpose(0, 1).contiguous()]


def _plain_verify(s):
    n, k, v = s["n"], s["k"], s["v"]
    p, x = s["p"], s["x"].long()
    px = p[:, :k].gather(2, x[..., None])[..., 0].double()
    qx = torch.ones_like(px) if s["q"] is None else s["q"].gather(2, x[..., None])[..., 0].double()
    ok = s["u"].double() * qx < px
    a = ok.long().cumprod(dim=1).sum(dim=1)                                    # accepted drafts
    b = torch.arange(n, device="cuda")
    row = p[b, a].double()
    j = torch.clamp_max(a, k - 1)
    if s["q"] is None:
        sub = torch.zeros_like(row).scatter_(1, x[b, j][:, None], math.inf)
    else:
        sub = s["q"][b, j].double()
    left = torch.clamp_min(torch.where((a < k)[:, None], row - sub, row), 0)
    left = torch.where((left.sum(dim=1) > 0)[:, None], left, row)
    c = left.cumsum(dim=1)
    over = c > s["us"].double()[:, None] * c[:, -1:]
    over[:, -1] = True
    pick = over.to(torch.uint8).argmax(dim=1)
    at = torch.arange(k + 1, device="cuda")
    out = torch.cat([x, x[:, :1]], dim=1)
    out = torch.where(at < a[:, None], out, torch.where(at == a[:, None], pick[:, None], torch.full_like(out, -1)))
    return [out.to(torch.int32), (a + 1).to(torch.int32)]


# ---- the framework's calls -------------------------------------------------------------------

def _own(s):
    from kimi_delta_attention_06_gb300 import kda

    kind = s["kind"]
    if kind == "verify":
        return list(kda.verify_draft(s["p"], s["q"], s["x"], s["u"], s["us"]))
    if kind == "prefill":
        return list(kda.latent_prefill(s["q"], s["k"], s["v"], s["r"], s["cu_q_host"], s["cu_k_host"], s["scale"],
                                       causal=True, cu_q=s["cu_q"], cu_k=s["cu_k"], want_lse=True))
    dtype = kda.KDA_CACHE_BF16 if s["cache"] == "bf16" else kda.KDA_CACHE_E4M3
    if kind == "decode":
        return list(kda.latent_decode(s["q"], s["pages"], dtype, s["table"], s["lens"], s["scale"], want_lse=True))
    if kind == "append":
        kda.latent_append(s["c"], s["r"], s["pages"], dtype, s["slots"])
    return list(kda.latent_gather(s["pages"], dtype, s["table"], s["cu_host"], cu_seqlens=s["cu"],
                                  start_pos=s.get("start")))


def run(state):
    if own:
        return _own(state)
    return {"append": _plain_append, "gather": _plain_gather, "decode": _plain_decode, "prefill": _plain_prefill,
            "verify": _plain_verify}[state["kind"]](state)


def work(case):
    kind = case["kind"]
    if kind == "verify":
        # the rows that the answer needs: the target's, and the draft's of a sequence that stopped
        rows = 2 if case["draft"] else 1
        n, k, v = case["n"], case["k"], case["v"]
        return {"bytes": 4 * n * (rows * v + 5 * k + 2), "flops": n * v * rows}
    lens = _lens(case)
    if kind == "prefill":
        h, pre = case["h"], case["prefix"]
        pairs = sum(x * pre + x * (x + 1) // 2 for x in lens)
        tq, tk = sum(lens), sum(lens) + pre * case["n"]
        return {"bytes": 2 * (tq * h * (DN + DR + DV) + tk * h * (DN + DV) + tk * DR) + 4 * tq * h,
                "flops": 2 * pairs * h * (DN + DR + DV)}
    T, row = sum(lens), ROW[case["cache"]]
    if kind == "append":
        return {"bytes": T * (2 * ROW["bf16"] + row + 4), "flops": 0}
    if kind == "gather":
        return {"bytes": T * (ROW["bf16"] + row), "flops": 0}
    h, k = case["h"], case["k"]
    return {"bytes": T * row + case["n"] * k * h * (2 * (DC + DR) + 2 * DC + 4),
            "flops": 2 * T * k * h * (2 * DC + DR)}


# ---- in 64 bits, from the definitions --------------------------------------------------------

def _exact_rows(c, r, cache):
    """The values a cache row holds, by searching each latent's nearest code among all codes."""
    c = c.double()
    if cache == "e4m3":
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
        c = torch.sign(c) * torch.where(take_lo, codes[lo], codes[hi]) * s
    return c, r.double()


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


def exact(case, seed):
    s = prepare(case, seed)
    kind = case["kind"]
    if kind == "verify":
        return None
    if kind == "append":
        if s["c"].shape[0] > 200000:
            return None
        return list(_exact_rows(s["c"], s["r"], s["cache"]))
    flat = s["pages"].view(-1, ROW[s["cache"]]) if "pages" in s else None
    if kind == "gather":
        outs = []
        for n in range(s["n"]):
            t = torch.arange(int(s["cu_host"][n + 1] - s["cu_host"][n]), device="cuda")
            outs.append(flat[s["table"][n].long()[t // s["page"]] * s["page"] + t % s["page"]])
        return list(_exact_read(torch.cat(outs), s["cache"]))
    if kind == "decode":
        n, k, h = s["n"], s["k"], s["h"]
        o = torch.zeros(n, k, h, DC, dtype=torch.float64, device="cuda")
        lse = torch.full((n, k, h), -math.inf, dtype=torch.float64, device="cuda")
        for i in range(n):
            L = int(s["lens"][i])
            t = torch.arange(L, device="cuda")
            c, r = _exact_read(flat[s["table"][i].long()[t // s["page"]] * s["page"] + t % s["page"]], s["cache"])
            for j in range(k):
                see = L - (k - 1 - j)
                if see > 0:
                    x = s["q"][i, j].double() @ torch.cat([c[:see], r[:see]], dim=1).T * s["scale"]
                    o[i, j], lse[i, j] = torch.softmax(x, dim=1) @ c[:see], torch.logsumexp(x, dim=1)
        return [o, lse]
    h = s["h"]
    o = torch.zeros(*s["q"].shape[:2], DV, dtype=torch.float64, device="cuda")
    lse = torch.full(s["q"].shape[:2], -math.inf, dtype=torch.float64, device="cuda")
    for n in range(s["n"]):
        q0, q1, k0, k1 = (int(s[c][n + e]) for c in ("cu_q_host", "cu_k_host") for e in (0, 1))
        hide = torch.ones(q1 - q0, k1 - k0, dtype=torch.bool, device="cuda").triu(k1 - k0 - (q1 - q0) + 1)
        for head in range(h):
            key = torch.cat([s["k"][k0:k1, head], s["r"][k0:k1]], dim=1).double()
            x = (s["q"][q0:q1, head].double() @ key.T * s["scale"]).masked_fill(hide, -math.inf)
            o[q0:q1, head] = torch.softmax(x, dim=1) @ s["v"][k0:k1, head].double()
            lse[q0:q1, head] = torch.logsumexp(x, dim=1)
    return [o, lse]

"""GPU parity of the latent cache and the latent attention against plain fp64 forms."""
import math

import pytest
import torch

from kimi_delta_attention_06_gb300 import kda
from tests import _latent as L

pytestmark = pytest.mark.gpu
DEV = "cuda"
CACHES = [pytest.param(kda.KDA_CACHE_BF16, id="bf16"), pytest.param(kda.KDA_CACHE_E4M3, id="e4m3")]


@pytest.fixture(scope="module", autouse=True)
def _built():
    from kimi_delta_attention_06_gb300 import build
    build.build()


def _ok():
    assert kda.kda_device_status() == kda.KDA_OK


# ---- the cache -------------------------------------------------------------------------------

def _extreme_rows():
    """Latent rows at the ends of the types' ranges, with ties, zeros, NaN and infinities."""
    g = L.gen(3)
    c = torch.randn(12, L.DC, generator=g)
    c[1] = 0.0
    c[2] *= 1e-38
    c[3] *= 3e37
    c[4] = torch.linspace(-448, 448, L.DC)                     # many halfway cases
    c[5, 17], c[5, 400] = math.nan, math.inf
    c[6, 3] = -math.inf
    c[7] = 7.0 * 2.0 ** -20                                    # the largest value of a scale exactly
    c[8, 0] = 2.0 ** 127
    c[9] = 2.0 ** -133                                         # a denormal
    c[10] = -0.0
    c[11, 5] = 100.0
    return c.to(torch.bfloat16)


@pytest.mark.parametrize("dtype", CACHES)
def test_append_writes_the_defined_bytes(dtype):
    c = _extreme_rows()
    r = torch.randn(c.shape[0], L.DR, generator=L.gen(4)).to(torch.bfloat16)
    page, P = 16, 3
    slots = torch.tensor([47, 0, 5, 16, 31, 32, 2, 40, -1, 7, 1, 9], dtype=torch.int32)
    cache = torch.full((P, page, L.ROW[dtype]), 0xA5, dtype=torch.uint8, device=DEV)
    kda.latent_append(c.to(DEV), r.to(DEV), cache, dtype, slots.to(DEV))
    _ok()
    want = torch.full((P * page, L.ROW[dtype]), 0xA5, dtype=torch.uint8)
    rows = L.pack(c, r, dtype)
    for i, s in enumerate(slots.tolist()):
        if s >= 0:
            want[s] = rows[i]
    got = cache.cpu().view(P * page, -1)
    if dtype == kda.KDA_CACHE_E4M3:                            # either NaN code stands for NaN
        for x in (got, want):
            codes = x[:, :L.DC]
            codes[(codes & 127) == 127] = 127
    assert torch.equal(got, want)


@pytest.mark.parametrize("dtype", CACHES)
@pytest.mark.parametrize("T,page,fused", [(1, 16, False), (129, 48, True), (1000, 64, True)])
def test_append_then_gather_returns_the_values(dtype, T, page, fused):
    g = L.gen(T)
    c, r = L.latents(g, T, loud=3.0)
    both = torch.cat([c, r, c[:, :24]], dim=1).to(DEV)         # rows of a wider projection
    cd, rd = (both[:, :L.DC], both[:, L.DC:L.DC + L.DR]) if fused else (c.to(DEV), r.to(DEV))
    lens = [T // 3, 0, T - T // 3]
    before = [5, 0, page]
    need = [-(-(a + b) // page) for a, b in zip(lens, before)]
    table = torch.zeros(3, max(need), dtype=torch.int32)
    perm = torch.randperm(sum(need), generator=g)
    at, slots = 0, []
    for n in range(3):
        table[n, :need[n]] = perm[at:at + need[n]].to(torch.int32)
        at += need[n]
        slots += [int(table[n, p // page]) * page + p % page for p in range(before[n], before[n] + lens[n])]
    cache = kda.latent_cache(sum(need), page, dtype)
    kda.latent_append(cd, rd, cache, dtype, torch.tensor(slots, dtype=torch.int32, device=DEV))
    cu = torch.tensor([0, lens[0], lens[0], T], dtype=torch.int32)
    gc, gr = kda.latent_gather(cache, dtype, table.to(DEV), cu, start_pos=torch.tensor(before, dtype=torch.int32, device=DEV))
    _ok()
    want_c, want_r = L.unpack(L.pack(c, r, dtype), dtype)
    assert torch.equal(gc.cpu().double(), want_c) and torch.equal(gr.cpu().double(), want_r)


@pytest.mark.parametrize("dtype", CACHES)
def test_gather_whole_sequences_into_strided_rows(dtype):
    lens, page = [70, 1, 0, 33], 16
    cache, table, held = L.paged(lens, page, dtype, seed=9)
    T = sum(lens)
    wide = torch.full((T, 640), float("nan"), device=DEV, dtype=torch.bfloat16)
    cu = torch.tensor([0, 70, 71, 71, 104], dtype=torch.int32)
    kda.kda_latent_gather(cache.to(DEV), dtype, table.to(DEV), None, cu.to(DEV), cu, 4, T, wide[:, 64:576], wide[:, :64])
    _ok()
    assert torch.equal(wide[:, 64:576].cpu().double(), torch.cat([h[0] for h in held]))
    assert torch.equal(wide[:, :64].cpu().double(), torch.cat([h[1] for h in held]))
    assert torch.isnan(wide[:, 576:]).all()


@pytest.mark.parametrize("dtype", CACHES)
def test_bad_indices_are_reported_and_skipped(dtype):
    page, P = 16, 2
    c, r = L.latents(L.gen(1), 3)
    cache = kda.latent_cache(P, page, dtype)
    kda.latent_append(c.to(DEV), r.to(DEV), cache, dtype, torch.tensor([1, P * page, 2], dtype=torch.int32, device=DEV))
    assert kda.kda_device_status() == kda.KDA_ERR_INVALID_ARG
    rows = L.pack(c, r, dtype)
    flat = cache.cpu().view(P * page, -1)
    assert torch.equal(flat[[1, 2]], rows[[0, 2]]) and not flat[[0, 3]].any()
    # gather: a page past the pool, a negative page, and a position past the table
    table = torch.tensor([[0, 9], [-3, 1]], dtype=torch.int32, device=DEV)
    cu = torch.tensor([0, 20, 40], dtype=torch.int32)
    out_c = torch.full((40, L.DC), 7.0, device=DEV, dtype=torch.bfloat16)
    out_r = torch.full((40, L.DR), 7.0, device=DEV, dtype=torch.bfloat16)
    kda.kda_latent_gather(cache, dtype, table, torch.tensor([0, 13], dtype=torch.int32, device=DEV), cu.to(DEV), cu, 2,
                          40, out_c, out_r)
    assert kda.kda_device_status() == kda.KDA_ERR_INVALID_ARG
    left = (out_c == 7.0).all(dim=1).cpu()
    assert not left[:16].any() and left[16:23].all() and not left[23:39].any() and left[39]
    _ok()


# ---- absorbed attention ------------------------------------------------------------------------

def _decode(lens, K, H, page, dtype, seed, scale=192 ** -0.5, q_std=1.0, junk=None, loud=1.0, edit=None):
    cache, table, held = L.paged(lens, page, dtype, seed, loud=loud, junk=junk)
    q = (torch.randn(len(lens), K, H, L.DC + L.DR, generator=L.gen(seed + 1)) * q_std).to(torch.bfloat16)
    if edit:
        edit(q, cache, table, held)
    out, lse = kda.latent_decode(q.to(DEV), cache.to(DEV), dtype, table.to(DEV),
                                 torch.tensor(lens, dtype=torch.int32, device=DEV), scale, want_lse=True)
    _ok()
    rows = []
    for n, length in enumerate(lens):
        key = torch.cat(held[n], dim=1)
        for j in range(K):
            for h in range(H):
                rows.append(L.attend(q[n, j, h].double(), key, held[n][0], scale, length - (K - 1 - j)))
    L.check_rows(out.view(-1, L.DC), lse.view(-1), rows)
    return q, cache, table, out, lse


@pytest.mark.parametrize("dtype", CACHES)
@pytest.mark.parametrize("lens,K,H,page", [
    ([1], 1, 1, 16),
    ([0, 1, 2, 63, 64, 65], 1, 3, 16),          # empty, one, around a tile
    ([0, 1, 2, 3, 130], 4, 4, 32),              # queries that see nothing
    ([700, 33, 257], 1, 32, 48),                # pages that no tile divides
    ([300, 64, 129], 4, 32, 64),                # 128 rows
    ([90, 400], 3, 20, 128),
    ([500], 8, 64, 16),                         # 512 rows
    ([6000, 5], 1, 16, 64),                     # one long, one short
    ([2500], 2, 8, 1024),
])
def test_decode(dtype, lens, K, H, page):
    _decode(lens, K, H, page, dtype, seed=sum(lens) + K + H)


@pytest.mark.parametrize("dtype", CACHES)
@pytest.mark.parametrize("scale,q_std", [(192 ** -0.5, 30.0), (0.0, 1.0), (-0.07, 4.0), (1e-3, 1.0)])
def test_decode_scales(dtype, scale, q_std):
    """Sharp, flat, negated and nearly flat scores; the sharp ones move the running maximum far."""
    _decode([333, 1500], 2, 16, 64, dtype, seed=5, scale=scale, q_std=q_std)


@pytest.mark.parametrize("dtype", CACHES)
def test_decode_growing_scores(dtype):
    """Every tile holds a larger score than all before it, by far."""
    def edit(q, cache, table, held):
        for n in range(2):
            T = held[n][0].shape[0]
            r = torch.arange(T, dtype=torch.float64)[:, None] / 16 * torch.ones(1, L.DR, dtype=torch.float64)
            r = r.to(torch.bfloat16)
            held[n][1][:] = r.double()
            for t in range(T):
                at = L.DC if dtype else 2 * L.DC
                cache[table[n, t // 64], t % 64, at:at + 128] = r[t].view(torch.uint8)
        q[..., L.DC:] = 1.0
    _decode([900, 200], 1, 8, 64, dtype, seed=8, edit=edit)


@pytest.mark.parametrize("dtype", CACHES)
def test_decode_ignores_what_lies_past_the_end(dtype):
    """NaN bytes in the rest of the last pages, and in the latents of drafted tokens that earlier
    queries do not see."""
    _decode([1, 65, 100, 16], 1, 8, 16, dtype, seed=11, junk=0xFF)
    _decode([130, 64], 2, 32, 48, dtype, seed=12, junk=0x7F)

    lens, K, H, page = [70, 3], 3, 4, 16
    cache, table, held = L.paged(lens, page, dtype, seed=13)
    q = torch.randn(2, K, H, 576, generator=L.gen(14)).to(torch.bfloat16)
    for n, length in enumerate(lens):                          # the last token's latent is NaN
        cache[table[n, (length - 1) // page], (length - 1) % page, :L.DC] = 0xFF
    out, lse = kda.latent_decode(q.to(DEV), cache.to(DEV), dtype, table.to(DEV),
                                 torch.tensor(lens, dtype=torch.int32, device=DEV), 0.07, want_lse=True)
    _ok()
    for n, length in enumerate(lens):
        assert torch.isnan(out[n, K - 1].float()).any() and torch.isnan(lse[n, K - 1]).all()
        key = torch.cat(held[n], dim=1)
        rows = [L.attend(q[n, j, h].double(), key, held[n][0], 0.07, length - (K - 1 - j))
                for j in range(K - 1) for h in range(H)]
        L.check_rows(out[n, :K - 1].reshape(-1, L.DC), lse[n, :K - 1].reshape(-1), rows)


def test_decode_reports_bad_lengths_and_pages():
    cache, table, held = L.paged([40, 20, 30], 16, 0, seed=2)
    q = torch.randn(3, 1, 4, 576, generator=L.gen(1)).to(torch.bfloat16)
    lens = torch.tensor([40, -1, 30], dtype=torch.int32, device=DEV)
    out, lse = kda.latent_decode(q.to(DEV), cache.to(DEV), 0, table.to(DEV), lens, 0.07, want_lse=True)
    assert kda.kda_device_status() == kda.KDA_ERR_INVALID_ARG
    assert not out[1].any() and torch.isinf(lse[1]).all()      # counts as empty
    for n in (0, 2):
        L.check_rows(out[n, 0], lse[n, 0], [L.attend(q[n, 0, h].double(), torch.cat(held[n], 1), held[n][0], 0.07,
                                                     [40, 0, 30][n]) for h in range(4)])
    bad = table.clone()
    bad[0, 1] = 12345                                          # a page past the pool
    lens = torch.tensor([40, 20, 30], dtype=torch.int32, device=DEV)
    out2, _ = kda.latent_decode(q.to(DEV), cache.to(DEV), 0, bad.to(DEV), lens, 0.07)
    assert kda.kda_device_status() == kda.KDA_ERR_INVALID_ARG
    assert torch.equal(out2[2], out[2])                        # other sequences are unharmed
    _ok()


@pytest.mark.parametrize("dtype", CACHES)
def test_decode_repeats_bit_for_bit_and_on_another_stream(dtype):
    lens = [5000, 1, 900, 64, 0, 2222]
    cache, table, _ = L.paged(lens, 64, dtype, seed=20)
    q = torch.randn(6, 2, 32, 576, generator=L.gen(21)).to(torch.bfloat16).to(DEV)
    cache, table, ln = cache.to(DEV), table.to(DEV), torch.tensor(lens, dtype=torch.int32, device=DEV)
    a = kda.latent_decode(q, cache, dtype, table, ln, 0.07, want_lse=True)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        b = kda.latent_decode(q, cache, dtype, table, ln, 0.07, want_lse=True)
        c = kda.latent_decode(q, cache, dtype, table, ln, 0.07, want_lse=True)
    s.synchronize()
    _ok()
    for x in (b, c):
        assert torch.equal(a[0], x[0]) and torch.equal(a[1], x[1])


def test_decode_in_a_captured_graph_follows_new_lengths():
    lens = [100, 900]
    cache, table, held = L.paged(lens, 64, 0, seed=23)
    q = torch.randn(2, 1, 32, 576, generator=L.gen(24)).to(torch.bfloat16)
    qd, cache, table = q.to(DEV), cache.to(DEV), table.to(DEV)
    ln = torch.tensor([1, 1], dtype=torch.int32, device=DEV)
    out = torch.empty(2, 1, 32, 512, device=DEV, dtype=torch.bfloat16)
    lse = torch.empty(2, 1, 32, device=DEV)
    call = lambda: kda.kda_latent_decode(qd, cache, 0, table, ln, 2, 1, 32, 0.07, out, lse)
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        call()
    s.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        call()
    for now in ([100, 900], [7, 64], [0, 899]):
        ln.copy_(torch.tensor(now, dtype=torch.int32))
        g.replay()
        torch.cuda.synchronize()
        _ok()
        L.check_rows(out.view(-1, 512), lse.view(-1), [L.attend(q[n, 0, h].double(), torch.cat(held[n], 1), held[n][0],
                                                                0.07, now[n]) for n in range(2) for h in range(32)])


def test_decode_cache_offsets_past_32_bits():
    """Pages at both ends of a cache of more than 2^32 bytes."""
    page, P = 64, 60000                                        # 60000 * 64 * 1152 B = 4.4 GB
    small, table, held = L.paged([150], page, 0, seed=31)
    cache = torch.zeros(P, page, 1152, dtype=torch.uint8, device=DEV)
    where = torch.tensor([P - 1, 0, P - 2], dtype=torch.int32)
    for i in range(3):
        cache[int(where[i])] = small[int(table[0, i])].to(DEV)
    q = torch.randn(1, 1, 16, 576, generator=L.gen(32)).to(torch.bfloat16)
    out, lse = kda.latent_decode(q.to(DEV), cache, 0, where[None].to(DEV), torch.tensor([150], dtype=torch.int32, device=DEV),
                                 0.07, want_lse=True)
    _ok()
    L.check_rows(out[0, 0], lse[0, 0], [L.attend(q[0, 0, h].double(), torch.cat(held[0], 1), held[0][0], 0.07, 150)
                                        for h in range(16)])


# ---- expanded attention ------------------------------------------------------------------------

def _prefill(lens_q, lens_k, H, seed, causal=True, layout="dense", scale=192 ** -0.5, q_std=1.0, edit=None, rows=None):
    g = L.gen(seed)
    tq, tk = sum(lens_q), sum(lens_k)
    q = (torch.randn(tq, H, 192, generator=g) * q_std).to(torch.bfloat16)
    k = torch.randn(tk, H, 128, generator=g).to(torch.bfloat16)
    v = torch.randn(tk, H, 128, generator=g).to(torch.bfloat16)
    r = torch.randn(tk, 64, generator=g).to(torch.bfloat16)
    if edit:
        edit(q, k, v, r)
    if layout == "joint":
        kv = torch.cat([k, v], dim=2).to(DEV)
        kd, vd = kv[..., :128], kv[..., 128:]
    elif layout == "heads":
        kd, vd = (x.transpose(0, 1).contiguous().to(DEV).transpose(0, 1) for x in (k, v))
    else:
        kd, vd = k.to(DEV), v.to(DEV)
    rd = torch.cat([r, r], dim=1).to(DEV)[:, 64:] if layout == "joint" else r.to(DEV)
    cq = torch.tensor([0] + list(torch.tensor(lens_q).cumsum(0)), dtype=torch.int32)
    ck = torch.tensor([0] + list(torch.tensor(lens_k).cumsum(0)), dtype=torch.int32)
    out, lse = kda.latent_prefill(q.to(DEV), kd, vd, rd, cq, ck, scale, causal=causal, want_lse=True)
    _ok()
    for n in range(len(lens_q)):
        a, b = int(cq[n]), int(ck[n])
        Lq, Lk = lens_q[n], lens_k[n]
        pick = range(Lq) if rows is None else sorted({i for i in rows if i < Lq} | {Lq - 1})
        for h in range(H) if rows is None else {0, H - 1}:
            key = torch.cat([k[b:b + Lk, h], r[b:b + Lk]], dim=1).double()
            res = [L.attend(q[a + i, h].double(), key, v[b:b + Lk, h].double(), scale,
                            max(0, i + 1 + Lk - Lq) if causal else Lk) for i in pick]
            L.check_rows(out[a:a + Lq, h][list(pick)], lse[a:a + Lq, h][list(pick)], res)
    return out, lse


@pytest.mark.parametrize("lens_q,lens_k,H,causal,layout", [
    ([1], [1], 1, True, "dense"),
    ([127, 1, 129], [127, 1, 129], 2, True, "joint"),
    ([64, 128, 256], [64, 128, 256], 3, True, "heads"),
    ([5, 0, 130], [200, 7, 130], 2, True, "dense"),            # a chunk after a prefix; no queries
    ([40, 3], [10, 0], 2, True, "joint"),                      # more queries than keys: rows that see nothing
    ([33, 200], [300, 64], 2, False, "heads"),
    ([257, 255], [513, 255], 1, True, "joint"),
])
def test_prefill(lens_q, lens_k, H, causal, layout):
    _prefill(lens_q, lens_k, H, seed=sum(lens_q) + H, causal=causal, layout=layout)


def test_prefill_long_rows_sampled():
    _prefill([2100], [2100], 4, seed=3, layout="joint", rows=[0, 1, 127, 128, 255, 256, 1000, 1999])
    _prefill([300, 700], [4000, 1700], 2, seed=4, rows=[0, 63, 64, 255, 299, 512])


@pytest.mark.parametrize("scale,q_std", [(192 ** -0.5, 30.0), (0.0, 1.0), (-0.07, 4.0)])
def test_prefill_scales(scale, q_std):
    _prefill([300], [400], 2, seed=6, scale=scale, q_std=q_std)


def test_prefill_growing_scores():
    def edit(q, k, v, r):
        r[:] = (torch.arange(r.shape[0], dtype=torch.float32)[:, None] / 16).to(torch.bfloat16)
        q[..., 128:] = 1.0
    _prefill([600], [600], 2, seed=7, edit=edit)


def test_prefill_ignores_unseen_keys_and_values():
    """NaN and infinite keys and values: rows before them are untouched, rows from them on are NaN."""
    def clean(q, k, v, r):
        pass
    base, base_lse = _prefill([300], [300], 2, seed=9, edit=clean)

    def edit(q, k, v, r):
        v[150], k[260] = float("nan"), float("inf")
        v[290, 0, 3] = float("-inf")
    g = L.gen(9)
    q = torch.randn(300, 2, 192, generator=g).to(torch.bfloat16)
    k = torch.randn(300, 2, 128, generator=g).to(torch.bfloat16)
    v = torch.randn(300, 2, 128, generator=g).to(torch.bfloat16)
    r = torch.randn(300, 64, generator=g).to(torch.bfloat16)
    edit(q, k, v, r)
    cu = torch.tensor([0, 300], dtype=torch.int32)
    out, lse = kda.latent_prefill(*(x.to(DEV) for x in (q, k, v, r)), cu, cu, 192 ** -0.5, want_lse=True)
    _ok()
    key = torch.cat([k, r[:, None].expand(-1, 2, -1)], dim=2).double()
    for h in range(2):
        rows = [L.attend(q[i, h].double(), key[:, h], v[:, h].double(), 192 ** -0.5, i + 1) for i in range(150)]
        L.check_rows(out[:150, h], lse[:150, h], rows)
    assert torch.isnan(out[150:].float()).all()
    assert torch.isfinite(lse[150:260]).all()                  # keys up to 259 are finite


def test_prefill_on_another_stream_repeats():
    g = L.gen(15)
    mk = lambda *s: torch.randn(*s, generator=g).to(torch.bfloat16).to(DEV)
    q, k, v, r = mk(500, 4, 192), mk(700, 4, 128), mk(700, 4, 128), mk(700, 64)
    cq, ck = torch.tensor([0, 200, 500], dtype=torch.int32), torch.tensor([0, 250, 700], dtype=torch.int32)
    a, al = kda.latent_prefill(q, k, v, r, cq, ck, 0.07, want_lse=True)
    cqd, ckd = cq.to(DEV), ck.to(DEV)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        b, bl = kda.latent_prefill(q, k, v, r, cq, ck, 0.07, cu_q=cqd, cu_k=ckd, want_lse=True)
    s.synchronize()
    _ok()
    assert torch.equal(a, b) and torch.equal(al, bl)

"""A small hybrid decoder served speculatively: one KDA layer and one latent-attention layer, from
prompt to accepted tokens, through the package's entry points.

It shows how the calls fit together; the weights are random and the projections around the kernels
plain torch.  Per sequence the model keeps a KDA state (fixed size, a slot of a pool) and the latent
cache's pages (they grow).

  prompt    kda.prefill, kda.latent_append, kda.latent_prefill (expanded form; a second prompt chunk
            reads its cached prefix back with kda.latent_gather and expands it)
  step      the last token and K drafted ones enter together:
            kda.kda_decode_multi (verify), kda.latent_append, kda.latent_decode (absorbed form),
            kda.verify_draft, kda.kda_decode_multi (commit of the accepted prefix).
            Cache rows of rejected tokens are written over by the next step.

  python -m kimi_delta_attention_06_gb300.hybrid_step [--seqs 8] [--prompt 1000] [--draft 3] [--steps 20]
"""
from __future__ import annotations

import argparse
import time

import torch
import torch.nn.functional as F

from . import build, kda

DC, DR, DN, DV = kda.KDA_LATENT_DIM, kda.KDA_LATENT_ROPE, 128, 128


def _rms(x):
    """x over its root mean square, in fp32 (a factor rounded to bf16 would shift whole rows)."""
    x = x.float()
    return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6)


class HybridModel:
    """Random weights of a two-layer hybrid: H heads of 128, vocabulary V."""

    def __init__(self, vocab: int = 1024, width: int = 256, heads: int = 4, seed: int = 0, device="cuda"):
        g = torch.Generator(device=device).manual_seed(seed)
        mk = lambda *s: (torch.randn(*s, generator=g, device=device) / s[-2] ** 0.5).to(torch.bfloat16)
        self.V, self.M, self.H, self.device = vocab, width, heads, device
        self.embed = torch.randn(vocab, width, generator=g, device=device).to(torch.bfloat16)
        self.kda_in = mk(width, heads * 3 * 128)
        self.kda_gate = mk(width, heads * 128)
        self.kda_beta = mk(width, heads)
        self.kda_out = mk(heads * 128, width)
        self.lat_q = mk(width, heads * (DN + DR))
        self.lat_kv = mk(width, DC + DR)
        self.lat_uk = mk(heads, DC, DN)
        self.lat_uv = mk(heads, DC, DV)
        self.lat_out = mk(heads * DV, width)
        self.scale = (DN + DR) ** -0.5

    def kda_inputs(self, x):
        """q, k, v, log_alpha, beta of hidden rows x [T, M]."""
        T = x.shape[0]
        q, k, v = (x @ self.kda_in).view(T, self.H, 3, 128).unbind(2)
        q, k = (F.normalize(t.float(), dim=-1).to(torch.bfloat16) for t in (q, k))
        la = -F.softplus((x @ self.kda_gate).float().view(T, self.H, 128) - 2.0)
        return q, k, v.contiguous(), la.contiguous(), torch.sigmoid((x @ self.kda_beta).float()).to(torch.bfloat16)

    def latent(self, x):
        """The fused projection's rows: normalised latent and position key, slices of one tensor."""
        row = x @ self.lat_kv
        row = torch.cat([_rms(row[:, :DC]).to(row.dtype), row[:, DC:]], dim=1)
        return row[:, :DC], row[:, DC:]

    def expand(self, c):
        """Per-head keys and values [T, H, 128] of latents [T, 512], slices of one tensor."""
        kv = torch.einsum("tc,hcd->thd", c, torch.cat([self.lat_uk, self.lat_uv], dim=2))
        return kv[..., :DN], kv[..., DN:]

    def absorb(self, q):
        """q [.., H, 192] -> [.., H, 576]: W_uk^T q_nope, then the position part."""
        return torch.cat([torch.einsum("...hd,hcd->...hc", q[..., :DN], self.lat_uk), q[..., DN:]], dim=-1).contiguous()

    def probs(self, x):
        return torch.softmax(_rms(x) @ self.embed.t().float() * 0.25, dim=-1)


class HybridServer:
    """States, pages and lengths of N sequences."""

    def __init__(self, model: HybridModel, seqs: int, max_tokens: int, page: int = 64,
                 cache_dtype: int = kda.KDA_CACHE_E4M3):
        m = self.m = model
        self.N, self.page, self.cache_dtype = seqs, page, cache_dtype
        pages = -(-max_tokens // page)
        self.cache = kda.latent_cache(seqs * pages, page, cache_dtype, device=m.device)
        g = torch.Generator().manual_seed(1)
        self.table = torch.randperm(seqs * pages, generator=g).to(torch.int32).view(seqs, pages).to(m.device)
        self.state = torch.zeros(seqs, m.H, 128, 128, device=m.device)
        self.lens = torch.zeros(seqs, dtype=torch.int32, device=m.device)
        self.room = pages * page                               # tokens that a sequence's pages hold
        self.most = 0                                          # upper bound of the lengths, kept on the host

    def _take(self, tokens: int):
        """Refuse a step of `tokens` a sequence that the pages do not hold (an index past the table would be a fault on
        the GPU).  The bound counts every entered token as accepted; the lengths are read back only where it is reached."""
        if self.most + tokens > self.room:
            self.most = int(self.lens.max()) if self.N else 0
            if self.most + tokens > self.room:
                raise ValueError(f"{tokens} more tokens do not fit: a sequence holds {self.most} of {self.room}")
        self.most += tokens

    def _slots(self, seq, pos):
        """Cache rows of tokens at positions pos of sequences seq."""
        return (self.table[seq, pos // self.page] * self.page + pos % self.page).to(torch.int32)

    def prompt(self, tokens):
        """Enter the next chunk of every sequence's prompt (a list of N 1-D token tensors);
        returns the target's distribution [N, V] after each."""
        m, dev = self.m, self.m.device
        lens = torch.tensor([t.numel() for t in tokens], dtype=torch.int32)
        if len(tokens) != self.N:
            raise ValueError(f"{self.N} sequences, got the tokens of {len(tokens)}")
        cu_host = F.pad(lens.cumsum(0), (1, 0)).to(torch.int32)
        before = self.lens.cpu()
        total = before + lens
        if self.N and int(total.max()) > self.room:
            raise ValueError(f"the prompt does not fit: a sequence would hold {int(total.max())} of {self.room} tokens")
        self.most = int(total.max()) if self.N else 0
        cu_k_host = F.pad(total.cumsum(0), (1, 0)).to(torch.int32)
        seq = torch.repeat_interleave(torch.arange(self.N), lens.long()).to(dev)
        pos = (torch.cat([torch.arange(int(n)) for n in lens]).to(dev) + self.lens[seq]).long()
        x = m.embed[torch.cat(list(tokens)).to(dev).long()]
        o, state, _ = kda.prefill(*m.kda_inputs(x), cu_host, init_state=self.state)
        self.state = state
        x = x + o.flatten(1) @ m.kda_out
        c, r = m.latent(x)
        kda.latent_append(c, r, self.cache, self.cache_dtype, self._slots(seq, pos))
        # (the cached rows, this chunk's among them: what later steps will see)
        c, r = kda.latent_gather(self.cache, self.cache_dtype, self.table, cu_k_host)
        k, v = m.expand(c)
        q = (x @ m.lat_q).view(-1, m.H, DN + DR)
        o, _ = kda.latent_prefill(q, k, v, r, cu_host, cu_k_host, m.scale)
        x = x + o.flatten(1) @ m.lat_out
        self.lens = total.to(dev)
        return m.probs(x[cu_host[1:].to(dev).long() - 1])

    def step(self, last, drafts, draft_probs, u_accept, u_sample):
        """One speculative step: last [N] and drafts [N, K] enter, and the sequences advance by the
        accepted drafts and one drawn token.  Returns (tokens [N, K + 1], num_tokens [N])."""
        m = self.m
        N, K = drafts.shape
        K1 = K + 1
        if N != self.N:
            raise ValueError(f"{self.N} sequences, got the drafts of {N}")
        self._take(K1)
        ids = torch.cat([last[:, None], drafts], dim=1)
        x = m.embed[ids.long()].view(N * K1, m.M)
        kin = [t.view(N, K1, *t.shape[1:]) for t in m.kda_inputs(x)]
        o = torch.empty(N, K1, m.H, 128, device=x.device, dtype=torch.bfloat16)
        kda.kda_decode_multi(*kin, self.state, N, None, None, 0, o, kda.KDA_OUT_BF16, N, K1, m.H, 128, 128)
        x = x + o.flatten(2).view(N * K1, -1) @ m.kda_out
        c, r = m.latent(x)
        pos = self.lens.long()[:, None] + torch.arange(K1, device=x.device)
        seq = torch.arange(N, device=x.device)[:, None].expand(N, K1)
        kda.latent_append(c, r, self.cache, self.cache_dtype, self._slots(seq, pos).reshape(-1))
        q = m.absorb((x @ m.lat_q).view(N, K1, m.H, DN + DR))
        o, _ = kda.latent_decode(q, self.cache, self.cache_dtype, self.table, self.lens + K1, m.scale)
        o = torch.einsum("nkhc,hcd->nkhd", o, m.lat_uv)
        x = x + o.flatten(2).view(N * K1, -1) @ m.lat_out
        p = m.probs(x).view(N, K1, m.V)
        tokens, num = kda.verify_draft(p, draft_probs, drafts, u_accept, u_sample)
        # commit: num_tokens counts the accepted drafts and the drawn token, which is as many of the
        # entered tokens (the last one and the accepted drafts) as the state moves by
        kda.kda_decode_multi(*kin, self.state, N, None, num, 1, o.new_empty(N, K1, m.H, 128), kda.KDA_OUT_BF16, N, K1,
                             m.H, 128, 128)
        self.lens = self.lens + num
        return tokens, num


def main(argv=None):
    ap = argparse.ArgumentParser()
    ap.add_argument("--seqs", type=int, default=8)
    ap.add_argument("--prompt", type=int, default=1000)
    ap.add_argument("--draft", type=int, default=3, help="drafted tokens a step")
    ap.add_argument("--steps", type=int, default=20)
    a = ap.parse_args(argv)
    build.build()
    g = torch.Generator(device="cuda").manual_seed(3)
    m = HybridModel()
    srv = HybridServer(m, a.seqs, a.prompt + (a.steps + 1) * (a.draft + 1))
    rand = lambda *s: torch.rand(*s, generator=g, device="cuda")
    prompts = [torch.randint(0, m.V, (max(1, a.prompt - 7 * n),), device="cuda", generator=g) for n in range(a.seqs)]
    p = srv.prompt(prompts)
    last = torch.multinomial(p, 1, generator=g)[:, 0].to(torch.int32)
    # a draft model that knows nothing of the text: the target's distribution after the prompt, blurred
    q = (0.5 * p + 0.5 / m.V)[:, None].expand(-1, a.draft, -1).contiguous()
    kept = 0
    torch.cuda.synchronize()
    t = time.perf_counter()
    for _ in range(a.steps):
        drafts = torch.multinomial(q.view(-1, m.V), 1, generator=g).view(a.seqs, a.draft).to(torch.int32)
        tokens, num = srv.step(last, drafts, q, rand(a.seqs, a.draft), rand(a.seqs))
        last = tokens.gather(1, (num - 1).long()[:, None])[:, 0]
        kept += int(num.sum())
    torch.cuda.synchronize()
    t = time.perf_counter() - t
    if kda.kda_device_status() != kda.KDA_OK:
        raise SystemExit("device status")
    print(f"{a.seqs} sequences, {a.steps} steps of {a.draft} drafted tokens: {kept} tokens in {t * 1e3:.1f} ms "
          f"({kept / a.steps / a.seqs:.2f} a step and sequence)")


if __name__ == "__main__":
    main()

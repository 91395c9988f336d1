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
  tree step the last token and a tree of drafted ones enter together: kda.decode_tree,
            kda.latent_append_rope (a node's place in the cache is not its position in the text),
            kda.latent_decode_tree, kda.verify_draft (a token drawn after each node; the path goes on
            while it is one of the node's children), kda.kda_decode_multi and kda.latent_append_rope
            (commit of the path), kda.token_logprobs.
A model with `rotary` turns its position parts: kda.latent_append_rope then stands wherever
kda.latent_append is written above.

  python -m kimi_delta_attention_06_gb300.hybrid_step [--seqs 8] [--prompt 1000] [--draft 3] [--steps 20]
                                                      [--branches 4] [--rotary 10000]
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
    """Random weights of a two-layer hybrid: H heads of 128, vocabulary V; position parts are rotated where the
    base of their frequencies, `rotary`, is not 0."""

    def __init__(self, vocab: int = 1024, width: int = 256, heads: int = 4, seed: int = 0, device="cuda", rotary: float = 0.0):
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
        # (pair i turns by position / rotary^(2 i / DR); angles of 0 leave the pairs as they are)
        self.rotary = rotary != 0.0
        pair = torch.arange(DR // 2, dtype=torch.float64) * 2 / DR
        self.inv_freq = (rotary ** -pair if self.rotary else torch.zeros_like(pair)).float().to(device)

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

    def logits(self, x):
        return _rms(x) @ self.embed.t().float() * 0.25

    def probs(self, x):
        return torch.softmax(self.logits(x), dim=-1)


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

    def _append(self, x, slots, pos, q=None):
        """Write the rows of hidden x [T, M] to the cache; where the model has positions, their keys are rotated, and so are
        the position parts of the queries q [T, H, DN + DR] where given, in place."""
        m = self.m
        c, r = m.latent(x)
        if not m.rotary:
            kda.latent_append(c, r, self.cache, self.cache_dtype, slots)
            return
        qr = None if q is None else q[..., DN:]
        kda.latent_append_rope(c, r, self.cache, self.cache_dtype, slots, pos.reshape(-1).to(torch.int32), m.inv_freq, qr, qr)

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
        q = (x @ m.lat_q).view(-1, m.H, DN + DR)
        self._append(x, self._slots(seq, pos), pos, q)
        # (the cached rows, this chunk's among them: what later steps will see)
        c, r = kda.latent_gather(self.cache, self.cache_dtype, self.table, cu_k_host)
        k, v = m.expand(c)
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
        pos = self.lens.long()[:, None] + torch.arange(K1, device=x.device)
        seq = torch.arange(N, device=x.device)[:, None].expand(N, K1)
        q = (x @ m.lat_q).view(N * K1, m.H, DN + DR)
        self._append(x, self._slots(seq, pos).reshape(-1), pos, q)
        q = m.absorb(q.view(N, K1, m.H, DN + DR))
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

    def step_tree(self, last, drafts, parents, u_sample, top: int = 0):
        """One speculative step over a tree: place 0 holds last [N], place 1 + j drafts[:, j] [N, K], whose parent is place
        parents[:, j] (in [0, j]; negative: no draft there).  A token is drawn after every node, with its u_sample
        [N, K + 1], so what is kept follows the target's distribution whatever the drafts are; siblings are distinct
        tokens (of equal ones the first counts).  Returns (tokens [N, K + 1]: the path's drawn tokens, then -1; num_tokens
        [N]; token_logprobs of `tokens` with `top` alternatives, [N, K + 1, ..] each)."""
        m = self.m
        N, K = drafts.shape
        K1 = K + 1
        if N != self.N:
            raise ValueError(f"{self.N} sequences, got the drafts of {N}")
        if parents.shape != drafts.shape or u_sample.shape != (N, K1):
            raise ValueError(f"parents [{N}, {K}] and u_sample [{N}, {K1}], got {list(parents.shape)} and {list(u_sample.shape)}")
        if K1 > kda.KDA_TREE_MAX_NODES:
            raise ValueError(f"a tree has at most {kda.KDA_TREE_MAX_NODES} nodes, got {K1}")
        self._take(K1)
        dev = last.device
        place = torch.arange(K1, device=dev)
        up = F.pad(torch.where(parents < 0, -2, parents), (1, 0), value=-1).to(torch.int32).contiguous()
        node = up >= -1
        ids = torch.where(node, torch.cat([last[:, None], drafts], dim=1), 0)
        # a node's depth: the length of its path, by jumps twice as far each time
        depth, jump = (up >= 0).long(), up.long().clamp(0, K1 - 1)
        for _ in range(K1.bit_length()):
            depth, jump = depth + depth.gather(1, jump), jump.gather(1, jump)
        x0 = m.embed[ids.long()].view(N * K1, m.M)
        kin = [t.view(N, K1, *t.shape[1:]) for t in m.kda_inputs(x0)]
        o = kda.decode_tree(*kin, self.state, up)
        x1 = x0 + o.flatten(2).view(N * K1, -1) @ m.kda_out
        seq = torch.arange(N, device=dev)[:, None].expand(N, K1)
        at = self.lens.long()[:, None] + place
        q = (x1 @ m.lat_q).view(N * K1, m.H, DN + DR)
        self._append(x1, torch.where(node, self._slots(seq, at), -1).view(-1), self.lens.long()[:, None] + depth, q)
        q = m.absorb(q.view(N, K1, m.H, DN + DR))
        o, _ = kda.latent_decode_tree(q, self.cache, self.cache_dtype, self.table, self.lens + K1, up, m.scale)
        o = torch.einsum("nkhc,hcd->nkhd", o, m.lat_uv)
        logits = m.logits(x1 + o.flatten(2).view(N * K1, -1) @ m.lat_out)
        none = torch.empty(N * K1, 0, device=dev)
        drawn, _ = kda.verify_draft(torch.softmax(logits, dim=-1)[:, None], None, none.to(torch.int32), none, u_sample.reshape(-1))
        drawn = drawn.view(N, K1)
        # the path: from each node to its child that holds the drawn token, K1 where there is none
        child = (up[:, None, :] == place[None, :, None]) & (ids[:, None, :] == drawn[:, :, None]) & (place > place[:, None])
        nxt = F.pad(torch.where(child, place, K1).amin(dim=2), (0, 1), value=K1)
        path = torch.zeros(N, K1, dtype=torch.long, device=dev)
        for i in range(1, K1):
            path[:, i] = nxt.gather(1, path[:, i - 1:i])[:, 0]
        on = path < K1
        num = on.sum(dim=1).to(torch.int32)
        path = torch.where(on, path, 0)
        # commit: the path's tokens move the state, and their cache rows take the places after the sequence
        rows = (seq * K1 + path).view(-1)
        kin = [t.flatten(0, 1)[rows].view(t.shape) for t in kin]
        kda.kda_decode_multi(*kin, self.state, N, None, num, 1, o.new_empty(N, K1, m.H, 128), kda.KDA_OUT_BF16, N, K1,
                             m.H, 128, 128)
        self._append(x1[rows], torch.where(on, self._slots(seq, at), -1).view(-1), at)
        tokens = torch.where(on, drawn.gather(1, path), -1)
        scores = kda.token_logprobs(logits[rows], tokens.view(-1), top)
        self.lens = self.lens + num
        return tokens, num, tuple(None if s is None else s.view(N, K1, *s.shape[1:]) for s in scores)


def main(argv=None):
    ap = argparse.ArgumentParser()
    ap.add_argument("--seqs", type=int, default=8)
    ap.add_argument("--prompt", type=int, default=1000)
    ap.add_argument("--draft", type=int, default=3, help="drafted tokens a step")
    ap.add_argument("--steps", type=int, default=20)
    ap.add_argument("--branches", type=int, default=1, help="chains of --draft tokens a step, which hang on the last token as a tree")
    ap.add_argument("--rotary", type=float, default=0.0, help="base of the rotary frequencies of the position parts (0: none)")
    a = ap.parse_args(argv)
    nodes = a.branches * a.draft
    if a.branches < 1 or a.branches > 1 and not 0 < nodes < kda.KDA_TREE_MAX_NODES:
        ap.error(f"--branches: a tree of 2 to {kda.KDA_TREE_MAX_NODES} nodes, the last token's among them")
    build.build()
    g = torch.Generator(device="cuda").manual_seed(3)
    m = HybridModel(rotary=a.rotary)
    srv = HybridServer(m, a.seqs, a.prompt + (a.steps + 1) * (nodes + 1))
    rand = lambda *s: torch.rand(*s, generator=g, device="cuda")
    prompts = [torch.randint(0, m.V, (max(1, a.prompt - 7 * n),), device="cuda", generator=g) for n in range(a.seqs)]
    p = srv.prompt(prompts)
    last = torch.multinomial(p, 1, generator=g)[:, 0].to(torch.int32)
    # a draft model that knows nothing of the text: the target's distribution after the prompt, blurred
    q = (0.5 * p + 0.5 / m.V)[:, None].expand(-1, a.draft, -1).contiguous()
    kept, lp = 0, 0.0
    places = torch.arange(a.draft * a.branches, device="cuda").view(a.draft, a.branches)      # level by level
    parents = F.pad(places[:-1] + 1, (0, 0, 1, 0)).view(1, -1).expand(a.seqs, -1).contiguous() if a.draft else None
    torch.cuda.synchronize()
    t = time.perf_counter()
    for _ in range(a.steps):
        if a.branches > 1:                                     # the branches of a level are distinct tokens
            drafts = torch.multinomial(q.view(-1, m.V), a.branches, generator=g).view(a.seqs, nodes).to(torch.int32)
            tokens, num, scores = srv.step_tree(last, drafts, parents, rand(a.seqs, nodes + 1))
            last = tokens.gather(1, (num - 1).long()[:, None])[:, 0]
            kept += int(num.sum())
            lp += float(scores[0].sum())                       # (places past the path count 0)
            continue
        drafts = torch.multinomial(q.view(-1, m.V), 1, generator=g).view(a.seqs, a.draft).to(torch.int32)
        tokens, num = srv.step(last, drafts, q, rand(a.seqs, a.draft), rand(a.seqs))
        last = tokens.gather(1, (num - 1).long()[:, None])[:, 0]
        kept += int(num.sum())
    torch.cuda.synchronize()
    t = time.perf_counter() - t
    if kda.kda_device_status() != kda.KDA_OK:
        raise SystemExit("device status")
    print(f"{a.seqs} sequences, {a.steps} steps of {nodes} drafted tokens: {kept} tokens in {t * 1e3:.1f} ms "
          f"({kept / a.steps / a.seqs:.2f} a step and sequence)" + (f", {lp / kept:.2f} a token's log probability" if a.branches > 1 else ""))


if __name__ == "__main__":
    main()

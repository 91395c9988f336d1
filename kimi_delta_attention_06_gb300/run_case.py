"""Run one KDA workload a few times through the C ABI (for profilers and quick timing).

  python -m kimi_delta_attention_06_gb300.run_case --what prefill --T 8192 [--H 32] [--D 128] [--reps 2]
  python -m kimi_delta_attention_06_gb300.run_case --what varlen [--H 32] [--D 128] [--reps 2]
      (prefill / varlen also take --decay channel|head|none: KDA, Gated DeltaNet, DeltaNet;
       prefill / varlen --segments P run kda_chunk_prefill_segmented(_ex) with P segments)
  python -m kimi_delta_attention_06_gb300.run_case --what decode --N 512 [--H 32] [--D 128] [--reps 2]
  python -m kimi_delta_attention_06_gb300.run_case --what decode_multi --N 512 --K 4 [--commit 1] [--reps 2]
  python -m kimi_delta_attention_06_gb300.run_case --what prep --T 145408 [--reps 2]     (input preparation)
  python -m kimi_delta_attention_06_gb300.run_case --what outnorm --T 145408 [--reps 2]  (output norm)
  python -m kimi_delta_attention_06_gb300.run_case --what latent_append --T 145408 [--cache e4m3] [--reps 2]
  python -m kimi_delta_attention_06_gb300.run_case --what latent_gather --T 145408 [--cache e4m3] [--reps 2]
  python -m kimi_delta_attention_06_gb300.run_case --what latent_decode --N 64 --T 16384 [--K 1] [--H 32] [--cache bf16]
      (absorbed latent attention of K tokens of N sequences of T cached tokens each, pages of 64)
  python -m kimi_delta_attention_06_gb300.run_case --what latent_prefill --T 8192 [--H 32]
  python -m kimi_delta_attention_06_gb300.run_case --what verify --N 256 --K 4 [--vocab 131072]

Inputs are the seeded synthetic tensors of workloads.py, generated on the GPU
(varlen: 16 packed sequences of log-uniform length, about 280k tokens).
Prints the CUDA-event time of each repetition and the median rate of the
repetitions after the first.
"""
from __future__ import annotations

import argparse

import torch

from . import build, kda, workloads


def latent_case(a, dev, stream):
    """The run, its description and its count of units for the latent and verification cases."""
    g = torch.Generator(device=dev).manual_seed(7)
    rn = lambda *s: torch.randn(*s, generator=g, device=dev).to(torch.bfloat16)
    if a.what == "verify":
        p = torch.softmax(torch.randn(a.N, a.K + 1, a.vocab, generator=g, device=dev) * 2, -1)
        q = torch.softmax(p[:, :a.K].log() + 0.5 * torch.randn(a.N, a.K, a.vocab, generator=g, device=dev), -1)
        x = torch.multinomial(q.view(-1, a.vocab), 1, generator=g).view(a.N, a.K).to(torch.int32)
        u, us = torch.rand(a.N, a.K, generator=g, device=dev), torch.rand(a.N, generator=g, device=dev)
        return (lambda: kda.verify_draft(p, q, x, u, us, stream=stream)), f"{a.N} sequences x {a.K} drafts of {a.vocab}", a.N
    if a.what == "latent_prefill":
        q, kv, r = rn(a.T, a.H, 192), rn(a.T, a.H, 256), rn(a.T, 64)
        cu = torch.tensor([0, a.T], dtype=torch.int32)
        cud = cu.to(dev)
        return (lambda: kda.latent_prefill(q, kv[..., :128], kv[..., 128:], r, cu, cu, 192 ** -0.5, cu_q=cud, cu_k=cud,
                                           stream=stream)), f"{a.T} tokens x {a.H} heads, causal", a.T
    dt = kda.KDA_CACHE_E4M3 if a.cache == "e4m3" else kda.KDA_CACHE_BF16
    n = a.N if a.what == "latent_decode" else 1
    per = -(-a.T // 64)
    table = torch.randperm(n * per, generator=g, device=dev).to(torch.int32).view(n, per)
    cache = kda.latent_cache(n * per, 64, dt, device=dev)
    t = torch.arange(a.T, device=dev)
    slots = (table.long()[:, t // 64] * 64 + t % 64).to(torch.int32)
    c, r = rn(a.T, 512), rn(a.T, 64)
    for i in range(n):
        kda.latent_append(c, r, cache, dt, slots[i], stream=stream)
    if a.what == "latent_append":
        return (lambda: kda.latent_append(c, r, cache, dt, slots[0], stream=stream)), f"{a.T} tokens, {a.cache}", a.T
    if a.what == "latent_gather":
        cu = torch.tensor([0, a.T], dtype=torch.int32)
        cud = cu.to(dev)
        return (lambda: kda.latent_gather(cache, dt, table, cu, cu_seqlens=cud, stream=stream)), f"{a.T} tokens, {a.cache}", a.T
    q = rn(n, a.K, a.H, 576)
    lens = torch.full((n,), a.T, dtype=torch.int32, device=dev)
    return (lambda: kda.latent_decode(q, cache, dt, table, lens, 192 ** -0.5, stream=stream)), \
        f"{n} sequences of {a.T} cached tokens ({n * a.T * cache.shape[2] / 1e9:.3f} GB), {a.K} x {a.H} rows, {a.cache}", n * a.K


def main(argv=None):
    ap = argparse.ArgumentParser()
    ap.add_argument("--what", choices=["prefill", "varlen", "decode", "decode_multi", "prep", "outnorm", "latent_append",
                                       "latent_gather", "latent_decode", "latent_prefill", "verify"],
                    default="prefill")
    ap.add_argument("--cache", choices=["bf16", "e4m3"], default="e4m3", help="latent cache rows")
    ap.add_argument("--vocab", type=int, default=131072, help="verify: vocabulary size")
    ap.add_argument("--K", type=int, default=4, help="tokens per sequence (decode_multi, latent_decode), drafts (verify)")
    ap.add_argument("--commit", type=int, default=0, help="decode_multi: 1 writes the states back")
    ap.add_argument("--decay", choices=["channel", "head", "none"], default="channel",
                    help="prefill decay layout (per channel = KDA, per head = Gated DeltaNet, none = DeltaNet)")
    ap.add_argument("--T", type=int, default=8192)
    ap.add_argument("--N", type=int, default=512)
    ap.add_argument("--H", type=int, default=32)
    ap.add_argument("--D", type=int, default=128)
    ap.add_argument("--ckpt", type=int, default=32768)
    ap.add_argument("--reps", type=int, default=2)
    ap.add_argument("--segments", type=int, default=0, help="prefill: segments of kda_chunk_prefill_segmented")
    a = ap.parse_args(argv)
    build.build()
    dev = torch.device("cuda", 0)
    stream = torch.cuda.current_stream()
    if a.what in ("prefill", "varlen"):
        if a.what == "prefill":
            c = workloads.single_case(a.T, seed=2, device=dev, H=a.H, D=a.D, ckpt_stride=a.ckpt)
        else:
            c = workloads.varlen_case(device=dev, H=a.H, D=a.D, ckpt_stride=a.ckpt)
        T, N = c.T, c.N
        cu = c.cu_seqlens.to(dev)
        decay = {"channel": kda.KDA_DECAY_CHANNEL, "head": kda.KDA_DECAY_HEAD, "none": kda.KDA_DECAY_NONE}[a.decay]
        la = {kda.KDA_DECAY_CHANNEL: c.log_alpha, kda.KDA_DECAY_HEAD: c.log_alpha[:, :, 0].contiguous(),
              kda.KDA_DECAY_NONE: None}[decay]
        out = torch.empty(T, a.H, a.D, device=dev, dtype=torch.bfloat16)
        fin = torch.empty(N, a.H, a.D, a.D, device=dev)
        nck = kda.kda_ckpt_count(c.cu_seqlens, a.ckpt)
        ck = torch.empty(max(nck, 1), a.H, a.D, a.D, device=dev)

        def run():
            if a.segments > 0 and a.what == "varlen":
                kda.kda_chunk_prefill_segmented_ex(c.q, c.k, c.v, la, c.beta, c.init_state, c.cu_seqlens, N, T, a.H,
                                                   a.D, a.D, out, kda.KDA_OUT_BF16, fin, ck if nck else None, a.ckpt,
                                                   decay, None, a.segments, stream=stream)
            elif a.segments > 0 and a.what == "prefill":
                kda.kda_chunk_prefill_segmented(c.q, c.k, c.v, la, c.beta, c.init_state, T, a.H, a.D, a.D, out,
                                                kda.KDA_OUT_BF16, fin, ck if nck else None, a.ckpt, decay, 0,
                                                a.segments, stream=stream)
            else:
                kda.kda_chunk_prefill_ex(c.q, c.k, c.v, la, c.beta, c.init_state, cu, c.cu_seqlens, N, T, a.H,
                                         a.D, a.D, out, kda.KDA_OUT_BF16, fin, ck if nck else None, a.ckpt, decay,
                                         stream=stream)
        units, count = f"{T} tokens, {N} sequences, decay {a.decay}, segments {a.segments}", T
    elif a.what in ("prep", "outnorm"):
        g = torch.Generator(device=dev).manual_seed(6)
        T, H, D = a.T, a.H, a.D
        cu_host = torch.tensor([0, T], dtype=torch.int32)
        cu = cu_host.to(dev)
        if a.what == "prep":
            xs = [torch.randn(T, H, D, generator=g, device=dev).to(torch.bfloat16) for _ in range(3)]
            w = torch.randn(3, H, D, 4, generator=g, device=dev) * 0.5
            ar = torch.randn(T, H, D, generator=g, device=dev) - 2.0
            br = torch.randn(T, H, generator=g, device=dev).to(torch.bfloat16)
            outs = [torch.empty(T, H, D, device=dev, dtype=torch.bfloat16) for _ in range(3)]
            la = torch.empty(T, H, D, device=dev)
            be = torch.empty(T, H, device=dev, dtype=torch.bfloat16)

            def run():
                kda.kda_prepare_inputs(xs[0], xs[1], xs[2], w, None, ar, br, cu, cu_host, 1, T, H, D, 1,
                                       outs[0], outs[1], outs[2], la, be, stream)
            nbytes = T * H * (3 * 2 * D + 4 * D + 2) * 2          # read and write the same bytes
        else:
            o = torch.randn(T, H, D, generator=g, device=dev).to(torch.bfloat16)
            gam = torch.rand(H, D, generator=g, device=dev) + 0.5
            y = torch.empty_like(o)

            def run():
                kda.kda_output_norm(o, kda.KDA_OUT_BF16, gam, 1e-6, y, T, H, D, stream)
            nbytes = T * H * D * 2 * 2
        units, count = f"{T} tokens x {H} heads ({nbytes / 1e9:.3f} GB moved)", T
    elif a.what.startswith("latent") or a.what == "verify":
        run, units, count = latent_case(a, dev, stream)
    elif a.what == "decode_multi":
        d = workloads.decode_case(N=a.N, H=a.H, D=a.D, steps=a.K, seed=4, device=dev)
        tok = {key: torch.stack([s[key] for s in d.steps], dim=1).contiguous()
               for key in ("q", "k", "v", "log_alpha", "beta")}
        out = torch.empty(a.N, a.K, a.H, a.D, device=dev, dtype=torch.bfloat16)

        def run():
            kda.kda_decode_multi(tok["q"], tok["k"], tok["v"], tok["log_alpha"], tok["beta"], d.state, a.N, None,
                                 None, a.commit, out, kda.KDA_OUT_BF16, a.N, a.K, a.H, a.D, a.D, stream=stream)
        units, count = f"{a.N} sequences x {a.K} tokens, commit={a.commit}", a.N * a.K
    else:
        d = workloads.decode_case(N=a.N, H=a.H, D=a.D, steps=1, seed=4, device=dev)
        s = d.steps[0]
        out = torch.empty(a.N, a.H, a.D, device=dev, dtype=torch.bfloat16)

        def run():
            kda.kda_decode_step(s["q"], s["k"], s["v"], s["log_alpha"], s["beta"], d.state, out,
                                kda.KDA_OUT_BF16, a.N, a.H, a.D, a.D, stream)
        units, count = f"{a.N} sequences", a.N
    times = []
    for i in range(a.reps):
        e0 = torch.cuda.Event(enable_timing=True)
        e1 = torch.cuda.Event(enable_timing=True)
        e0.record(stream)
        run()
        e1.record(stream)
        torch.cuda.synchronize()
        times.append(e0.elapsed_time(e1))
        print(f"{a.what} rep {i}: {times[-1]:.3f} ms ({units})")
    if len(times) > 1:
        med = sorted(times[1:])[(len(times) - 1) // 2]
        print(f"{a.what} median of reps 1..{len(times) - 1}: {med:.3f} ms = {count / med * 1e3:.4g} "
              f"{'sequences' if a.what == 'decode' else 'tokens'}/s")
    st = kda.kda_device_status()
    if st != 0:
        raise SystemExit(f"device status {st}")


if __name__ == "__main__":
    main()

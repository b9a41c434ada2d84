"""One draft-verify step of a small decoder on the block-FP8 operators.

Every sequence has some tokens in an E4M3 cache and k drafted tokens; the step
runs the k + 1 new tokens of all sequences through the layers and the head,
and verifies the drafts:

    fp8_rmsnorm_quant -> fp8_block_gemm (q, k, v) -> fp8_kv_append ->
    fp8_kv_attention -> fp8_act_quant -> fp8_block_gemm (out) ->
    fp8_rmsnorm_quant (adds the residual) -> fp8_block_gemm (gate, up) ->
    fp8_silu_mul_quant -> fp8_block_gemm (down)            per layer, then
    fp8_rmsnorm_quant -> fp8_block_gemm (vocabulary) -> verify_drafts

Weights are random and there is no positional encoding: the example shows the
calls, their buffers and a CUDA graph around them.

    python examples/verify_step.py                      # small, on cuda:0
    python examples/verify_step.py --hidden 5120 --mlp 8704 --heads 24 --kv-heads 4 \
        --layers 4 --vocab 151936 --batch 34 --drafts 2 --context 4096
"""
from __future__ import annotations

import argparse
import os
import sys
from dataclasses import dataclass

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from block_scaled_fp8_act_gb300 import fp8act  # noqa: E402


@dataclass
class Config:
    hidden: int = 512
    mlp: int = 1024
    heads: int = 8
    kv_heads: int = 2
    head_dim: int = 64
    layers: int = 2
    vocab: int = 1000
    batch: int = 3
    drafts: int = 2
    context: int = 100
    page: int = 16
    seed: int = 0


class Decoder:
    """Random block-FP8 weights, a paged cache per layer, and the buffers of a step of fixed shape."""

    def __init__(self, c: Config):
        self.c = c
        g = torch.Generator(device="cuda").manual_seed(c.seed)

        def linear(n, k):
            w = (torch.randn((n, k), device="cuda", generator=g) / k ** 0.5).bfloat16()
            return fp8act.fp8_weight_quant(w)

        def norm():
            return (1.0 + 0.1 * torch.randn(c.hidden, device="cuda", generator=g)).bfloat16()

        width = c.heads * c.head_dim
        self.kv_width = c.kv_heads * c.head_dim
        self.layers = [{"norm1": norm(), "qkv": linear(width + 2 * self.kv_width, c.hidden),
                        "out": linear(c.hidden, width), "norm2": norm(), "gate_up": linear(2 * c.mlp, c.hidden),
                        "down": linear(c.hidden, c.mlp)} for _ in range(c.layers)]
        self.norm, self.head = norm(), linear(c.vocab, c.hidden)
        self.embed = torch.randn((c.vocab, c.hidden), device="cuda", generator=g).bfloat16()

        n = c.drafts + 1
        per = -(-(c.context + n) // c.page)
        pages = c.batch * per
        self.table = torch.randperm(pages, device="cuda", generator=g).view(c.batch, per).to(torch.int32)
        self.caches = [fp8act.kv_cache(pages, c.kv_heads, c.page, c.head_dim) for _ in range(c.layers)]
        self.cu_q = torch.arange(c.batch + 1, device="cuda", dtype=torch.int32) * n
        self.kv_lens = torch.full((c.batch,), c.context + n, device="cuda", dtype=torch.int32)
        at = torch.arange(c.context + n, device="cuda")
        slots = self.table[:, at // c.page].long() * c.page + at % c.page  # of every position
        self.slots = slots[:, c.context:].reshape(-1).contiguous()
        for cache in self.caches:  # what earlier steps cached
            kv = torch.randn((2, c.batch * c.context, c.kv_heads, c.head_dim), device="cuda", generator=g).bfloat16()
            fp8act.fp8_kv_append(kv[0], kv[1], slots[:, :c.context].reshape(-1).contiguous(), cache)
        self.workspace = torch.empty(fp8act.kv_attention_workspace(n, c.heads, self.caches[0]), dtype=torch.uint8,
                                     device="cuda")

    def logits(self, tokens: torch.Tensor) -> torch.Tensor:
        """bf16 [batch, drafts + 1, vocab] of the new tokens int64 [batch, drafts + 1]."""
        c, n = self.c, tokens.shape[1]
        x, residual = self.embed[tokens.reshape(-1)], None
        width = c.heads * c.head_dim
        for w, cache in zip(self.layers, self.caches):
            if residual is None:
                q, sa, residual = *fp8act.fp8_rmsnorm_quant(x, w["norm1"]), x
            else:
                q, sa, residual = fp8act.fp8_rmsnorm_quant(x, w["norm1"], residual=residual)
            qkv = fp8act.fp8_block_gemm(q, sa, *w["qkv"])
            heads = qkv[:, :width].unflatten(1, (c.heads, c.head_dim))
            k, v = (t.unflatten(1, (c.kv_heads, c.head_dim)) for t in qkv[:, width:].split(self.kv_width, 1))
            fp8act.fp8_kv_append(k, v, self.slots, cache)
            o = fp8act.fp8_kv_attention(heads, cache, self.table, self.kv_lens, self.cu_q, max_q_len=n,
                                        workspace=self.workspace)
            x = fp8act.fp8_block_gemm(*fp8act.fp8_act_quant(o.view(-1, width)), *w["out"])
            q, sa, residual = fp8act.fp8_rmsnorm_quant(x, w["norm2"], residual=residual)
            q, sa = fp8act.fp8_silu_mul_quant(fp8act.fp8_block_gemm(q, sa, *w["gate_up"]))
            x = fp8act.fp8_block_gemm(q, sa, *w["down"])
        q, sa, _ = fp8act.fp8_rmsnorm_quant(x, self.norm, residual=residual)
        return fp8act.fp8_block_gemm(q, sa, *self.head).view(c.batch, n, c.vocab)

    def step(self, last, drafts, draft_logits, uniform, noise, temperature):
        """Verify drafts int32 [batch, k] after the tokens `last` int32 [batch]: (accepted, tokens, accept_prob, logits)."""
        logits = self.logits(torch.cat([last.unsqueeze(1), drafts], 1).long())
        return *fp8act.verify_drafts(logits, drafts, uniform, noise, temperature, draft_logits=draft_logits), logits


def inputs(c: Config, seed: int):
    """Last tokens, drafts with the logits they were drawn from, random numbers, temperatures."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    last = torch.randint(0, c.vocab, (c.batch,), device="cuda", generator=g).to(torch.int32)
    draft_logits = torch.randn((c.batch, c.drafts, c.vocab), device="cuda", generator=g).bfloat16()
    race = torch.empty(draft_logits.shape, device="cuda").exponential_(generator=g)
    drafts = (draft_logits.float().softmax(-1) / race).argmax(-1).to(torch.int32)
    uniform = torch.rand((c.batch, c.drafts), device="cuda", generator=g)
    noise = torch.empty((c.batch, c.vocab), device="cuda").exponential_(generator=g).clamp_(min=1e-20)
    return last, drafts, draft_logits, uniform, noise, torch.ones(c.batch, device="cuda")


def main() -> None:
    p = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    for f in Config.__dataclass_fields__.values():
        p.add_argument("--" + f.name.replace("_", "-"), type=int, default=f.default)
    p.add_argument("--steps", type=int, default=20)
    a = vars(p.parse_args())
    steps = a.pop("steps")
    c = Config(**a)
    fp8act.load(build=True)
    decoder = Decoder(c)
    state = inputs(c, c.seed + 1)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        decoder.step(*state)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        accepted, tokens, prob, _ = decoder.step(*state)
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    graph.replay()
    start.record()
    for _ in range(steps):
        graph.replay()
    end.record()
    torch.cuda.synchronize()
    assert fp8act.check_status() == 0
    print(f"{start.elapsed_time(end) / steps * 1e3:.1f} us a step of {c.batch} x {c.drafts + 1} tokens, "
          f"{c.layers} layers, {c.context} cached tokens a sequence")
    print("accepted", accepted.tolist(), "mean acceptance probability", round(float(prob.mean()), 3))
    print("tokens", tokens.tolist()[:4])


if __name__ == "__main__":
    main()

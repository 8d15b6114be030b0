"""A prompt and decode steps through a whole decoder layer: attention over a paged
cache and the routed-expert feed-forward, with the norms round both blocks.

    python examples/decoder_layer.py        # a small layer on cuda:0, a prompt and a few tokens

Per token, with x the residual stream (fp32), all on one stream and without a
host synchronisation:

    h  = rms(x; w_in)                                  BlockNorm
    q, k, v = h W_qkv                                  Linear
    norm the heads of q and k (head_norm), rotate both
    by the position, cache k and v                     KVCache.append
    o  = attention over the cache                      KVCache.attend
    x  = x + rms(o W_o; w_attn_out); h = rms(x; w_mid) Linear, BlockNorm
    y  = routed experts + shared expert of h           MoELayer.decode
    x  = x + rms(y; w_moe_out); h = rms(x; w_next)     BlockNorm

The last norm's output is the next layer's input. A prompt goes the same way in chunks
(prefill), with KVCache.attend_chunk and MoELayer.prefill_chunk.
"""
from __future__ import annotations

import os
import sys

import numpy as np
import torch

if __name__ == "__main__":
    sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import quantized_routed_expert_moe_gb300 as moe
import seeded_inputs as si


class DecoderLayer:
    """One decoder layer for one sequence. ``layer`` is a canonical MoE layer
    (as MoELayer takes it) with bf16 activations; the attention weights are seeded."""

    def __init__(self, layer, n_heads: int, n_kv_heads: int, head_dim: int, max_tokens: int, page_size: int = 16,
                 cache=torch.bfloat16, seed: int = 0, device: str = "cuda:0", head_norm: bool = False, max_chunk: int = 1):
        H = layer.spec.hidden
        g = torch.Generator(device=device).manual_seed(seed)

        def randn(*shape, scale=1.0):
            return torch.randn(*shape, generator=g, device=device) * scale
        self.heads, self.kv_heads, self.d = n_heads, n_kv_heads, head_dim
        bf16 = torch.bfloat16
        self.w_qkv = randn((n_heads + 2 * n_kv_heads) * head_dim, H, scale=H ** -0.5).to(bf16)
        self.w_o = randn(H, n_heads * head_dim, scale=(n_heads * head_dim) ** -0.5).to(bf16)
        w = [1 + 0.1 * randn(H) for _ in range(5)]   # w_in, w_attn_out, w_mid, w_moe_out, w_next
        self.first = moe.BlockNorm(H, w_pre=w[0])
        self.after_attention = moe.BlockNorm(H, w_post=w[1], w_pre=w[2])
        self.after_experts = moe.BlockNorm(H, w_post=w[3], w_pre=w[4])
        self.qkv_proj, self.o_proj = moe.Linear(self.w_qkv), moe.Linear(self.w_o)
        self.q_norm, self.k_norm = [1 + 0.1 * randn(head_dim) for _ in range(2)] if head_norm else (None, None)
        self.experts = moe.MoELayer(layer, max_tokens=max_chunk)
        # pages in an order of their own, as an allocator that serves many sequences would give them
        n_pages = -(-max_tokens // page_size)
        self.table = torch.randperm(n_pages, generator=g, device=device).to(torch.int32)[None]
        pages = torch.zeros(2, n_pages, n_kv_heads, page_size, head_dim, device=device, dtype=bf16).to(cache)
        scale = None if cache is bf16 else np.full(n_kv_heads, 8 / 448, np.float32)
        self.kv = moe.KVCache(pages[0], pages[1], n_heads=n_heads, k_scale=scale, v_scale=scale,
                              inv_freq=np.array([10000.0 ** (-2.0 * i / head_dim) for i in range(head_dim // 2)]))
        self.position = torch.zeros(1, dtype=torch.int32, device=device)
        self.length = torch.zeros(1, dtype=torch.int32, device=device)
        self.one_chunk = torch.arange(2, dtype=torch.int32, device=device)   # times its tokens: where it starts and ends
        # buffers of a step: a caller that serves tokens allocates nothing
        self.h, self.h_mid, self.h_next = (torch.empty(1, H, device=device, dtype=bf16) for _ in range(3))
        self.q_rot, self.o = (torch.empty(1, n_heads, head_dim, device=device, dtype=bf16) for _ in range(2))
        self.y = torch.empty(H, device=device, dtype=bf16)
        self.qkv = torch.empty(1, self.w_qkv.shape[0], device=device, dtype=bf16)
        self.attn = torch.empty(1, H, device=device, dtype=bf16)

    def step(self, x, stream=None):
        """One token: x [1, H] fp32 residual, updated in place; returns the next layer's
        input [1, H] bf16. Nothing is read back to the host. All of it runs on one stream,
        torch's current one by default; x has to be ready there."""
        with torch.cuda.stream(torch.cuda.current_stream() if stream is None else stream):
            self.length.add_(1)
            self.first.run(x, h=self.h)
            self.qkv_proj.run(self.h, self.qkv)
            self.q, self.k, self.v = self.qkv.view(1, -1, self.d).split([self.heads, self.kv_heads, self.kv_heads], 1)
            self.kv.append(self.q, self.k, self.v, self.position, self.table, self.q_rot, q_norm=self.q_norm,
                           k_norm=self.k_norm)
            self.kv.attend(self.q_rot, self.table, self.length, self.o)
            self.o_proj.run(self.o.view(1, -1), self.attn)
            self.after_attention.run(x, self.attn, x, self.h_mid)
            self.experts.decode(self.h_mid, self.y, stream=torch.cuda.current_stream())
            self.after_experts.run(x, self.y[None], x, self.h_next)
            self.position.add_(1)
        return self.h_next

    def prefill(self, x, stream=None):
        """A chunk of a prompt, at most max_chunk tokens: x [T, H] fp32 residual, updated in
        place; returns the next layer's input [T, H] bf16. Chunks follow one another and come
        before the steps that continue them. As for a step, all of it runs on one stream,
        without a host synchronisation; what it returns is that stream's."""
        with torch.cuda.stream(torch.cuda.current_stream() if stream is None else stream):
            T, H = x.shape

            def new(*shape):
                return torch.empty(*shape, device=x.device, dtype=torch.bfloat16)
            h, h_mid, h_next, attn, y = (new(T, H) for _ in range(5))
            qkv, q_rot, o = new(T, self.w_qkv.shape[0]), new(T, self.heads, self.d), new(T, self.heads, self.d)
            positions = self.position + torch.arange(T, dtype=torch.int32, device=x.device)
            self.length.add_(T)
            self.first.run(x, h=h)
            self.qkv_proj.run(h, qkv)
            q, k, v = qkv.view(T, -1, self.d).split([self.heads, self.kv_heads, self.kv_heads], 1)
            self.kv.append(q, k, v, positions, self.table, q_rot, seq=torch.zeros_like(positions), q_norm=self.q_norm,
                           k_norm=self.k_norm)
            self.kv.attend_chunk(q_rot, self.one_chunk * T, self.table, self.length, o)
            self.o_proj.run(o.view(T, -1), attn)
            self.after_attention.run(x, attn, x, h_mid)
            self.experts.prefill_chunk(h_mid, T, y, stream=torch.cuda.current_stream())
            self.after_experts.run(x, y, x, h_next)
            self.position.add_(T)
        # what the chunk went through, for who wants to look
        self.chunk = dict(h=h, q=q, k=k, v=v, q_rot=q_rot, o=o, attn=attn, h_mid=h_mid, y=y)
        return h_next

    def close(self):
        self.experts.close()
        self.kv.close()


def main(tokens: int = 20):
    spec = si.LayerSpec(hidden=512, inter=256, n_experts=32, top_k=8)   # bf16 activations
    prompt = 48
    layer = DecoderLayer(si.gen_layer(0, 0, spec), n_heads=8, n_kv_heads=2, head_dim=64, max_tokens=prompt + tokens,
                         head_norm=True, max_chunk=32)
    x = torch.randn(prompt, spec.hidden, device="cuda:0", generator=torch.Generator("cuda:0").manual_seed(2))
    for chunk in x.split(32):
        h = layer.prefill(chunk)
        print(f"{len(chunk)} tokens of the prompt: next input of the last {h[-1, :3].float().tolist()}")
    x = torch.randn(1, spec.hidden, device="cuda:0", generator=torch.Generator("cuda:0").manual_seed(1))
    for t in range(tokens):
        h = layer.step(x)
        print(f"token {t}: residual rms {float(x.square().mean().sqrt()):.4f}, next input {h[0, :3].float().tolist()}")
    status, bits = layer.kv.health()
    assert status == 0, bits
    layer.close()


if __name__ == "__main__":
    main()

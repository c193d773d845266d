"""One decode step of a transformer block around the MoE layer, on one GPU.

    python examples/decode_block.py [--batch 4] [--steps 16] [--layers 2] [--cache bf16|nvfp4]

Every layer runs, for the next token of each sequence of a batch,

    qkv   = W_qkv x                                   nvfp4_linear
    q, cache <- rotary(q), rotary(k), v               kv_append
    a     = attention(q, cache)                       paged_decode_attention
    y     = W_o a                                     nvfp4_linear
    r, x  = r + s * norm(y), norm(r)                  residual_norm
    y     = MoE(x)                                    router_logits, decode_routed
    r, x  = r + s * gate * norm(y), norm(r)           residual_norm

and the last x gives the next-token logits (nvfp4_linear, float32). The step reads positions and
lengths from device tensors, so one CUDA graph serves every step. With --cache nvfp4 the keys and
values are kept in four bits. The weights are random: the program shows the calls, their order and
their buffers.
"""
from __future__ import annotations

import argparse
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402

from nvfp4_mixture_experts_02_gb300 import ftmoe  # noqa: E402

EPS = 1e-6
KV_GSCALE = 0.005   # of a four-bit cache: block scales up to 448 reach magnitudes of 6 * 448 * 0.005 = 13


class Layer:
    """The weights of one block (NvFP4Linear and NvFP4Experts objects, bf16 vectors)."""

    def __init__(self, w_qkv, w_o, w_router, experts, attn_post, moe_pre, moe_post, moe_gate, next_pre,
                 k, shared=None):
        self.w_qkv, self.w_o, self.w_router, self.experts = w_qkv, w_o, w_router, experts
        self.attn_post, self.moe_pre = attn_post, moe_pre
        self.moe_post, self.moe_gate, self.next_pre = moe_post, moe_gate, next_pre
        self.k, self.shared = k, shared


class DecodeStep:
    """The step's buffers for `batch` sequences; `step(x_in)` runs it on the current stream."""

    def __init__(self, layers, caches, table, rope, Hq, first_pre, w_logits, batch, scale=1.0):
        dev, H = first_pre.device, first_pre.shape[0]
        Hkv, D = caches[0].heads
        bf, f32 = dict(dtype=torch.bfloat16, device=dev), dict(dtype=torch.float32, device=dev)
        self.layers, self.caches, self.table, self.rope = layers, caches, table, rope
        self.Hq, self.Hkv, self.D, self.scale = Hq, Hkv, D, scale
        self.first_pre, self.w_logits = first_pre, w_logits
        self.positions = torch.zeros(batch, dtype=torch.int32, device=dev)
        self.lengths = torch.ones(batch, dtype=torch.int32, device=dev)
        self.x, self.r = torch.empty((batch, H), **bf), torch.empty((batch, H), **f32)
        self.qkv = torch.empty((batch, Hq + 2 * Hkv, D), **bf)
        self.q, self.a = torch.empty((batch, Hq, D), **bf), torch.empty((batch, Hq, D), **bf)
        self.lse = torch.empty((batch, Hq), **f32)
        self.y = torch.empty((batch, H), **bf)
        self.logits = torch.empty((batch, w_logits.N), **f32)
        # one workspace for all of the step's calls: its flags can be read after a replay of the captured step
        sizes = [ftmoe.paged_attention_workspace_bytes(batch, D)]
        for layer in layers:
            e = layer.experts
            sizes.append(ftmoe.workspace_bytes(batch, layer.k, e.E, e.H, e.I, layer.shared is not None))
            sizes += [ftmoe.nvfp4_linear_workspace_bytes(batch, w.K) for w in (layer.w_qkv, layer.w_o, w_logits)]
        self.workspace = torch.zeros(max(sizes), dtype=torch.uint8, device=dev)

    def step(self, x_in):
        """x_in bf16 [batch, H], the new tokens' embeddings -> logits f32 [batch, N]; positions and
        lengths advance."""
        Hq, Hkv, ws = self.Hq, self.Hkv, self.workspace
        # the residual stream begins as the embedding, in float32
        ftmoe.residual_norm(x_in, None, w_pre=self.first_pre, eps=EPS, res_out=self.r, x_out=self.x)
        for layer, cache in zip(self.layers, self.caches):
            qkv = self.qkv
            ftmoe.nvfp4_linear(self.x, layer.w_qkv, out=qkv.view(qkv.shape[0], -1), workspace=ws)
            q, k, v = qkv.split([Hq, Hkv, Hkv], 1)
            ftmoe.kv_append(k, v, cache, self.table, self.positions, q=q, rope=self.rope, q_out=self.q,
                            workspace=ws)
            ftmoe.paged_decode_attention(self.q, cache, self.table, self.lengths, out=self.a, lse=self.lse,
                                         workspace=ws)
            ftmoe.nvfp4_linear(self.a.view(self.a.shape[0], -1), layer.w_o, out=self.y, workspace=ws)
            ftmoe.residual_norm(self.y, self.r, w_post=layer.attn_post, w_pre=layer.moe_pre,
                                scale=self.scale, eps=EPS, res_out=self.r, x_out=self.x)
            scores, _ = ftmoe.router_logits(self.x, layer.w_router)
            ftmoe.decode_routed(self.x, scores, layer.k, layer.experts, layer.shared, out=self.y,
                                workspace=ws)
            ftmoe.residual_norm(self.y, self.r, w_post=layer.moe_post, w_pre=layer.next_pre,
                                gate=layer.moe_gate, scale=self.scale, eps=EPS, res_out=self.r,
                                x_out=self.x)
        ftmoe.nvfp4_linear(self.x, self.w_logits, out=self.logits, workspace=ws)
        self.positions.add_(1)
        self.lengths.add_(1)
        return self.logits


def rotary_table(rows, dim, device):
    inv = 10000.0 ** (-torch.arange(0, dim, 2, dtype=torch.float64) / dim)
    angle = torch.arange(rows, dtype=torch.float64)[:, None] * inv
    return torch.cat([angle.cos(), angle.sin()], 1).float().to(device)


def random_matrix(N, K, device):
    """Random codes under block scales around 2^-6: entries of about 1/sqrt(K) at K = 1024."""
    codes = torch.randint(0, 256, (N, K // 2), dtype=torch.uint8, device=device)
    scales = torch.randint(0x28, 0x38, (N, K // 16), dtype=torch.uint8, device=device)
    return ftmoe.NvFP4Linear(codes, scales, torch.full((1,), 0.03, device=device))


def random_model(batch, n_layers, device, H=1024, Hq=8, Hkv=2, D=128, E=16, k=4, I=512, vocabulary=1000,
                 page=16, room=256, cache="bf16"):
    ones = lambda: torch.ones(H, dtype=torch.bfloat16, device=device)  # noqa: E731
    byte = lambda *s: torch.randint(0, 256, s, dtype=torch.uint8, device=device)  # noqa: E731
    block = lambda *s: torch.randint(0x28, 0x38, s, dtype=torch.uint8, device=device)  # noqa: E731
    g = torch.full((E,), 0.03, device=device)
    layers, caches = [], []
    width = room // page
    table = torch.randperm(batch * width, device=device).to(torch.int32).view(batch, width)
    for _ in range(n_layers):
        experts = ftmoe.NvFP4Experts(byte(E, 2 * I, H // 2), block(E, 2 * I, H // 16), g,
                                     byte(E, H, I // 2), block(E, H, I // 16), g)
        layers.append(Layer(random_matrix((Hq + 2 * Hkv) * D, H, device), random_matrix(H, Hq * D, device),
                            (0.03 * torch.randn(E, H, device=device)).bfloat16(), experts, ones(), ones(),
                            ones(), ones(), ones(), k))
        pool = lambda w, t: torch.zeros((batch * width, page, Hkv, w), dtype=t, device=device)  # noqa: E731
        if cache == "nvfp4":
            codes, scales = (lambda: pool(D // 2, torch.uint8)), (lambda: pool(D // 16, torch.uint8))
            caches.append(ftmoe.NvFP4KVCache(codes(), codes(), scales(), scales(), KV_GSCALE, KV_GSCALE))
        else:
            caches.append(ftmoe.PagedKVCache(pool(D, torch.bfloat16), pool(D, torch.bfloat16)))
    return DecodeStep(layers, caches, table, rotary_table(room, D, device), Hq, ones(),
                      random_matrix(vocabulary, H, device), batch, scale=0.5)


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--batch", type=int, default=4)
    ap.add_argument("--steps", type=int, default=16)
    ap.add_argument("--layers", type=int, default=2)
    ap.add_argument("--cache", choices=("bf16", "nvfp4"), default="bf16")
    args = ap.parse_args()
    device = torch.device("cuda")
    torch.manual_seed(0)
    model = random_model(args.batch, args.layers, device, cache=args.cache)
    embedding = torch.randn(1000, model.x.shape[1], device=device).bfloat16()
    x_in = embedding[:args.batch].clone()
    model.step(x_in)   # one eager step before the capture: per-device set-up
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        tokens = model.step(x_in).argmax(1)
        x_in.copy_(embedding[tokens])
    begin, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    torch.cuda.synchronize()
    begin.record()
    for _ in range(args.steps):
        graph.replay()
    end.record()
    torch.cuda.synchronize()
    assert ftmoe.get_error(model.workspace) == 0
    print(f"{args.steps} steps of {args.layers} layers for {args.batch} sequences: "
          f"{begin.elapsed_time(end) / args.steps * 1e3:.1f} us a step, last tokens {tokens.tolist()}")


if __name__ == "__main__":
    main()

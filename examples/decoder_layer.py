"""A decoder layer of a mixture-of-experts model over the paged NVFP4 cache:
ragged prompts in one pass, then tokens one by one from a CUDA graph.

    python examples/decoder_layer.py

Per call: NVFP4 query/key/value projection, append (head norms, rotary
positions, quantization into the pages), attention over the cache, NVFP4 output
projection, then the router, the experts' two grouped products and the weighted
combine.  The weights are random; the norms around the two blocks are PyTorch's.
"""

import os
import sys
from dataclasses import dataclass

import torch
import torch.nn.functional as F

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import nvfp4_router_gate_gb300 as R  # noqa: E402

PAGE = 64


@dataclass
class Batch:
    """Where the rows of x belong: int32 tensors on the GPU."""
    positions: torch.Tensor     # [T] place of each token in its sequence
    slots: torch.Tensor         # [T] place of each token in the cache
    page_table: torch.Tensor    # [B, max_pages]
    kv_lens: torch.Tensor       # [B] tokens of each sequence, this call's included
    cu_q: torch.Tensor = None   # [B + 1] rows of each sequence (None: one each)
    max_q: int = None


class DecoderLayer:
    def __init__(self, dim=512, heads=16, kv_heads=2, head_dim=128, experts=16, top_k=4, inner=256, n_pages=256,
                 max_pos=4096, max_tokens=1024, max_seqs=16, seed=0):
        gen = torch.Generator(device="cuda").manual_seed(seed)

        def weight(*shape):
            return (torch.randn(*shape, generator=gen, device="cuda") * shape[-1] ** -0.5).bfloat16()

        self.heads, self.kv_heads, self.head_dim, self.top_k = heads, kv_heads, head_dim, top_k
        self.inner, self.max_tokens = inner, max_tokens
        self.qkv = R.Nvfp4Linear(weight((heads + 2 * kv_heads) * head_dim, dim), max_tokens, torch.bfloat16)
        self.proj = R.Nvfp4Linear(weight(dim, heads * head_dim), max_tokens, torch.bfloat16)
        self.q_norm, self.k_norm = torch.ones(2, head_dim, device="cuda").unbind()
        self.cos, self.sin = R.rope_table(max_pos, head_dim)
        # a normed head of `head_dim` channels has entries up to about 6; values are projections of normed rows
        self.kv = R.Nvfp4KVCache(n_pages, kv_heads, head_dim, PAGE, k_gsa=8.0 / 2688, v_gsa=8.0 / 2688, n_heads=heads,
                                 max_tokens=max_tokens, max_seqs=max_seqs)
        self.gate = R.RouterGate(weight(experts, dim), torch.zeros(experts), k=top_k, max_tokens=max_tokens)
        self.up = R.nvfp4_pack_experts(weight(experts, 2 * inner, dim))
        self.down = R.nvfp4_pack_experts(weight(experts, dim, inner))
        self.moe_ws = R.new_workspace(max(R.nvfp4_moe_gemm_workspace_size(max_tokens, dim, experts, top_k),
                                          R.nvfp4_moe_gemm_workspace_size(max_tokens * top_k, inner, experts, 1)))

    def attention(self, x, b):
        """The attention block's heads [T, heads, head_dim] for normed rows x, which join the cache."""
        T, H, KV = x.shape[0], self.heads, self.kv_heads
        qkv = self.qkv(x).view(T, H + 2 * KV, self.head_dim)
        q = self.kv.append(qkv[:, :H], qkv[:, H:H + KV], qkv[:, H + KV:], b.positions, b.slots, self.cos, self.sin,
                           q_weight=self.q_norm, k_weight=self.k_norm)
        return q, self.kv.attend(q, b.page_table, b.kv_lens, cu_q=b.cu_q, max_q=b.max_q)[0]

    def experts(self, x):
        T = x.shape[0]
        ids, w = self.gate(x)
        a, g = R.nvfp4_moe_gemm(x, ids, *self.up, out_dtype=torch.bfloat16, workspace=self.moe_ws).chunk(2, dim=-1)
        h = (F.silu(a) * g).reshape(T * self.top_k, self.inner)
        y = R.nvfp4_moe_gemm(h, ids.reshape(-1, 1), *self.down, out_dtype=torch.bfloat16, workspace=self.moe_ws)
        return R.nvfp4_moe_combine(y.view(T, self.top_k, -1), w).bfloat16()

    def __call__(self, x, b):
        heads = self.attention(F.rms_norm(x, x.shape[-1:]), b)[1]
        x = x + self.proj(heads.flatten(1))
        return x + self.experts(F.rms_norm(x, x.shape[-1:]))


class Sequences:
    """Pages of a few sequences, handed out in order; lengths on host and GPU."""

    def __init__(self, n, max_len):
        per = -(-max_len // PAGE)
        self.table = torch.arange(n * per, dtype=torch.int32, device="cuda").view(n, per).flip(0).contiguous()
        self.lens = torch.zeros(n, dtype=torch.int32, device="cuda")

    def place(self, seq, pos):
        return (self.table[seq.long(), (pos // PAGE).long()] * PAGE + pos % PAGE).int()

    def prompts(self, n_q):
        """The batch that adds n_q[b] tokens to sequence b."""
        n = torch.tensor(n_q, dtype=torch.int32, device="cuda")
        cu = F.pad(n.cumsum(0), (1, 0)).int()
        seq = torch.repeat_interleave(torch.arange(len(n_q), device="cuda"), n.long())
        pos = (torch.arange(int(cu[-1]), device="cuda") - cu[seq] + self.lens[seq]).int()
        self.lens += n
        return Batch(pos, self.place(seq, pos), self.table, self.lens, cu, max(n_q))

    def step(self):
        """The batch that adds a token to every sequence; may be captured in a graph."""
        pos = self.lens.clone()
        slots = self.place(torch.arange(len(pos), device="cuda"), pos)
        self.lens += 1
        return Batch(pos, slots, self.table, self.lens)


def main(n_q=(300, 17, 128, 1), steps=8):
    layer, seqs = DecoderLayer(), Sequences(len(n_q), 512)
    x = torch.randn(sum(n_q), 512, device="cuda", dtype=torch.bfloat16)
    y = layer(x, seqs.prompts(list(n_q)))
    rows = y[torch.tensor(n_q).cumsum(0).cuda() - 1].clone()          # the last token of each prompt
    # a decode step: warmed up on a side stream with a copy of the lengths, captured, replayed
    before = seqs.lens.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        layer(rows, seqs.step())
    torch.cuda.current_stream().wait_stream(side)
    seqs.lens.copy_(before)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        rows.copy_(layer(rows, seqs.step()))
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    start.record()
    for _ in range(steps):
        graph.replay()
    end.record()
    end.synchronize()
    assert layer.kv.status() == 0 and layer.gate.status() == 0
    print("prompts of %s tokens, then %d steps of %d sequences: %.1f us a step, lengths %s" % (
        list(n_q), steps, len(n_q), 1e3 * start.elapsed_time(end) / steps, seqs.lens.tolist()))
    return layer, seqs, rows


if __name__ == "__main__":
    main()

"""One attention layer served from a paged cache, with the library's calls only.

    python examples/attention_serving.py

Projections (FP16 weights), prompts of different lengths attended to together,
their keys and values written to pages, each prompt forked into several
samples that share its full pages, a few tokens decoded for every sample, and
the samples' pages given back and the cache compacted.
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import compensated_fp32_projection_gb300 as cf  # noqa: E402

HIDDEN, HEADS, KV_HEADS, DIM, PAGE = 512, 8, 2, 64, 16


def ints(values, device):
    return torch.tensor(values, dtype=torch.int32, device=device)


class Layer:
    """y = W_o attention(W_q x, W_k x, W_v x): FP32 activations, FP16 weights."""

    def __init__(self, seed, device):
        g = torch.Generator().manual_seed(seed)
        width = (HEADS + 2 * KV_HEADS) * DIM
        self.w_qkv = (torch.randn(width, HIDDEN, generator=g) * HIDDEN ** -0.5).half().to(device)
        self.w_o = (torch.randn(HIDDEN, HEADS * DIM, generator=g) * 0.05).half().to(device)

    def qkv(self, x):
        """q, k and v as parts of one projection's output: strided, not copied."""
        y = cf.comp_gemm_f32x16_ws(x, self.w_qkv).view(x.shape[0], HEADS + 2 * KV_HEADS, DIM)
        return y[:, :HEADS], y[:, HEADS:HEADS + KV_HEADS], y[:, HEADS + KV_HEADS:]

    def out(self, attended):
        return cf.comp_gemm_f32x16_ws(attended.reshape(-1, HEADS * DIM), self.w_o)


class Cache:
    """Pages of keys and values and the tables that say whose they are."""

    def __init__(self, pages, rows, width, device):
        self.k, self.v = (torch.zeros(pages, KV_HEADS, PAGE, DIM, dtype=torch.float16, device=device)
                          for _ in range(2))
        self.table = torch.full((rows, width), -1, dtype=torch.int32, device=device)
        self.lengths = torch.zeros(rows, dtype=torch.int32, device=device)
        self.refs = torch.zeros(pages, dtype=torch.int32, device=device)

    def write(self, k, v, rows, cu=None):
        """New tokens of some rows: pages for them, then the tokens."""
        new = torch.ones_like(rows) if cu is None else cu[1:] - cu[:-1]
        want = self.lengths.index_add(0, rows, new)
        left = cf.comp_kv_reserve(self.table, want, self.refs, PAGE, self.table, self.refs)[2]
        cf.comp_kv_append_f32(k, v, self.k, self.v, self.table[rows].contiguous(), self.lengths[rows].contiguous(), cu)
        self.lengths.copy_(want)
        return left

    def fork(self, parents, children):
        return cf.comp_kv_fork(self.k, self.v, self.table, self.lengths, self.refs, parents, children, self.table,
                               self.lengths, self.refs)[3]

    def free(self, rows):
        cf.comp_kv_free(self.table, self.lengths, self.refs, rows, self.table, self.lengths, self.refs)

    def compact(self):
        return cf.comp_kv_compact(self.k, self.v, self.table, self.refs, self.table, self.refs)[3]


def serve(lens=(200, 57), samples=3, steps=5, seed=0, device="cuda"):
    """Returns what was computed: the prompts' outputs, each step's (its inputs
    too), free pages left after the forks, and pages in use before and after."""
    g = torch.Generator().manual_seed(seed)
    layer, cache = Layer(seed, device), Cache(256, len(lens) * (samples + 1), 32, device)
    prompts = torch.randn(sum(lens), HIDDEN, generator=g).to(device)
    cu = ints([0, *torch.tensor(lens).cumsum(0).tolist()], device)
    rows = ints(range(len(lens)), device)

    q, k, v = layer.qkv(prompts)
    prompt_out = layer.out(cf.comp_attn_f32(q, k, v, cu, cu))
    cache.write(k, v, rows, cu)

    children = ints(range(len(lens), len(lens) * (samples + 1)), device)
    left = cache.fork(rows.repeat_interleave(samples), children)
    tokens, outs = [], []
    for _ in range(steps):
        x = torch.randn(len(children), HIDDEN, generator=g).to(device)
        q, k, v = layer.qkv(x)
        cache.write(k, v, children)
        attended = torch.empty(len(children), HEADS, DIM, device=device)
        for i, n in enumerate(lens):  # the samples of a prompt share its full pages
            mine = slice(i * samples, (i + 1) * samples)
            of = children[mine]
            cf.comp_attn_decode_f32x16(q[mine], cache.k, cache.v, cache.table[of], cache.lengths[of],
                                       shared=n // PAGE, out=attended[mine])
        tokens.append(x)
        outs.append(layer.out(attended))
    before = int((cache.refs > 0).sum())
    cache.free(children)
    live = cache.compact()
    return {"layer": layer, "prompts": prompts, "prompt_out": prompt_out, "tokens": tokens, "outs": outs,
            "left": int(left), "before": before, "live": int(live), "cache": cache}


if __name__ == "__main__":
    r = serve()
    torch.cuda.synchronize()
    print(f"prompts {tuple(r['prompt_out'].shape)}, {len(r['outs'])} steps of {tuple(r['outs'][0].shape)}; "
          f"{r['left']} pages free after the forks, {r['before']} in use, "
          f"{r['live']} after the samples were given back")

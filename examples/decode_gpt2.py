"""Greedy decoding with a GPT-2-small-shaped model on the library's kernels.

    python examples/decode_gpt2.py --batch 4 --new 256 --cache int8 --budget 128

Every step of a token runs on the library: the int8 lookup, the W4 matmuls
(GELU and residual fused), the append to the paged cache, the attention over
it (which also accumulates each position's weight), the int8 head, and the log
probabilities with the next token.  Once a sequence holds --budget positions
beyond --keep, the positions that attention weighed least are evicted and their
pages reused.  LayerNorm and the position embedding, which the library does not
have, are a few torch operations.  The weights are random (seeded), so the text
means nothing.
"""
from __future__ import annotations

import argparse
import os
import sys
import time

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import synth  # noqa: E402
import w4_block_dequant_amd as w4  # noqa: E402

HEADS, DIM = 12, 64  # of GPT-2 small: 768 wide
DTYPES = {"fp32": torch.float32, "fp16": torch.float16, "bf16": torch.bfloat16,
          "int8": torch.int8}


class Model:
    """GPT-2-small shapes; weights prepacked K-major, head and lookup token-major."""

    def __init__(self, layers: int = synth.GPT2_LAYERS, vocab: int = synth.GPT2_VOCAB,
                 device: str = "cuda:0", keep_canonical: bool = False):
        self.device, self.vocab, self.layers = torch.device(device), vocab, []

        def up(a):
            return torch.from_numpy(a).to(self.device)

        for layer in range(layers):
            slots = []
            for slot, (K, N) in enumerate(synth.GPT2_SHAPES):
                packed = w4.w4_quantize_pack(up(synth.weights(K, N, synth.CFG_GPT2_DECODE, layer, slot)))
                slots.append((w4.w4_prepack_kmajor(*packed),
                              up(synth.bias(N, synth.CFG_GPT2_DECODE, layer, slot)),
                              packed if keep_canonical else None))
            self.layers.append(slots)
        Q, self.hs = w4.i8_quantize_head(up(synth.head_table(synth.GPT2_HIDDEN, vocab)))
        self.Qt = w4.i8_prepack_head(Q, vocab)
        gen = torch.Generator(device=self.device).manual_seed(synth.SEED)
        self.positions = torch.randn((4096, synth.GPT2_HIDDEN), generator=gen,
                                     device=self.device) * synth.SIGMA_W


def norm(x):
    """LayerNorm without gain and offset."""
    x = x - x.mean(1, keepdim=True)
    return x * torch.rsqrt(x.square().mean(1, keepdim=True) + 1e-5)


class Cache:
    """One set of pools for each layer and one page table for all of them."""

    def __init__(self, model: Model, batch: int, length: int, dtype: str, page: int = 16):
        dev, self.page, self.batch = model.device, page, batch
        # twice the pages that the sequences need: an eviction copies to fresh ones
        cols = -(-length // page)
        pages = 2 * batch * cols
        shape = (pages, HEADS, page, DIM)
        self.pools = []
        for _ in model.layers:
            pool = {n: torch.zeros(shape, dtype=DTYPES[dtype], device=dev) for n in "KV"}
            pool["weight"] = torch.zeros(shape[:3], device=dev)
            pool["k_scale"] = pool["v_scale"] = None
            if dtype == "int8":
                pool["k_scale"], pool["v_scale"] = (torch.zeros(shape[:3], device=dev)
                                                    for _ in range(2))
            self.pools.append(pool)
        self.free = list(range(pages))[::-1]
        self.owned = [[] for _ in range(batch)]
        self.table = torch.full((batch, cols), -1, dtype=torch.int32)  # on the host
        self.on_gpu = self.table.to(dev)
        self.lens = torch.zeros(batch, dtype=torch.int32, device=dev)
        self.length = 0  # of every sequence
        self.seq = torch.arange(batch, dtype=torch.int32, device=dev)

    def grow(self):
        """Room for one more position of every sequence."""
        if self.length % self.page == 0:
            for b in range(self.batch):
                page = self.free.pop()
                self.table[b, len(self.owned[b])] = page
                self.owned[b].append(page)
            self.on_gpu = self.table.to(self.on_gpu.device)
        self.length += 1

    def evict(self, keep: int, recent: int):
        """Leave each sequence and head `keep` positions; the old pages go back."""
        need = -(-keep // self.page)
        fresh = [[self.free.pop() for _ in range(need)] for _ in range(self.batch)]
        table = torch.full_like(self.table, -1)
        table[:, :need] = torch.tensor(fresh, dtype=torch.int32)
        on_gpu = table.to(self.on_gpu.device)
        for p in self.pools:
            _, lens = w4.kv_evict(p["K"], p["V"], p["weight"], self.on_gpu, self.lens, keep,
                                  recent, on_gpu, k_scale=p["k_scale"], v_scale=p["v_scale"],
                                  max_len=self.length)
        self.lens.copy_(lens)
        for b in range(self.batch):
            self.free += self.owned[b]
            self.owned[b] = fresh[b]
        self.table, self.on_gpu, self.length = table, on_gpu, keep


def step(model: Model, cache: Cache, tokens: torch.Tensor, position: int) -> torch.Tensor:
    """One token of every sequence: appends it to the cache, returns the logits [batch, vocab]."""
    cache.grow()
    at = cache.lens.clone()
    cache.lens += 1
    x = w4.i8_embed_kmajor(tokens, model.Qt, model.hs, synth.GPT2_HIDDEN)
    x = x + model.positions[position]
    width = HEADS * DIM
    for (qkv, out, fc, proj), p in zip(model.layers, cache.pools):
        y = w4.w4_matmul_kmajor(norm(x), *qkv[0], qkv[1])
        q, k, v = (y[:, i * width:(i + 1) * width].unflatten(1, (HEADS, DIM)) for i in range(3))
        pools = dict(k_scale=p["k_scale"], v_scale=p["v_scale"], weight=p["weight"])
        w4.kv_append(k, v, p["K"], p["V"], cache.on_gpu, cache.seq, at, **pools)
        a = w4.kv_attend(q, p["K"], p["V"], cache.on_gpu, cache.lens, max_len=cache.length,
                         **pools)
        x = w4.w4_matmul_kmajor(a.reshape(-1, width), *out[0], out[1], residual=x)
        h = w4.w4_matmul_kmajor(norm(x), *fc[0], fc[1], act="gelu")
        x = w4.w4_matmul_kmajor(h, *proj[0], proj[1], residual=x)
    return w4.i8_head_logits_rows(norm(x), model.Qt, model.hs)


def generate(model: Model, prompt: torch.Tensor, new: int, dtype: str = "bf16",
             budget: int = 128, keep: int = 256, recent: int = 32):
    """prompt int64 [batch, length] -> (tokens [batch, new], their log probabilities and the
    entropies [batch, new], the cache).  The prompt is fed token by token."""
    batch, length = prompt.shape
    cache = Cache(model, batch, min(length + new, keep + budget), dtype)
    tokens, logprobs, entropies = [], [], []
    for i in range(length + new - 1):
        if cache.length == keep + budget:
            cache.evict(keep, recent)
        logits = step(model, cache, prompt[:, i].contiguous() if i < length else tokens[-1], i)
        if i >= length - 1:
            _, entropy, ids, best = w4.lp_logprobs(logits, None, 1)
            tokens.append(ids[:, 0].contiguous())
            logprobs.append(best[:, 0])
            entropies.append(entropy)
    return (torch.stack(tokens, 1), torch.stack(logprobs, 1), torch.stack(entropies, 1), cache)


def main():
    ap = argparse.ArgumentParser(description=__doc__,
                                 formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--batch", type=int, default=4)
    ap.add_argument("--prompt", type=int, default=synth.GPT2_PROMPT)
    ap.add_argument("--new", type=int, default=256)
    ap.add_argument("--layers", type=int, default=synth.GPT2_LAYERS)
    ap.add_argument("--cache", choices=list(DTYPES), default="bf16")
    ap.add_argument("--keep", type=int, default=128)
    ap.add_argument("--budget", type=int, default=64)
    ap.add_argument("--recent", type=int, default=32)
    a = ap.parse_args()
    model = Model(a.layers)
    prompt = torch.from_numpy(synth.tokens(a.batch * a.prompt, model.vocab, synth.CFG_GPT2_DECODE))
    prompt = prompt.reshape(a.batch, a.prompt).to(model.device)
    args = (model, prompt, a.new, a.cache, a.budget, a.keep, a.recent)
    generate(model, prompt, 2, a.cache, a.budget, a.keep, a.recent)  # first launches
    torch.cuda.synchronize()
    began = time.perf_counter()
    tokens, logprobs, entropies, cache = generate(*args)
    torch.cuda.synchronize()
    spent = time.perf_counter() - began
    steps = a.prompt + a.new - 1
    print(f"{steps} steps of {a.batch} sequences in {spent:.3f} s: {steps * a.batch / spent:.0f} "
          f"tokens/s, {1e3 * spent / steps:.3f} ms a step; cache {a.cache}, {cache.length} positions "
          f"held of {steps}")
    print(f"mean log probability {float(logprobs.mean()):.4f}, mean entropy "
          f"{float(entropies.mean()):.4f}, first tokens {tokens[:, :8].tolist()}")


if __name__ == "__main__":
    main()

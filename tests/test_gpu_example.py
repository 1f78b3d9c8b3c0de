"""The decoding example: its logits against a dense 64-bit model, and its evictions.

The reference runs the same dequantized weights and the same tokens with all
keys and values in 64 bits.  Tolerance: each matmul is within 1e-5 of
sum |x w|, which for these weights is some 30 times its result; eight of them
and the head follow each other in two layers, so logits may be off by
9 * 30 * 1e-5 of the largest.  The cache's own rounding adds 2^-9 (bf16), 2^-12
(fp16) or 1/254 (int8) of a value, attenuated like any noise of that size that
enters once a layer.
"""
import math
import os
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, os.path.join(ROOT, "examples"))

import decode_gpt2 as ex  # noqa: E402
import synth  # noqa: E402
import w4_block_dequant_amd as w4  # noqa: E402

VOCAB = 4096
ROUNDING = {"fp32": 0.0, "fp16": 2.0 ** -12, "bf16": 2.0 ** -9, "int8": 1 / 254}


@pytest.fixture(scope="module")
def model():
    return ex.Model(layers=2, vocab=VOCAB, keep_canonical=True)


def dense_logits(model, tokens):
    """fp64 [batch, length, vocab] of the whole sequences."""
    B, T = tokens.shape
    H, D = ex.HEADS, ex.DIM
    table = model.Qt[:, :synth.GPT2_HIDDEN].double() * model.hs.double()[:, None]
    x = table[tokens] + model.positions[:T].double()

    def norm(x):
        x = x - x.mean(-1, keepdim=True)
        return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-5)

    mask = torch.full((T, T), -math.inf, dtype=torch.float64, device=x.device).triu(1)
    for slots in model.layers:
        W = [w4.w4_dequantize(*s[2]).double() for s in slots]
        b = [s[1].double() for s in slots]
        q, k, v = (t.reshape(B, T, H, D).transpose(1, 2) for t in (norm(x) @ W[0] + b[0]).chunk(3, -1))
        s = torch.matmul(q, k.transpose(2, 3).contiguous()) / math.sqrt(D) + mask
        a = torch.matmul(torch.softmax(s, -1), v.contiguous())
        x = x + a.transpose(1, 2).reshape(B, T, H * D) @ W[1] + b[1]
        h = norm(x) @ W[2] + b[2]
        h = 0.5 * h * (1 + torch.tanh(math.sqrt(2 / math.pi) * (h + 0.044715 * h ** 3)))
        x = x + h @ W[3] + b[3]
    return norm(x) @ table.t()


@pytest.mark.parametrize("dtype", list(ROUNDING))
def test_steps_match_a_dense_model(model, dtype):
    print("example", dtype, flush=True)
    B, T = 3, 45
    tokens = torch.from_numpy(synth.tokens(B * T, VOCAB, 77)).reshape(B, T).to(model.device)
    ref = dense_logits(model, tokens)
    cache = ex.Cache(model, B, T, dtype)
    far = 0.0
    for t in range(T):
        logits = ex.step(model, cache, tokens[:, t].contiguous(), t).double()
        far = max(far, float((logits - ref[:, t]).abs().max() / ref[:, t].abs().max()))
        lp, entropy, ids, best = w4.lp_logprobs(logits.float(), tokens[:, t].contiguous(), 3)
        p = torch.log_softmax(logits, 1)
        assert torch.allclose(lp.double(), p.gather(1, tokens[:, t:t + 1])[:, 0], atol=1e-4)
        assert torch.equal(ids[:, 0], logits.argmax(1))
        assert torch.allclose(entropy.double(), -(p.exp() * p).sum(1), atol=1e-4)
    bound = 9 * 30 * 1e-5 + 4 * ROUNDING[dtype]
    print(f"  off by {far:.2e} of the largest logit, bound {bound:.2e}", flush=True)
    assert far <= bound
    # a step's attention adds 1 over a sequence's positions, for each head
    for p in cache.pools:
        total = float(p["weight"].double().sum())
        assert abs(total - B * ex.HEADS * T) <= 1e-5 * B * ex.HEADS * T


@pytest.mark.parametrize("dtype", ["bf16", "int8"])
def test_generation_with_evictions(model, dtype):
    """Lengths stay within keep + budget, no page is lost, results stay finite and repeat."""
    print("example eviction", dtype, flush=True)
    prompt = torch.from_numpy(synth.tokens(2 * 20, VOCAB, 78)).reshape(2, 20).to(model.device)
    runs = [ex.generate(model, prompt, 90, dtype, budget=24, keep=40, recent=8) for _ in range(2)]
    for tokens, logprobs, entropies, cache in runs:
        assert tokens.shape == (2, 90) and (tokens >= 0).all() and (tokens < VOCAB).all()
        assert torch.isfinite(logprobs).all() and torch.isfinite(entropies).all()
        assert (logprobs <= 0).all() and (entropies >= 0).all()
        assert (entropies <= math.log(VOCAB) + 1e-4).all()
        assert 40 <= cache.length <= 64
        assert cache.lens.tolist() == [cache.length] * 2
        owned = [p for pages in cache.owned for p in pages]
        assert sorted(owned + cache.free) == list(range(cache.pools[0]["K"].shape[0]))
    assert torch.equal(runs[0][0], runs[1][0]) and torch.equal(runs[0][1], runs[1][1])


def test_evicting_nothing_changes_nothing(model):
    """keep as long as the sequence: the copy on other pages gives the same logits."""
    T = 33
    tokens = torch.from_numpy(synth.tokens(2 * (T + 1), VOCAB, 79)).reshape(2, T + 1).to(model.device)
    logits = []
    for move in (False, True):
        cache = ex.Cache(model, 2, T + 1, "fp16")
        for t in range(T):
            ex.step(model, cache, tokens[:, t].contiguous(), t)
        if move:
            cache.evict(T, 4)
        logits.append(ex.step(model, cache, tokens[:, T].contiguous(), T))
    assert torch.equal(logits[0], logits[1])

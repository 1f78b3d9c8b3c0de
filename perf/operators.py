"""What a decode step does beside its weight matmuls: cases, plain forms and 64-bit values.

Four operators stand between the QKV matmul and the next token: the append of
new keys and values to a paged cache, the attention of one new token over it,
the eviction of the positions that attention weighs least, and the log
probabilities read off the head's logits.  With ``own`` false ``run`` computes
them in elementary torch operations in 32 bits; with ``own`` true it calls
the library.

A cache is two pools K, V [pages, kv heads, page size, head dim] (fp32, fp16,
bf16, or int8 with one fp32 scale for each token and head) and a table int32
[sequences, columns]: position t of sequence b is slot t % page size of page
table[b, t // page size]; entries past a sequence's length are -1.  Pools are
drawn whole: slots past a length hold what a freed page held.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
DTYPES = {"fp32": torch.float32, "fp16": torch.float16, "bf16": torch.bfloat16,
          "int8": torch.int8}
BYTES = {"fp32": 4, "fp16": 2, "bf16": 2, "int8": 1}


def listed():
    return [
        # GPT-2 small (12 heads of 64): the first token after a 58-token prompt, one sequence;
        # twelve such calls in a token, so the launch is what counts
        _attend("attend gpt2 first token", "fp32", 1, 12, 12, 64, 16, 59),
        # the 3.8B dense widths (32 heads of 96), one user near the end of a 4k context
        _attend("attend dense one user", "bf16", 1, 32, 32, 96, 64, 4095),
        # the same model, a batch of users at every length up to 4k, int8 cache
        _attend("attend dense batch int8", "int8", 16, 32, 32, 96, 16, 4096, ragged=True),
        # shared key/value heads (4 queries to each), four very long documents: the largest pass
        _attend("attend long documents", "bf16", 4, 32, 8, 128, 128, 131072),
        # shared heads (8 to each), ragged batch, weights accumulated for a later eviction,
        # a window that starts past the first positions
        _attend("attend weighing window", "fp16", 31, 24, 3, 128, 32, 8191, ragged=True,
                window=6000, weigh=True),
        # one decode step of 64 users into an int8 cache (read back as its values)
        _append("append decode int8", "int8", 64, 64, 32, 96, 16, 16),
        # a prompt of 2000 tokens for each of 4 users, shared heads of 128
        _append("append prompts", "bf16", 8000, 4, 8, 128, 64, 2000),
        # GPT-2's 1024-token context cut to half for 4 users, fp32 cache
        _evict("evict gpt2 context", "fp32", 4, 12, 64, 16, 1024, 512, 64),
        # the 3.8B widths: 8 users at every length up to 4k, at most 1500 rows kept
        _evict("evict dense batch", "bf16", 8, 32, 96, 64, 4096, 1500, 128, ragged=True),
        # the head's last row: next token and its log probability, one user
        _logprobs("logprobs next token", 1, 50257, 1),
        # a 58-token prompt scored with five alternatives each, some tokens forbidden
        _logprobs("logprobs prompt", 58, 50257, 5, masked=True),
        # a long document scored against a larger vocabulary, twenty alternatives
        _logprobs("logprobs document", 2048, 100003, 20),
    ]


def _attend(name, dtype, batch, heads, kv_heads, dim, page, length, ragged=False, window=0,
            weigh=False):
    return {"name": name, "op": "attend", "dtype": dtype, "batch": batch, "heads": heads,
            "kv_heads": kv_heads, "dim": dim, "page": page, "length": length, "ragged": ragged,
            "window": window, "weigh": weigh}


def _append(name, dtype, rows, batch, kv_heads, dim, page, length):
    return {"name": name, "op": "append", "dtype": dtype, "rows": rows, "batch": batch,
            "kv_heads": kv_heads, "dim": dim, "page": page, "length": length,
            "ragged": rows == batch}


def _evict(name, dtype, batch, kv_heads, dim, page, length, keep, recent, ragged=False):
    return {"name": name, "op": "evict", "dtype": dtype, "batch": batch, "kv_heads": kv_heads,
            "dim": dim, "page": page, "length": length, "keep": keep, "recent": recent,
            "ragged": ragged}


def _logprobs(name, rows, vocab, top, masked=False, pad=0):
    return {"name": name, "op": "logprobs", "rows": rows, "vocab": vocab, "top": top,
            "masked": masked, "pad": pad}


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["attend", "attend", "append", "evict", "logprobs"])
    if op == "logprobs":
        vocab = _log(rng, 2000, 160000)
        rows = _log(rng, 1, max(1, min(2048, 200_000_000 // vocab)))
        case = _logprobs(None, rows, vocab, rng.choice([0, 1, 3, 8, 20, 37, 64]),
                         rng.random() < 0.3, rng.choice([0, 0, 1, 47]))
    else:
        dim = rng.choice([64, 96, 128, 128, 40, 80, 120, 256])
        page = rng.choice([16, 32, 64, 256])
        dtype = rng.choice(["fp32", "fp16", "bf16", "int8"])
        kv_heads = rng.choice([1, 2, 3, 5, 8, 12, 32])
        group = rng.choice([1, 1, 2, 4, 5, 8, 16, 20]) if op == "attend" else 1
        # positions whose keys and values cost no more than the largest listed pass, in bytes
        # and in products
        most = 1_800_000_000 // (kv_heads * dim * max(2 * BYTES[dtype], group))
        if op == "attend":
            length = _log(rng, 1, min(131072, most))
            batch = _log(rng, 1, max(1, min(96, most // length)))
            case = _attend(None, dtype, batch, kv_heads * group, kv_heads, dim, page, length,
                           rng.random() < 0.6, rng.choice([0, 0, 0, 1 + length // 3]),
                           rng.random() < 0.3)
        elif op == "append":
            length = _log(rng, 1, min(4000, most))
            batch = _log(rng, 1, max(1, min(128, most // (8 * length))))
            rows = batch * (length if rng.random() < 0.4 else 1)
            case = _append(None, dtype, rows, batch, kv_heads, dim, page, length)
        else:
            length = _log(rng, 16, min(32768, most // 8))
            batch = _log(rng, 1, max(1, min(32, most // (8 * length))))
            keep = max(1, int(length * rng.uniform(0.1, 0.9)))
            case = _evict(None, rng.choice(["fp32", "fp16", "bf16"]), batch, kv_heads, dim, page,
                          length, keep, int(keep * rng.uniform(0, 0.6)), rng.random() < 0.5)
    del case["name"]
    return case


# ---- inputs ------------------------------------------------------------------
def _lengths(case):
    """The batch's lengths: all of them `length`, or spread evenly over 1..length."""
    B, L = case["batch"], case["length"]
    if not case.get("ragged") or B == 1:
        return [L] * B
    return [1 + (L - 1) * i // (B - 1) for i in range(B)]


def _attended(case):
    w = case["window"]
    return sum(min(n, w) if w else n for n in _lengths(case))


def _pool(shape, dtype, gen):
    """One pool (and its scales, of int8) of normal values."""
    if dtype == "int8":
        codes = torch.randint(-127, 128, shape, generator=gen, device=DEV, dtype=torch.int8)
        return codes, torch.rand(shape[:3], generator=gen, device=DEV) * 0.02 + 0.005
    return torch.randn(shape, generator=gen, device=DEV, dtype=DTYPES[dtype]), None


def _table(pages_of, cols, gen_cpu, first=0):
    """Shuffled pages for each sequence, -1 past what it needs."""
    total = int(sum(pages_of))
    order = torch.randperm(total, generator=gen_cpu).to(torch.int32) + first
    table = torch.full((len(pages_of), cols), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(pages_of):
        table[b, :n] = order[at:at + n]
        at += n
    return table.to(DEV), total


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    cpu = torch.Generator().manual_seed(seed)
    st = dict(case)
    if case["op"] == "logprobs":
        M, N = case["rows"], case["vocab"]
        logits = torch.randn((M, N + case["pad"]), generator=gen, device=DEV) * 3.0
        if case["masked"]:
            logits[torch.rand(logits.shape, generator=gen, device=DEV) < 0.3] = -math.inf
        st["logits"] = logits[:, :N]
        st["tokens"] = torch.randint(0, N, (M,), generator=gen, device=DEV)
        return st
    H, D, ps, B = case["kv_heads"], case["dim"], case["page"], case["batch"]
    lens = [_lengths(case)[i] for i in torch.randperm(B, generator=cpu).tolist()]
    cols = -(-case["length"] // ps)
    table, pages = _table([-(-n // ps) for n in lens], cols, cpu)
    spare = 0
    if case["op"] == "evict":
        cols_out = -(-min(case["keep"], case["length"]) // ps)
        st["table_out"], spare = _table([-(-min(n, case["keep"]) // ps) for n in lens], cols_out,
                                        cpu, first=pages)
    shape = (pages + spare, H, ps, D)
    st["K"], st["k_scale"] = _pool(shape, case["dtype"], gen)
    st["V"], st["v_scale"] = _pool(shape, case["dtype"], gen)
    st["table"] = table
    st["lens"] = torch.tensor(lens, dtype=torch.int32, device=DEV)
    st["weight"] = None
    if case["op"] == "attend":
        st["q"] = torch.randn((B, case["heads"], D), generator=gen, device=DEV) * 2.0
        st["starts"] = None
        if case["window"]:
            st["starts"] = (st["lens"] - case["window"]).clamp_min(0)
        if case["weigh"]:
            st["weight"] = torch.rand(shape[:3], generator=gen, device=DEV)
    elif case["op"] == "append":
        # keys and values are columns of a fused QKV product's rows
        R = case["rows"]
        qkv = torch.randn((R, 3 * H * D), generator=gen, device=DEV)
        st["k"] = qkv[:, H * D:2 * H * D].unflatten(1, (H, D))
        st["v"] = qkv[:, 2 * H * D:].unflatten(1, (H, D))
        per = R // B
        seq = torch.arange(R, dtype=torch.int32) // per
        at = torch.tensor(lens, dtype=torch.int32)[seq.long()] - per + torch.arange(R, dtype=torch.int32) % per
        mix = torch.randperm(R, generator=cpu) if per == 1 else torch.arange(R)
        st["seq"], st["at"] = seq[mix].to(DEV), at[mix].to(DEV)
        st["weight"] = torch.rand(shape[:3], generator=gen, device=DEV)
    else:
        # accumulated weights are heavy-tailed: a few positions take most
        st["weight"] = torch.rand(shape[:3], generator=gen, device=DEV).clamp_min(1e-6).pow(-1.5)
        st["kept"] = torch.empty((B, H, case["keep"]), dtype=torch.int32, device=DEV)
        st["lens_out"] = torch.empty(B, dtype=torch.int32, device=DEV)
    return st


# ---- one pass ------------------------------------------------------------------
def run(s):
    return {"attend": _run_attend, "append": _run_append, "evict": _run_evict,
            "logprobs": _run_logprobs}[s["op"]](s)


def _values(pool, scale):
    """What an int8 pool stands for; other pools as they are."""
    return pool if scale is None else pool.float() * scale[..., None]


def _rows(pool, scale, table):
    """The pool's rows by sequence and head, fp32 [B, H, columns * page size, D]."""
    x = _values(pool[table.long().clamp_min(0)],
                None if scale is None else scale[table.long().clamp_min(0)]).float()
    B, C, H, ps, D = x.shape
    return x.permute(0, 2, 1, 3, 4).reshape(B, H, C * ps, D)


def _run_attend(s):
    if own:
        import w4_block_dequant_amd as w4
        out = w4.kv_attend(s["q"], s["K"], s["V"], s["table"], s["lens"], starts=s["starts"],
                           k_scale=s["k_scale"], v_scale=s["v_scale"], weight=s["weight"])
        return (out,) if s["weight"] is None else (out, s["weight"])
    table, D, H = s["table"], s["dim"], s["kv_heads"]
    k = _rows(s["K"], s["k_scale"], table)
    B, _, T, _ = k.shape
    q = s["q"].reshape(B, H, -1, D)
    sc = torch.matmul(q, k.transpose(2, 3)) * (1.0 / math.sqrt(D))
    del k
    t = torch.arange(T, device=DEV)
    seen = t < s["lens"][:, None]
    if s["starts"] is not None:
        seen &= t >= s["starts"][:, None]
    sc = sc.masked_fill(~seen[:, None, None, :], -math.inf)
    top = sc.amax(-1, keepdim=True)
    p = torch.exp(sc - torch.where(top == -math.inf, torch.zeros_like(top), top))
    p = p / p.sum(-1, keepdim=True).clamp_min(1e-30)
    out = torch.matmul(p, _rows(s["V"], s["v_scale"], table)).reshape(B, -1, D)
    if s["weight"] is None:
        return (out,)
    add = p.sum(2).reshape(B, H, -1, s["page"]).transpose(1, 2)  # [B, columns, H, page size]
    s["weight"].index_put_((table.long().clamp_min(0),), add, accumulate=True)
    return out, s["weight"]


def _stored(x, dtype):
    """Rows as the cache's type holds them, and int8's scales."""
    if dtype != "int8":
        return x.to(DTYPES[dtype]), None
    scale = x.abs().amax(-1) / 127.0
    codes = torch.round(x / torch.where(scale == 0, torch.ones_like(scale), scale)[..., None])
    return codes.clamp(-127, 127).to(torch.int8), scale


def _run_append(s):
    if own:
        import w4_block_dequant_amd as w4
        w4.kv_append(s["k"], s["v"], s["K"], s["V"], s["table"], s["seq"], s["at"],
                     k_scale=s["k_scale"], v_scale=s["v_scale"], weight=s["weight"])
    else:
        at = s["at"].long()
        page, slot = s["table"][s["seq"].long(), at // s["page"]].long(), at % s["page"]
        k, ks = _stored(s["k"], s["dtype"])
        v, vs = _stored(s["v"], s["dtype"])
        s["K"][page, :, slot] = k
        s["V"][page, :, slot] = v
        if ks is not None:
            s["k_scale"][page, :, slot] = ks
            s["v_scale"][page, :, slot] = vs
        s["weight"][page, :, slot] = 0.0
    return _values(s["K"], s["k_scale"]), _values(s["V"], s["v_scale"]), s["weight"]


def _run_evict(s):
    if own:
        import w4_block_dequant_amd as w4
        w4.kv_evict(s["K"], s["V"], s["weight"], s["table"], s["lens"], s["keep"], s["recent"],
                    s["table_out"], kept=s["kept"], lens_out=s["lens_out"])
        return s["K"], s["V"], s["weight"], s["kept"], s["lens_out"]
    table, keep, ps = s["table"].long().clamp_min(0), s["keep"], s["page"]
    B, H = table.shape[0], s["kv_heads"]
    w = s["weight"][table].permute(0, 2, 1, 3).reshape(B, H, -1)  # [B, H, T]
    T = w.shape[2]
    t, n = torch.arange(T, device=DEV), s["lens"].long()[:, None, None]
    recent = min(s["recent"], keep)
    # the newest rows first, then by weight, then by position; nothing past the length
    w = torch.where(t >= n - recent, torch.full_like(w, math.inf), w)
    w = torch.where((n <= keep), torch.full_like(w, math.inf), w)
    w = torch.where(t >= n, torch.full_like(w, -math.inf), w)
    order = torch.sort(w, dim=2, descending=True, stable=True).indices[:, :, :keep]
    m = s["lens"].long().clamp_max(keep)
    i = torch.arange(order.shape[2], device=DEV)
    order = torch.where(i < m[:, None, None], order, torch.full_like(order, T))
    order = torch.sort(order, dim=2).values
    live = (i < m[:, None])[:, None, :].expand(B, H, -1)
    s["kept"].fill_(-1)
    s["kept"][:, :, :order.shape[2]] = torch.where(live, order, torch.full_like(order, -1))
    s["lens_out"].copy_(m)
    b, h, j = live.nonzero(as_tuple=True)
    src = order[b, h, j]
    page, slot = table[b, src // ps], src % ps
    page_to, slot_to = s["table_out"].long()[b, j // ps], j % ps
    s["K"][page_to, h, slot_to] = s["K"][page, h, slot]
    s["V"][page_to, h, slot_to] = s["V"][page, h, slot]
    s["weight"][page_to, h, slot_to] = s["weight"][page, h, slot]
    return s["K"], s["V"], s["weight"], s["kept"], s["lens_out"]


def _run_logprobs(s):
    if own:
        import w4_block_dequant_amd as w4
        return w4.lp_logprobs(s["logits"], s["tokens"], s["top"])
    x = s["logits"]
    top = x.amax(1, keepdim=True)
    e = torch.exp(x - top)
    total = e.sum(1, keepdim=True)
    log_total = torch.log(total)
    logprob = (x.gather(1, s["tokens"][:, None]) - top - log_total)[:, 0]
    # a forbidden token has no share: 0 * -inf is taken as 0
    d = torch.where(x == -math.inf, torch.zeros_like(x), x - top)
    entropy = (log_total - (e * d).sum(1, keepdim=True) / total)[:, 0]
    if s["top"] == 1:  # amax and the lowest index that has it
        ids = torch.where(x == top, torch.arange(x.shape[1], device=DEV), x.shape[1]).amin(1, keepdim=True)
        best = top
    else:
        best, ids = torch.sort(x, dim=1, descending=True, stable=True)
        best, ids = best[:, :s["top"]], ids[:, :s["top"]]
    return logprob, entropy, ids, best - top - log_total


# ---- work and 64-bit values --------------------------------------------------------
def work(case):
    """Bytes: every input read once, every output written once; flops: multiplies and adds."""
    if case["op"] == "logprobs":
        M, N, k = case["rows"], case["vocab"], case["top"]
        return {"bytes": 4 * M * N + M * (8 + 8 + 12 * k), "flops": 5 * M * N}
    H, D, B = case["kv_heads"], case["dim"], case["batch"]
    row = D * BYTES[case["dtype"]] + (4 if case["dtype"] == "int8" else 0)
    if case["op"] == "attend":
        n = _attended(case)
        return {"bytes": n * H * (2 * row + (8 if case["weigh"] else 0))
                + B * case["heads"] * D * 8, "flops": 4 * n * case["heads"] * D}
    if case["op"] == "append":
        n = case["rows"] * H
        return {"bytes": n * (8 * D + 2 * row + 4), "flops": n * 2 * D}
    lens = _lengths(case)
    out = sum(min(n, case["keep"]) for n in lens)
    return {"bytes": H * (4 * sum(lens) + out * (4 * row + 8) + 4 * B * case["keep"]), "flops": H * sum(lens)}


def exact(case, seed):
    """What run returns, from the definitions in 64 bits, one sequence or head after the other."""
    s = prepare(case, seed)
    if case["op"] == "logprobs":
        logprob, entropy, best = [], [], []
        for row, token in zip(s["logits"], s["tokens"].tolist()):
            x = row.double()
            lse = torch.logsumexp(x, 0)
            lp = x - lse
            logprob.append(lp[token])
            entropy.append(-torch.special.xlogy(lp.exp(), lp.exp()).sum())
            best.append(torch.topk(lp, case["top"]).values)
        return torch.stack(logprob), torch.stack(entropy), None, torch.stack(best)
    ps, H, D = case["page"], case["kv_heads"], case["dim"]
    table, lens = s["table"].cpu().numpy(), s["lens"].tolist()
    if case["op"] == "attend":
        outs = []
        for b, n in enumerate(lens):
            lo = max(0, n - case["window"]) if case["window"] else 0
            heads = []
            pages = torch.from_numpy(table[b, :-(-n // ps)]).long().to(DEV)
            for h in range(H):
                k, v = s["K"][pages, h].double(), s["V"][pages, h].double()
                if s["k_scale"] is not None:
                    k = k * s["k_scale"][pages, h].double()[..., None]
                    v = v * s["v_scale"][pages, h].double()[..., None]
                k, v = k.reshape(-1, D)[lo:n], v.reshape(-1, D)[lo:n]
                q = s["q"][b].reshape(H, -1, D)[h].double()
                p = torch.softmax(q @ k.t().contiguous() / math.sqrt(D), dim=1)
                heads.append(p @ v)
                if s["weight"] is not None:
                    if h == 0 and b == 0:
                        total = s["weight"].double()
                    t = torch.arange(lo, n, device=DEV)
                    total[pages[t // ps], h, t % ps] += p.sum(0)
            outs.append(torch.cat(heads))
        out = torch.stack(outs)
        return (out,) if s["weight"] is None else (out, total)
    if case["op"] == "append":
        seq, at = s["seq"].cpu().numpy(), s["at"].cpu().numpy()
        page = torch.from_numpy(table[seq, at // ps]).long().to(DEV)
        slot = torch.from_numpy(at % ps).long().to(DEV)
        got = []
        for x, pool, scale in ((s["k"], s["K"], s["k_scale"]), (s["v"], s["V"], s["v_scale"])):
            y, x = pool.double(), x.double()
            if scale is not None:
                y = y * scale.double()[..., None]
                step = x.abs().amax(-1, keepdim=True) / 127
                x = torch.round(x / step) * step
            else:
                x = x.to(pool.dtype).double()
            y[page, :, slot] = x
            got.append(y)
        w = s["weight"].double()
        w[page, :, slot] = 0
        return got[0], got[1], w
    K, V, weight = s["K"].clone(), s["V"].clone(), s["weight"].clone()
    out, host = s["table_out"].cpu().numpy(), s["weight"].cpu().numpy()
    for b, n in enumerate(lens):
        for h in range(H):
            w = host[table[b, :-(-n // ps)], h].reshape(-1)[:n]
            keep = min(n, case["keep"])
            recent = min(case["recent"], keep)
            order = np.lexsort((np.arange(n - recent), -w[:n - recent].astype(np.float64)))
            old = np.sort(np.concatenate([order[:keep - recent], np.arange(n - recent, n)]))
            new = np.arange(keep)
            a, c = (torch.from_numpy(np.asarray(i, dtype=np.int64)).to(DEV)
                    for i in (table[b, old // ps], old % ps))
            x, y = (torch.from_numpy(np.asarray(i, dtype=np.int64)).to(DEV)
                    for i in (out[b, new // ps], new % ps))
            for pool in (K, V, weight):
                pool[x, h, y] = pool[a, h, c]
    return K, V, weight, None, None

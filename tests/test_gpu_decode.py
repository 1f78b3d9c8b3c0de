"""The paged cache's operators and the log probabilities against their formulas in 64 bits.

Tolerances are worst-case fp32 bounds of the formulas (eps = 2^-24 relative to
each rounding): a score carries (head_dim + 8) eps of sum |q k| plus 4 eps of
itself; a softmax weight twice that and its sums' chains; an output the same
relative to sum p |v|.  Copies, positions, ids and stored codes are exact.
Slots and pages that nothing owns hold NaN, table entries past a length hold
ids that no pool has.
"""
import math

import numpy as np
import pytest
import torch

import w4_block_dequant_amd as w4

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
EPS = 2.0 ** -24
DTYPES = {"fp32": torch.float32, "fp16": torch.float16, "bf16": torch.bfloat16,
          "int8": torch.int8}


def note(msg):
    print(msg, flush=True)


def status():
    return torch.zeros(1, dtype=torch.int32, device=DEV)


class Cache:
    """A paged cache in host memory (values in 64 bits beside the stored ones)."""

    def __init__(self, dtype, lens, heads, dim, ps, seed, weight=False, spare=2, amp=1.0):
        g = np.random.default_rng([seed, heads, dim, ps])
        self.dtype, self.lens, self.heads, self.dim, self.ps = dtype, list(lens), heads, dim, ps
        need = [-(-n // ps) for n in lens]
        cols = max(need + [0]) + 1
        pages = sum(need) + spare
        order = g.permutation(pages)
        self.table = np.full((len(lens), cols), 0x7FFFFFF0, np.int64)
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = order[at:at + n]
            at += n
        self.free = order[at:]
        shape = (pages, heads, ps, dim)
        live = np.zeros((pages, ps), bool)
        for b, n in enumerate(lens):
            for t0 in range(0, n, ps):
                live[self.table[b, t0 // ps], :min(ps, n - t0)] = True
        live = torch.from_numpy(live)[:, None, :].expand(shape[:3])
        gt = torch.Generator().manual_seed(seed)

        def pool():
            if dtype == "int8":
                x = torch.randint(-127, 128, shape, generator=gt, dtype=torch.int8)
                s = torch.rand(shape[:3], generator=gt) * 0.03 * amp + 0.001
                s[~live] = math.nan
                return x, s
            x = (torch.randn(shape, generator=gt) * amp).to(DTYPES[dtype])
            x[~live] = math.nan
            return x, None

        self.K, self.ks = pool()
        self.V, self.vs = pool()
        self.weight = torch.rand(shape[:3], generator=gt) if weight else None

    def on_gpu(self):
        up = [None if t is None else t.to(DEV) for t in (self.K, self.V, self.ks, self.vs,
                                                           self.weight)]
        return up, torch.from_numpy(self.table.astype(np.int32)).to(DEV)

    def rows(self, b, h, which):
        """fp64 [len, dim] of one sequence and head."""
        n = self.lens[b]
        pages = torch.from_numpy(self.table[b, :-(-n // self.ps)])
        pool, scale = (self.K, self.ks) if which == "k" else (self.V, self.vs)
        x = pool[pages, h].double()
        if scale is not None:
            x = x * scale[pages, h].double()[..., None]
        return x.reshape(-1, self.dim)[:n]


def attend_reference(c, q, starts, scale):
    """(out, tolerance, weights added, their tolerance) in 64 bits."""
    B, Hq, D = q.shape
    G = Hq // c.heads
    out = torch.zeros((B, Hq, D), dtype=torch.float64)
    tol = torch.full((B, Hq, D), 1e-37, dtype=torch.float64)
    add = torch.zeros(c.K.shape[:3], dtype=torch.float64)
    add_tol = torch.zeros_like(add)
    for b in range(B):
        n, lo = c.lens[b], max(0, starts[b]) if starts is not None else 0
        if lo >= n:
            continue
        for h in range(c.heads):
            k, v = c.rows(b, h, "k")[lo:], c.rows(b, h, "v")[lo:]
            qq = q[b, h * G:(h + 1) * G].double()
            s = (qq @ k.t()) * scale
            worst = (qq.abs() @ k.abs().t()).amax(1) * abs(scale)
            off = (D + 8) * EPS * worst + 4 * EPS * s.abs().amax(1)
            rel = 2 * off + EPS * (32 + (n - lo) / 64)
            p = torch.softmax(s, 1)
            out[b, h * G:(h + 1) * G] = p @ v
            tol[b, h * G:(h + 1) * G] += (p @ v.abs()) * rel[:, None]
            t = torch.arange(lo, n)
            page = torch.from_numpy(c.table[b])[t // c.ps]
            add[page, h, t % c.ps] = p.sum(0)
            add_tol[page, h, t % c.ps] = (p * rel[:, None]).sum(0)
    return out, tol, add, add_tol


def run_attend(c, Hq, seed, starts=None, scale=None, weigh=False, amp=1.0, max_len=0, fused=False):
    g = torch.Generator().manual_seed(seed)
    B, D = len(c.lens), c.dim
    q = torch.randn((B, Hq, D), generator=g) * amp
    (K, V, ks, vs, w), table = c.on_gpu()
    lens = torch.tensor(c.lens, dtype=torch.int32, device=DEV)
    st = None if starts is None else torch.tensor(starts, dtype=torch.int32, device=DEV)
    qd = q.to(DEV)
    if fused:  # q as the first columns of wider rows, not 16-byte aligned
        wide = torch.full((B, Hq * D + 37), math.nan, device=DEV)
        wide[:, 1:1 + Hq * D] = qd.reshape(B, -1)
        qd = wide[:, 1:1 + Hq * D].unflatten(1, (Hq, D))
    bad = status()
    out = torch.full((B, Hq, D), math.nan, device=DEV)
    before = None if w is None else w.clone()
    got = w4.kv_attend(qd, K, V, table, lens, starts=st, scale=scale, max_len=max_len, k_scale=ks,
                       v_scale=vs, weight=w if weigh else None, out=out, d_status=bad)
    assert got is out
    torch.cuda.synchronize()
    assert int(bad) == 0
    ref, tol, add, add_tol = attend_reference(c, q, starts, D ** -0.5 if scale is None else scale)
    err = (out.cpu().double() - ref).abs()
    assert torch.isfinite(out).all()
    note(f"  max err/tol {float((err / tol).max()) if err.numel() else 0:.3f}")
    assert (err <= tol).all()
    if weigh:
        want = c.weight.double() + add
        werr = (w.cpu().double() - want).abs()
        lim = add_tol + 2 * EPS * want
        note(f"  weights max err/tol {float((werr / lim).max()):.3f}")
        assert (werr <= lim).all()
        same = add == 0
        assert torch.equal(w.cpu()[same], c.weight[same])
    elif w is not None:
        assert torch.equal(w, before)
    return out


EDGE_LENS = [0, 1, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 200]


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("Hq,H,D,ps", [(12, 12, 64, 16), (4, 4, 96, 32), (8, 2, 128, 16),
                                       (10, 2, 40, 64), (3, 1, 8, 16), (16, 1, 256, 16),
                                       (40, 2, 120, 32), (5, 5, 24, 4096), (6, 3, 160, 128)])
def test_attend_edge_lengths(dtype, Hq, H, D, ps):
    note(f"attend {dtype} heads {Hq}/{H} dim {D} page {ps}")
    run_attend(Cache(dtype, EDGE_LENS, H, D, ps, 3, weight=True), Hq, 4, weigh=True, fused=True)


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("weigh", [False, True])
def test_attend_windows(dtype, weigh):
    """First positions inside, at and past the length: rows left empty give zeros."""
    note(f"attend windows {dtype}")
    lens = [300, 300, 300, 300, 40, 1, 0, 513]
    starts = [0, 1, 299, 300, 41, -5, 3, 500]
    c = Cache(dtype, lens, 2, 64, 16, 5, weight=True)
    out = run_attend(c, 6, 6, starts=starts, weigh=weigh)
    for b in (3, 4, 6):
        assert not out[b].any()


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("Hq,H,D,n", [(2, 2, 96, 5000), (8, 1, 128, 9001), (32, 4, 64, 2049)])
def test_attend_long(dtype, Hq, H, D, n):
    note(f"attend long {dtype} {Hq}/{H} {D} {n}")
    run_attend(Cache(dtype, [n, 7, n // 3], H, D, 64, 7, weight=True), Hq, 8, weigh=True)


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("amp", [0.0, 30.0, 1e-30])
def test_attend_peaked_and_flat(dtype, amp):
    """Queries that pick one position, weigh all alike, or are tiny."""
    note(f"attend amplitude {amp} {dtype}")
    run_attend(Cache(dtype, [700, 33], 2, 64, 16, 9, weight=True), 4, 10, amp=amp, weigh=True)


@pytest.mark.parametrize("dtype", list(DTYPES))
def test_attend_scale_and_bound_on_lengths(dtype):
    note(f"attend scale, max_len {dtype}")
    run_attend(Cache(dtype, [100, 257, 3], 2, 64, 16, 11), 2, 12, scale=0.5, max_len=257)
    run_attend(Cache(dtype, [100, 257, 3], 2, 64, 16, 11), 2, 12, scale=-0.25, max_len=10 ** 6)


@pytest.mark.parametrize("seqs", [1, 2, 300])
def test_attend_many_sequences(seqs):
    note(f"attend {seqs} sequences")
    lens = [(37 * i) % 90 for i in range(seqs)]
    run_attend(Cache("bf16", lens, 3, 64, 32, 13, weight=True), 6, 14, weigh=True)


def test_attend_repeats_bit_for_bit():
    c = Cache("bf16", [3000, 900, 1], 2, 128, 64, 15, weight=True)
    a = run_attend(c, 8, 16)
    b = run_attend(c, 8, 16)
    assert torch.equal(a, b)


def test_attend_reports_bad_lengths_and_pages():
    """What the host cannot see: a length past the table, a negative one, a foreign page id."""
    note("attend bad lengths")
    c = Cache("fp32", [64, 40, 64], 2, 64, 16, 17)
    (K, V, *_), table = c.on_gpu()
    table = table[:, :4].contiguous()
    q = torch.randn((3, 2, 64), generator=torch.Generator().manual_seed(1)).to(DEV)
    bad = status()
    lens = torch.tensor([1000, -3, 64], dtype=torch.int32, device=DEV)
    out = w4.kv_attend(q, K, V, table, lens, d_status=bad)
    assert int(bad) == w4.W4_ERR_BAD_SHAPE
    full = torch.tensor([64, 0, 64], dtype=torch.int32, device=DEV)
    assert torch.equal(out, w4.kv_attend(q, K, V, table, full))
    assert not out[1].any()
    # max_len cuts as the table does
    bad.zero_()
    out = w4.kv_attend(q, K, V, table, full, max_len=16, d_status=bad)
    assert int(bad) == w4.W4_ERR_BAD_SHAPE
    cut = torch.tensor([16, 0, 16], dtype=torch.int32, device=DEV)
    ref = w4.kv_attend(q, K, V, table, cut)
    assert torch.allclose(out, ref, rtol=1e-5, atol=1e-6)
    # positions of a page that the pool does not have take no part
    c.table[0, 1] = c.K.shape[0]
    c.table[2, 3] = -1
    table = torch.from_numpy(c.table[:, :4].astype(np.int32)).to(DEV).contiguous()
    bad.zero_()
    out = w4.kv_attend(q, K, V, table, full, d_status=bad).cpu().double()
    assert int(bad) == w4.W4_ERR_BAD_SHAPE
    for b, gone in ((0, 1), (2, 3)):
        pages = torch.from_numpy(np.delete(c.table[b, :4], gone))
        for h in range(2):
            k, v = (x[pages, h].double().reshape(-1, 64) for x in (c.K, c.V))
            p = torch.softmax(k @ q[b, h].cpu().double() / 8, 0)
            assert torch.allclose(out[b, h], p @ v, rtol=1e-4, atol=1e-5)


def test_attend_pool_past_32_bit_offsets():
    """Pages whose bytes lie past 2^32, one on each side of the line."""
    pages, H, ps, D = 66000, 8, 64, 128  # 4.3e9 elements of one byte
    note("attend pool past 2^32")
    K = torch.empty((pages, H, ps, D), dtype=torch.int8, device=DEV)
    V = torch.empty_like(K)
    ks = torch.full((pages, H, ps), 0.01, device=DEV)
    vs = torch.full((pages, H, ps), 0.02, device=DEV)
    g = torch.Generator(device=DEV).manual_seed(2)
    used = torch.tensor([65999, 0, 32768, 65536, 40000], device=DEV)
    for pool in (K, V):
        pool[used] = torch.randint(-127, 128, (5, H, ps, D), generator=g, device=DEV,
                                   dtype=torch.int8)
    q = torch.randn((1, 2 * H, D), generator=g, device=DEV)
    table = used.to(torch.int32)[None].contiguous()
    n = 4 * ps + 9
    out = w4.kv_attend(q, K, V, table, torch.tensor([n], dtype=torch.int32, device=DEV),
                       k_scale=ks, v_scale=vs).double()
    k, v = (x[used].transpose(0, 1).reshape(H, -1, D)[:, :n].double() for x in (K, V))
    s = (q.double().reshape(H, 2, 1, D) * k[:, None] * 0.01).sum(-1) / math.sqrt(D)
    ref = (torch.softmax(s, -1)[..., None] * v[:, None] * 0.02).sum(2).reshape(1, 2 * H, D)
    assert torch.allclose(out, ref, rtol=1e-4, atol=1e-4 * float(ref.abs().max()))
    # a row appended to the last page arrives there
    x = torch.randn((1, H, D), generator=g, device=DEV)
    at = torch.tensor([5], dtype=torch.int32, device=DEV)
    w4.kv_append(x, x, K, V, table, torch.zeros(1, dtype=torch.int32, device=DEV), at, k_scale=ks,
                 v_scale=vs)
    assert torch.equal(ks[65999, :, 5], x[0].abs().amax(-1) / 127)
    assert int(K[65999, :, 5].abs().amax()) == 127


def test_attend_on_another_stream_and_in_a_graph():
    """A side stream has a workspace of its own; a captured call replays on new lengths."""
    note("attend stream and graph")
    c = Cache("bf16", [2000, 31], 2, 64, 16, 19, weight=True)
    (K, V, _, _, w), table = c.on_gpu()
    q = torch.randn((2, 8, 64), generator=torch.Generator().manual_seed(3)).to(DEV)
    lens = torch.tensor(c.lens, dtype=torch.int32, device=DEV)
    ref = w4.kv_attend(q, K, V, table, lens)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = w4.kv_attend(q, K, V, table, lens)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got, ref)
    out = torch.empty_like(ref)
    ws = torch.empty(1 << 22, dtype=torch.uint8, device=DEV)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        w4.kv_attend(q, K, V, table, lens, weight=w, out=out, workspace=ws)
    for n in (2000, 1, 777, 0, 1999):
        lens[0] = n
        w.zero_()
        ws.fill_(0x5A)
        graph.replay()
        w2 = torch.zeros_like(w)
        ref = w4.kv_attend(q, K, V, table, lens, weight=w2)
        assert torch.equal(out, ref) and torch.equal(w, w2)


@pytest.mark.parametrize("dtype", ["int8", "bf16"])
def test_attend_and_append_with_arrays_off_16_bytes(dtype):
    """Scales, weights, lengths and the table need 4-byte alignment only."""
    note(f"attend off alignment {dtype}")
    c = Cache(dtype, [300, 45], 2, 40, 16, 41, weight=True)
    (K, V, ks, vs, w), table = c.on_gpu()
    q = torch.randn((2, 4, 40), generator=torch.Generator().manual_seed(42)).to(DEV)
    lens = torch.tensor(c.lens, dtype=torch.int32, device=DEV)

    def shifted(t):
        if t is None:
            return None
        wide = torch.zeros(t.numel() + 1, dtype=t.dtype, device=DEV)
        wide[1:] = t.reshape(-1)
        return wide[1:].view(t.shape)

    w1, w2 = w.clone(), shifted(w)
    ref = w4.kv_attend(q, K, V, table, lens, k_scale=ks, v_scale=vs, weight=w1)
    got = w4.kv_attend(shifted(q), K, V, shifted(table), shifted(lens), k_scale=shifted(ks),
                       v_scale=shifted(vs), weight=w2, out=shifted(torch.zeros_like(ref)))
    assert torch.equal(ref, got) and torch.equal(w1, w2)
    x = torch.randn((2, 2, 40), generator=torch.Generator().manual_seed(43)).to(DEV)
    seq = torch.tensor([1, 0], dtype=torch.int32, device=DEV)
    at = torch.tensor([44, 7], dtype=torch.int32, device=DEV)
    K2, V2, ks2, vs2 = K.clone(), V.clone(), shifted(ks), shifted(vs)
    w4.kv_append(x, x, K, V, table, seq, at, k_scale=ks, v_scale=vs, weight=w1)
    w4.kv_append(shifted(x), shifted(x), K2, V2, shifted(table), shifted(seq), shifted(at),
                 k_scale=ks2, v_scale=vs2, weight=w2)
    assert torch.equal(bits(K), bits(K2)) and torch.equal(bits(V), bits(V2))
    assert torch.equal(w1, w2)
    if ks is not None:
        assert torch.equal(bits(ks), bits(ks2)) and torch.equal(bits(vs), bits(vs2))


def test_append_and_evict_in_a_graph():
    """Captured once, replayed on new rows, places, lengths and weights."""
    note("append and evict graph")
    c = Cache("bf16", [90, 40], 2, 64, 16, 44, weight=True, spare=8)
    (K, V, _, _, w), table = c.on_gpu()
    x = torch.randn((2, 2, 64), device=DEV)
    seq = torch.tensor([0, 1], dtype=torch.int32, device=DEV)
    at = torch.tensor([89, 39], dtype=torch.int32, device=DEV)
    lens = torch.tensor(c.lens, dtype=torch.int32, device=DEV)
    out = torch.tensor(c.free[:6].reshape(2, 3).astype(np.int32), device=DEV)
    kept = torch.empty((2, 2, 48), dtype=torch.int32, device=DEV)
    new = torch.empty(2, dtype=torch.int32, device=DEV)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        w4.kv_append(x, x, K, V, table, seq, at, weight=w)
        w4.kv_evict(K, V, w, table, lens, 48, 5, out, kept=kept, lens_out=new)
    g = torch.Generator(device=DEV).manual_seed(45)
    for n in (90, 33, 64, 0):
        x.normal_(generator=g)
        w.uniform_(generator=g)
        lens[0] = n
        at[0] = max(n - 1, 0)
        K2, V2, w2 = K.clone(), V.clone(), w.clone()
        graph.replay()
        w4.kv_append(x, x, K2, V2, table, seq, at, weight=w2)
        kept2, new2 = w4.kv_evict(K2, V2, w2, table, lens, 48, 5, out)
        assert torch.equal(kept, kept2) and torch.equal(new, new2)
        assert torch.equal(bits(K), bits(K2)) and torch.equal(bits(V), bits(V2))
        assert torch.equal(bits(w), bits(w2))


# ---- append --------------------------------------------------------------------
def stored(x, dtype):
    if dtype != "int8":
        return x.to(DTYPES[dtype]), None
    s = x.abs().amax(-1) / np.float32(127)
    q = torch.round(x / torch.where(s == 0, torch.ones_like(s), s)[..., None])
    return q.clamp(-127, 127).to(torch.int8), s


def bits(t):
    return t.contiguous().view(torch.uint8).cpu()


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("H,D,ps,R", [(12, 64, 16, 5), (1, 8, 16, 3), (3, 96, 32, 70),
                                      (2, 256, 64, 9), (5, 40, 16, 33)])
@pytest.mark.parametrize("offset", [0, 1])
def test_append_rows(dtype, H, D, ps, R, offset):
    """Rows of a fused product, in any order, some skipped; everything else stays as it was."""
    note(f"append {dtype} {H}x{D} page {ps} rows {R} offset {offset}")
    lens = [100, 3, 2 * ps]
    c = Cache(dtype, lens, H, D, ps, 21, weight=True)
    (K, V, ks, vs, w), table = c.on_gpu()
    g = torch.Generator().manual_seed(22)
    width = H * D
    wide = torch.randn((R, 3 * width + 4 + offset), generator=g)
    wide[0, offset + width:] = 0.0                    # a zero row
    wide[1, offset + width:offset + 2 * width] *= 1e-3
    wide[R - 1, offset + 2 * width:] *= 1e4
    k = wide[:, offset + width:offset + 2 * width].unflatten(1, (H, D))
    v = wide[:, offset + 2 * width:offset + 3 * width].unflatten(1, (H, D))
    wd = wide.to(DEV)
    kd = wd[:, offset + width:offset + 2 * width].unflatten(1, (H, D))
    vd = wd[:, offset + 2 * width:offset + 3 * width].unflatten(1, (H, D))
    places = [(b, t) for b, n in enumerate(lens) for t in range(n)]
    pick = torch.randperm(len(places), generator=g)[:R].tolist()
    seq = torch.tensor([places[i][0] for i in pick], dtype=torch.int32)
    at = torch.tensor([places[i][1] for i in pick], dtype=torch.int32)
    seq[2] = -1
    bad = status()
    w4.kv_append(kd, vd, K, V, table, seq.to(DEV), at.to(DEV), k_scale=ks, v_scale=vs, weight=w,
                 d_status=bad)
    torch.cuda.synchronize()
    assert int(bad) == 0
    want = [c.K.clone(), c.V.clone(), None if c.ks is None else c.ks.clone(),
            None if c.vs is None else c.vs.clone(), c.weight.clone()]
    for r in range(R):
        if seq[r] < 0:
            continue
        page, slot = int(c.table[int(seq[r]), int(at[r]) // ps]), int(at[r]) % ps
        for j, x in enumerate((k[r], v[r])):
            val, s = stored(x, dtype)
            want[j][page, :, slot] = val
            if s is not None:
                want[2 + j][page, :, slot] = s
        want[4][page, :, slot] = 0.0
    for name, a, b in zip(("K", "V", "k_scale", "v_scale", "weight"), (K, V, ks, vs, w), want):
        if b is not None:
            assert torch.equal(bits(a), bits(b)), name


def test_append_int8_ties_and_extremes():
    """Half-way codes go to even; subnormal and huge rows keep their scale."""
    note("append int8 ties")
    D = 64
    x = torch.zeros((4, 1, D))
    x[0, 0] = torch.arange(D) - 31.5
    x[0, 0, 0] = 127.0
    x[1, 0] = torch.linspace(-1, 1, D) * 3e38
    x[2, 0] = torch.linspace(-1, 1, D) * 1e-40
    x[3, 0, 5] = -2.0
    K = torch.zeros((1, 1, 16, D), dtype=torch.int8, device=DEV)
    V = torch.zeros_like(K)
    ks = torch.zeros((1, 1, 16), device=DEV)
    vs = torch.zeros_like(ks)
    z = torch.zeros(4, dtype=torch.int32, device=DEV)
    at = torch.arange(4, dtype=torch.int32, device=DEV)
    w4.kv_append(x.to(DEV), -x.to(DEV), K, V, torch.zeros((1, 1), dtype=torch.int32, device=DEV),
                 z, at, k_scale=ks, v_scale=vs)
    for pool, sc, sign in ((K, ks, 1), (V, vs, -1)):
        codes, s = stored(sign * x[:, 0], "int8")
        assert torch.equal(pool[0, 0, :4].cpu(), codes)
        assert torch.equal(sc[0, 0, :4].cpu(), s)


@pytest.mark.parametrize("dtype", list(DTYPES))
def test_append_reports_and_skips_bad_places(dtype):
    note(f"append bad places {dtype}")
    c = Cache(dtype, [40, 20], 2, 64, 16, 23, weight=True)
    c.table[1, 1] = -7
    (K, V, ks, vs, w), table = c.on_gpu()
    x = torch.randn((5, 2, 64), generator=torch.Generator().manual_seed(5)).to(DEV)
    seq = torch.tensor([2, 0, 0, 1, -1], dtype=torch.int32, device=DEV)
    at = torch.tensor([0, 16 * c.table.shape[1], -1, 17, 10 ** 6], dtype=torch.int32, device=DEV)
    before = [bits(t) for t in (K, V, w)]
    bad = status()
    w4.kv_append(x, x, K, V, table, seq, at, k_scale=ks, v_scale=vs, weight=w, d_status=bad)
    assert int(bad) == w4.W4_ERR_BAD_SHAPE
    for t, b in zip((K, V, w), before):
        assert torch.equal(bits(t), b)


@pytest.mark.parametrize("dtype", list(DTYPES))
def test_append_nonfinite(dtype):
    note(f"append non-finite {dtype}")
    c = Cache(dtype, [16], 1, 64, 16, 24)
    (K, V, ks, vs, _), table = c.on_gpu()
    x = torch.ones((1, 1, 64), device=DEV)
    x[0, 0, 3], x[0, 0, 4], x[0, 0, 5] = math.nan, math.inf, -math.inf
    zero = torch.zeros(1, dtype=torch.int32, device=DEV)
    bad = status()
    w4.kv_append(x, x, K, V, table, zero, zero, k_scale=ks, v_scale=vs, d_status=bad)
    if dtype == "int8":
        assert int(bad) == w4.W4_ERR_NONFINITE
    else:
        row = K[int(c.table[0, 0]), 0, 0].float()
        assert int(bad) == 0
        assert torch.isnan(row[3]) and row[4] == math.inf and row[5] == -math.inf
        assert torch.equal(row[6:], torch.ones_like(row[6:]))


# ---- eviction --------------------------------------------------------------------
def evict_reference(w, n, keep, recent):
    """Old positions that stay, ascending (w: the weights of the n positions)."""
    if n <= keep:
        return np.arange(n)
    r = min(recent, keep)
    x = np.where(np.isnan(w[:n - r]), -np.inf, w[:n - r].astype(np.float64))
    # NaN lies below every number, -infinity among them
    order = np.lexsort((np.arange(n - r), np.isnan(w[:n - r]), -x))
    return np.sort(np.concatenate([order[:keep - r], np.arange(n - r, n)])).astype(np.int64)


def run_evict(c, keep, recent, max_len=0):
    """Evict and check everything: positions, copied rows, and that the rest is untouched."""
    B, H, ps, D = len(c.lens), c.heads, c.ps, c.dim
    cols_out = max(1, -(-keep // ps))
    total = c.K.shape[0]
    need = [-(-min(n, keep) // ps) for n in c.lens]
    extra = sum(need)

    def grow(t):
        if t is None:
            return None
        more = torch.zeros((extra,) + t.shape[1:], dtype=t.dtype)
        return torch.cat([t, more])

    host = [grow(t) for t in (c.K, c.V, c.ks, c.vs, c.weight)]
    K, V, ks, vs, w = [None if t is None else t.to(DEV) for t in host]
    table_out = np.full((B, cols_out), -9, np.int32)
    at = total
    for b, m in enumerate(need):
        table_out[b, :m] = np.arange(at, at + m)[::-1]
        at += m
    table = torch.from_numpy(c.table.astype(np.int32)).to(DEV)
    lens = torch.tensor(c.lens, dtype=torch.int32, device=DEV)
    bad = status()
    kept, lens_out = w4.kv_evict(K, V, w, table, lens, keep, recent,
                                 torch.from_numpy(table_out).to(DEV), k_scale=ks, v_scale=vs,
                                 max_len=max_len, d_status=bad)
    torch.cuda.synchronize()
    assert int(bad) == 0
    assert lens_out.cpu().tolist() == [min(n, keep) for n in c.lens]
    got = kept.cpu().numpy()
    want = [t if t is None else t.clone() for t in host]
    for b, n in enumerate(c.lens):
        pages = c.table[b, :-(-n // ps)]
        for h in range(H):
            old = evict_reference(c.weight[pages, h].reshape(-1)[:n].numpy(), n, keep, recent)
            m = min(n, keep)
            assert np.array_equal(got[b, h, :m], old), (b, h)
            assert (got[b, h, m:] == -1).all()
            new = np.arange(m)
            src, dst = c.table[b, old // ps], table_out[b, new // ps].astype(np.int64)
            for t in want:
                if t is not None:
                    t[dst, h, new % ps] = t[src, h, old % ps]
    for name, a, b in zip(("K", "V", "k_scale", "v_scale", "weight"), (K, V, ks, vs, w), want):
        if b is not None:
            assert torch.equal(bits(a), bits(b)), name


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("H,D,ps", [(2, 64, 16), (3, 96, 32), (1, 8, 64), (2, 40, 16)])
def test_evict_edge_lengths(dtype, H, D, ps):
    note(f"evict {dtype} {H}x{D} page {ps}")
    lens = [0, 1, 15, 16, 17, 40, 41, 64, 100, 333]
    for keep, recent in ((40, 7), (1, 0), (1, 5), (33, 33), (64, 0)):
        run_evict(Cache(dtype, lens, H, D, ps, 25, weight=True), keep, recent)


@pytest.mark.parametrize("kind", ["equal", "few", "nan", "inf", "zeros", "ascending", "descending"])
def test_evict_ties_and_odd_weights(kind):
    note(f"evict weights {kind}")
    c = Cache("bf16", [700, 257, 64], 2, 64, 16, 26, weight=True)
    g = torch.Generator().manual_seed(27)
    w = c.weight
    if kind == "equal":
        w.fill_(0.25)
    elif kind == "few":
        w.copy_(torch.randint(0, 3, w.shape, generator=g).float())
    elif kind == "nan":
        w[torch.rand(w.shape, generator=g) < 0.7] = math.nan
        w[torch.rand(w.shape, generator=g) < 0.1] = -math.inf
    elif kind == "inf":
        w[torch.rand(w.shape, generator=g) < 0.3] = math.inf
    elif kind == "zeros":  # -0 and +0 tie
        w.copy_(torch.where(torch.rand(w.shape, generator=g) < 0.5, 0.0, -0.0))
    else:
        for b, n in enumerate(c.lens):
            t = torch.arange(n)
            page = torch.from_numpy(c.table[b])[t // 16]
            w[page, :, t % 16] = (t if kind == "ascending" else n - t).float()[:, None]
    for keep, recent in ((100, 30), (250, 0), (699, 1)):
        run_evict(c, keep, recent)


@pytest.mark.parametrize("n,keep,recent", [(5000, 2000, 100), (40000, 9001, 64),
                                           (70001, 70000, 0), (140000, 3, 1)])
def test_evict_long(n, keep, recent):
    note(f"evict long {n} -> {keep}")
    run_evict(Cache("int8", [n, n // 2], 1, 8, 64, 28, weight=True), keep, recent, max_len=n)


def test_evict_reports_bad_pages():
    note("evict bad pages")
    c = Cache("fp32", [64], 1, 64, 16, 29, weight=True, spare=4)
    (K, V, _, _, w), table = c.on_gpu()
    table[0, 2] = -1
    out = torch.tensor([[int(c.free[0]), 10 ** 6]], dtype=torch.int32, device=DEV)
    before = bits(K[table[0, :2].long()])
    bad = status()
    kept, lens_out = w4.kv_evict(K, V, w, table, torch.tensor([64], dtype=torch.int32, device=DEV),
                                 32, 16, out, d_status=bad)
    assert int(bad) == w4.W4_ERR_BAD_SHAPE
    assert int(lens_out) == 32
    assert torch.equal(bits(K[table[0, :2].long()]), before)
    assert not set(range(32, 48)) & set(kept[0, 0].cpu().tolist())


# ---- log probabilities ---------------------------------------------------------
def lp_check(x, tokens, top, ld_pad=0, offset=0, d_status=None):
    M, N = x.shape
    wide = torch.full((M, N + ld_pad + offset), 77.0, device=DEV)
    wide[:, offset:offset + N] = x.to(DEV)
    view = wide[:, offset:offset + N]
    lp, ent, ids, best = w4.lp_logprobs(view, None if tokens is None else tokens.to(DEV), top,
                                        d_status=d_status)
    torch.cuda.synchronize()
    d = x.double()
    m = d.amax(1, keepdim=True)
    m0 = torch.where(m == -math.inf, torch.zeros_like(m), m)
    S = torch.exp(d - m0).sum(1, keepdim=True)
    logS = torch.log(S)
    # relative to the maximum: at 3e38 even 64 bits would absorb log S
    rel = torch.where(d == -math.inf, d, d - m0)
    chain = 16 + N / 256
    p = torch.exp(rel - logS)
    # a forbidden token has -infinity, also where the whole row is forbidden; so has one whose
    # log probability no fp32 number reaches
    logp = torch.where(d == -math.inf, d, rel - logS)
    logp = torch.where(logp.float() == -math.inf, torch.full_like(d, -math.inf), logp)
    dist = torch.where(d == -math.inf, torch.zeros_like(d), (d - m0).abs())
    p = torch.where(m == -math.inf, torch.zeros_like(p), p)
    # each term of S carries eps (|x - m| + 2), its sum the chain
    s_rel = EPS * ((p * dist).sum(1) + chain)
    tol_s = 2 * s_rel + 4 * EPS * logS[:, 0].abs()
    ent_ref = torch.where(m[:, 0] == -math.inf, torch.zeros(M, dtype=torch.float64),
                          (p * torch.where(p == 0, torch.zeros_like(d), logS - rel)).sum(1))
    ent_tol = tol_s + EPS * (p * dist * (dist + chain + 4)).sum(1) + 2 * s_rel * (p * dist).sum(1)
    assert ((ent.cpu().double() - ent_ref).abs() <= ent_tol + 1e-37).all()

    def close(got, want, far):
        gone = want == -math.inf
        assert torch.equal(got.cpu().double() == -math.inf, gone)
        lim = tol_s.reshape((-1,) + (1,) * (want.dim() - 1)) + 3 * EPS * far + 1e-37
        err = (got.cpu().double() - want).abs()
        assert (err[~gone] <= lim.expand_as(err)[~gone]).all()

    if tokens is None:
        assert lp is None
    else:
        at = tokens[:, None]
        close(lp, logp.gather(1, at)[:, 0], dist.gather(1, at)[:, 0])
    order = np.lexsort((np.broadcast_to(np.arange(N), (M, N)), -x.numpy().astype(np.float64)))
    order = torch.from_numpy(order[:, :top].copy())
    assert ids.shape == (M, top) and torch.equal(ids.cpu(), order)
    if top:
        close(best, logp.gather(1, order), dist.gather(1, order))


@pytest.mark.parametrize("N", [1, 2, 3, 63, 64, 65, 255, 257, 1000, 4097, 50257, 100003, 200001])
@pytest.mark.parametrize("M", [1, 3])
@pytest.mark.parametrize("top", [0, 1, 5, 20, 64])
def test_logprobs_sizes(M, N, top):
    g = torch.Generator().manual_seed(N + M)
    note(f"logprobs {M}x{N} top {top}")
    x = torch.randn((M, N), generator=g) * 3
    lp_check(x, torch.randint(0, N, (M,), generator=g), min(top, N))


@pytest.mark.parametrize("M,N,top", [(58, 50257, 5), (300, 8191, 20), (1500, 1021, 3),
                                     (2600, 97, 7)])
@pytest.mark.parametrize("pad,offset", [(0, 0), (47, 1), (3, 0), (64, 3)])
def test_logprobs_rows_and_strides(M, N, top, pad, offset):
    note(f"logprobs {M}x{N} top {top} pad {pad} offset {offset}")
    g = torch.Generator().manual_seed(M)
    x = torch.randn((M, N), generator=g) * 3
    lp_check(x, torch.randint(0, N, (M,), generator=g), top, pad, offset)


def lp_rows(kind, N, g):
    x = torch.randn((6, N), generator=g)
    if kind == "masked":
        x[torch.rand(x.shape, generator=g) < 0.9] = -math.inf
        x[1] = -math.inf
        x[2] = -math.inf
        x[2, N // 2] = 1.5
        x[3, 3:] = -math.inf
    elif kind == "lowest":  # masks of the type's lowest value
        x[torch.rand(x.shape, generator=g) < 0.9] = torch.finfo(torch.float32).min
        x[1] = torch.finfo(torch.float32).min
        x[2, :] = torch.finfo(torch.float32).min
        x[2, 7 % N] = torch.finfo(torch.float32).max
    elif kind == "equal":
        x[:3] = 0.0
        x[3:] = -7.25
        x[4, N - 1] = -7.0
    elif kind == "ties":
        x = torch.randint(-3, 3, (6, N), generator=g).float()
        x[0] = torch.where(torch.rand(N, generator=g) < 0.5, 0.0, -0.0)
    elif kind == "ascending":
        x[:] = torch.arange(N) * 0.001
    elif kind == "descending":
        x[:] = torch.arange(N) * -0.001
    elif kind == "wide":
        x *= 1e4
        x[1] *= 1e25
    elif kind == "saw":  # largest entries in one stretch, others of one residue
        x[0, ::64] += 50
        x[1, 128:160] += 50
        x[2, -70:] += torch.arange(70) * 1.0
        x[3, :70] += torch.arange(70) * 1.0
    return x


@pytest.mark.parametrize("kind", ["masked", "lowest", "equal", "ties", "ascending", "descending",
                                  "wide", "saw"])
@pytest.mark.parametrize("N", [97, 3000, 50257, 131072])
@pytest.mark.parametrize("top", [1, 20, 64])
def test_logprobs_odd_rows(kind, N, top):
    note(f"logprobs rows {kind} {N} top {top}")
    g = torch.Generator().manual_seed(31)
    x = lp_rows(kind, N, g)
    bad = status()
    lp_check(x, torch.randint(0, N, (6,), generator=g), top, d_status=bad)
    lp_check(x.repeat(60, 1), torch.randint(0, N, (360,), generator=g), top, d_status=bad)
    assert int(bad) == 0


@pytest.mark.parametrize("M,N", [(4, 50257), (400, 1000), (4, 30)])
def test_logprobs_reports_nonfinite_rows_and_bad_tokens(M, N):
    note(f"logprobs non-finite {M}x{N}")
    g = torch.Generator().manual_seed(33)
    x = torch.randn((M, N), generator=g)
    x[1, N // 3] = math.nan
    x[2, N - 1] = math.inf
    tokens = torch.randint(0, N, (M,), generator=g)
    bad = status()
    lp, ent, ids, best = w4.lp_logprobs(x.to(DEV), tokens.to(DEV), 9, d_status=bad)
    assert int(bad) == w4.W4_ERR_NONFINITE
    for r in (1, 2):
        assert torch.isnan(lp[r]) and torch.isnan(ent[r]) and torch.isnan(best[r]).all()
        assert (ids[r] == -1).all()
    fine = [r for r in range(M) if r not in (1, 2)]
    lp_check(x[fine], tokens[fine], 9)
    assert torch.isfinite(lp[fine]).all() and torch.isfinite(ent[fine]).all()
    x[1], x[2] = 0.5, 0.25
    tokens[0], tokens[3] = N, -1
    bad.zero_()
    lp, ent, _, _ = w4.lp_logprobs(x.to(DEV), tokens.to(DEV), 0, d_status=bad)
    assert int(bad) == w4.W4_ERR_BAD_SHAPE
    assert torch.isnan(lp[0]) and torch.isnan(lp[3]) and torch.isfinite(lp[1])
    assert torch.isfinite(ent).all()


def test_logprobs_without_tokens_and_empty():
    lp_check(torch.randn((2, 300), generator=torch.Generator().manual_seed(1)), None, 4)
    lp, ent, ids, best = w4.lp_logprobs(torch.empty((0, 50), device=DEV),
                                        torch.empty(0, dtype=torch.int64, device=DEV), 3)
    assert lp.shape == (0,) and ent.shape == (0,) and ids.shape == (0, 3) and best.shape == (0, 3)


def test_logprobs_in_a_graph():
    note("logprobs graph")
    for M in (1, 40):
        x = torch.randn((M, 50257), device=DEV)
        tokens = torch.zeros(M, dtype=torch.int64, device=DEV)
        ws = torch.full((1 << 22,), 0x5A, dtype=torch.uint8, device=DEV)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = w4.lp_logprobs(x, tokens, 10, workspace=ws)
        for i in range(4):
            x.normal_()
            ws.fill_(i)
            graph.replay()
            for a, b in zip(got, w4.lp_logprobs(x, tokens, 10)):
                assert torch.equal(a, b)


# ---- refusals of the binding (the host checks of the C entry points need no GPU) ----
def test_empty_calls():
    K = torch.zeros((1, 2, 16, 64), device=DEV)
    none = torch.empty(0, dtype=torch.int32, device=DEV)
    table = torch.empty((0, 3), dtype=torch.int32, device=DEV)
    q = torch.empty((0, 4, 64), device=DEV)
    assert w4.kv_attend(q, K, K, table, none).shape == (0, 4, 64)
    w4.kv_append(torch.empty((0, 2, 64), device=DEV), torch.empty((0, 2, 64), device=DEV), K, K,
                 table, none, none)
    kept, lens_out = w4.kv_evict(K, K, torch.zeros((1, 2, 16), device=DEV), table, none, 4, 0,
                                 table)
    assert kept.shape == (0, 2, 4) and lens_out.shape == (0,)
    # a table without columns: every sequence is empty
    q = torch.ones((2, 4, 64), device=DEV)
    lens = torch.zeros(2, dtype=torch.int32, device=DEV)
    out = w4.kv_attend(q, K, K, torch.empty((2, 0), dtype=torch.int32, device=DEV), lens)
    assert not out.any()


def test_binding_refuses():
    K = torch.zeros((2, 2, 16, 64), device=DEV)
    table = torch.zeros((1, 2), dtype=torch.int32, device=DEV)
    lens = torch.ones(1, dtype=torch.int32, device=DEV)
    q = torch.zeros((1, 4, 64), device=DEV)
    for exc, call in [
        (TypeError, lambda: w4.kv_attend(q.half(), K, K, table, lens)),
        (TypeError, lambda: w4.kv_attend(q, K, K.half(), table, lens)),
        (TypeError, lambda: w4.kv_attend(q, K.double(), K.double(), table, lens)),
        (TypeError, lambda: w4.kv_attend(q, K, K, table.long(), lens)),
        (TypeError, lambda: w4.kv_attend(q.cpu(), K, K, table, lens)),
        (ValueError, lambda: w4.kv_attend(q[:, :, :32], K, K, table, lens)),
        (ValueError, lambda: w4.kv_attend(q, K, K[:1], table, lens)),
        (ValueError, lambda: w4.kv_attend(q, K, K, table, lens.expand(3).contiguous())),
        (ValueError, lambda: w4.kv_attend(q, K.to(torch.int8), K.to(torch.int8), table, lens)),
        (ValueError, lambda: w4.kv_attend(q.transpose(1, 2).contiguous().transpose(1, 2), K, K,
                                          table, lens)),
        (ValueError, lambda: w4.kv_attend(q, K, K, table, lens, weight=K[:, :, :, 0])),
        (ValueError, lambda: w4.kv_attend(q, K, K, table, lens, out=q[:, :2].contiguous())),
        (w4.W4Error, lambda: w4.kv_attend(q[:, :3], K, K, table, lens)),
        (w4.W4Error, lambda: w4.kv_attend(q, K, K, table, lens, max_len=-1)),
        (ValueError, lambda: w4.kv_append(q, q, K, K, table, lens, lens)),
        (ValueError, lambda: w4.kv_evict(K, K, None, table, lens, 1, 0, table)),
        (w4.W4Error, lambda: w4.kv_evict(K, K, torch.zeros((2, 2, 16), device=DEV), table, lens,
                                         0, 0, table)),
        (w4.W4Error, lambda: w4.kv_evict(K, K, torch.zeros((2, 2, 16), device=DEV), table, lens,
                                         20, 0, table[:, :1].contiguous())),
        (TypeError, lambda: w4.lp_logprobs(q[0].half())),
        (ValueError, lambda: w4.lp_logprobs(q)),
        (ValueError, lambda: w4.lp_logprobs(q[0].t())),
        (ValueError, lambda: w4.lp_logprobs(q[0], lens.long())),
        (w4.W4Error, lambda: w4.lp_logprobs(q[0], None, 65)),
        (w4.W4Error, lambda: w4.lp_logprobs(q[0], None, -1)),
        (w4.W4Error, lambda: w4.lp_logprobs(q[0, :, :3], None, 4)),
    ]:
        with pytest.raises(exc):
            call()
    torch.cuda.synchronize()

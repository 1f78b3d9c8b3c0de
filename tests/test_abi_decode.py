"""Host-side checks of the paged cache's and the log probabilities' entry points (no GPU call)."""
import ctypes

import pytest
import torch

import w4_block_dequant_amd as w4

LIB = w4.library()
A = 1 << 12  # a fake, 4 KiB-aligned "device address": never dereferenced
OK, NULL, SHAPE, ALIGN, WS = (w4.W4_OK, w4.W4_ERR_NULL_PTR, w4.W4_ERR_BAD_SHAPE,
                              w4.W4_ERR_MISALIGNED, w4.W4_ERR_WORKSPACE)


def cache(**over):
    f = dict(k=A, v=A, k_scale=None, v_scale=None, weight=None, pages=100, heads=4, page_size=16,
             head_dim=64, dtype=2)
    f.update(over)
    return w4.KvCache(*f.values())


def attend(c=None, q=A, q_stride=None, q_heads=8, table=A, seqs=2, cols=10, lens=A, starts=None,
           max_len=0, out=A, ws=A, wsb=1 << 40, d_status=None):
    c = cache() if c is None else c
    stride = q_heads * c.head_dim if q_stride is None else q_stride
    return LIB.kv_check_attend_args(ctypes.byref(c), q, stride, q_heads, table, seqs, cols, lens,
                                    starts, max_len, out, ws, wsb, d_status)


def test_cache_description():
    assert attend() == OK
    assert LIB.kv_check_attend_args(None, A, 512, 8, A, 2, 10, A, None, 0, A, A, 0, None) == NULL
    for bad in (dict(dtype=4), dict(dtype=-1), dict(pages=0), dict(pages=1 << 31), dict(heads=0),
                dict(page_size=8), dict(page_size=24), dict(page_size=8192), dict(page_size=0),
                dict(head_dim=0), dict(head_dim=12), dict(head_dim=264),
                dict(pages=(1 << 31) - 1, heads=65536)):
        assert attend(cache(**bad)) == SHAPE, bad
    for size in (16, 32, 4096):
        assert attend(cache(page_size=size)) == OK
    assert attend(cache(k=None)) == NULL
    assert attend(cache(dtype=3)) == NULL                       # int8 without scales
    assert attend(cache(dtype=3, k_scale=A, v_scale=A)) == OK
    assert attend(cache(k=A + 8)) == ALIGN
    assert attend(cache(weight=A + 2)) == ALIGN


def test_attend_arguments():
    assert attend(q_heads=6) == SHAPE
    assert attend(q_heads=0) == SHAPE
    assert attend(q_stride=511) == SHAPE
    assert attend(q_stride=513) == OK
    assert attend(seqs=-1) == SHAPE
    assert attend(cols=-1) == SHAPE
    assert attend(max_len=-1) == SHAPE
    assert attend(max_len=(1 << 30) + 1) == SHAPE
    assert attend(seqs=1 << 30) == SHAPE
    for name in ("q", "table", "lens", "out"):
        assert attend(**{name: None}) == NULL
    for name in ("q", "table", "lens", "starts", "out", "d_status"):
        assert attend(**{name: A + 2}) == ALIGN
    assert attend(seqs=0, q=None, table=None, lens=None, out=None, ws=None, wsb=0) == OK
    assert attend(cols=0, table=None) == OK


def test_attend_workspace():
    c = cache(weight=A)
    need = LIB.kv_attend_workspace_bytes(ctypes.byref(c), 2, 8, 160)
    assert need > 0
    assert attend(c, ws=None, wsb=0) == WS
    assert attend(c, wsb=need - 1) == WS
    assert attend(c, wsb=need) == OK
    assert attend(c, ws=A + 16, wsb=need) == ALIGN
    assert LIB.kv_attend_workspace_bytes(ctypes.byref(cache(head_dim=7)), 2, 8, 160) == 0
    # enough for any smaller bound on the lengths too
    for weight in (None, A):
        for dtype in (0, 2):
            c = cache(weight=weight, dtype=dtype)
            for seqs, heads in ((1, 4), (3, 8), (40, 64)):
                sizes = [LIB.kv_attend_workspace_bytes(ctypes.byref(c), seqs, heads, n)
                         for n in (1, 15, 160, 1000, 5000, 131072)]
                assert sizes == sorted(sizes)


def append(c=None, k=A, ks=256, v=A, vs=256, rows=3, table=A, seqs=2, cols=10, seq=A, at=A,
           d_status=None):
    return LIB.kv_append(ctypes.byref(cache() if c is None else c), k, ks, v, vs, rows, table, seqs,
                         cols, seq, at, d_status, None)


def test_append_arguments():
    assert append(rows=0, k=None, v=None, table=None, seq=None, at=None) == OK
    assert append(cache(head_dim=7)) == SHAPE
    assert append(ks=255) == SHAPE
    assert append(vs=255) == SHAPE
    assert append(rows=-1) == SHAPE
    assert append(rows=1 << 31) == SHAPE
    assert append(seqs=-1) == SHAPE
    for name in ("k", "v", "table", "seq", "at"):
        assert append(**{name: None}) == NULL
        assert append(**{name: A + 2}) == ALIGN


def evict(c=None, table=A, seqs=2, cols=10, lens=A, max_len=0, keep=40, recent=8, out=A,
          cols_out=3, kept=A, lens_out=A, d_status=None):
    return LIB.kv_evict(ctypes.byref(cache(weight=A) if c is None else c), table, seqs, cols, lens,
                        max_len, keep, recent, out, cols_out, kept, lens_out, d_status, None)


def test_evict_arguments():
    assert evict(seqs=0, table=None, lens=None, out=None, kept=None, lens_out=None) == OK
    assert evict(cache()) == NULL                                # no weights
    assert evict(keep=0) == SHAPE
    assert evict(recent=-1) == SHAPE
    assert evict(cols_out=2) == SHAPE                            # 32 slots for 40 rows
    assert evict(max_len=(1 << 24) + 1) == SHAPE
    assert evict(seqs=20000) == SHAPE
    for name in ("table", "lens", "out", "kept", "lens_out"):
        assert evict(**{name: None}) == NULL
        assert evict(**{name: A + 2}) == ALIGN


def logprobs(x=A, M=3, N=100, ld=100, tokens=A, top=5, lp=A, ent=A, ids=A, best=A, ws=A,
             wsb=1 << 40, d_status=None):
    return LIB.lp_check_logprobs_args(x, M, N, ld, tokens, top, lp, ent, ids, best, ws, wsb,
                                      d_status)


def test_logprobs_arguments():
    assert logprobs() == OK
    assert logprobs(M=0, x=None, tokens=None, lp=None, ent=None, ids=None, best=None, N=0, ld=0) == OK
    for bad in (dict(M=-1), dict(N=-1), dict(N=0), dict(ld=99), dict(top=-1), dict(top=65),
                dict(top=5, N=4), dict(N=1 << 31, ld=1 << 31), dict(M=1 << 31)):
        assert logprobs(**bad) == SHAPE, bad
    assert logprobs(x=None) == NULL
    assert logprobs(tokens=None) == NULL
    assert logprobs(tokens=None, lp=None) == OK
    assert logprobs(ids=None) == NULL
    assert logprobs(ids=None, best=None, top=0) == OK
    assert logprobs(ent=None) == OK
    assert logprobs(tokens=A + 4) == ALIGN
    assert logprobs(ids=A + 4) == ALIGN
    for name in ("x", "lp", "ent", "best", "d_status"):
        assert logprobs(**{name: A + 2}) == ALIGN
    for M, N, top in ((1, 50257, 1), (1, 50257, 20), (58, 50257, 5), (4, 200001, 64)):
        need = LIB.lp_logprobs_workspace_bytes(M, N, top)
        if need:
            assert logprobs(M=M, N=N, ld=N, top=top, wsb=need - 1) == WS
            assert logprobs(M=M, N=N, ld=N, top=top, ws=None, wsb=0) == WS
            assert logprobs(M=M, N=N, ld=N, top=top, ws=A + 16, wsb=need) == ALIGN
        assert logprobs(M=M, N=N, ld=N, top=top, wsb=need) == OK


@pytest.mark.skipif(torch.cuda.is_available(), reason="needs a machine without a GPU")
def test_well_formed_calls_reach_the_device_check():
    assert append() == w4.W4_ERR_DEVICE
    assert evict() == w4.W4_ERR_DEVICE
    assert LIB.lp_logprobs(A, 3, 100, 100, A, 5, A, A, A, A, A, 1 << 40, None, None) == w4.W4_ERR_DEVICE

"""Rotary positions and the 8-bit cache without a GPU: what the C ABI and the
wrappers refuse before anything is enqueued, sizes, frequencies."""
import ctypes
import math

import pytest
import torch

import bit_quantized_attention_sage_b200 as sage
from bit_quantized_attention_sage_b200 import build, kvcache

P = ctypes.c_void_p(1 << 16)
ODD = ctypes.c_void_p((1 << 16) + 1)
S3 = (ctypes.c_longlong * 3)(4096, 1024, 128)
NEG = (ctypes.c_longlong * 3)(4096, -1, 128)


@pytest.fixture(scope="module")
def L():
    build.build()
    return sage.lib()


def cache(**kw):
    a = dict(k_i8=1 << 16, k_scale=1 << 16, v_f8=1 << 16, v_exp=1 << 16, weight=1 << 16, n_pages=8,
             heads=2, D=128)
    a.update(kw)
    return ctypes.byref(kvcache._Cache(*a.values()))


def seqs(**kw):
    a = dict(pages=1 << 16, lengths=1 << 16, B=2, max_pages=4)
    a.update(kw)
    return ctypes.byref(kvcache._Seqs(*a.values()))


def query(**kw):
    a = dict(q=1 << 16, q_strides=S3, q_lens=None, type=0, H=4, Nq=1, max_len=256, scale=0.1)
    a.update(kw)
    return ctypes.byref(kvcache._Query(*a.values()))


BAD_CACHE = [dict(k_i8=None), dict(k_i8=(1 << 16) + 8), dict(v_f8=None), dict(k_scale=None),
             dict(v_exp=None), dict(weight=(1 << 16) + 2), dict(n_pages=0), dict(heads=0),
             dict(heads=65536), dict(D=96)]
BAD_SEQS = [dict(pages=None), dict(lengths=None), dict(lengths=(1 << 16) + 2), dict(B=0),
            dict(B=65536), dict(max_pages=0), dict(max_pages=(1 << 24) + 1)]


def calls(L):
    """The cache's entry points as functions of (cache, seqs)."""
    yield lambda c, s: L.sage_cache_append(c, s, P, P, 0, 1, S3, S3, None, None, None)
    yield lambda c, s: L.sage_cache_read(c, s, 1, None, None, P, P, None, None)
    yield lambda c, s: L.sage_cache_attn(c, s, query(), 0, 0, 0, 0, P, S3, None, P, 1 << 40, None)
    yield lambda c, s: L.sage_cache_weights(c, s, query(), 0, 0, 0, 0, P, 0, None)
    yield lambda c, s: L.sage_cache_evict(c, s, 64, 0, 0, None, 0, P, P, P, 1 << 40, None)


def test_bad_caches_and_sequences(L):
    for f in calls(L):
        for kw in BAD_CACHE:
            assert f(cache(**kw), seqs()) == 1, kw
        for kw in BAD_SEQS:
            assert f(cache(), seqs(**kw)) == 1, kw
        assert f(None, seqs()) == 1 and f(cache(), None) == 1
        # pages * heads past 2^30
        assert f(cache(n_pages=(1 << 29) + 1), seqs()) == 2


def test_append_arguments(L):
    def call(k=P, v=P, type=0, n=1, ks=S3, vs=S3, nn=None, sh=None):
        return L.sage_cache_append(cache(), seqs(), k, v, type, n, ks, vs, nn, sh, None)

    for kw in (dict(k=None), dict(v=None), dict(k=ODD), dict(type=2), dict(type=-1), dict(n=0),
               dict(ks=None), dict(vs=NEG), dict(nn=ODD), dict(sh=ODD)):
        assert call(**kw) == 1, kw


def test_read_arguments(L):
    def call(n=1, st=None, sh=None, k=P, v=P, w=None, c=None):
        return L.sage_cache_read(c or cache(), seqs(), n, st, sh, k, v, w, None)

    for kw in (dict(n=0), dict(st=ODD), dict(sh=ctypes.c_void_p(4100)), dict(k=None), dict(v=ODD),
               dict(w=ODD), dict(w=P, c=cache(weight=None))):
        assert call(**kw) == 1, kw


def test_attention_arguments(L):
    def call(q=None, mask=0, mb=0, win=0, sink=0, out=P, os=S3, lse=None, ws=P, nb=1 << 40):
        return L.sage_cache_attn(cache(), seqs(), q or query(), mask, mb, win, sink, out, os, lse, ws, nb,
                                 None)

    for kw in (dict(q=query(q=None)), dict(q=query(q=65537)), dict(q=query(q_strides=NEG)),
               dict(q=query(q_lens=65538)), dict(q=query(type=2)), dict(q=query(H=3)),
               dict(q=query(H=0)), dict(q=query(Nq=0)), dict(q=query(Nq=(1 << 24) + 1)),
               dict(q=query(max_len=-1)), dict(q=query(max_len=257)),
               dict(q=query(scale=float("nan"))), dict(q=query(scale=float("inf"))),
               dict(q=query(scale=-1.0)), dict(mask=4), dict(mask=-1), dict(mask=2),
               dict(mask=3, mb=0, win=1), dict(mask=3, mb=1, win=0), dict(mask=3, mb=1, win=1, sink=-1),
               dict(out=None), dict(out=ODD), dict(os=NEG), dict(lse=ODD)):
        assert call(**kw) == 1, kw
    assert L.sage_cache_weights(cache(weight=None), seqs(), query(), 0, 0, 0, 0, P, 0, None) == 1
    assert L.sage_cache_weights(cache(), seqs(), query(), 0, 0, 0, 0, None, 0, None) == 1
    assert L.sage_cache_weights(cache(), seqs(), query(), 2, 0, 0, 0, P, 0, None) == 1


def test_evict_arguments_and_workspace(L):
    need = L.sage_cache_evict_workspace_bytes(2, 2, 128, 100, 1)
    # a place for every survivor; in place two staged pages a sequence and
    # head: codes, weights, scale, exponent
    assert L.sage_cache_evict_workspace_bytes(2, 2, 128, 100, 0) == 2 * 2 * 100 * 4
    assert need == 1600 + -(-(2 * 2 * 2 * (2 * 64 * 128 + 64 * 4 + 4 + 1)) // 16) * 16
    for a in ((0, 2, 128, 100), (2, 0, 128, 100), (2, 2, 96, 100), (2, 2, 128, 0)):
        assert L.sage_cache_evict_workspace_bytes(*a, 1) == 0

    def call(keep=100, sink=0, recent=0, po=None, width=0, kept=P, lo=P, ws=P, nb=need, c=None):
        return L.sage_cache_evict(c or cache(), seqs(), keep, sink, recent, po, width, kept, lo, ws, nb,
                                  None)

    for kw in (dict(keep=0), dict(sink=-1), dict(recent=-1), dict(sink=60, recent=41), dict(po=P, width=1),
               dict(po=ODD, width=2), dict(po=P, width=2, nb=1599), dict(kept=None), dict(lo=None), dict(ws=None), dict(nb=need - 1),
               dict(ws=ctypes.c_void_p(4100)), dict(c=cache(weight=None))):
        assert call(**kw) == 1, kw


def test_rope_arguments(L):
    def call(x=P, y=P, type=0, B=1, H=1, N=1, D=64, R=64, xs=S3, ys=S3, pos=P, p64=1, ps=0, f=P, amp=1.0):
        return L.sage_rope(x, y, type, B, H, N, D, R, xs, ys, pos, p64, ps, f, amp, 0, 0, None)

    for kw in (dict(x=None), dict(y=ODD), dict(type=3), dict(type=2, x=ctypes.c_void_p(65538)), dict(B=0),
               dict(B=65536), dict(H=65536), dict(N=0), dict(R=63), dict(R=66), dict(R=-2), dict(xs=NEG),
               dict(ys=None), dict(pos=None), dict(pos=ctypes.c_void_p(65540)), dict(ps=-1), dict(f=None),
               dict(amp=float("inf"))):
        assert call(**kw) == 1, kw
    assert call(D=4096, R=2050) == 2
    assert L.sage_rope_tables(4, 3, P, 1, P, 1.0, P, P, None) == 1
    assert L.sage_rope_tables(4, 4, P, 1, P, 1.0, None, P, None) == 1


def test_frequencies():
    f, amp = sage.rope_freqs(8, 100.0, device="cpu")
    assert amp == 1.0 and torch.allclose(f, 100.0 ** -torch.tensor([0, 0.25, 0.5, 0.75]).double(),
                                         rtol=1e-15)
    g, _ = sage.rope_freqs(8, 100.0, ("linear", 4), device="cpu")
    assert torch.allclose(g * 4, f, rtol=1e-15)
    # ntk: the lowest frequency becomes that of linear scaling, the highest stays
    g, _ = sage.rope_freqs(8, 100.0, ("ntk", 4), device="cpu")
    assert g[0] == 1 and math.isclose(g[-1], f[-1] / 4, rel_tol=1e-12)
    # yarn: fast pairs keep their frequency, slow ones are divided
    f, _ = sage.rope_freqs(64, device="cpu")
    g, amp = sage.rope_freqs(64, scaling=("yarn", 8, 4096), device="cpu")
    turns = 4096 * f / (2 * math.pi)
    assert torch.equal(g[turns > 32], f[turns > 32])
    assert torch.allclose(g[turns < 1] * 8, f[turns < 1], rtol=1e-15)
    mid = (turns > 1) & (turns < 32)
    assert ((g < f) & (g > f / 8))[mid].all() and math.isclose(amp, 0.1 * math.log(8) + 1)
    for bad in ((7,), (0,), (8, -1.0), (8, 1e4, ("linear", 0)), (8, 1e4, ("linear",)), (8, 1e4, ("none", 2)),
                (8, 1e4, ("yarn", 2)), (8, 1e4, ("yarn", 2, 100, 1, 1)), (8, 1e4, ("ntk", math.inf))):
        with pytest.raises(ValueError):
            sage.rope_freqs(*bad, device="cpu")


def test_cpu_tensors_are_refused():
    x = torch.zeros((1, 2, 3, 64), dtype=torch.bfloat16)
    f, _ = sage.rope_freqs(64, device="cpu")
    with pytest.raises(ValueError):
        sage.rope(x, torch.arange(3), f)
    with pytest.raises(ValueError):
        sage.rope_tables(torch.arange(3), f)
    with pytest.raises(ValueError):
        sage.KVCache8(4, 2, 64, device="cpu")
    with pytest.raises(ValueError):
        kvcache._mask(("window", 1, 2))


def test_weights_that_vector_loads_cannot_read(L):
    # the prune reads four weights at a time
    for f in calls(L):
        assert f(cache(weight=(1 << 16) + 4), seqs()) == 1
        assert f(cache(weight=(1 << 16) + 8), seqs()) == 1


def test_evict_must_not_write_the_lengths_it_reads(L):
    s = ctypes.c_void_p(1 << 16)
    assert L.sage_cache_evict(cache(), seqs(lengths=1 << 16), 64, 0, 0, None, 0, P, s, P, 1 << 40,
                              None) == 1


def test_more_heads_than_blocks(L):
    # a decode call's join has a block for each of B * heads
    c = cache(n_pages=1, heads=65535)
    assert L.sage_cache_attn(c, seqs(B=65535, max_pages=100), query(H=65535, max_len=6400), 0, 0, 0, 0,
                             P, S3, None, P, 1 << 60, None) == 2


def test_rows_are_needed_where_they_are_read(L):
    # a query without rows is refused by the attention; the weights take it,
    # without q and lse, and refuse what is wrong with the rest
    for kw in (dict(H=0), dict(Nq=0), dict(H=0, Nq=0)):
        assert L.sage_cache_attn(cache(), seqs(), query(**kw), 0, 0, 0, 0, P, S3, None, P, 1 << 40, None) == 1
    for kw in (dict(H=-2), dict(Nq=-1), dict(Nq=0, type=2), dict(H=0, q_lens=65538), dict(Nq=0, max_len=257),
               dict(Nq=0, scale=float("nan"))):
        assert L.sage_cache_weights(cache(), seqs(), query(**kw), 0, 0, 0, 0, P, 0, None) == 1, kw
    assert L.sage_cache_weights(cache(weight=None), seqs(), query(Nq=0), 0, 0, 0, 0, None, 0, None) == 1
    assert L.sage_cache_weights(cache(), seqs(), None, 0, 0, 0, 0, P, 0, None) == 1
    assert L.sage_cache_attn(cache(), seqs(), None, 0, 0, 0, 0, P, S3, None, P, 1 << 40, None) == 1


def test_outputs_over_their_inputs():
    # against the elements themselves, of strided views of one buffer
    import random
    rng = random.Random(1)
    for dt in (torch.float32, torch.bfloat16):
        base = torch.zeros(2000, dtype=dt)
        index = torch.arange(2000)
        seen = [0, 0]
        for _ in range(3000):
            shape = [rng.randint(1, 3) for _ in range(4)]

            def view():
                step, at = [0, 0, 0], shape[3] + rng.randint(0, 2)
                for i in rng.sample(range(3), 3):
                    step[i], at = at, at * shape[i] + rng.randint(0, 1)
                if rng.random() < 0.5:
                    step = [rng.randint(0, 40) for _ in range(3)]
                return (*step, 1), rng.randint(0, 60)

            sx, ox = view()
            sy, oy = view()
            if rng.random() < 0.5:
                sy = sx
            x, y = (torch.as_strided(base, shape, s, o) for s, o in ((sx, ox), (sy, oy)))
            ix, iy = (torch.as_strided(index, shape, s, o) for s, o in ((sx, ox), (sy, oy)))
            want = not torch.equal(ix, iy) and bool(set(ix.flatten().tolist()) & set(iy.flatten().tolist()))
            assert kvcache._meets(x, kvcache._strides(x), y, kvcache._strides(y)) == want
            seen[want] += 1
        assert min(seen) > 500
    # heads of one fused projection are apart, far buffers too
    qkv = torch.zeros((2, 2040, 3, 24, 128), dtype=torch.bfloat16)
    q, k, v = (qkv[:, :, i].transpose(1, 2) for i in range(3))
    far = torch.zeros((2, 24, 2040, 128), dtype=torch.bfloat16)
    for y, want in ((k, False), (v, False), (far, False), (q, False), (q[:, :, 1:], True)):
        x = q[:, :, :y.shape[2]]
        assert kvcache._meets(x, kvcache._strides(x), y, kvcache._strides(y)) == want
        assert kvcache._meets(y, kvcache._strides(y), x, kvcache._strides(x)) == want

"""The paged 8-bit cache where calls differ from the ordinary: query rows of
uneven size, many and empty sequences, one head cut into many shares, pages
past 2^31 bytes, long prunes, bad pages, captured weights and prunes."""
import numpy as np
import pytest
import torch

import bit_quantized_attention_sage_b200 as sage
import cache_ref as ref
from test_gpu_kvcache import check_attn, dev, filled, ok

pytestmark = pytest.mark.gpu


def randn(shape, seed, dtype=torch.bfloat16):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).to(dtype).cuda()


def check_weights(c, q, lse, tab, lengths, q_lens, mask, got, scale=None, absent=()):
    """As in test_weights: a term's exponent carries the score's error and the
    fp32 argument's, |t| <= 64."""
    D = q.shape[3]
    r = ref.attention(c, q, tab, lengths, q_lens, mask, D ** -0.5 if scale is None else scale,
                      lse.double().cpu().numpy())
    E, W = r[3], r[4]
    d = (D / 16 + 6) * 2.0 ** -22 * (E.max() + 16) + 2.0 ** -18
    got = got.double().cpu().numpy()
    for b, x in enumerate(lengths):
        t = np.arange(x)
        at = (tab[b][t // 64], slice(None), t % 64)
        assert (np.abs(got[at] - W[at]) <= W[at] * d + 1e-30).all()


# 10: one power of two for all rows; 45: rows keep their own
@pytest.mark.parametrize("spread", [10, 45])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("mask", [None, "causal", ("window", 7, 3, 20)])
def test_weights_of_rows_of_uneven_size(D, spread, mask):
    lengths, n, G = [150, 10, 300], 40, 4  # 160 rows: two blocks of them
    kv, tab, _ = filled(lengths, 1, D, spread, weight=True)
    c = ref.Cache(kv)
    q = torch.randn((3, G, n, D), generator=torch.Generator().manual_seed(1))
    e = torch.randint(-spread, 1, (3, G, n, 1), generator=torch.Generator().manual_seed(2))
    q = torch.ldexp(q, e)
    q[:, 1, ::5] = 0.0
    q = q.to(torch.bfloat16).cuda()
    _, lse = sage.cache_attn(q, kv, dev(tab), dev(lengths), mask, return_lse=True)
    sage.cache_weights(q, kv, lse, dev(tab), dev(lengths), mask, accumulate=False)
    ok()
    check_weights(c, q, lse, tab, lengths, [n] * 3, mask, kv.weight)


@pytest.mark.parametrize("n", [1, 3, 6])
def test_many_sequences(n):
    # more than a block's threads look up at once; a third of them empty, the
    # first and the last among these
    B, G, D = 700, 4, 64
    rng = np.random.default_rng(n)
    lengths = rng.integers(0, 150, B) * (rng.random(B) > 0.33)
    lengths[0] = lengths[-1] = 0
    lengths = lengths.tolist()
    q_lens = rng.integers(0, n + 1, B).tolist()
    kv, tab, _ = filled(lengths, 1, D, n, weight=True)
    c = ref.Cache(kv)
    q = randn((B, G, n, D), n)
    out = torch.full_like(q, 3.0)
    lse = torch.full(q.shape[:3], 3.0, device="cuda")
    for max_len in (None, 1):
        sage.cache_attn(q, kv, dev(tab), dev(lengths), "causal", q_lens=dev(q_lens), out=out, lse=lse,
                        max_len=max_len)
        ok()
        check_attn(c, q, out, lse, tab, lengths, q_lens, "causal", D ** -0.5, untouched=3.0)
        sage.cache_weights(q, kv, lse, dev(tab), dev(lengths), "causal", q_lens=dev(q_lens),
                           accumulate=False, max_len=max_len)
        ok()
        check_weights(c, q, lse, tab, lengths, q_lens, "causal", kv.weight)


@pytest.mark.parametrize("n", [1, 3])
def test_many_sequences_in_shares(n):
    # a page table wide enough that blocks share the pages of all heads
    B, G, D = 700, 4, 64
    rng = np.random.default_rng(n)
    lengths = rng.integers(0, 150, B) * (rng.random(B) > 0.33)
    lengths[0], lengths[1:200], lengths[-1] = 0, 0, 0
    lengths[350] = 5000
    lengths = lengths.tolist()
    q_lens = rng.integers(0, n + 1, B)
    q_lens[350] = n
    q_lens = q_lens.tolist()
    kv, tab, _ = filled(lengths, 1, D, n, weight=True)
    tab = np.pad(tab, ((0, 0), (0, 20)), constant_values=-7)
    c = ref.Cache(kv)
    q = randn((B, G, n, D), n)
    out = torch.full_like(q, 3.0)
    lse = torch.full(q.shape[:3], 3.0, device="cuda")
    sage.cache_attn(q, kv, dev(tab), dev(lengths), "causal", q_lens=dev(q_lens), out=out, lse=lse)
    sage.cache_weights(q, kv, lse, dev(tab), dev(lengths), "causal", q_lens=dev(q_lens),
                       accumulate=False)
    ok()
    check_attn(c, q, out, lse, tab, lengths, q_lens, "causal", D ** -0.5, untouched=3.0)
    check_weights(c, q, lse, tab, lengths, q_lens, "causal", kv.weight)


@pytest.mark.parametrize("G,n", [(1, 1), (8, 1), (16, 1), (5, 3), (8, 4)])
@pytest.mark.parametrize("D", [64, 128])
def test_one_head_in_many_shares(D, G, n):
    lengths = [9000]
    kv, tab, _ = filled(lengths, 1, D, G, weight=True)
    c = ref.Cache(kv)
    q = randn((1, G, n, D), n)
    o, lse = sage.cache_attn(q, kv, dev(tab), dev(lengths), "causal", return_lse=True)
    sage.cache_weights(q, kv, lse, dev(tab), dev(lengths), "causal", accumulate=False)
    ok()
    check_attn(c, q, o, lse, tab, lengths, [n], "causal", D ** -0.5)
    check_weights(c, q, lse, tab, lengths, [n], "causal", kv.weight)


def test_pages_past_two_gigabytes():
    # the same tokens in pages 0 .. and in pages whose codes lie past 2^31
    # bytes: every result has the same bits
    D, P = 128, 300000
    far = sage.KVCache8(P, 1, D, track_weight=True)
    near = sage.KVCache8(8, 1, D, track_weight=True)
    tabs = [dev([[P - 1, 3, P - 5], [270000, P - 2, 262144]]), dev([[0, 1, 2], [3, 4, 5]])]
    k, v = randn((2, 1, 150, D), 1), randn((2, 1, 150, D), 2)
    before, lengths = dev([0, 0]), dev([150, 131])
    res = []
    for kv, tab in zip((far, near), tabs):
        r = []
        sage.cache_append(kv, k, v, tab, before, n_new=lengths)
        for n in (1, 4, 20):
            q = randn((2, 2, n, D), n)
            o, lse = sage.cache_attn(q, kv, tab, lengths, "causal", return_lse=True)
            sage.cache_weights(q, kv, lse, tab, lengths, "causal")
            r += [o, lse]
        r += list(sage.cache_read(kv, tab, lengths, 150, weights=True))
        r += list(sage.cache_evict(kv, tab, lengths, 100, sink=2, recent=20))
        r += list(sage.cache_read(kv, tab, r[-1], 100, weights=True))
        ok()
        res.append(r)
    for a, b in zip(*res):
        assert torch.equal(a, b)


@pytest.mark.parametrize("length,keep", [(70000, 1000), (65536, 65535), (70001, 69000)])
def test_long_prunes(length, keep):
    # up to and past the weights that the selection keeps in shared memory
    kv, tab, _ = filled([length], 1, 64, 7, weight=True)
    w = torch.rand(kv.weight.shape, generator=torch.Generator().manual_seed(3))
    kv.weight.copy_(torch.where(w < 0.3, 0.125, w))
    c = ref.Cache(kv)
    kept, n_out = sage.cache_evict(kv, dev(tab), dev([length]), keep, sink=100, recent=200)
    ok()
    assert n_out.tolist() == [keep]
    idx, K, S, V, E, W = c.evict(tab[0], length, keep, 100, 200, 0)
    assert np.array_equal(kept[0, 0].cpu().numpy(), idx)
    got, pg = ref.Cache(kv), tab[0][:-(-keep // 64)].astype(np.int64)
    assert np.array_equal(got.k[pg, 0], K) and np.array_equal(got.s[pg, 0], S)
    assert np.array_equal(got.v[pg, 0], V) and np.array_equal(got.e[pg, 0], E)
    assert np.array_equal(got.w[pg, 0], W)


@pytest.mark.parametrize("bad", [-1, 1 << 30])
def test_bad_pages_are_recorded_and_absent(bad):
    # (each kernel asks page_id and leaves a page alone that it refuses)
    D, n = 64, 200
    kv = sage.KVCache8(16, 2, D, track_weight=True)
    names = ("k_i8", "k_scale", "v_f8", "v_exp", "weight")
    good = np.arange(8, dtype=np.int32).reshape(2, 4)
    tab = good.copy()
    tab[0, 1] = bad
    k, v = randn((2, 2, n, D), 1), randn((2, 2, n, D), 2)
    for x in names[:-1]:
        getattr(kv, x).fill_(3)
    sage.cache_append(kv, k, v, dev(tab), dev([0, 0]))
    assert sage.sync_status() == 1
    for x in names[:-1]:  # page 1 and those of no sequence
        assert (getattr(kv, x)[[1, 8, 15]].float() == 3).all()
    alone = sage.KVCache8(16, 2, D)
    sage.cache_append(alone, k, v, dev(good), dev([0, 0]))
    ok()
    used = [0, 2, 3, 4, 5, 6, 7]
    for x in names[:-1]:
        assert torch.equal(getattr(kv, x)[used], getattr(alone, x)[used])
    kr, vr = sage.cache_read(kv, dev(tab), dev([n, n]), n)
    assert sage.sync_status() == 1
    assert not kr[0, :, 64:128].any() and not vr[0, :, 64:128].any()
    assert kr[0, :, :64].any() and kr[1, :, 64:128].any()
    for rows in (1, 9):  # 2 and 18 query rows
        q = randn((2, 4, rows, D), rows)
        lse = torch.zeros(q.shape[:3], device="cuda")
        kv.weight.fill_(5.0)
        sage.cache_weights(q, kv, lse, dev(tab), dev([n, n]), accumulate=False)
        assert sage.sync_status() == 1
        assert (kv.weight[[1, 8, 15]] == 5).all()
        c = ref.Cache(alone)
        check_weights(c, q[1:], lse[1:], good[1:], [n], [rows], None, kv.weight)
    sage.cache_evict(kv, dev(good), dev([n, n]), 130, pages_out=dev([[8, bad, 10], [11, 12, 13]]))
    assert sage.sync_status() == 1
    assert (kv.k_i8[[14, 15]] == 3).all() and (kv.v_f8[9] == 3).all()
    sage.cache_evict(kv, dev(tab), dev([n, n]), 130)
    assert sage.sync_status() == 1
    assert (kv.k_i8[[14, 15]] == 3).all()


def test_captured_weights_and_prune():
    # a replay reads the lengths and the cache as they are then
    B, H, Hkv, D, n, keep = 3, 8, 2, 128, 5, 70
    lengths = [300, 64, 129]
    kv, tab, _ = filled(lengths, Hkv, D, 11, weight=True)
    t, ln, q = dev(tab), dev(lengths), randn((B, H, n, D), 4)
    names = ("k_i8", "k_scale", "v_f8", "v_exp", "weight")

    def step():
        o, lse = sage.cache_attn(q, kv, t, ln, "causal", return_lse=True)
        sage.cache_weights(q, kv, lse, t, ln, "causal")
        kept, n_out = sage.cache_evict(kv, t, ln, keep, sink=3, recent=9)
        ln.copy_(n_out)
        return o, kept, n_out

    start = [getattr(kv, x).clone() for x in names]

    def restore(lengths):
        for x, s in zip(names, start):
            getattr(kv, x).copy_(s)
        ln.copy_(dev(lengths))

    want = []
    for ls in (lengths, [200, 64, 1]):
        restore(ls)
        r = [x.clone() for x in step()]
        want.append(r + [getattr(kv, x).clone() for x in names])
    ok()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = step()
    for ls, w in zip((lengths, [200, 64, 1]), want):
        restore(ls)
        g.replay()
        ok()
        for a, b in zip(list(out) + [getattr(kv, x) for x in names], w):
            assert torch.equal(a.view(torch.uint8) if a.is_floating_point() else a,
                               b.view(torch.uint8) if b.is_floating_point() else b)


def test_calls_on_two_streams():
    # each call's scratch is its stream's
    kv, tab, _ = filled([4000, 300], 2, 64, 13, weight=True)
    t, ln = dev(tab), dev([4000, 300])
    qs = [randn((2, 4, n, 64), n) for n in (1, 6, 40)]
    want = [sage.cache_attn(q, kv, t, ln, "causal", return_lse=True) for q in qs]
    w = [sage.cache_weights(q, kv, l, t, ln, "causal", weight=torch.zeros_like(kv.weight))
         for q, (_, l) in zip(qs, want)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for i in range(12):
        s = streams[i % 2]
        with torch.cuda.stream(s):
            q = qs[i % 3]
            o, l = sage.cache_attn(q, kv, t, ln, "causal", return_lse=True)
            x = sage.cache_weights(q, kv, l, t, ln, "causal", weight=torch.zeros_like(kv.weight))
            got.append((i % 3, o, l, x))
    torch.cuda.synchronize()
    ok()
    for i, o, l, x in got:
        assert torch.equal(o, want[i][0]) and torch.equal(l, want[i][1]) and torch.equal(x, w[i])


def test_refusals_of_the_wrappers():
    kv = sage.KVCache8(4, 2, 64, track_weight=True)
    bare = sage.KVCache8(4, 2, 64)
    t, ln = dev([[0, 1]]), dev([0])
    q = torch.zeros((1, 4, 1, 64), dtype=torch.bfloat16, device="cuda")
    k = q[:, :2]
    lse = torch.zeros((1, 4, 1), device="cuda")
    odd = torch.zeros(4 * 2 * 64 + 1, device="cuda")[1:].view(4, 2, 64)
    for f in (lambda: sage.cache_append(kv, q, q, t, ln),
              lambda: sage.cache_append(kv, k.float(), k.float(), t, ln),
              lambda: sage.cache_append(kv, k, k.half(), t, ln),
              lambda: sage.cache_append(kv, k, k, t.long(), ln),
              lambda: sage.cache_append(kv, k, k, t, ln.cpu()),
              lambda: sage.cache_append(kv, k, k, t, ln, n_new=dev([1, 1])),
              lambda: sage.cache_append(kv, k, k, t, ln, k_shift=torch.zeros(64, device="cuda")),
              lambda: sage.cache_append(kv, k.transpose(2, 3), k.transpose(2, 3), t, ln),
              lambda: sage.cache_read(bare, t, ln, 1, weights=True),
              lambda: sage.cache_attn(q[:, :3], kv, t, ln),
              lambda: sage.cache_attn(q.float(), kv, t, ln),
              lambda: sage.cache_attn(q, kv, t, ln, "diagonal"),
              lambda: sage.cache_attn(q, kv, t, ln, lse=lse.half()),
              lambda: sage.cache_attn(q, kv, t, ln, out=q[:, :2]),
              lambda: sage.cache_weights(q, bare, lse, t, ln),
              lambda: sage.cache_weights(q, kv, lse[:, :2], t, ln),
              lambda: sage.cache_weights(q, kv, lse, t, ln, weight=kv.weight[:2]),
              lambda: sage.cache_evict(bare, t, ln, 1),
              lambda: sage.cache_evict(kv, t, ln, 4, sink=3, recent=2),
              lambda: sage.cache_evict(kv, t, ln, 100, pages_out=dev([[2]]))):
        with pytest.raises(ValueError):
            f()
    with pytest.raises(sage.SageError):  # refused by the library: not 16-byte aligned
        sage.cache_weights(q, kv, lse, t, ln, weight=odd)
    with pytest.raises(sage.SageError):  # a workspace that is too small
        big = sage.KVCache8(64, 1, 64)
        sage.cache_attn(q, big, dev([list(range(64))]), dev([4000]),
                        workspace=torch.zeros(64, dtype=torch.uint8, device="cuda"))
    ok()


@pytest.mark.parametrize("n,B,length", [(1, 37, 4700), (1, 1, 9000), (40, 3, 2000)])
def test_what_follows_sees_the_whole_result(n, B, length):
    # heads that no block cuts leave the join nothing to do; the copy behind
    # the call still waits for the attention
    kv, tab, _ = filled([length] * B, 8, 128, 3)
    t, ln, q = dev(tab), dev([length] * B), randn((B, 8, n, 128), 5)
    want = sage.cache_attn(q, kv, t, ln, "causal")
    torch.cuda.synchronize()
    out = torch.empty_like(q)
    for _ in range(50):
        out.zero_()
        sage.cache_attn(q, kv, t, ln, "causal", out=out)
        got = out.clone()
        assert torch.equal(got, want)
    ok()


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("n", [3, 7, 20])  # 6 and 14 rows, 40
@pytest.mark.parametrize("length", [100, 9000])
def test_a_row_that_is_not_finite_stays_alone(D, n, length):
    G, bad = 2, 1
    kv, tab, _ = filled([length], 2, D, n, weight=True)
    t, ln = dev(tab), dev([length])
    q = randn((1, 2 * G, n, D), n)
    want, wl = sage.cache_attn(q, kv, t, ln, "causal", return_lse=True)
    ww = sage.cache_weights(q, kv, wl, t, ln, "causal", accumulate=False).clone()
    for value in (float("nan"), float("inf")):
        p = q.clone()
        p[0, 1, bad, 5] = value
        o, lse = sage.cache_attn(p, kv, t, ln, "causal", return_lse=True)
        w = sage.cache_weights(p, kv, lse, t, ln, "causal", accumulate=False)
        ok()
        rest = torch.ones(o.shape[:3], dtype=torch.bool, device="cuda")
        rest[0, 1, bad] = False
        assert torch.equal(o[rest], want[rest]) and torch.equal(lse[rest], wl[rest])
        if value != value:
            assert torch.isnan(o[0, 1, bad]).all() and torch.isnan(lse[0, 1, bad])
        # the other key head, and the keys behind the row
        at = np.arange(length - n + bad + 1, length)
        pg, slot = torch.from_numpy(tab[0][at // 64]).long(), torch.from_numpy(at % 64)
        assert torch.equal(w[pg, 0, slot], ww[pg, 0, slot])
        every = torch.from_numpy(tab[0]).long()
        full = every[:length // 64]
        assert torch.equal(w[full, 1], ww[full, 1])
        if value != value:
            assert torch.isnan(w[full, 0]).all()


def test_any_call_may_be_the_first(monkeypatch):
    from bit_quantized_attention_sage_b200 import kvcache
    kv = sage.KVCache8(64, 2, 64)
    q = randn((1, 4, 1, 64), 1)
    t, ln, f = dev([list(range(64))]), dev([0]), torch.ones(32, dtype=torch.float64, device="cuda")
    for call in (lambda: sage.cache_attn_workspace_bytes(kv, 1, 4, 1, 4096, "causal"),
                 lambda: sage.cache_attn(q, kv, t, ln),
                 lambda: sage.cache_append(kv, q[:, :2], q[:, :2], t, ln),
                 lambda: sage.cache_read(kv, t, ln, 1),
                 lambda: sage.rope(q, dev([3]), f),
                 lambda: sage.rope_tables(dev([3]), f)):
        monkeypatch.setattr(kvcache, "torch", None)
        kvcache._TYPES.clear()
        call()
    ok()

"""More of the paged 8-bit cache: odd page counts and empty queries in the
summed weights, prunes of subnormal keys and of shortened sequences, outputs
over their inputs."""
import numpy as np
import pytest
import torch

import bit_quantized_attention_sage_b200 as sage
import cache_ref as ref
from test_gpu_kvcache import check_attn, dev, filled, ok
from test_gpu_kvcache_edges import check_weights, randn

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D", [64, 128])
def test_weights_of_odd_page_counts(D):
    # a stretch of many heads that end on a lone page: each such tile's second
    # half is no page, whatever tile had its place in the rings before
    rng = np.random.default_rng(D)
    B, Hkv, n, G = 40, 12, 9, 2
    lengths = (64 * rng.choice([1, 2, 3, 4, 5], B) - rng.integers(0, 64, B)).tolist()
    kv, tab, _ = filled(lengths, Hkv, D, 2, weight=True)
    c = ref.Cache(kv)
    q = randn((B, Hkv * G, n, D), 3)
    _, lse = sage.cache_attn(q, kv, dev(tab), dev(lengths), "causal", return_lse=True)
    kv.weight.fill_(7.0)
    sage.cache_weights(q, kv, lse, dev(tab), dev(lengths), "causal", accumulate=False)
    ok()
    check_weights(c, q, lse, tab, lengths, [n] * B, "causal", kv.weight)
    used = torch.zeros(kv.weight.shape, dtype=torch.bool)
    for b, x in enumerate(lengths):
        t = np.arange(x)
        used[torch.from_numpy(tab[b][t // 64]).long(), :, torch.from_numpy(t % 64)] = True
    assert (kv.weight[~used.cuda()] == 7.0).all()


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("H,n", [(4, 0), (0, 3), (0, 0)])
def test_empty_queries_overwrite_the_weights(D, H, n):
    # the sum over no rows is zero; other slots and an accumulating call stay
    lengths = [0, 1, 64, 200, 5000]
    kv, tab, _ = filled(lengths, 2, D, 4, weight=True)
    kv.weight.copy_(torch.rand(kv.weight.shape) + 1)
    before = kv.weight.clone()
    q = torch.zeros((5, H, n, D), dtype=torch.bfloat16, device="cuda")
    lse = torch.zeros(q.shape[:3], device="cuda")
    q_lens = dev([n, 0, n, n, 0])
    for kw in ({}, {"q_lens": q_lens}):
        assert sage.cache_weights(q, kv, lse, dev(tab), dev(lengths), "causal", **kw) is kv.weight
        ok()
        assert torch.equal(kv.weight, before)
    for max_len in (None, 1):
        kv.weight.copy_(before)
        sage.cache_weights(q, kv, lse, dev(tab), dev(lengths), "causal", q_lens=q_lens,
                           accumulate=False, max_len=max_len)
        ok()
        want = before.clone()
        for b, x in enumerate(lengths):
            t = np.arange(x)
            want[torch.from_numpy(tab[b][t // 64]).long(), :, torch.from_numpy(t % 64)] = 0
        assert torch.equal(kv.weight, want)


@pytest.mark.parametrize("D", [64, 128])
def test_prune_of_subnormal_keys(D):
    # scales of a few last places: the new scale is rounded by more than the
    # codes' range allows for, and codes past it are held at +-127
    n, keep = 512, 128
    kv, tab, _ = filled([n], 2, D, 5, weight=True)
    pg = torch.from_numpy(tab[0]).long()
    g = torch.Generator().manual_seed(1)
    top = torch.randint(1, 8, kv.weight.shape, generator=g)
    code = torch.randint(-127, 128, kv.k_i8.shape, generator=g)
    kv.k_i8.copy_((code.sign() * (code.abs() % (top[..., None] + 1))).to(torch.int8))
    # multiples of the least fp32 number, 2^-149: 7 of 55 .. 61 of them / 127
    # round to 3, and 7 * 55 / 3 is past 127
    steps = torch.randint(55, 62, kv.k_scale.shape, generator=g).to(torch.int32)
    kv.k_scale.copy_(steps.view(torch.float32))
    kv.weight[pg] = torch.rand((len(pg), 2, 64), generator=g).cuda()
    c = ref.Cache(kv)
    sage.cache_evict(kv, dev(tab), dev([n]), keep)
    ok()
    got, p = ref.Cache(kv), tab[0][:2].astype(np.int64)
    for h in range(2):
        _, K, S, _, _, _ = c.evict(tab[0], n, keep, 0, 0, h)
        assert np.array_equal(got.s[p, h], S)
        assert (np.abs(K) == 127).any()
        assert np.array_equal(got.k[p, h], K)


@pytest.mark.parametrize("case", ["itself", "token_on", "token_back", "other_head_order", "fused"])
@pytest.mark.parametrize("n", [1, 2, 300])
def test_outputs_over_their_inputs(case, n):
    # every form gives what an output of its own does, and leaves the rest of
    # the buffer alone
    B, H, D, lengths = 2, 4, 64, [3000, 70]
    kv, tab, _ = filled(lengths, 2, D, n)
    f, _ = sage.rope_freqs(D)
    pos = torch.arange(n, device="cuda") * 100
    t, ln = dev(tab), dev(lengths)
    for call in (lambda x, out=None: sage.rope(x, pos, f, layout="half", out=out),
                 lambda x, out=None: sage.cache_attn(x, kv, t, ln, "causal", out=out),
                 lambda x, out=None: sage.cache_attn(x, kv, t, ln, "causal", out=out, return_lse=True)[0]):
        base = randn((B, n + 1, 3, H, D), n)
        q = base[:, :n, 0].transpose(1, 2)
        out = {"itself": q, "token_on": base[:, 1:, 0].transpose(1, 2),
               "token_back": q, "other_head_order": base[:, :n, :2].reshape(B, n, 2 * H, D),
               "fused": base[:, :n, 1].transpose(1, 2)}[case]
        if case == "token_back":
            q = base[:, 1:, 0].transpose(1, 2)
        if case == "other_head_order":  # rows of q as heads of the result
            flat = base.view(-1)
            q = torch.as_strided(flat, (B, H, n, D), (3 * H * D * (n + 1), D, 3 * H * D, 1))
            out = torch.as_strided(flat, (B, H, n, D), (3 * H * D * (n + 1), D * n, D, 1))
        want, rest = call(q), base.clone()
        rest_out = torch.as_strided(rest, out.shape, out.stride(), out.storage_offset())
        rest_out.copy_(want)
        assert call(q, out) is out
        ok()
        assert torch.equal(out, want) and torch.equal(base, rest)


@pytest.mark.parametrize("place", ["in", "out"])
def test_prune_of_a_shortened_sequence(place):
    # a page whose scales are larger than its tokens need (larger ones were
    # taken back) gets those its tokens need; a page with scales of its own
    # tokens keeps its values
    D, B = 64, 1
    kv = sage.KVCache8(10, 2, D, track_weight=True)
    tab = np.array([[4, 1, 7, 2]], np.int32)
    large, small = randn((B, 2, 70, D), 1) * 100, randn((B, 2, 246, D), 2)
    sage.cache_append(kv, large, large, dev(tab), dev([0]))
    sage.cache_append(kv, small, small, dev(tab), dev([10]))  # shortened to 10 tokens
    sage.cache_append(kv, small, small, dev(tab), dev([3]))   # to 3
    lengths, keep = [249], 192
    kv.weight.zero_()
    for i in range(3):
        kv.weight[int(tab[0, i])] = 1.0
    c = ref.Cache(kv)
    assert c.k[4, 0, 3:].max() < 127  # the large tokens' scale
    po = None if place == "in" else np.array([[9, 8, 6]], np.int32)
    kept, _ = sage.cache_evict(kv, dev(tab), dev(lengths), keep, pages_out=None if po is None else dev(po))
    ok()
    got = ref.Cache(kv)
    pg = (tab if po is None else po)[0][:3].astype(np.int64)
    for h in range(2):
        assert kept[0, h].tolist() == list(range(192))
        _, K, S, V, E, _ = c.evict(tab[0], lengths[0], keep, 0, 0, h)
        assert np.array_equal(got.k[pg, h], K) and np.array_equal(got.s[pg, h], S)
        assert np.array_equal(got.v[pg, h], V) and np.array_equal(got.e[pg, h], E)
    # whole pages of their own scales: the key of absmax has code 127, so the new
    # scale is s fp32(127 / 127); a largest value just above 448 2^e was rounded
    # down to 448 2^e, whose least exponent is e, so value codes may double
    own = tab[0][1:3].astype(np.int64)
    assert np.array_equal(got.k[pg[1:]], c.k[own]) and np.array_equal(got.s[pg[1:]], c.s[own])
    val = [x.v * np.exp2(x.e.astype(np.float64))[..., None, None] for x in (got, c)]
    assert np.array_equal(val[0][pg[1:]], val[1][own])


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("G,n", [(1, 1), (8, 1), (8, 2), (5, 4), (9, 2)])
def test_one_long_head(D, G, n):
    # a hundred shares and more of one head, more than 32 ranges of keys
    lengths = [70001]
    kv, tab, _ = filled(lengths, 1, D, G, weight=True)
    c = ref.Cache(kv)
    q = randn((1, G, n, D), n)
    o, lse = sage.cache_attn(q, kv, dev(tab), dev(lengths), "causal", return_lse=True)
    sage.cache_weights(q, kv, lse, dev(tab), dev(lengths), "causal", accumulate=False)
    ok()
    check_attn(c, q, o, lse, tab, lengths, [n], "causal", D ** -0.5)
    check_weights(c, q, lse, tab, lengths, [n], "causal", kv.weight)

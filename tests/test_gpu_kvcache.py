"""The paged 8-bit cache against plain 64-bit implementations: what enters it
bit for bit, attention over it, the summed weights and the prune."""
import math

import numpy as np
import pytest
import torch

import bit_quantized_attention_sage_b200 as sage
import cache_ref as ref

pytestmark = pytest.mark.gpu
DTS = {"bf16": torch.bfloat16, "fp16": torch.float16}


def dev(a, dt=torch.int32):
    return torch.as_tensor(np.asarray(a)).to(dt).cuda()


def ok():
    assert sage.sync_status() == 0


def filled(lengths, Hkv, D, seed, dtype=torch.bfloat16, spare=0, weight=False, vscale=1.0):
    """A cache with `lengths` tokens a sequence, appended by the library, its
    reference copy, the page table; unused slots hold garbage (NaN codes)."""
    rng = np.random.default_rng(seed)
    tab, P, left = ref.make_pages(lengths, rng, spare)
    kv = sage.KVCache8(P, Hkv, D, track_weight=weight)
    kv.k_i8.random_(-128, 128)
    kv.v_f8.fill_(0x7F)
    kv.k_scale.fill_(float("nan"))
    n = max(1, max(lengths))
    g = torch.Generator().manual_seed(seed)
    k = (torch.randn((len(lengths), Hkv, n, D), generator=g) +
         2 * torch.randn((1, Hkv, 1, D), generator=g)).to(dtype).cuda()
    v = (torch.randn((len(lengths), Hkv, n, D), generator=g) * vscale).to(dtype).cuda()
    sage.cache_append(kv, k, v, dev(tab), dev([0] * len(lengths)), n_new=dev(lengths))
    for b, x in enumerate(lengths):  # slots behind the end: anything, NaN among it
        if x % 64:
            kv.v_f8[int(tab[b, x // 64]), :, x % 64:] = 0xFF
            kv.k_i8[int(tab[b, x // 64]), :, x % 64:] = -128
    ok()
    return kv, tab, left


# ---------------------------------------------------------------- append and read

@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("before,n", [([0], 1), ([0, 63, 64, 5], 1), ([0, 1, 60], 2),
                                      ([3, 0, 64], 63), ([7, 0, 130], 64), ([63, 1, 0], 65),
                                      ([10, 200], 200)])
def test_append_is_exact(D, before, n):
    rng = np.random.default_rng(n)
    B, Hkv = len(before), 3
    tab, P, _ = ref.make_pages([x + n for x in before], rng)
    kv = sage.KVCache8(P, Hkv, D, track_weight=True)
    kv.weight.fill_(7.0)
    want = ref.Cache(kv)
    g = torch.Generator().manual_seed(n * D)
    steps = [(x, b0) for x, b0 in ((max(before), [0] * B), (n, before))]
    for i, (m, b0) in enumerate(steps):
        if m == 0:
            continue
        nn = before if i == 0 else [n - (j % 2) * (n // 2) for j in range(B)]
        # the second call's tokens are larger for some heads: their page's
        # scale grows and its codes move; others stay
        f = torch.tensor([1.0, 30.0, 0.1])[None, :, None, None] if i else 1.0
        k = (torch.randn((B, Hkv, m, D), generator=g) * f).to(torch.bfloat16).cuda()
        v = (torch.randn((B, Hkv, m, D), generator=g) * f).to(torch.bfloat16).cuda()
        sage.cache_append(kv, k, v, dev(tab), dev(b0), n_new=dev(nn))
        want.append(k, v, tab, b0, nn)
        ok()
        want.same(kv)
    sage.cache_append(kv, k, v, dev(tab), dev(b0), n_new=dev(nn))  # again: nothing changes
    ok()
    want.same(kv)


@pytest.mark.parametrize("kind", ["fp16", "shift", "strided", "odd_strides", "zero", "tiny", "huge",
                                  "ties"])
def test_append_kinds(kind):
    B, Hkv, n, D = 2, 2, 150, 64
    rng = np.random.default_rng(3)
    tab, P, _ = ref.make_pages([n + 70] * B, rng)
    kv = sage.KVCache8(P, Hkv, D)
    want = ref.Cache(kv)
    g = torch.Generator().manual_seed(5)
    dt = torch.float16 if kind == "fp16" else torch.bfloat16
    k = torch.randn((B, Hkv, n, D), generator=g)
    v = torch.randn((B, Hkv, n, D), generator=g)
    shift = None
    if kind == "shift":
        k += 3 * torch.randn((1, Hkv, 1, D), generator=g)
        shift = k.mean((0, 2)).contiguous().cuda()
    if kind == "zero":
        k[:, 0, :80], v[:, 1, 64:] = 0, 0
    if kind == "tiny":
        k, v = k * 1e-38, v * 1e-12
    if kind == "huge":
        k, v = k * 1e37, v * 1e37
    if kind == "ties":  # quotients that are exact halves: absmax 127, steps of 1/2
        k = torch.randint(-254, 255, k.shape, generator=g) / 2.0
        k[:, :, ::32, 0] = 127.0
        v = torch.randint(-896, 897, v.shape, generator=g) / 2.0
    k, v = k.to(dt).cuda(), v.to(dt).cuda()
    if kind == "strided":
        k = k.transpose(1, 2).contiguous().transpose(1, 2)
        v = v.transpose(1, 2).contiguous().transpose(1, 2)
    if kind == "odd_strides":
        k = torch.nn.functional.pad(k, (1, 2))[..., 1:-2]
    sage.cache_append(kv, k, v, dev(tab), dev([70, 3]), k_shift=shift)
    want.append(k, v, tab, [70, 3], [n, n], shift)
    ok()
    want.same(kv)


def test_read_returns_the_values_of_the_codes():
    lengths = [0, 1, 64, 130]
    kv, tab, _ = filled(lengths, 2, 128, 1, weight=True)
    kv.weight.copy_(torch.rand(kv.weight.shape))
    c = ref.Cache(kv)
    starts = [0, 0, 60, 65]
    shift = torch.randn(2, 128).cuda()
    k, v, w = sage.cache_read(kv, dev(tab), dev(lengths), 70, starts=dev(starts), weights=True)
    ks, _ = sage.cache_read(kv, dev(tab), dev(lengths), 70, starts=dev(starts), k_shift=shift)
    ok()
    for b, x in enumerate(lengths):
        for h in range(2):
            K, V = c.tokens(tab[b], x, h)
            m = max(0, min(70, x - starts[b]))
            s = slice(starts[b], starts[b] + m)
            assert np.array_equal(k[b, h, :m].cpu().numpy(), K[s].astype(np.float32))
            assert np.array_equal(v[b, h, :m].cpu().numpy(), V[s].astype(np.float32))
            assert not k[b, h, m:].any() and not v[b, h, m:].any() and not w[b, h, m:].any()
            t = np.arange(starts[b], starts[b] + m)
            assert np.array_equal(w[b, h, :m].cpu().numpy(), c.w[tab[b][t // 64], h, t % 64])
            sh = (K[s].astype(np.float32) + shift[h].cpu().numpy())
            assert np.array_equal(ks[b, h, :m].cpu().numpy(), sh)


# ---------------------------------------------------------------- attention

def check_attn(c, q, o, lse, tab, lengths, q_lens, mask, scale, untouched=None):
    """Tolerance of O: half a step of its type; 2^-11 of the weights' fp16
    rounding on sum p |v|; the fp32 scores' error d (the products are exact;
    D / 16 accumulation steps, the scale's two products and the exponent's
    argument, each at most 2 units of 2^-23 of the sum of magnitudes) once in
    the numerator and once in the sum; exp2's 2^-21 and the sums' n 2^-23."""
    B, H, N, D = q.shape
    O, L, A, E, _ = ref.attention(c, q, tab, lengths, q_lens, mask, scale)
    got, gl = o.double().cpu().numpy(), lse.double().cpu().numpy()
    d = (D / 16 + 6) * 2.0 ** -22 * (E + 16)
    n = max(lengths) + 16
    rel = 2.0 ** -11 + 2 * d + 2.0 ** -20 + n * 2.0 ** -23
    for b in range(B):
        m = q_lens[b]
        tol = ref.half_step(O[b, :, :m], q.dtype) + A[b, :, :m] * rel[b, :, :m, None] + \
            torch.finfo(q.dtype).tiny
        err = np.abs(got[b, :, :m] - O[b, :, :m])
        assert (err <= tol).all(), "O: worst excess %.3g" % (err - tol).max()
        none = np.isneginf(L[b, :, :m])
        assert np.array_equal(np.isneginf(gl[b, :, :m]), none)
        le = np.abs(gl[b, :, :m][~none] - L[b, :, :m][~none])
        lt = (d[b, :, :m] + 2.0 ** -19 + n * 2.0 ** -23 + 2.0 ** -22 * 64)[~none]
        assert (le <= lt).all(), "lse: worst excess %.3g" % (le - lt).max()
        if untouched is not None:
            assert (o[b, :, m:] == untouched).all() and (lse[b, :, m:] == untouched).all()


MASKS = [None, "causal", ("block_causal", 50), ("window", 1, 40, 3), ("window", 30, 2, 70)]


@pytest.mark.parametrize("D,G,dt", [(128, 1, "bf16"), (128, 4, "fp16"), (64, 3, "bf16"),
                                    (64, 8, "fp16"), (128, 7, "bf16")])
@pytest.mark.parametrize("mask", MASKS)
@pytest.mark.parametrize("n", [1, 5, 70])
def test_attention_small(D, G, dt, mask, n):
    lengths = [0, 1, 63, 64, 65, 200]
    kv, tab, _ = filled(lengths, 2, D, D + G)
    c = ref.Cache(kv)
    q = torch.randn((len(lengths), 2 * G, n, D), generator=torch.Generator().manual_seed(n)).to(DTS[dt]).cuda()
    q_lens = [n, n, n - n // 2, n, max(0, n - 1), n]
    out = torch.full_like(q, 3.0)
    lse = torch.full(q.shape[:3], 3.0, device="cuda")
    o = sage.cache_attn(q, kv, dev(tab), dev(lengths), mask, q_lens=dev(q_lens), out=out, lse=lse)
    ok()
    assert o is out
    check_attn(c, q, o, lse, tab, lengths, q_lens, mask, D ** -0.5, untouched=3.0)


@pytest.mark.parametrize("max_len", [None, 3000, 1000, 1])
@pytest.mark.parametrize("n,G,D", [(1, 4, 128), (3, 1, 64), (40, 2, 128), (300, 1, 64)])
def test_attention_ranges(n, G, D, max_len):
    # several KV ranges a tile; a bound that is too small only costs time
    lengths = [3000, 1777]
    kv, tab, _ = filled(lengths, 1, D, n)
    c = ref.Cache(kv)
    q = torch.randn((2, G, n, D), generator=torch.Generator().manual_seed(n)).to(torch.bfloat16).cuda()
    for mask in ("causal", ("window", 100, 3, 130)):
        o, lse = sage.cache_attn(q, kv, dev(tab), dev(lengths), mask, max_len=max_len, scale=0.2,
                                 return_lse=True)
        ok()
        check_attn(c, q, o, lse, tab, lengths, [n, n], mask, 0.2)


@pytest.mark.parametrize("n", [1, 100])
def test_attention_uneven_scales(n):
    # pages whose values differ by 2^70, and a query row of far larger size
    lengths, D = [500], 128
    kv, tab, _ = filled(lengths, 2, D, 9)
    for i, e in enumerate((-40, 30, -20, 0, 25, -5, 12, -33)):
        kv.v_exp[int(tab[0, i])] = e
        kv.k_scale[int(tab[0, i])] *= 4.0 ** (i % 3 - 1)
    kv.v_f8[int(tab[0, 2])] = 0  # a page of zero values
    kv.v_exp[int(tab[0, 2])] = -40
    c = ref.Cache(kv)
    q = torch.randn((1, 2, n, D), generator=torch.Generator().manual_seed(4)).to(torch.bfloat16).cuda()
    q[0, 1] *= 8
    q[0, 0, 0] = 0
    o, lse = sage.cache_attn(q, kv, dev(tab), dev(lengths), None, scale=0.05, return_lse=True)
    ok()
    check_attn(c, q, o, lse, tab, lengths, [n], None, 0.05)


@pytest.mark.parametrize("n", [1, 90])
def test_attention_strides(n):
    lengths, D, H = [300, 77], 128, 4
    kv, tab, _ = filled(lengths, 2, D, 2)
    c = ref.Cache(kv)
    g = torch.Generator().manual_seed(6)
    base = torch.randn((2, n, H, D + 3), generator=g).to(torch.bfloat16).cuda()
    q = base[..., 1:D + 1].transpose(1, 2)  # odd offset and strides
    out = torch.zeros((2, n, H, D + 1), dtype=torch.bfloat16, device="cuda")[..., 1:].transpose(1, 2)
    lse = torch.empty((2, H, n), device="cuda")
    sage.cache_attn(q, kv, dev(tab), dev(lengths), "causal", out=out, lse=lse)
    ok()
    check_attn(c, q, out, lse, tab, lengths, [n, n], "causal", D ** -0.5)
    one = q[:1, :, :1].expand(2, H, n, D)  # broadcast queries
    o, lse = sage.cache_attn(one, kv, dev(tab), dev(lengths), None, return_lse=True)
    ok()
    check_attn(c, one, o, lse, tab, lengths, [n, n], None, D ** -0.5)


@pytest.mark.parametrize("n", [1, 80])
def test_attention_shared_pages_and_a_bad_page(n):
    # two sequences read one prefix; a page id that is none counts as absent
    kv, tab, _ = filled([200, 200], 2, 64, 8)
    tab[1, :2] = tab[0, :2]
    c = ref.Cache(kv)
    q = torch.randn((2, 2, n, 64), generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).cuda()
    o, lse = sage.cache_attn(q, kv, dev(tab), dev([200, 200]), None, return_lse=True)
    ok()
    check_attn(c, q, o, lse, tab, [200, 200], [n, n], None, 0.125)
    bad = tab.copy()
    bad[1, 1] = 1 << 20
    o2, lse2 = sage.cache_attn(q, kv, dev(bad), dev([200, 200]), None, return_lse=True)
    assert sage.sync_status() == 1 and sage.sync_status() == 0
    assert torch.equal(o2[0], o[0]) and torch.equal(lse2[0], lse[0])
    # the same keys without that page: its tokens taken out of the table
    short = np.concatenate([tab[1:, :1], tab[1:, 2:]], 1)
    check_attn(c, q[1:], o2[1:], lse2[1:], short, [136], [n], None, 0.125)


# ---------------------------------------------------------------- weights

@pytest.mark.parametrize("D,G,n", [(128, 1, 1), (64, 4, 1), (128, 3, 33), (64, 2, 150)])
@pytest.mark.parametrize("mask", MASKS)
def test_weights(D, G, n, mask):
    lengths = [0, 1, 64, 300]
    kv, tab, _ = filled(lengths, 2, D, G, weight=True)
    c = ref.Cache(kv)
    q = torch.randn((4, 2 * G, n, D), generator=torch.Generator().manual_seed(n)).to(torch.bfloat16).cuda()
    q_lens = [n, n, max(0, n - 1), n]
    lse = torch.zeros(q.shape[:3], device="cuda")
    sage.cache_attn(q, kv, dev(tab), dev(lengths), mask, q_lens=dev(q_lens), lse=lse)
    kv.weight.fill_(0.5)
    kv.weight[int(tab[3, 4]), :, 300 % 64:] = float("nan")  # behind the end: not touched
    sage.cache_weights(q, kv, lse, dev(tab), dev(lengths), mask, q_lens=dev(q_lens))
    ok()
    W = ref.attention(c, q, tab, lengths, q_lens, mask, D ** -0.5, lse.double().cpu().numpy())
    E, W = W[3], W[4]
    # a term's exponent: the score's error and the fp32 argument's, |t| <= 64
    d = (D / 16 + 6) * 2.0 ** -22 * (E.max() + 16) + 2.0 ** -18
    got = kv.weight.double().cpu().numpy()
    for b, x in enumerate(lengths):
        t = np.arange(x)
        at = (tab[b][t // 64], slice(None), t % 64)
        w = W[tab[b][t // 64], :, t % 64]
        assert (np.abs(got[at] - 0.5 - w) <= w * d + 2.0 ** -23 + 1e-30).all()
    assert torch.isnan(kv.weight[int(tab[3, 4]), :, 300 % 64:]).all()
    over = sage.cache_weights(q, kv, lse, dev(tab), dev(lengths), mask, q_lens=dev(q_lens),
                              weight=torch.full_like(kv.weight, 9.0), accumulate=False, max_len=1)
    ok()
    used = np.zeros(W.shape, bool)
    for b, x in enumerate(lengths):
        t = np.arange(x)
        used[tab[b][t // 64], :, t % 64] = True
    o = over.double().cpu().numpy()
    assert (o[~used] == 9.0).all()
    assert (np.abs(o - W)[used] <= W[used] * d + 1e-30).all()


# ---------------------------------------------------------------- evict

@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("keep,sink,recent", [(1, 0, 0), (64, 0, 0), (100, 10, 30), (100, 60, 40),
                                              (129, 0, 128), (300, 1, 1)])
@pytest.mark.parametrize("place", ["in", "out"])
def test_evict(D, keep, sink, recent, place):
    lengths = [0, 1, 64, 129, 500, 1000]
    nb, B, Hkv = -(-keep // 64), len(lengths), 2
    kv, tab, left = filled(lengths, Hkv, D, keep, spare=nb * B, weight=True)
    g = torch.Generator().manual_seed(keep)
    w = torch.rand(kv.weight.shape, generator=g)
    kv.weight.copy_(torch.where(w < 0.5, 0.25, w))  # many equal ones
    # uneven scales: survivors of one page come from pages of other scales
    kv.k_scale.mul_(torch.rand(kv.k_scale.shape, generator=g).cuda() + 0.5)
    kv.v_exp.add_(torch.randint(-3, 4, kv.v_exp.shape, generator=g).to(torch.int8).cuda())
    c = ref.Cache(kv)
    po = None if place == "in" else np.asarray(left[:nb * B], np.int32).reshape(B, nb)
    snap = {x: getattr(kv, x).clone() for x in ("k_i8", "k_scale", "v_f8", "v_exp", "weight")}
    kept, n_out = sage.cache_evict(kv, dev(tab), dev(lengths), keep, sink, recent,
                                   pages_out=None if po is None else dev(po))
    ok()
    assert n_out.tolist() == [min(x, keep) for x in lengths]
    got = ref.Cache(kv)
    for b, x in enumerate(lengths):
        n = min(x, keep)
        for h in range(Hkv):
            if n == 0:
                assert (kept[b, h] == -1).all()
                continue
            idx, K, S, V, E, W = c.evict(tab[b], x, keep, sink, recent, h)
            assert np.array_equal(kept[b, h, :n].cpu().numpy(), idx)
            assert (kept[b, h, n:] == -1).all()
            pg = (tab if po is None else po)[b][:-(-n // 64)].astype(np.int64)
            if place == "in" and x <= keep:
                for nme, t in snap.items():
                    assert torch.equal(getattr(kv, nme)[pg, h].view(torch.uint8),
                                       t[pg, h].view(torch.uint8))
                continue
            assert np.array_equal(got.k[pg, h], K) and np.array_equal(got.s[pg, h], S)
            assert np.array_equal(got.v[pg, h], V) and np.array_equal(got.e[pg, h], E)
            assert np.array_equal(got.w[pg, h], W)


def test_evict_orders_every_weight():
    # infinities, NaN (largest) and negative zero (a zero)
    kv, tab, _ = filled([200], 1, 64, 3, weight=True)
    w = torch.zeros(200)
    w[50], w[60], w[70], w[80], w[20] = math.inf, math.nan, 1e30, 1e-40, -0.0
    flat = torch.zeros(256)
    flat[:200] = w
    kv.weight[torch.from_numpy(tab[0]).long(), 0] = flat.view(4, 64).cuda()
    kept, _ = sage.cache_evict(kv, dev(tab), dev([200]), 6)
    ok()
    assert kept[0, 0].tolist() == [0, 1, 50, 60, 70, 80]


# ---------------------------------------------------------------- a run of them

def stream_step(kv, tab, q, k, v, pos, f, lengths, scratch):
    n = k.shape[2]
    kr = sage.rope(k, pos, f, layout="half")
    sage.cache_append(kv, kr, v, tab, lengths)
    lengths.add_(n)
    qr = sage.rope(q, pos, f, layout="half")
    o, lse = sage.cache_attn(qr, kv, tab, lengths, "causal", return_lse=True)
    sage.cache_weights(qr, kv, lse, tab, lengths, "causal")
    return o


def test_steps_together_and_captured():
    """Rotate, append, attend, sum weights, prune, go on: against plain 64-bit
    attention over the cache's own values; then the step as a captured graph."""
    B, H, Hkv, D, cap = 2, 4, 2, 64, 8
    rng = np.random.default_rng(0)
    tab = dev(rng.permutation(B * cap).reshape(B, cap))
    kv = sage.KVCache8(B * cap, Hkv, D, track_weight=True)
    f, _ = sage.rope_freqs(D)
    g = torch.Generator().manual_seed(0)
    lengths = dev([0, 0])

    def inputs(n):
        return [torch.randn((B, h, n, D), generator=g).to(torch.bfloat16).cuda() for h in (H, Hkv, Hkv)]

    pos = torch.arange(300, device="cuda")
    q, k, v = inputs(300)
    o = stream_step(kv, tab, q, k, v, pos, f, lengths, None)
    ok()
    c = ref.Cache(kv)
    qr = sage.rope(q, pos, f, layout="half")
    _, lse = sage.cache_attn(qr, kv, tab, lengths, "causal", return_lse=True)
    check_attn(c, qr, o, lse, tab.cpu().numpy(), [300, 300], [300, 300], "causal", D ** -0.5)
    # every row's weights sum to one
    total = kv.weight.double().sum((0, 2))
    assert (total - B * 2 * 300).abs().max() < 1e-3
    kept, n_out = sage.cache_evict(kv, tab, lengths, 128, sink=4, recent=32)
    lengths.copy_(n_out)
    assert lengths.tolist() == [128, 128]
    # tokens one at a time, eager and as a replayed graph, agree
    q, k, v = inputs(1)
    pos1 = dev([300], torch.int64)
    state = [t.clone() for t in (kv.k_i8, kv.k_scale, kv.v_f8, kv.v_exp, kv.weight, lengths)]
    eager = []
    for i in range(3):
        eager.append(stream_step(kv, tab, q, k, v, pos1 + i, f, lengths, None).clone())
    ok()
    end = [t.clone() for t in (kv.k_i8, kv.k_scale, kv.v_f8, kv.v_exp, kv.weight, lengths)]
    here = (kv.k_i8, kv.k_scale, kv.v_f8, kv.v_exp, kv.weight, lengths)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    p = pos1.clone()
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr, stream=s):
        og = stream_step(kv, tab, q, k, v, p, f, lengths, None)
    for t, x in zip(here, state):
        t.copy_(x)
    for i in range(3):
        p.copy_(pos1 + i)
        gr.replay()
        assert torch.equal(og, eager[i])
    ok()
    for t, x in zip(here, end):
        assert torch.equal(t, x)


def test_other_stream_and_two_graphs():
    # scratch of a call on another stream is that stream's; two captured
    # calls keep scratch of their own
    lengths = [3000]
    kv, tab, _ = filled(lengths, 2, 128, 5)
    t, ln = dev(tab), dev(lengths)
    qs = [torch.randn((1, 2, 2, 128), generator=torch.Generator().manual_seed(i)).to(torch.bfloat16).cuda()
          for i in range(4)]
    want = [sage.cache_attn(q, kv, t, ln, None) for q in qs]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = []
    for q in qs:
        got.append(sage.cache_attn(q, kv, t, ln, None, stream=s))
        torch.empty(1 << 20, dtype=torch.uint8, device="cuda").fill_(255)  # would reuse freed scratch
    s.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    graphs = []
    for q in qs[:2]:
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            o = sage.cache_attn(q, kv, t, ln, None)
        graphs.append((gr, o))
    for _ in range(3):
        for gr, _ in graphs:
            gr.replay()
    torch.cuda.synchronize()
    for (gr, o), b in zip(graphs, want):
        assert torch.equal(o, b)
    ok()


def test_bad_lengths_are_recorded():
    kv, tab, _ = filled([100], 1, 64, 1)
    q = torch.zeros((1, 1, 1, 64), dtype=torch.bfloat16, device="cuda")
    sage.cache_attn(q, kv, dev(tab), dev([-3]))
    assert sage.sync_status() == 1
    sage.cache_append(kv, q.expand(1, 1, 100, 64), q.expand(1, 1, 100, 64), dev(tab), dev([100]))
    assert sage.sync_status() == 1 and sage.sync_status() == 0  # past the page table

"""Attention over pages whose value exponents lie far apart: what a page adds
to a row's sum of weights must not depend on the size of its values."""
import numpy as np
import pytest
import torch

import bit_quantized_attention_sage_b200 as sage
import cache_ref as ref
from test_gpu_kvcache import check_attn, dev, filled, ok

pytestmark = pytest.mark.gpu

# exponents of the pages in turn; 113 is that of values of about 1e37
PATTERNS = {
    "first": lambda i, n: 113 if i == 0 else -40,
    "last": lambda i, n: 113 if i == n - 1 else -40,
    "middle": lambda i, n: 113 if i == n // 2 else -40,
    "up": lambda i, n: -40 + 153 * i // max(1, n - 1),
    "down": lambda i, n: 113 - 153 * i // max(1, n - 1),
    "mixed": lambda i, n: (-40, 113, 0, 20, 52, 53, 54, 100, -7)[i * 5 % 9],
}


def spread_exponents(kv, tab, length, pattern):
    n = -(-length // 64)
    for i in range(n):
        kv.v_exp[int(tab[i])] = PATTERNS[pattern](i, n)


def randq(shape, seed):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).to(torch.bfloat16).cuda()


# one row and 16 (few-row kernel), 40 and 300 (many-row kernel, one and two tiles)
@pytest.mark.parametrize("n,G", [(1, 1), (1, 8), (4, 4), (20, 2), (300, 1)])
@pytest.mark.parametrize("pattern", sorted(PATTERNS))
@pytest.mark.parametrize("D", [64, 128])
def test_exponents_far_apart(D, pattern, n, G):
    lengths = [500, 3000, 64, 130]  # a block a head, shares, one page, a page and two tokens
    kv, tab, _ = filled(lengths, 1, D, n + G)
    for b, x in enumerate(lengths):
        spread_exponents(kv, tab[b], x, pattern)
    c = ref.Cache(kv)
    q = randq((4, G, n, D), 5)
    for mask, max_len in ((None, None), ("causal", 1000)):
        o, lse = sage.cache_attn(q, kv, dev(tab), dev(lengths), mask, max_len=max_len, return_lse=True)
        ok()
        check_attn(c, q, o, lse, tab, lengths, [n] * 4, mask, D ** -0.5)


@pytest.mark.parametrize("n", [1, 40])
@pytest.mark.parametrize("pattern", ["first", "last", "mixed"])
def test_one_head_in_many_shares(pattern, n):
    lengths, D = [9000], 128
    kv, tab, _ = filled(lengths, 1, D, 3)
    spread_exponents(kv, tab[0], lengths[0], pattern)
    c = ref.Cache(kv)
    q = randq((1, 2, n, D), 6)
    o, lse = sage.cache_attn(q, kv, dev(tab), dev(lengths), "causal", return_lse=True)
    ok()
    check_attn(c, q, o, lse, tab, lengths, [n], "causal", D ** -0.5)


@pytest.mark.parametrize("n", [1, 40])
@pytest.mark.parametrize("swap", [False, True])
def test_huge_values_beside_zeros(swap, n):
    # as they come through append: a page of values of 1e37, one of zeros
    # whose keys score 10 (in powers of two) higher
    D, lengths = 64, [128]
    kv = sage.KVCache8(2, 1, D)
    k = torch.zeros((1, 1, 128, D))
    v = torch.zeros_like(k)
    big, small = (slice(64, 128), slice(0, 64)) if swap else (slice(0, 64), slice(64, 128))
    k[..., small, 0] = 10 * np.log(2)
    v[..., big, :] = 1e37 * torch.randn((64, D), generator=torch.Generator().manual_seed(1))
    tab = np.array([[1, 0]], np.int32)
    sage.cache_append(kv, k.to(torch.bfloat16).cuda(), v.to(torch.bfloat16).cuda(), dev(tab), dev([0]))
    assert sorted(kv.v_exp.flatten().tolist())[0] == -40 and kv.v_exp.max() > 110
    c = ref.Cache(kv)
    q = torch.zeros((1, 1, n, D), dtype=torch.bfloat16, device="cuda")
    q[..., 0] = 1.0
    o, lse = sage.cache_attn(q, kv, dev(tab), dev(lengths), scale=1.0, return_lse=True)
    ok()
    check_attn(c, q, o, lse, tab, lengths, [n], None, 1.0)

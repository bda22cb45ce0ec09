"""More of the paged 8-bit cache: odd page counts in the summed weights."""
import numpy as np
import pytest
import torch

import bit_quantized_attention_sage_b200 as sage
import cache_ref as ref
from test_gpu_kvcache import dev, filled, ok
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

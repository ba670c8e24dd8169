"""Attention over 8-bit pages at the ends of what queries and keys may be."""
import numpy as np
import pytest
import torch

from test_gpu_paged import BF16, close, ints
from test_gpu_paged8 import Pool8

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("lengths,n,G", [([40], [1], 1), ([700, 33], [1, 1], 8), ([90, 700], [3, 5], 8)])
@pytest.mark.parametrize("q_size,k_size", [(1e36, 9e11), (3e38, 9e11), (-1e38, 1e9), (3e38, 1e-9), (1e-38, 9e11), (1e-38, 1e-9)])
def test_large_queries_beside_large_keys_in_other_channels(d, lengths, n, G, q_size, k_size):
    """Keys have channel 0 alone and queries all others: every product is 0, whatever the powers of two on both sides multiply to."""
    p = Pool8(lengths, n, 2, d, 16)
    t = sum(lengths)
    g = torch.Generator("cuda").manual_seed(1)
    k = torch.zeros(t, 2, d, device="cuda", dtype=BF16)
    k[::3, :, 0] = k_size
    v = torch.randn(t, 2, d, generator=g, device="cuda").to(BF16)
    p.cache.append(k, v, ints(np.concatenate([[0], np.cumsum(lengths)])))
    p.sync_back()
    q = torch.full((sum(n), 2 * G, d), q_size, device="cuda", dtype=BF16)
    q[:, :, 0] = 0
    close(p, *p.cache.attend(q, p.cu_t, return_lse=True), p.oracle(q), BF16)

"""Decode over the paged cache with scores so large that fp32 holds them in steps of several
units: every weight but the largest key's is 0 there, so the output is that key's value."""
import numpy as np
import pytest
import torch

import __graft_entry__
from gpu_helpers import f64
from oracle import qcache as Q
from test_gpu_qcache import ints

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def K():
    __graft_entry__.build()
    from long_context_anchor_gb300 import kascade
    return kascade


@pytest.mark.parametrize("prefix", [None, 64])
@pytest.mark.parametrize("dtype,d", [(BF, 128), (F32, 64)])
@pytest.mark.parametrize("exponent", [20, 22, 23, 24, 25, 26, 27, 28, 30, 40])
def test_one_key_has_the_weight(K, dtype, d, exponent, prefix):
    rng = np.random.default_rng(exponent)
    n, bs, B = 150, 32, 8
    k = rng.choice([-1.0, 1.0], (n, 1, d))
    v = rng.standard_normal((n, 1, d))
    blocks = -(-n // bs)
    table = np.tile(np.arange(blocks), (B, 1))
    pages = torch.zeros((blocks, 1, bs // 16, 18 * d), dtype=torch.uint8, device="cuda")
    dev = lambda x: torch.from_numpy(x).to(dtype).cuda()
    K.qcache_append(dev(k), dev(v), ints(np.arange(n)), pages)
    kept, vals = Q.rows_of(pages.cpu().numpy(), table[0], n, 0, d, 1.0, 1.0)
    assert np.array_equal(np.sign(kept), k[:, 0]) and np.ptp(np.abs(kept)) == 0
    # query b is `best[b]`'s key times a power of two (signs of keys: another key's product is
    # below by two elements' at least, 2^(exponent + 1) / sqrt(d) in the score)
    best = rng.choice(n, B, replace=False)
    q = dev(kept[best][:, None] * 2.0 ** exponent)
    args = (q, pages, ints(table), ints([n] * B))
    got = (K.qcache_dense_decode(*args) if prefix is None
           else K.qcache_prefix_decode(*args, prefix, always=True))
    want = vals[best]
    assert not torch.isnan(got).any()
    # the weight and the sum are the same number: the division and the output round
    assert (np.abs(f64(got[:, 0]) - want) <= (2.0 ** -8 if dtype == BF else 2.0 ** -22) * np.abs(want)).all()
    if prefix is None:
        out, idx = K.qcache_anchor_decode(*args, 4)
        assert torch.equal(out, got) and all(best[b] in idx[b, 0].tolist() for b in range(B))

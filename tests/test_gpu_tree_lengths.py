"""paged_attn_tree over the longest cache that a table of 32-bit positions holds."""

from __future__ import annotations

import numpy as np
import pytest

from gpu_util import from_dev, to_dev_i32
from test_gpu_tree_attn import gb  # noqa: F401

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.mark.parametrize("Hq", [1, 16])  # one row tile, two
@pytest.mark.parametrize("own", [0, 32])
def test_a_cache_of_2_31_tokens(gb, Hq, own):
    """2^31 - 32 cached tokens, all in one block, and a star of 16 nodes in another.  Cached keys
    have score 0, a node's own key `own`: it then weighs e^32 against 2^31, and what other nodes'
    keys would add shows.  Sums of probabilities and of values are whole numbers below 2^24 in
    every range (2^24 steps of 128 keys over 150 CTAs), so that fp32 holds them exactly."""
    D, n, L = 64, 16, 2 ** 31 - 32
    rng = np.random.default_rng(Hq + own)
    v = rng.integers(-1, 2, (2, 1, 16, D)).astype(np.float64)
    k = torch.zeros(2, 1, 16, D, dtype=torch.bfloat16, device="cuda")
    q = torch.zeros(1, Hq, n, D, dtype=torch.bfloat16, device="cuda")
    q[..., 0] = 8
    k[1, :, :, 0] = own / 8
    table = torch.zeros(1, 2 ** 27 - 1, dtype=torch.int32, device="cuda")
    table[0, -1] = 1
    o, lse = gb.paged_attn_tree(q, k, torch.from_numpy(v).to("cuda", torch.bfloat16), table,
                                to_dev_i32(np.array([L])), to_dev_i32(np.full((1, n), -1)), L + n, scale=1.0)
    torch.cuda.synchronize()
    assert gb.attn_device_status() == (gb.ATTN_OK, 0)
    weight = np.exp(np.float64(own))
    want = (L / 16 * v[0, 0].sum(0) + weight * v[1, 0]) / (L + weight)  # [n, D]
    # the result's rounding; 150 ranges put together, whose weights and sums are off by 2^-18 each at most
    # (an LSE of some 16 and e to the difference of two, the same for all channels)
    assert (np.abs(from_dev(o)[0] - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -14).all()
    assert (np.abs(from_dev(lse)[0] - np.log(L + weight)) <= 2.0 ** -16).all()

"""Draws from rows whose mass lies in very many tokens of little weight."""
import numpy as np
import pytest

from streaming_persistent_sm_b200 import wpk as W

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("below", [10.5, 11.0, 11.3, 11.75, 12.1, 12.5, 12.9, 13.2])
def test_draws_near_the_borders_of_small_tokens(below):
    """One token of weight 1 and 2^17 of w = exp(-below), 2^-15 to 2^-19.  The draw u falls (u total - 1) / w tokens
    behind the first one.  Weights are held as multiples of 2^-45, so w may be off by 2^-45, which moves that by
    (1 - u) 2^-45 / w^2 tokens; numbers u are taken that fall further than twice that from a border between two
    tokens, but nearer than (1 - u) 2^-22 / w: what a weight that is right to 2^-22 would leave open."""
    import torch

    rng = np.random.default_rng(70)
    n, B = 1 << 17, 512
    z = np.float32(-below)
    w = np.exp(np.float64(z))
    total = 1.0 + n * w
    u = rng.random(1 << 22, dtype=np.float32)
    x = (u.astype(np.float64) * total - 1.0) / w
    off = np.abs(x - np.rint(x))
    rest = 1.0 - u.astype(np.float64)
    take = (x > 0.5) & (x < n - 0.5) & (off > 2 * rest * 2.0 ** -45 / w ** 2) & (off < rest * 2.0 ** -22 / w)
    u, x = u[take][:B], x[take][:B]
    assert len(u) == B
    logits = torch.full((B, n + 1), float(z), device="cuda")
    logits[:, 0] = 0.0
    tok = W.sample(logits, torch.from_numpy(u).cuda()).cpu().numpy()
    assert (tok == np.floor(x).astype(int) + 1).all(), (tok != np.floor(x).astype(int) + 1).mean()

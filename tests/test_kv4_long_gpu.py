"""Runs of tokens in which one block goes through more tiles than its rings hold, against float64 NumPy."""
import numpy as np
import pytest

from streaming_persistent_sm_b200 import wpk as W
from tests import operators_ref as R
from tests.test_kv4_gpu import DTYPES, _i32, _torch
from tests.test_kv4_spread_gpu import _near, _to

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("sizes", ["even", "growing", "spread"])
@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("dtype", DTYPES)
def test_blocks_of_many_tiles(dtype, hd, sizes):
    """608 sequences of one new token and 64 heads fill every SM twice over, so no keys are split: up to 34 tiles of
    64 keys a block.  They repeat eight sequences, whose pages they share, and must answer the same bits.  Values are
    of one size, or grow by a factor of 1.5 every 64 keys, or differ by 10^8 (10^4 in fp16) from token to token."""
    torch = _torch()
    rng = np.random.default_rng(60)
    heads, page = 64, 48
    lens = np.array([2170, 1281, 1280, 1279, 65, 1, 2000, 1344])
    blocks = -(-int(lens.max()) // page)
    n = blocks * page
    v = rng.standard_normal((8, n, 1, hd))
    if sizes == "growing":
        v *= 1e-3 * 1.5 ** (np.arange(n) // 64)[:, None, None]
    elif sizes == "spread":
        top = 2 if dtype == "float16" else 4
        v *= 10.0 ** rng.uniform(-top, top, (8, n, 1, 1))
    (kt, k64), (vt, v64) = _to(rng.standard_normal((8, n, 1, hd)), dtype), _to(v, dtype)
    c = W.KV4Cache(8 * blocks, 1, hd, page)
    table = _i32(rng.permutation(8 * blocks).reshape(8, blocks))
    c.append(kt.reshape(-1, 1, hd), vt.reshape(-1, 1, hd), _i32([0] * 8), table)
    q, q64 = _to(rng.standard_normal((8, heads, hd)), dtype)
    pos, times = _i32(lens - 1), 76
    got = c.attention(q.repeat(times, 1, 1), pos.repeat(times), table.repeat(times, 1)).reshape(times, 8, heads, hd)
    assert torch.equal(got, got[:1].expand_as(got))
    for b in range(8):
        _near(got[0, b:b + 1], q64[b:b + 1], R.held(k64[b]), R.held(v64[b]), int(lens[b]) - 1, dtype, hd ** -0.5)


def test_many_sequences_without_a_bound_of_their_runs():
    """Without max_new any of 1100 sequences might bring all 66000 tokens; the answers are those with the bound."""
    torch = _torch()
    rng = np.random.default_rng(61)
    B, n, kv, group, hd = 1100, 60, 8, 4, 64
    c = W.KV4Cache(B, kv, hd, 64)
    table, pos = _i32(rng.permutation(B)[:, None]), _i32(np.zeros(B))
    ip = _i32(np.arange(B + 1) * n)
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    rows = lambda heads: torch.randn(B * n, heads, hd, generator=g, device="cuda").bfloat16()  # noqa: E731
    c.append(rows(kv), rows(kv), pos, table, indptr=ip)
    q = rows(kv * group)
    want = c.attention(q, pos, table, indptr=ip, max_new=n)
    assert torch.equal(c.attention(q, pos, table, indptr=ip), want)
    assert want.isfinite().all() and (want != 0).any(-1).all()

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


@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("dtype", DTYPES)
def test_a_million_keys_in_one_block(dtype, hd):
    """640 sequences of 2^20 keys (they share their pages) leave no keys to split: a warp sums 2^18 of them.  All rows
    of V are the same, so the answer is that row.  It is off by half a step of the type, by the rounding of the
    weights times V's scale (2^-11 for bf16 and fp16, 2^-21 for fp32, of the part s c), and by sums of up to 2^15 terms,
    numerator and denominator, whose roundings to nearest have either sign: n of them add up to 8 sqrt(n) 2^-24 or
    more with a probability below 1e-13.  Sums that are cut off instead lose n 2^-24 and more: 4e-3."""
    torch = _torch()
    n, B = 1 << 20, 640
    dt = getattr(torch, dtype)
    c = W.KV4Cache(n // 64, 1, hd, 64)
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    row = torch.full((hd,), 0.93, dtype=dt, device="cuda")
    row[0] = -0.21
    k = torch.randn(n, 1, hd, generator=g, device="cuda").to(dt)
    table = torch.arange(n // 64, dtype=torch.int32, device="cuda")[None]
    c.append(k, row.expand(n, 1, hd).contiguous(), _i32([0]), table)
    q = torch.randn(B, 4, hd, generator=g, device="cuda").to(dt)
    got = c.attention(q, _i32([n - 1] * B), table.repeat(B, 1)).double().cpu().numpy()
    want = R.held(row.double().cpu().numpy())
    half = torch.finfo(dt).eps / 2
    weight, sums = 2.0 ** -21 if dtype == "float32" else 2.0 ** -11, 8 * 2.0 ** 7.5 * 2.0 ** -24
    part = want - want.min()
    tol = half * np.abs(want) + weight * part + 2 * sums * (part + abs(want.min()) + np.abs(want))
    assert (np.abs(got - want) <= tol).all(), float(np.abs(got - want).max())

"""Attention over the 4-bit cache where sizes differ by many powers of ten between neighbouring queries, keys and
values, against float64 NumPy: what a query does not see, or weighs by nothing, must not change its answer."""
import numpy as np
import pytest

from streaming_persistent_sm_b200 import wpk as W
from tests import operators_ref as R
from tests.test_kv4_gpu import DTYPES, _check_attention, _i32, _torch
from tests.test_kv4_runs_gpu import _check, _wide

pytestmark = pytest.mark.gpu


def _to(x, dtype):
    """x in dtype on the GPU, and its values there in 64 bits."""
    torch = _torch()
    t = torch.from_numpy(np.asarray(x, np.float32)).to(getattr(torch, dtype))
    return t.cuda(), t.double().numpy()


def _cache(k, v, dtype, page=64):
    """A cache with the tokens k, v [n, kv, hd] of one sequence, its table, and what it holds."""
    n, kv, hd = k.shape
    blocks = -(-n // page)
    c = W.KV4Cache(blocks, kv, hd, page)
    table = _i32(np.arange(blocks)[None, ::-1].copy())
    (kt, k64), (vt, v64) = _to(k, dtype), _to(v, dtype)
    c.append(kt, vt, _i32([0]), table)
    return c, table, R.held(k64), R.held(v64)


@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
def test_neighbouring_queries_keep_their_own_sizes(dtype, hd):
    """Queries of 1, 1e-3, 1e-6 and 1e-9 in one block of rows, each attended over keys of the inverse size, where
    its logits are of ordinary size."""
    rng = np.random.default_rng(50)
    n, size = 130, np.array([1.0, 1e-3, 1e-6, 1e-9])
    q, q64 = _to(rng.standard_normal((1, 4, hd)) * size[:, None], dtype)
    v = rng.standard_normal((n, 1, hd))
    for i, s in enumerate(size):
        c, table, k64, v64 = _cache(rng.standard_normal((n, 1, hd)) / s, v, dtype)
        got = c.attention(q, _i32([n - 1]), table)
        _check_attention(got[:, i:i + 1], q64[:, i:i + 1], [(k64, v64)], [n - 1], [1], dtype, hd ** -0.5)


@pytest.mark.parametrize("bad", [np.inf, -np.inf, np.nan])
@pytest.mark.parametrize("dtype", DTYPES)
def test_a_query_that_is_not_finite_keeps_to_itself(dtype, bad):
    """Beside queries of 1e4 over keys of 1e-4, and as small ones over large keys."""
    rng = np.random.default_rng(51)
    n, hd = 70, 64
    v = rng.standard_normal((n, 1, hd))
    for size in (1e4, 1e-3):
        x = rng.standard_normal((2, 4, hd)) * size
        x[0, 2, 7] = bad
        q, q64 = _to(x, dtype)
        c, table, k64, v64 = _cache(rng.standard_normal((n, 1, hd)) / size, v, dtype)
        got = c.attention(q, _i32([n - 2]), table)
        assert got[0, 2].isnan().all()
        keep = [0, 1, 3]
        _check_attention(got[:, keep], q64[:, keep], [(k64, v64)], [n - 2], [2], dtype, hd ** -0.5)


@pytest.mark.parametrize("many", [False, True], ids=["few_rows_kernel", "many_rows_kernel"])
@pytest.mark.parametrize("dtype", DTYPES)
def test_values_that_are_all_one_large_number(dtype, many):
    """Rows of V without any range have the scale 0, so that nothing but their offset is of any size."""
    rng = np.random.default_rng(52)
    n, hd, large = 3000, 64, 2.0 ** (15 if dtype == "float16" else 60)
    c, table, k64, v64 = _cache(rng.standard_normal((n, 1, hd)) * 0.1, np.full((n, 1, hd), -large), dtype)
    new = 20 if many else 1
    q, q64 = _to(rng.standard_normal((new, 4, hd)), dtype)
    got = c.attention(q, _i32([n - new]), _wide(table, 64) if many else table)
    (_check if many else _check_attention)(got, q64, [(k64, v64)], [n - new], [new], dtype, hd ** -0.5)


def _near(got, q64, k, v, past, dtype, scale):
    """The bound of test_kv4_runs_gpu's _check for one sequence, and half of the type's least step: results below the
    normal range (2^-14 for fp16) are multiples of it (2^-24), so their rounding is off by half of it however small
    they are."""
    torch = _torch()
    info = torch.finfo(getattr(torch, dtype))
    half = info.eps / 2
    want, bulk, reach = R.attention(q64, k, v, past, scale)
    logit = (2 * 2.0 ** -12 if dtype == "bfloat16" else 2.0 ** -22) + (q64.shape[-1] + 24) * 2.0 ** -24
    weight = {"bfloat16": 2 * 2.0 ** -12, "float16": 2.0 ** -12, "float32": 2.0 ** -22}[dtype] + 1.01 * logit * (1 + reach)
    tol = half * np.abs(want) + 2 * weight[..., None] * (bulk + np.abs(want)) * (1 + half) + info.smallest_normal * half
    err = np.abs(got.double().cpu().numpy() - want)
    assert (err <= tol).all(), (float((err - tol).max()), float(err.max()))


KERNELS = [(d, m) for d in DTYPES for m in (False, True)]  # dtype, many rows
HUGE = {"float32": 1e18, "bfloat16": 1e18, "float16": 1.5e4}
TINY = {"float32": 1.0, "bfloat16": 1.0, "float16": 1e-6}


@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("dtype,many", KERNELS)
def test_a_huge_value_changes_no_query_that_does_not_weigh_it(dtype, hd, many):
    """The values of tokens 70 and 100 are huge.  Queries before them do not see them; those behind see their keys
    at logits some 60 below the others', so that they weigh 1e-26."""
    rng = np.random.default_rng(53)
    n, group = 140, 2
    u = rng.choice([-1.0, 1.0], hd)
    k = rng.standard_normal((n, 1, hd)) * 0.1
    v = rng.standard_normal((n, 1, hd)) * TINY[dtype]
    k[[70, 100], 0] = -60.0 * hd ** -0.5 * u
    v[[70, 100]] *= HUGE[dtype] / TINY[dtype]
    q, q64 = _to(u + 0.1 * rng.standard_normal((n, group, hd)), dtype)
    c, table, k64, v64 = _cache(k, v, dtype)
    got = c.attention(q, _i32([0]), _wide(table, 64) if many else table)
    _near(got, q64, k64, v64, 0, dtype, hd ** -0.5)


@pytest.mark.parametrize("dtype,many", KERNELS)
def test_a_huge_value_fades_when_larger_logits_come(dtype, many):
    """A huge value of weight 1 among the first keys, whose logits the later keys pass by 60: what it weighs then is
    nothing, and the small values behind it, up to a second huge one of weight nothing, are the answer."""
    rng = np.random.default_rng(54)
    n, hd = 1500, 64
    u = rng.choice([-1.0, 1.0], hd)
    k = rng.standard_normal((n, 1, hd)) * 0.1 + np.where(np.arange(n) < 300, -60.0 * hd ** -0.5, 0.0)[:, None, None] * u
    v = rng.standard_normal((n, 1, hd)) * TINY[dtype]
    v[[3, 700]] *= HUGE[dtype] / TINY[dtype]
    k[700] = -120.0 * hd ** -0.5 * u
    new = 20 if many else 1
    q, q64 = _to(u + 0.1 * rng.standard_normal((new, 4, hd)), dtype)
    c, table, k64, v64 = _cache(k, v, dtype)
    got = c.attention(q, _i32([n - new]), _wide(table, 64) if many else table)
    _near(got, q64, k64, v64, n - new, dtype, hd ** -0.5)


@pytest.mark.parametrize("many", [False, True], ids=["few_rows_kernel", "many_rows_kernel"])
@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
def test_a_huge_key_changes_no_query_that_does_not_weigh_it(dtype, hd, many):
    """The keys of tokens 70 and 100 are huge.  Queries before them do not see them; those behind see them at logits
    of -1e13 and less, so their exact weights are zeros and the answers are those without these tokens."""
    rng = np.random.default_rng(55)
    n, group, at = 140, 2, [70, 100]
    u = rng.choice([-1.0, 1.0], hd)
    k = rng.standard_normal((n, 1, hd))
    k[at, 0] = -1e13 * u
    v = rng.standard_normal((n, 1, hd))
    q, q64 = _to(u + 0.1 * rng.standard_normal((n, group, hd)), dtype)
    c, table, k64, v64 = _cache(k, v, dtype)
    got = c.attention(q, _i32([0]), _wide(table, 64) if many else table)
    there = np.setdiff1d(np.arange(n), at)
    _near(got[there], q64[there], k64[there], v64[there], 0, dtype, hd ** -0.5)

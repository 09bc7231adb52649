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

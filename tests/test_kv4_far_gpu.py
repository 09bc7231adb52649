"""Sequences of 2^29 positions and more, of which few have a page: the last ones are appended, read and attended."""
import numpy as np
import pytest

from streaming_persistent_sm_b200 import wpk as W
from tests import operators_ref as R
from tests.test_kv4_gpu import _check_attention, _i32, _rows, _torch

pytestmark = pytest.mark.gpu


def _far(page, first, n, kv, hd, dtype, rng):
    """n rows appended from position `first` on, pages for the positions from the page before on."""
    torch = _torch()
    blocks = (first + n - 1) // page + 1
    table = torch.full((1, blocks), -1, dtype=torch.int32, device="cuda")
    have = (n + page - 1) // page + 1
    lo = blocks - have
    table[0, lo:] = _i32(np.arange(have)[::-1].copy())
    c = W.KV4Cache(have, kv, hd, page)
    k, k64 = _rows(rng, n, kv, hd, dtype)
    v, v64 = _rows(rng, n, kv, hd, dtype)
    c.append(k, v, _i32([first]), table)
    return c, table, R.held(k64), R.held(v64), max(lo * page, 0)


@pytest.mark.parametrize("page,first", [(16, 2 ** 29 + 21), (32, 2 ** 30 + 21), (48, 3 * 2 ** 29 + 21),
                                        (16, 2 ** 31 - 100)])
def test_far_positions_hold_their_rows_and_are_attended(page, first):
    torch = _torch()
    rng = np.random.default_rng(page)
    n, kv, hd = 60, 2, 64
    c, table, k64, v64, lo = _far(page, first, n, kv, hd, "bfloat16", rng)
    gk, gv = c.read(_i32([first]), table, n, dtype=torch.float32)
    assert np.array_equal(gk.cpu().numpy(), k64.astype(np.float32))
    assert np.array_equal(gv.cpu().numpy(), v64.astype(np.float32))
    q, q64 = _rows(rng, 1, 2 * kv, hd, "bfloat16")
    got = c.attention(q, _i32([first + n - 1]), table)
    # rows of the first page in front of them were never appended: zeros, seen as keys
    pad = np.zeros((first - lo, kv, hd))
    k64, v64 = np.concatenate([pad, k64]), np.concatenate([pad, v64])
    _check_attention(got, q64, [(k64, v64)], [len(k64) - 1], [1], "bfloat16", hd ** -0.5)

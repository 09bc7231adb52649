"""Attention over the 4-bit cache for runs of tokens (many query rows a kv head), against float64 NumPy."""
import numpy as np
import pytest

from streaming_persistent_sm_b200 import wpk as W
from tests import operators_ref as R
from tests.test_kv4_gpu import DTYPES, _filled, _i32, _indptr, _positions, _rows, _table, _torch

pytestmark = pytest.mark.gpu


def _wide(table, page):
    """The table with room for 2^17 tokens a sequence, without pages there: the tcgen05 kernel takes calls
    of many rows over many keys, and it counts the keys that a table could name."""
    torch = _torch()
    more = (1 << 17) // page - table.shape[1]
    return torch.cat([table, torch.full((table.shape[0], more), -1, dtype=torch.int32, device="cuda")], 1)


def _check(got, q64, kvs, past, counts, dtype, scale):
    """|error| <= half a step of the output's type, and of the arithmetic (`bulk` and `reach` are
    R.attention's: the weighted sizes of the values' parts, the largest logit's sum of sizes).
    bf16: Q and K rounded to fp16 (2^-12 each) move a logit by 2 * 2^-12 reach, so a weight by e^d - 1
    < 1.01 d; the weights are rounded by 2^-12, the values too.  fp16: Q to 2^-22, the weights to
    2^-12.  fp32: Q and the weights to 2^-22.  All: a logit's sum of hd products and about 24 further
    roundings of 2^-24 of its terms' sizes.  Both sums of the quotient carry what a weight is off."""
    torch = _torch()
    got = got.double().cpu().numpy()
    half = torch.finfo(getattr(torch, dtype)).eps / 2
    at = np.concatenate([[0], np.cumsum(counts)])
    for b, (k, v) in enumerate(kvs):
        x = q64[at[b]:at[b + 1]]
        want, bulk, reach = R.attention(x, k, v, past[b], scale)
        logit = (2 * 2.0 ** -12 if dtype == "bfloat16" else 2.0 ** -22) + (x.shape[-1] + 24) * 2.0 ** -24
        fixed = {"bfloat16": 2 * 2.0 ** -12, "float16": 2.0 ** -12, "float32": 2.0 ** -22}[dtype]
        weight = fixed + 1.01 * logit * (1 + reach)
        tol = half * np.abs(want) + 2 * weight[..., None] * (bulk + np.abs(want)) * (1 + half)
        err = np.abs(got[at[b]:at[b + 1]] - want)
        assert (err <= tol).all(), (b, float((err - tol).max()), float(err.max()))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("hd,kv,group,page,past,counts,rope", [
    (64, 1, 64, 64, [5], [1], False),                          # one token of many heads: 64 rows
    (64, 1, 3, 16, [0, 63, 64, 65], [16, 17, 43, 85], True),   # pages that end inside a tile; 129 rows and more
    (128, 2, 4, 48, [10, 0, 0, 200], [31, 0, 1, 33], True),    # a sequence without new tokens, one with one
    (64, 2, 7, 256, [255, 256], [20, 55], False),
    (64, 1, 4, 64, [2000], [100], True),                       # keys split over a cluster, its length odd
    (128, 1, 8, 128, [2047], [17], False),
])
def test_runs_match_float64(dtype, hd, kv, group, page, past, counts, rope):
    rng = np.random.default_rng(hd + group + page)
    lens = [p + c for p, c in zip(past, counts)]
    c, table, kvs = _filled(rng, lens, kv, hd, page, dtype)
    q, q64 = _rows(rng, sum(counts), kv * group, hd, dtype)
    rt = W.rope_table(max(lens), hd, 500000.0) if rope else None
    got = c.attention(q, _i32(past), _wide(table, page), indptr=_indptr(counts), max_new=max(counts), rope=rt)
    if rope:
        q64 = R.rotate(q64, _positions(past, counts), rt.cpu().numpy())
    _check(got, q64, kvs, past, counts, dtype, hd ** -0.5)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("hd", [64, 128])
def test_runs_of_many_sequences_fill_the_gpu(dtype, hd):
    """Enough of them that no keys are split; their lengths and runs all differ."""
    rng = np.random.default_rng(36)
    B, kv, page = 80, 4, 64
    counts = rng.integers(0, 21, B)
    counts[3] = 20
    past = rng.integers(0, 120, B)
    c, table, kvs = _filled(rng, list(past + counts), kv, hd, page, dtype)
    more = _torch().full((B, 7 - table.shape[1]), 1 << 20, dtype=_torch().int32, device="cuda")
    q, q64 = _rows(rng, int(counts.sum()), 4 * kv, hd, dtype)
    got = c.attention(q, _i32(past), _torch().cat([table, more], 1), indptr=_indptr(counts), max_new=20)
    _check(got, q64, kvs, past, counts, dtype, hd ** -0.5)


@pytest.mark.parametrize("dtype", DTYPES)
def test_runs_with_values_and_queries_of_any_size(dtype):
    """Keys, values and queries whose sizes differ by powers of ten from token to token (within the
    type's range), growing and shrinking along the sequence."""
    torch = _torch()
    rng = np.random.default_rng(31)
    n, hd, top = 300, 64, 2 if dtype == "float16" else 12
    size = 10.0 ** rng.uniform(-top, top, (n, 1, 1))
    v = (rng.standard_normal((n, 1, hd)) * size).astype(np.float32)
    k = (rng.standard_normal((n, 1, hd)) * 10.0 ** rng.uniform(-3, 0, (n, 1, 1))).astype(np.float32)
    q = (rng.standard_normal((60, 3, hd)) * 10.0 ** rng.uniform(-3, 0, (60, 3, 1))).astype(np.float32)
    k, v, q = (torch.from_numpy(x).to(getattr(torch, dtype)) for x in (k, v, q))
    c = W.KV4Cache(5, 1, hd, 64)
    table = _i32([[3, 1, 0, 2, 4]])
    c.append(k.cuda(), v.cuda(), _i32([0]), table)
    got = c.attention(q.cuda(), _i32([n - 60]), _wide(table, 64))
    _check(got, q.double().numpy(), [(R.held(k.double().numpy()), R.held(v.double().numpy()))], [n - 60], [60],
           dtype, hd ** -0.5)


@pytest.mark.parametrize("dtype", DTYPES)
def test_runs_leave_out_pages_and_sequences_without_a_place(dtype):
    rng = np.random.default_rng(32)
    lens, new = [200] * 4, 30
    c, table, kvs = _filled(rng, lens, 2, 64, 16, dtype)
    t = table.clone()
    t[1, 3] = -1               # 16 keys of sequence 1 are gone
    t[2, :] = 1 << 30          # all of sequence 2's
    q, q64 = _rows(rng, 4 * new, 4, 64, dtype)
    got = c.attention(q, _i32([170, 170, 170, -1]), _wide(t, 16))  # sequence 3 is idle
    assert (got[2 * new:] == 0).all()
    k, v = kvs[1]
    there = np.r_[0:48, 64:200]
    _check(got[:2 * new], q64[:2 * new], [kvs[0], (k[there], v[there])], [170, 154], [new] * 2, dtype, 0.125)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("which", ["k", "v"])
def test_runs_keep_a_row_that_is_not_finite_to_the_queries_that_see_it(dtype, which):
    rng = np.random.default_rng(33)
    n = 150
    k, k64 = _rows(rng, n, 1, 64, dtype)
    v, v64 = _rows(rng, n, 1, 64, dtype)
    (k if which == "k" else v)[70, 0, 5] = float("nan")
    c = W.KV4Cache(3, 1, 64, 64)
    table = _i32([[0, 2, 1]])
    c.append(k, v, _i32([0]), table)
    q, q64 = _rows(rng, n, 2, 64, dtype)
    got = c.attention(q, _i32([0]), _wide(table, 64))
    assert got[70:].isnan().all() and not got[:70].isnan().any()
    _check(got[:70], q64[:70], [(R.held(k64[:70]), R.held(v64[:70]))], [0], [70], dtype, 0.125)
    q[3, 1, 0] = float("inf")  # a query that is not finite keeps to itself
    other = c.attention(q, _i32([0]), _wide(table, 64))
    assert other[3, 1].isnan().all()
    assert _torch().equal(other[:3], got[:3]) and _torch().equal(other[4:70], got[4:70])


def test_runs_stop_where_the_rotations_and_the_rows_do():
    torch = _torch()
    rng = np.random.default_rng(34)
    c, table, kvs = _filled(rng, [100], 1, 64, 64, "float32")
    q, q64 = _rows(rng, 60, 2, 64, "float32")
    rt = W.rope_table(90, 64, 500000.0)
    out = torch.full((60, 2, 64), 7.0, device="cuda")
    c.attention(q, _i32([40]), _wide(table, 64), indptr=_i32([0, 57]), max_new=60, rope=rt, out=out)
    assert (out[57:] == 7.0).all()               # behind the last sequence: left as they were
    assert (out[50:57] == 0.0).all()             # positions without a rotation
    _check(out[:50], R.rotate(q64[:50], np.arange(40, 90), rt.cpu().numpy()), kvs, [40], [50], "float32", 0.125)


@pytest.mark.parametrize("dtype", ["bfloat16", "float16"])
def test_runs_on_other_streams_captured_and_twice_at_once(dtype):
    torch = _torch()
    rng = np.random.default_rng(35)
    past, counts = [300, 0, 65], [40, 33, 64]
    c, table, _ = _filled(rng, [p + n for p, n in zip(past, counts)], 2, 64, 64, dtype)
    q, _ = _rows(rng, sum(counts), 8, 64, dtype)
    pos, ip, table = _i32(past), _indptr(counts), _wide(table, 64)
    run = lambda out: c.attention(q, pos, table, indptr=ip, max_new=64, out=out)  # noqa: E731
    want = run(None)
    outs = [torch.zeros_like(q) for _ in range(4)]
    streams = [torch.cuda.Stream() for _ in outs]
    torch.cuda.synchronize()
    for o, s in zip(outs, streams):
        with torch.cuda.stream(s):
            for _ in range(5):
                run(o)
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in outs)
    g = torch.cuda.CUDAGraph()
    outs[0].zero_()
    with torch.cuda.graph(g):
        run(outs[0])
    g.replay()
    assert torch.equal(outs[0], want)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("wide", [False, True], ids=["few_rows_kernel", "many_rows_kernel"])
@pytest.mark.parametrize("sign", [1, -1])
def test_logits_of_tens_of_millions(dtype, wide, sign):
    """Keys a_j u and queries b u with u of +-1: logits of 7e7 and more, those of two keys 3 % (2e6) apart,
    so each query answers with the value of one key, off only by the roundings of weights and values."""
    torch = _torch()
    rng = np.random.default_rng(37)
    n, hd = 24, 64
    u = rng.choice([-1.0, 1.0], hd)
    a = 3000.0 * 1.03 ** rng.permutation(n)
    to = lambda x: torch.from_numpy(x.astype(np.float32)).to(getattr(torch, dtype))  # noqa: E731
    k, q = to(a[:, None, None] * u), to(np.broadcast_to(sign * 3000.0 * u, (n, 4, hd)).copy())
    v, v64 = _rows(rng, n, 1, hd, dtype)
    c = W.KV4Cache(1, 1, hd, 64)
    table = _i32([[0]])
    c.append(k.cuda(), v, _i32([0]), table)
    got = c.attention(q.cuda(), _i32([0]), _wide(table, 64) if wide else table).double().cpu().numpy()
    want, bulk, _ = R.attention(q.double().numpy(), R.held(k.double().numpy()), R.held(v64), 0, 0.125)
    half = torch.finfo(getattr(torch, dtype)).eps / 2
    fixed = {"bfloat16": 2 * 2.0 ** -12, "float16": 2.0 ** -12, "float32": 2.0 ** -20}[dtype]
    assert (np.abs(got - want) <= half * np.abs(want) + 2 * fixed * (bulk + np.abs(want)) * (1 + half)).all()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("wide", [False, True], ids=["few_rows_kernel", "many_rows_kernel"])
def test_queries_and_keys_of_zeros_answer_means(dtype, wide):
    torch = _torch()
    rng = np.random.default_rng(38)
    n = 70
    v, v64 = _rows(rng, n, 1, 64, dtype)
    k, q = torch.zeros_like(v), torch.zeros(n, 4, 64, dtype=v.dtype, device="cuda")
    c = W.KV4Cache(2, 1, 64, 64)
    table = _i32([[1, 0]])
    c.append(k, v, _i32([0]), table)
    got = c.attention(q, _i32([0]), _wide(table, 64) if wide else table)
    _check(got, np.zeros((n, 4, 64)), [(np.zeros((n, 1, 64)), R.held(v64))], [0], [n], dtype, 0.125)

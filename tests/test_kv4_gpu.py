"""The 4-bit paged cache on the GPU: append, read and attention against float64 NumPy."""
import numpy as np
import pytest

from streaming_persistent_sm_b200 import wpk as W
from tests import operators_ref as R

pytestmark = pytest.mark.gpu

DTYPES = ["float32", "bfloat16", "float16"]


def _torch():
    import torch

    return torch


def _rows(rng, n, heads, hd, dtype, size=1.0):
    """Random rows in dtype (on the GPU) and their exact values."""
    torch = _torch()
    x = torch.from_numpy((rng.standard_normal((n, heads, hd)) * size).astype(np.float32)).to(getattr(torch, dtype))
    return x.cuda(), x.double().numpy()


def _i32(x):
    return _torch().tensor(np.asarray(x), dtype=_torch().int32, device="cuda")


def _table(rng, batch, blocks):
    return _i32(rng.permutation(batch * blocks).reshape(batch, blocks))


def _indptr(counts):
    return _i32(np.concatenate([[0], np.cumsum(counts)]))


def _positions(pos, counts):
    return np.concatenate([np.arange(p, p + c) for p, c in zip(pos, counts)]) if sum(counts) else np.zeros(0, int)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("hd,kv,page,counts,past,rope", [
    (64, 8, 64, [1], [600], True),
    (64, 1, 16, [1, 1, 1], [0, 15, 16], False),
    (64, 2, 64, [5, 0, 1, 130], [0, 7, 63, 1], True),
    (128, 3, 48, [47, 2, 96, 0, 33], [1, 47, 0, 3, 100], True),
    (128, 1, 256, [300], [0], False),
    (64, 3, 32, [2] * 40, list(range(40)), True),
])
def test_append_holds_the_exact_codes(dtype, hd, kv, page, counts, past, rope):
    torch = _torch()
    rng = np.random.default_rng(hd + kv + page)
    total = sum(counts)
    blocks = -(-max(p + c for p, c in zip(past, counts)) // page)
    c = W.KV4Cache(len(counts) * blocks, kv, hd, page)
    k, k64 = _rows(rng, total, kv, hd, dtype, 3.0)
    v, v64 = _rows(rng, total, kv, hd, dtype, 0.01)
    table, pos, ip = _table(rng, len(counts), blocks), _i32(past), _indptr(counts)
    rt = W.rope_table(blocks * page, hd, 500000.0) if rope else None
    c.append(k, v, pos, table, indptr=ip, rope=rt)
    if rope:
        k64 = R.rotate(k64, _positions(past, counts), rt.cpu().numpy())
    # s c + z is rounded once, to the type that is asked for
    for want_type in ("float32", dtype):
        gk, gv = c.read(pos, table, total, indptr=ip, dtype=getattr(torch, want_type))
        for got, x in ((gk, k64), (gv, v64)):
            want = torch.from_numpy(R.held(x).astype(np.float32)).to(getattr(torch, want_type))
            assert torch.equal(got.cpu(), want)


def test_append_rounds_ties_and_odd_rows_as_defined():
    torch = _torch()
    hd = 64
    rows = np.zeros((9, hd), np.float32)
    rows[0] = np.arange(hd) / 4.0            # quotients that are whole numbers and halves
    rows[0, 60:] = 15.0
    rows[0] = np.minimum(rows[0], 15.0)
    rows[1] = np.where(np.arange(hd) % 2, 7.5, 0.0)
    rows[1, 0] = 15.0
    rows[2] = -3.0                           # one value only: s = 0
    rows[3] = 1.0 + 2.0 ** -20               # one value that bf16 cannot hold
    rows[4] = np.linspace(-1e-30, 1e-30, hd)
    rows[5] = np.linspace(-3e37, 3e37, hd)
    rows[6] = np.linspace(1000.0, 1000.001, hd)
    rows[7] = np.linspace(-1000.001, -1000.0, hd)
    rows[8, 3] = -1e-3
    x = torch.from_numpy(rows[:, None]).cuda()
    c = W.KV4Cache(1, 1, hd, 16)
    table, pos = _i32([[0]]), _i32([0])
    c.append(x, -x, pos, table)
    k, v = c.read(pos, table, len(rows), dtype=torch.float32)
    assert np.array_equal(k.cpu().numpy()[:, 0], R.held(rows).astype(np.float32))
    assert np.array_equal(v.cpu().numpy()[:, 0], R.held(-rows.astype(np.float64)).astype(np.float32))


@pytest.mark.parametrize("bad", [np.nan, np.inf, -np.inf])
@pytest.mark.parametrize("rope", [False, True])
def test_rows_that_are_not_finite_read_as_nan_and_no_other_does(bad, rope):
    torch = _torch()
    rng = np.random.default_rng(3)
    k, _ = _rows(rng, 6, 2, 64, "float32")
    v, _ = _rows(rng, 6, 2, 64, "float32")
    k[2, 1, 40] = bad
    v[4, 0, 0] = bad
    c = W.KV4Cache(1, 2, 64, 16)
    table, pos = _i32([[0]]), _i32([0])
    c.append(k, v, pos, table, rope=W.rope_table(16, 64) if rope else None)
    gk, gv = (x.cpu().numpy() for x in c.read(pos, table, 6, dtype=torch.float32))
    for got, at in ((gk, (2, 1)), (gv, (4, 0))):
        nan = np.isnan(got).any(-1)
        assert nan[at] and np.isnan(got[at]).all() and nan.sum() == 1


def test_rows_without_a_place_are_dropped_and_read_as_zeros():
    torch = _torch()
    rng = np.random.default_rng(4)
    counts, past = [3, 4, 40, 2, 20], [0, -1, 0, 5, 30]  # sequence 1 is idle, 4 outgrows its table
    k, k64 = _rows(rng, sum(counts), 1, 64, "bfloat16")
    v, v64 = _rows(rng, sum(counts), 1, 64, "bfloat16")
    table = np.arange(5 * 3).reshape(5, 3)
    table[2, 1] = -1          # no page for positions 16 .. 31
    table[3, 0] = 99          # nor such a page
    c = W.KV4Cache(15, 1, 64, 16)
    t, pos, ip = _i32(table), _i32(past), _indptr(counts)
    before = c.pages.clone()
    c.append(k, v, pos, t, indptr=ip)
    gk, gv = (x.cpu().numpy() for x in c.read(pos, t, sum(counts), indptr=ip, dtype=torch.float32))
    p = _positions([max(x, 0) for x in past], counts)
    seq = np.repeat(np.arange(5), counts)
    there = (seq != 1) & (seq != 3) & (p < 48) & ~((seq == 2) & (p >= 16) & (p < 32))
    for got, x in ((gk, k64), (gv, v64)):
        assert np.array_equal(got[there], R.held(x[there]).astype(np.float32))
        assert (got[~there] == 0).all()
    used = {int(table[s, q // 16]) for s, q, on in zip(seq, p, there) if on}
    untouched = [b for b in range(15) if b not in used]
    assert torch.equal(c.pages[untouched], before[untouched])


def test_a_rope_table_ends_the_positions_that_are_appended_and_answered():
    torch = _torch()
    rng = np.random.default_rng(5)
    k, k64 = _rows(rng, 20, 1, 64, "float32")
    c = W.KV4Cache(2, 1, 64, 16)
    table, pos, rt = _i32([[1, 0]]), _i32([0]), W.rope_table(10, 64)
    c.append(k, k, pos, table, rope=rt)
    got, _ = c.read(pos, table, 20, dtype=torch.float32)
    want = R.held(R.rotate(k64[:10], np.arange(10), rt.cpu().numpy())).astype(np.float32)
    assert np.array_equal(got.cpu().numpy()[:10], want)
    assert (got.cpu().numpy()[10:] == 0).all()
    o = c.attention(k, pos, table, rope=rt)
    assert (o[10:] == 0).all() and (o[:10] != 0).any(-1).all()


def test_rows_behind_the_last_sequence_are_left_as_they_were():
    torch = _torch()
    rng = np.random.default_rng(6)
    q, _ = _rows(rng, 12, 4, 64, "bfloat16")
    k, _ = _rows(rng, 12, 2, 64, "bfloat16")
    c = W.KV4Cache(2, 2, 64, 16)
    table, pos, ip = _i32([[0], [1]]), _i32([0, 2]), _i32([0, 3, 7])
    c.append(k, k, pos, table, indptr=ip)
    out = torch.full_like(q, 7.0)
    c.attention(q, pos, table, indptr=ip, out=out)
    assert (out[7:] == 7.0).all() and (out[:7] != 7.0).any(-1).all()
    gk = torch.full((12, 2, 64), 5.0, dtype=torch.bfloat16, device="cuda")
    gv = torch.full_like(gk, 6.0)
    cs = W.wpk_kv4_cache(c.pages.data_ptr(), table.data_ptr(), 2, 2, 1, 2, 64, 16)
    W.wpk_kv4_read(cs, pos.data_ptr(), ip.data_ptr(), 12, gk.data_ptr(), gk.stride()[:2], gv.data_ptr(),
                   gv.stride()[:2], W.WPK_BF16, torch.cuda.current_stream().cuda_stream)
    assert (gk[7:] == 5.0).all() and (gv[7:] == 6.0).all() and (gk[:7] != 5.0).any()


def _filled(rng, lens, kv, hd, page, dtype, size=1.0, table=None):
    """A cache with lens[b] tokens of each sequence, its table, and the values it holds."""
    blocks = max(1, -(-max(lens) // page))
    c = W.KV4Cache(len(lens) * blocks, kv, hd, page)
    table = _table(rng, len(lens), blocks) if table is None else table
    k, k64 = _rows(rng, sum(lens), kv, hd, dtype, size)
    v, v64 = _rows(rng, sum(lens), kv, hd, dtype, size)
    c.append(k, v, _i32([0] * len(lens)), table, indptr=_indptr(lens))
    at = np.concatenate([[0], np.cumsum(lens)])
    return c, table, [(R.held(k64[a:b]), R.held(v64[a:b])) for a, b in zip(at[:-1], at[1:])]


def _check_attention(got, q64, kvs, past, counts, dtype, scale):
    """|error| <= half a step of the output's type, and of the arithmetic: each logit is a sum of hd
    products in fp32 (and of about 24 further roundings of 2^-24 of its terms' sizes), which changes
    a weight by e^d - 1 < 1.01 d; a weight is rounded to 2^-12 for bf16 (fp16 operand), to 2^-21 for
    fp32 (fp16 is held to the same, though one of its weights alone may be off by 2^-12).  The weights multiply s c and z of a value v = s c + z, not v: sum p (s c + |z|), which
    R.attention gives as `bulk`, is what a relative error of the weights can move the sum by.  Both
    sums of the quotient carry this."""
    torch = _torch()
    got = got.double().cpu().numpy()
    half = torch.finfo(getattr(torch, dtype)).eps / 2
    at = np.concatenate([[0], np.cumsum(counts)])
    for b, (k, v) in enumerate(kvs):
        x = q64[at[b]:at[b + 1]]
        want, bulk, reach = R.attention(x, k, v, past[b], scale)
        hd = x.shape[-1]
        weight = (2.0 ** -12 if dtype == "bfloat16" else 2.0 ** -21) + 1.01 * (hd + 24) * 2.0 ** -24 * (1 + reach)
        tol = half * np.abs(want) + 2 * weight[..., None] * (bulk + np.abs(want)) * (1 + half)
        err = np.abs(got[at[b]:at[b + 1]] - want)
        assert (err <= tol).all(), (b, float((err - tol).max()), float(err.max()))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("hd,kv,group,page,past,counts,rope", [
    (64, 2, 4, 64, [0], [1], False),                                # a single key
    (64, 1, 1, 16, [62, 63, 64, 65, 127, 511, 512, 513], [1] * 8, True),
    (64, 8, 4, 64, [623, 0, 300], [1] * 3, True),
    (128, 2, 8, 64, [700, 64, 5], [1] * 3, True),
    (128, 1, 3, 48, [47, 48, 1000], [1] * 3, False),
    (64, 2, 7, 32, [100, 3], [1, 1], True),
    (64, 1, 16, 64, [200], [1], False),                             # more heads than a row block
    (64, 2, 4, 64, [0, 130, 7, 0], [67, 5, 0, 1], True),            # runs of tokens, a sequence without any
    (128, 1, 5, 16, [0, 31], [130, 33], False),
    (64, 3, 2, 256, [255], [260], True),
])
def test_attention_matches_float64(dtype, hd, kv, group, page, past, counts, rope):
    rng = np.random.default_rng(hd * group + page)
    lens = [p + c for p, c in zip(past, counts)]
    c, table, kvs = _filled(rng, lens, kv, hd, page, dtype)
    q, q64 = _rows(rng, sum(counts), kv * group, hd, dtype)
    rt = W.rope_table(max(lens), hd, 500000.0) if rope else None
    got = c.attention(q, _i32(past), table, indptr=_indptr(counts), max_new=max(counts), rope=rt)
    if rope:
        q64 = R.rotate(q64, _positions(past, counts), rt.cpu().numpy())
    _check_attention(got, q64, kvs, past, counts, dtype, hd ** -0.5)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("hd", [64, 128])
def test_attention_over_a_long_axis_and_few_rows(dtype, hd):
    # one sequence over many CTAs of a cluster, its length odd; a scale of its own
    rng = np.random.default_rng(11)
    c, table, kvs = _filled(rng, [40001], 1, hd, 64, dtype)
    q, q64 = _rows(rng, 1, 2, hd, dtype)
    got = c.attention(q, _i32([40000]), table, scale=0.3)
    _check_attention(got, q64, kvs, [40000], [1], dtype, float(np.float32(0.3)))


@pytest.mark.parametrize("size", [1e-20, 1e-6, 3e4])
def test_attention_with_values_of_any_size(size):
    """Scales far from 1, a sequence whose values' sizes differ from token to token, rows that peak."""
    torch = _torch()
    rng = np.random.default_rng(12)
    n, hd = 200, 64
    k = rng.standard_normal((n, 1, hd)).astype(np.float32)
    v = (rng.standard_normal((n, 1, hd)) * size * 10.0 ** rng.uniform(-2, 2, (n, 1, 1))).astype(np.float32)
    q = rng.standard_normal((1, 4, hd)).astype(np.float32)
    c = W.KV4Cache(4, 1, hd, 64)
    table = _i32([[3, 1, 0, 2]])
    c.append(torch.from_numpy(k).cuda(), torch.from_numpy(v).cuda(), _i32([0]), table)
    got = c.attention(torch.from_numpy(q).cuda(), _i32([n - 1]), table)
    kvs = [(R.held(k.astype(np.float64)), R.held(v.astype(np.float64)))]
    _check_attention(got, q.astype(np.float64), kvs, [n - 1], [1], "float32", hd ** -0.5)


def test_attention_leaves_out_pages_and_sequences_without_a_place():
    torch = _torch()
    rng = np.random.default_rng(13)
    lens = [100, 100, 100, 100]
    c, table, kvs = _filled(rng, lens, 2, 64, 16, "float32")
    t = table.clone()
    t[1, 2] = -1               # 16 keys of sequence 1 are gone
    t[2, :] = 1 << 30          # all of sequence 2's
    q, q64 = _rows(rng, 4, 4, 64, "float32")
    pos = _i32([99, 99, 99, -1])  # and sequence 3 is idle
    got = c.attention(q, pos, t)
    assert (got[2:] == 0).all()
    k, v = kvs[1]
    gone = np.r_[0:32, 48:100]
    _check_attention(got[:2], q64[:2], [kvs[0], (k[gone], v[gone])], [99, 83], [1, 1], "float32", 0.125)


def test_attention_keeps_a_row_that_is_not_finite_to_the_queries_that_see_it():
    torch = _torch()
    rng = np.random.default_rng(14)
    k, k64 = _rows(rng, 70, 1, 64, "float32")
    v, v64 = _rows(rng, 70, 1, 64, "float32")
    v[40, 0, 1] = np.nan
    c = W.KV4Cache(2, 1, 64, 64)
    table = _i32([[0, 1]])
    c.append(k, v, _i32([0]), table)
    q, q64 = _rows(rng, 70, 2, 64, "float32")
    got = c.attention(q, _i32([0]), table)
    assert got[40:].isnan().all() and not got[:40].isnan().any()
    _check_attention(got[:40], q64[:40], [(R.held(k64[:40]), R.held(v64[:40]))], [0], [40], "float32", 0.125)


def test_strided_tensors_other_streams_and_captured_graphs():
    torch = _torch()
    rng = np.random.default_rng(15)
    B, H, kv, hd = 3, 8, 2, 64
    past = [70, 5, 129]
    c, table, kvs = _filled(rng, [p + 1 for p in past], kv, hd, 64, "bfloat16")
    packed, x64 = _rows(rng, B, H + 2 * kv, hd, "bfloat16")  # q, k and v of a token side by side
    q, k, v = packed[:, :H], packed[:, H:H + kv], packed[:, H + kv:]
    pos, rt = _i32(past), W.rope_table(256, hd)
    out = torch.zeros(B, 2 * H, hd, dtype=torch.bfloat16, device="cuda")[:, ::2]

    def step():
        c.append(k, v, pos, table, rope=rt)
        c.attention(q, pos, table, rope=rt, out=out)

    def check():
        at, cs = np.array(past), rt.cpu().numpy()
        k64 = R.held(R.rotate(x64[:, H:H + kv], at, cs))
        v64 = R.held(x64[:, H + kv:])
        new = [(np.concatenate([a[:p], k64[i:i + 1]]), np.concatenate([b[:p], v64[i:i + 1]]))
               for i, ((a, b), p) in enumerate(zip(kvs, past))]
        _check_attention(out, R.rotate(x64[:, :H], at, cs), new, past, [1] * B, "bfloat16", hd ** -0.5)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    check()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for _ in range(2):  # the same graph on new tokens
        fresh, x64 = _rows(rng, B, H + 2 * kv, hd, "bfloat16")
        packed.copy_(fresh)
        out.zero_()
        g.replay()
        check()


def test_two_runs_give_the_same_bits():
    rng = np.random.default_rng(16)
    c, table, _ = _filled(rng, [3000, 17], 2, 64, 64, "bfloat16")
    q, _ = _rows(rng, 2, 8, 64, "bfloat16")
    a, b = (c.attention(q, _i32([2999, 16]), table) for _ in range(2))
    assert _torch().equal(a, b)


def test_empty_calls_do_nothing():
    torch = _torch()
    c = W.KV4Cache(1, 1, 64, 16)
    table, pos = _i32([[0]]), _i32([0])
    x = torch.empty(0, 1, 64, device="cuda")
    c.append(x, x, pos, table)
    assert c.read(pos, table, 0)[0].shape == (0, 1, 64)
    assert c.attention(x, pos, table).shape == (0, 1, 64)


def test_python_refusals():
    torch = _torch()
    c = W.KV4Cache(2, 2, 64, 16)
    x = torch.zeros(4, 2, 64, device="cuda")
    table, pos = _i32([[0], [1]]), _i32([0, 0])
    c.append(x, x, pos, table)
    for call in [
        lambda: c.append(x, x[:3], pos, table),
        lambda: c.append(x, x.bfloat16(), pos, table),
        lambda: c.append(x.double(), x.double(), pos, table),
        lambda: c.append(x.cpu(), x, pos, table),
        lambda: c.append(x, x, pos.long(), table),
        lambda: c.append(x, x, pos[:1], table),
        lambda: c.append(x, x, pos, table.float()),
        lambda: c.append(x, x, pos, _i32([[0, 0], [1, 1]])[:, :1]),
        lambda: c.append(x, x, pos, table, indptr=_i32([0, 4])),
        lambda: c.append(x, x, pos, table, rope=torch.zeros(8, 32, device="cuda")),
        lambda: c.append(x[:3], x[:3], pos, table),
        lambda: c.append(x.transpose(1, 2), x, pos, table),
        lambda: c.attention(torch.zeros(4, 3, 64, device="cuda"), pos, table),
        lambda: c.attention(x, pos, table, scale=float("nan")),
        lambda: c.attention(x, pos, table, max_new=-1),
        lambda: c.attention(x, pos, table, out=x.bfloat16()),
        lambda: c.read(pos, table, 4, dtype=torch.float64),
        lambda: W.KV4Cache(2, 2, 96, 16),
        lambda: W.KV4Cache(2, 2, 64, 24),
        lambda: W.KV4Cache(0, 2, 64, 16),
    ]:
        with pytest.raises(W.WpkError):
            call()

"""wpk_sample against its definition in float64 NumPy."""
import numpy as np
import pytest

from streaming_persistent_sm_b200 import wpk as W
from tests import operators_ref as R

pytestmark = pytest.mark.gpu


def _dev(x, dtype=None):
    import torch

    return None if x is None else torch.as_tensor(np.asarray(x), dtype=dtype or torch.float32).cuda()


def _check(logits, u, dtype="float32", **kw):
    """Tokens and kept counts equal; a log-probability is a 64-bit value rounded to fp32 (half a
    step, 2^-24 of it), off by the masses' 2^-45 steps (2^-20 for 2^18 of them, in all 1e-6 of a
    mass of at least 1) before that."""
    import torch

    x = torch.from_numpy(np.asarray(logits, dtype=np.float32)).to(getattr(torch, dtype))
    z = x.double().numpy()
    i32 = torch.int32
    got = W.sample(x.cuda(), _dev(u), temperature=_dev(kw.get("temperature")), top_k=_dev(kw.get("top_k"), i32),
                   top_p=_dev(kw.get("top_p")), min_p=_dev(kw.get("min_p")), want_logprob=True, want_kept=True)
    tok, lp, kept = (t.cpu().numpy() for t in got)
    f = lambda n, d, b: float(np.float32(kw[n][b])) if kw.get(n) is not None else d  # noqa: E731
    for b in range(len(z)):
        want, wlp, ids = R.sample_row(z[b], float(np.float32(u[b])), f("temperature", 1.0, b), int(f("top_k", 0, b)),
                                      f("top_p", 1.0, b), f("min_p", 0.0, b))
        assert kept[b] == len(ids), (b, kept[b], len(ids))
        assert tok[b] == want, (b, tok[b], want)
        if np.isnan(wlp):
            assert np.isnan(lp[b])
        else:
            assert abs(lp[b] - wlp) <= 2.0 ** -24 * abs(wlp) + 1e-6, (b, lp[b], wlp)
    return tok


def _logits(rng, B, V, spread=2.0, peaks=20):
    z = rng.standard_normal((B, V)) * spread
    for b in range(B):
        at = rng.integers(0, V, peaks)
        z[b, at] += rng.exponential(4.0, peaks) + 4.0
    return z


@pytest.mark.parametrize("dtype", ["float32", "bfloat16", "float16"])
@pytest.mark.parametrize("B,V", [(1, 1), (3, 2), (5, 33), (4, 1000), (2, 8192), (3, 8193), (2, 32003), (1, 128256),
                                 (40, 20011), (2, 262144)])
def test_every_filter_alone_and_together(B, V, dtype):
    rng = np.random.default_rng(B * V)
    z, u = _logits(rng, B, V), rng.random(B, dtype=np.float32)
    T = rng.choice([0.5, 1.0, 1.7], B)
    k, p, m = rng.choice([1, 7, 50, 2000, 0], B), rng.choice([0.1, 0.9, 0.99, 1.0], B), rng.choice([0.0, 0.05, 0.5], B)
    for kw in (dict(), dict(temperature=T), dict(top_k=k), dict(temperature=T, top_p=p), dict(min_p=m),
               dict(temperature=T, top_k=k, top_p=p, min_p=m)):
        _check(z, u, dtype, **kw)


@pytest.mark.parametrize("V", [700, 50021])
def test_flat_rows_keep_many_tokens(V):
    # hardly any difference between tokens: borders deep in the row, buckets that overflow the sorted list
    rng = np.random.default_rng(V)
    z = rng.standard_normal((6, V)) * np.array([1e-3, 1e-5, 0.1, 1.0, 1e-3, 1e-5])[:, None]
    z[4:] += 30.0 * (np.arange(V) == 17)
    u = rng.random(6, dtype=np.float32)
    _check(z, u, top_p=[0.5, 0.9, 0.3, 0.99, 0.9, 1e-3])
    _check(z, u, top_k=[V // 2, V - 1, 13, V // 3, 2, V], temperature=[1.0, 1.0, 0.1, 3.0, 100.0, 1e6])
    _check(z, u, top_k=[V // 2] * 6, top_p=[0.5, 0.999, 0.25, 0.75, 0.0, 1.0])


@pytest.mark.parametrize("V", [64, 5000, 40000])
def test_ties_go_to_the_lowest_ids(V):
    rng = np.random.default_rng(V)
    z = rng.integers(0, 3, (5, V)).astype(np.float64)
    z[0] = 2.0                                    # one value only
    z[1] = np.where(np.arange(V) % 2, 0.0, -0.0)  # and zeros of both signs
    u = np.array([0.0, 0.25, 0.5, 0.999999, 1.0 - 2.0 ** -24], np.float32)
    _check(z, u, top_k=[V // 4, V // 2, 1, 5, V - 1])
    _check(z, u, top_p=[0.25, 0.5, 0.7, 0.9, 1e-6])
    _check(z, u, temperature=[0.0, 0.0, 0.0, -1.0, 1e-30])


def test_masked_rows():
    rng = np.random.default_rng(7)
    z = _logits(rng, 8, 9001)
    z[0, 10:] = -np.inf               # few tokens left
    z[1] = -np.inf
    z[1, 8999] = -40.0                # one
    z[2] = -np.inf                    # none
    z[3, rng.random(9001) < 0.99] = -3.4028234663852886e38  # masked by the type's lowest value
    z[4, 5] = np.nan
    z[5, 5] = np.inf
    z[6] = -3.4028234663852886e38     # all tokens at that value
    u = rng.random(8, dtype=np.float32)
    for kw in (dict(), dict(top_k=[20] * 8), dict(top_p=[0.9] * 8), dict(min_p=[0.1] * 8),
               dict(top_k=[500] * 8, top_p=[0.8] * 8, min_p=[0.01] * 8), dict(temperature=[0.0] * 8)):
        tok = _check(z, u, **kw)
        assert (tok[[2, 4, 5]] == -1).all()


def test_parameters_out_of_their_ranges():
    rng = np.random.default_rng(8)
    z = _logits(rng, 6, 3001)
    u = np.array([0.0, -1.0, 2.0, 1.0, 0.3, 0.7], np.float32)
    _check(z, u, top_k=[-5, 0, 3001, 10 ** 9, 1, 2], top_p=[2.0, 1.0, -1.0, 0.0, 5.0, 0.5],
           min_p=[-1.0, 2.0, 0.0, 1.0, 0.5, 1e-30], temperature=[1.0, 1e30, 1e-30, np.inf, 1.0, 2.0])


def test_draws_follow_the_distribution():
    # a grid of uniform numbers over one row: token i is drawn for its share of them, to the grid's step
    rng = np.random.default_rng(9)
    n, V = 4096, 50
    row = rng.standard_normal(V)
    u = (np.arange(n) + 0.5) / n
    tok = W.sample(_dev(np.tile(row, (n, 1))), _dev(u)).cpu().numpy()
    share = np.exp(row) / np.exp(row).sum()
    assert (np.abs(np.bincount(tok, minlength=V) / n - share) <= 1.0 / n + 1e-6).all()
    assert (np.diff(tok) >= 0).all()


def test_strides_streams_and_captured_graphs():
    import torch

    rng = np.random.default_rng(10)
    B, V = 5, 12345
    wide = torch.zeros(B, V + 7, device="cuda")
    x = wide[:, 3:3 + V]
    u, p, out = torch.zeros(B, device="cuda"), torch.full((B,), 0.8, device="cuda"), torch.zeros(
        B, dtype=torch.int32, device="cuda")

    def fill(seed):
        r = np.random.default_rng(seed)
        z, un = _logits(r, B, V).astype(np.float32), r.random(B, dtype=np.float32)
        x.copy_(torch.from_numpy(z))
        u.copy_(torch.from_numpy(un))
        return [R.sample_row(z[b], un[b], top_p=float(np.float32(0.8)))[0] for b in range(B)]

    want = fill(1)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        W.sample(x, u, top_p=p, out_tok=out)
    torch.cuda.current_stream().wait_stream(side)
    assert out.tolist() == want
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        W.sample(x, u, top_p=p, out_tok=out)
    for seed in (2, 3):
        want = fill(seed)
        g.replay()
        assert out.tolist() == want


def test_python_refusals():
    import torch

    x, u = torch.zeros(2, 100, device="cuda"), torch.zeros(2, device="cuda")
    W.sample(x, u)
    assert W.sample(x[:0], u[:0]).shape == (0,)
    for call in [
        lambda: W.sample(x.cpu(), u.cpu()),
        lambda: W.sample(x.double(), u),
        lambda: W.sample(x.t(), u),
        lambda: W.sample(x[0], u),
        lambda: W.sample(x, u.double()),
        lambda: W.sample(x, u[:1]),
        lambda: W.sample(x, None),
        lambda: W.sample(x, u, top_k=torch.zeros(2, device="cuda")),
        lambda: W.sample(x, u, top_p=torch.zeros(4, device="cuda")[::2]),
        lambda: W.sample(torch.zeros(1, 262145, device="cuda"), u[:1]),
        lambda: W.sample(torch.zeros(1, 0, device="cuda"), u[:1]),
        lambda: W.sample(x[:1].expand(2, 100), u),
        lambda: W.sample(x, u, out_tok=torch.zeros(2, device="cuda")),
    ]:
        with pytest.raises(W.WpkError):
            call()

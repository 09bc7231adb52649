"""What the operators outside the step program refuse, through the C ABI (no GPU needed: every call
here is refused before anything is launched; the addresses are never used)."""
import ctypes as C
import os

import pytest

from streaming_persistent_sm_b200 import wpk as W

P = 1 << 20  # an aligned address


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not os.path.exists(W.LIB_PATH):
        from streaming_persistent_sm_b200 import build

        build.build()
    return W.load_library()


def _cache(**kw):
    a = dict(pages_dev=P, block_table_dev=P, n_blocks=8, batch=2, max_blocks=4, n_kv_heads=2, head_dim=64,
             page_tokens=64)
    a.update(kw)
    return W.wpk_kv4_cache(*[a[n] for n, _ in W.wpk_kv4_cache._fields_])


def _refused(code, call, *words):
    with pytest.raises(W.WpkError) as e:
        call()
    assert e.value.code == code
    for w in words:
        assert w in str(e.value)


ARGS, SHAPE, UNSUPPORTED = W.WPK_ERR_INVALID_ARG, W.WPK_ERR_SHAPE, W.WPK_ERR_UNSUPPORTED


def test_page_bytes():
    assert W.wpk_kv4_page_bytes(64, 64) == 64 * 2 * 36
    assert W.wpk_kv4_page_bytes(128, 16) == 16 * 2 * 68
    for hd in (0, 32, 65, 96, 256):
        _refused(UNSUPPORTED, lambda: W.wpk_kv4_page_bytes(hd, 64), "head_dim")
    for page in (-16, 0, 8, 24, 272):
        _refused(ARGS, lambda: W.wpk_kv4_page_bytes(64, page), "page_tokens")
    assert W.load_library().wpk_kv4_page_bytes(64, 64, None) == ARGS


CALLS = {
    "append": lambda c, total=2, pos=P, dt=1, x=P, st=(128, 64), ip=0: W.wpk_kv4_append(
        c, pos, ip, total, x, st, x, st, dt, 0, 0, 0),
    "read": lambda c, total=2, pos=P, dt=1, x=P, st=(128, 64), ip=0: W.wpk_kv4_read(
        c, pos, ip, total, x, st, x, st, dt, 0),
    "attention": lambda c, total=2, pos=P, dt=1, x=P, st=(128, 64), ip=0: W.wpk_kv4_attention(
        c, pos, ip, total, 1, x, st, 2, dt, x, st),
}


@pytest.mark.parametrize("name", sorted(CALLS))
def test_cache_calls(name):
    call = CALLS[name]
    for field in ("pages_dev", "block_table_dev"):
        _refused(ARGS, lambda: call(_cache(**{field: None})), "null")
    for field in ("n_blocks", "batch", "max_blocks", "n_kv_heads"):
        for bad in (0, -1):
            _refused(ARGS, lambda: call(_cache(**{field: bad})), "positive")
    _refused(ARGS, lambda: call(_cache(pages_dev=P + 8)), "16-byte")
    _refused(UNSUPPORTED, lambda: call(_cache(head_dim=96)), "head_dim")
    _refused(ARGS, lambda: call(_cache(page_tokens=20)), "page_tokens")
    _refused(SHAPE, lambda: call(_cache(n_blocks=1 << 31)), "pages")
    _refused(SHAPE, lambda: call(_cache(max_blocks=1 << 25)), "positions")
    _refused(ARGS, lambda: call(_cache(), pos=None), "null")
    _refused(ARGS, lambda: call(_cache(), x=None), "null")
    _refused(ARGS, lambda: call(_cache(), x=P + 4), "aligned")
    _refused(ARGS, lambda: call(_cache(), dt=0, x=P + 8), "aligned")
    _refused(ARGS, lambda: call(_cache(), dt=3), "dtype")
    _refused(ARGS, lambda: call(_cache(), total=-2), "total")
    _refused(SHAPE, lambda: call(_cache(), total=3), "multiple")
    _refused(SHAPE, lambda: call(_cache(n_kv_heads=1 << 15), total=1 << 17), "rows")
    _refused(SHAPE, lambda: call(_cache(n_kv_heads=1 << 16)), "kv heads")
    for st in ((130, 64), (128, 66), (-128, 64), (128, -64)):
        _refused(ARGS, lambda: call(_cache(), st=st), "strides")


def test_append_and_attention_arguments():
    c = _cache()
    _refused(ARGS, lambda: W.wpk_kv4_append(c, P, 0, 2, P, (128, 64), P, (128, 64), 1, P, 0), "rope_positions")
    _refused(ARGS, lambda: W.wpk_kv4_append(c, P, 0, 2, P, (128, 64), P, (128, 64), 1, P + 8, 10), "rope")
    _refused(ARGS, lambda: W.wpk_kv4_append(c, P, 0, 2, P, (128, 64), P + 2, (128, 64), 1), "aligned")
    att = lambda **kw: W.wpk_kv4_attention(  # noqa: E731
        c, P, 0, 2, kw.get("max_new", 1), P, (128, 64), kw.get("heads", 4), 1, kw.get("out", P), (128, 64),
        scale=kw.get("scale", 0.0))
    for heads in (0, -2, 3):
        _refused(ARGS, lambda: att(heads=heads), "n_heads")
    _refused(ARGS, lambda: att(max_new=-1), "max_new")
    _refused(ARGS, lambda: att(out=None), "null")
    for scale in (-1.0, float("nan"), float("inf")):
        _refused(ARGS, lambda: att(scale=scale), "scale")


def test_sample_arguments():
    s = lambda **kw: W.wpk_sample(  # noqa: E731
        kw.get("x", P), kw.get("dt", 0), kw.get("batch", 2), kw.get("vocab", 100), kw.get("stride", 100),
        kw.get("u", P), kw.get("out", P))
    for name in ("x", "u", "out"):
        _refused(ARGS, lambda: s(**{name: None}), "null")
    _refused(ARGS, lambda: s(dt=7), "dtype")
    _refused(ARGS, lambda: s(batch=-1), "batch")
    _refused(ARGS, lambda: s(vocab=0), "vocab")
    _refused(UNSUPPORTED, lambda: s(vocab=262145, stride=262145), "vocab")
    _refused(ARGS, lambda: s(stride=99), "row_stride")
    _refused(ARGS, lambda: s(x=P + 2), "aligned")
    _refused(SHAPE, lambda: s(batch=1 << 29), "rows")


def test_messages_belong_to_the_thread():
    import threading

    _refused(UNSUPPORTED, lambda: W.wpk_kv4_page_bytes(96, 64))
    seen = []
    t = threading.Thread(target=lambda: seen.append(W.load_library().wpk_last_error(None)))
    t.start()
    t.join()
    assert seen == [b""] and b"head_dim" in W.load_library().wpk_last_error(None)
    assert C.sizeof(W.wpk_kv4_cache) == 48


def test_plans_over_4_bit_pages():
    import synth

    shape = synth.TINY
    build = lambda **kw: W.wpk_build_graph(W.model_cfg(shape), W.plan_cfg(3, 100, n_workers=16, **kw))  # noqa: E731
    for kw in (dict(), dict(mode=W.WPK_PER_OP_GRAPH, decode=W.WPK_DECODE_MMA),
               dict(mode=W.WPK_PER_OP_GRAPH, prefill=W.WPK_PREFILL_MMA)):
        _refused(UNSUPPORTED, lambda: build(kv_bits=4, **kw), "4-bit")
    for kw in (dict(kv_bits=8), dict(kv_bits=-4), dict(kv_bits=4, page_tokens=8), dict(kv_bits=4, page_tokens=24)):
        _refused(ARGS, lambda: build(mode=W.WPK_PER_OP_GRAPH, **kw))
    two = synth.TINY_TWO_STAGE
    _refused(UNSUPPORTED, lambda: W.wpk_build_graph(W.model_cfg(two), W.plan_cfg(
        2, 16, n_workers=16, mode=W.WPK_PER_OP_GRAPH, kv_bits=4)), "4-bit")
    h = build(mode=W.WPK_PER_OP_GRAPH, kv_bits=4, page_tokens=32)
    assert W.wpk_workspace_size(h)[1] == shape.n_layers * 3 * 4 * shape.n_kv_heads * 32 * 72
    W.wpk_destroy(h)
    h = build(mode=W.WPK_PER_OP_GRAPH, kv_bits=16, page_tokens=32)
    assert W.wpk_workspace_size(h)[1] == shape.n_layers * 3 * 4 * shape.n_kv_heads * 32 * 256
    W.wpk_destroy(h)


@pytest.mark.parametrize("device", ["cpu", "cpu:0", "meta"])
def test_a_cache_is_on_a_cuda_device(device):
    _refused(ARGS, lambda: W.KV4Cache(1, 1, 64, 16, device=device), "CUDA device", device)


@pytest.mark.parametrize("st", [(0, 64), (128, 0), (60, 64), (128, 32)])
def test_rows_that_are_written_do_not_overlap(st):
    c = _cache()
    _refused(ARGS, lambda: W.wpk_kv4_read(c, P, 0, 2, P, st, P, (128, 64), 1), "overlap")
    _refused(ARGS, lambda: W.wpk_kv4_read(c, P, 0, 2, P, (128, 64), P, st, 1), "overlap")
    _refused(ARGS, lambda: W.wpk_kv4_attention(c, P, 0, 2, 1, P, (128, 64), 2, 1, P, st), "overlap")

"""The 4-bit cache and sampling inside the framework's own steps: the engine against the oracle."""
import numpy as np
import pytest

import oracle
import synth
from streaming_persistent_sm_b200 import wpk as W
from tests import operators_ref as R
from tests.parity import MAX_ABS, REL_L2, run_teacher_forced

pytestmark = pytest.mark.gpu

S = synth.TINY
CTX = 96
KV4 = dict(mode=W.WPK_PER_OP_GRAPH, kv_bits=4)


class _Held4(oracle.llama.KVCache):
    """The oracle's cache, its rows as 4 bits hold them."""

    def write(self, layer, b, positions, k, v):
        super().write(layer, b, positions, R.held(k), R.held(v))


class _Decoder4(oracle.Decoder):
    def new_cache(self, batch, max_context, page_tokens=64, block_table=None):
        s = self.s
        return _Held4(s.n_layers, batch, max_context, s.n_kv_heads, s.head_dim, page_tokens, block_table)


@pytest.fixture(scope="module")
def weights():
    return synth.make_weights(S, seed=0)


@pytest.mark.parametrize("B,plan", [(1, {}), (3, dict(page_tokens=16)), (6, dict(page_tokens=32))])
def test_steps_over_4_bit_pages_match_the_oracle(weights, B, plan):
    eng = W.Engine(S, weights, B + 1, CTX, **KV4, **plan)  # a slot of the plan stays idle
    try:
        blocks = -(-CTX // (plan.get("page_tokens") or 64))
        table = np.random.default_rng(B).permutation((B + 1) * blocks).reshape(B + 1, blocks)
        W.wpk_set_block_table(eng.h, table)
        prompts = synth.make_prompts(S.vocab, B, 40, 7)
        for _ in range(2):  # a second batch of sequences over the same pages
            run_teacher_forced(eng, _Decoder4(S, weights), prompts, steps=24, max_context=CTX, check_every=6)
    finally:
        eng.close()


@pytest.mark.parametrize("plan", [dict(), KV4], ids=["megakernel", "kv4"])
def test_sampled_decoding(weights, plan):
    """Prompt, then steps whose tokens are drawn from their logits: the logits agree with the oracle fed the
    same tokens, and each token is the one that the definition draws from these logits."""
    import torch

    B, steps = 3, 12
    dec = (_Decoder4 if plan else oracle.Decoder)(S, weights)
    eng = W.Engine(S, weights, B, CTX, **plan)
    try:
        rng = np.random.default_rng(3)
        prompts = synth.make_prompts(S.vocab, B, 20, 9)
        kw = dict(temperature=[0.7, 1.0, 0.0], top_k=[50, 0, 0], top_p=[0.9, 0.95, 1.0], min_p=[0.0, 0.01, 0.0])
        dev = {n: torch.tensor(x, dtype=torch.int32 if n == "top_k" else torch.float32, device="cuda")
               for n, x in kw.items()}
        _, logits = eng.prefill(prompts, want_logits=True)
        cache = dec.new_cache(B, CTX)
        ref = dec.prefill(cache, prompts)
        u = rng.random((steps + 1, B), dtype=np.float32)
        tok = eng.sample(logits, torch.from_numpy(u[0]).cuda(), **dev)
        for s in range(steps + 1):
            z = logits.double().cpu().numpy()
            d = z - ref
            assert np.abs(d).max() <= MAX_ABS and (np.linalg.norm(d, axis=1) <= REL_L2 * np.linalg.norm(ref, axis=1)).all()
            f = lambda n, b: float(np.float32(kw[n][b]))  # noqa: E731
            want = [R.sample_row(z[b], float(u[s, b]), f("temperature", b), int(kw["top_k"][b]), f("top_p", b),
                                 f("min_p", b))[0] for b in range(B)]
            assert tok.cpu().tolist() == want, s
            if s == steps:
                break
            ref = dec.step(cache, tok.cpu().numpy())
            tok, logits = eng.step_sampled(torch.from_numpy(u[s + 1]).cuda(), in_tok=tok, **dev)
    finally:
        eng.close()


def test_codes_of_a_two_stage_frame_are_drawn_from_its_logits():
    import torch

    s = synth.TINY_TWO_STAGE
    eng = W.Engine(s, synth.make_weights(s, seed=0), 2, 16)
    try:
        _, logits = eng.prefill(synth.make_prompts(s.backbone.vocab, 2, 4, 1), want_logits=True)
        u = np.random.default_rng(4).random(logits.shape[:2], dtype=np.float32)
        k = torch.full(logits.shape[:2], 20, dtype=torch.int32, device="cuda")
        codes, lp = eng.sample(logits, torch.from_numpy(u).cuda(), top_k=k, want_logprob=True)
        assert codes.shape == lp.shape == logits.shape[:2]
        z = logits.double().cpu().numpy()
        for b in range(2):
            for c in range(s.n_codebooks):
                assert int(codes[b, c]) == R.sample_row(z[b, c], float(u[b, c]), top_k=20)[0]
        with pytest.raises(W.WpkError) as e:
            eng.step_sampled(torch.from_numpy(u).cuda())
        assert e.value.code == W.WPK_ERR_UNSUPPORTED
    finally:
        eng.close()


def test_codes_go_into_the_tensor_given():
    import torch

    s = synth.TINY_TWO_STAGE
    eng = W.Engine(s, synth.make_weights(s, seed=0), 2, 16)
    try:
        _, logits = eng.prefill(synth.make_prompts(s.backbone.vocab, 2, 4, 1), want_logits=True)
        u = torch.rand(logits.shape[:2], device="cuda")
        want = eng.sample(logits, u)
        into = torch.zeros(logits.shape[:2], dtype=torch.int32, device="cuda")
        got = eng.sample(logits, u, out_tok=into)
        assert torch.equal(into, want) and got.data_ptr() == into.data_ptr() and got.shape == want.shape
        with pytest.raises(W.WpkError):
            eng.sample(logits, u, out_tok=torch.zeros(into.t().shape, dtype=torch.int32, device="cuda").t())
    finally:
        eng.close()

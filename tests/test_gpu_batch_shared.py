"""Batched decode whose samples keep their common prefix once
(lf_batch_begin_shared) and the filtered generation
(lf_batch_generate_filtered): the paged append, the shared-prefix attention and
the filtered draw run together, step after step, as the engine uses them."""
import numpy as np
import pytest

import oracle
import paged_reference as ref
import synth
from gpu_helpers import REL_L2, assert_gates, note, rel_l2

pytestmark = pytest.mark.gpu


def run_shared(shape, seed, n_prompt, n_steps, B, gain_std=0.1, kv_fill=0):
    """As the batch tests: every sample teacher-forced on its own tokens
    against an oracle that ran the same prompt and those tokens."""
    from decode_persistent_sm_gb300 import Engine
    blob = synth.make_weights(shape, seed, gain_std=gain_std)
    prompt = synth.make_tokens(seed, n_prompt, shape.vocab)
    steps = [synth.make_tokens(seed * 100 + b, n_steps, shape.vocab) for b in range(B)]
    kv = synth.make_kv(shape, seed, kv_fill) if kv_fill else None
    orcs = []
    for _ in range(B):
        o = oracle.Oracle(shape, blob)
        if kv_fill:
            o.load_kv(kv, kv_fill)
        for t in prompt:
            o.step(int(t))
        orcs.append(o)
    rels, agree = [], []
    with Engine.from_shape(shape) as eng:
        eng.load_weights(blob)
        if kv_fill:
            eng.load_kv(kv, kv_fill)
        for t in prompt:
            eng.decode_step(int(t))
        eng.batch_begin_shared(B)
        assert eng.batch_info() == (B, kv_fill + n_prompt)
        for i in range(n_steps):
            toks = [int(steps[b][i]) for b in range(B)]
            got, am = eng.batch_step(toks)
            for b in range(B):
                want = orcs[b].step(toks[b])
                rels.append(note(got[b], want, am[b]))
                agree.append(am[b] == oracle.argmax(want))
        assert eng.batch_info() == (B, kv_fill + n_prompt + n_steps)
    return np.array(rels), np.array(agree)


@pytest.mark.parametrize("B,n_prompt", [(1, 12), (5, 20), (16, 64), (3, 65), (2, 0), (4, 120)])
def test_tiny(B, n_prompt):
    # the branch at the start, inside a page, on its border, and near the end of the context
    rels, agree = run_shared(synth.TINY, 3, n_prompt, 8, B)
    assert_gates(rels, agree, f"shared batch of {B} after {n_prompt}")


@pytest.mark.parametrize("lanes,delay", [(8, 0), (1, 2), (4, 3)])
def test_lanes_and_delays(lanes, delay):
    rels, agree = run_shared(synth.TINY.replace(n_lanes=lanes, dtp_delay=delay), 4, 9, 5, 3)
    assert_gates(rels, agree, f"shared batch, lanes={lanes} delay={delay}")


def test_six_layers_windows_crossed():
    # the windows of 16 and 8 keys slide out of the prefix while the samples run
    shape = synth.TINY.replace(n_layers=6, swa_window=(64, 0, 16, 0, 8, 0))
    rels, agree = run_shared(shape, 5, 70, 20, 4)
    assert_gates(rels, agree, "shared batch, 6 layers")


def test_same_function_as_the_separate_caches_and_the_engine_untouched():
    from decode_persistent_sm_gb300 import Engine
    shape = synth.TINY
    toks = synth.make_tokens(8, 40, shape.vocab)
    with Engine.from_shape(shape) as eng:
        eng.load_weights(synth.make_weights(shape, 8, gain_std=0.1))
        eng.prefill(toks[:30], logits=False)
        runs = []
        for begin in (eng.batch_begin, eng.batch_begin_shared, eng.batch_begin_shared):
            begin(3)
            runs.append([eng.batch_step([int(toks[30 + i]), int(toks[i]), 5 + i])[0] for i in range(8)])
        for sep, one, two in zip(*runs):
            assert np.array_equal(one, two)  # repeatable bit for bit
            for b in range(3):
                assert rel_l2(one[b], sep[b]) <= REL_L2
        eng.batch_end()
        after, _ = eng.decode_step(int(toks[30]))
        eng.set_position(30)
        again, _ = eng.decode_step(int(toks[30]))
        assert np.array_equal(after, again) and eng.position == 31


@pytest.mark.parametrize("begin", ["batch_begin", "batch_begin_shared"])
def test_filtered_generation_draws_what_its_logits_say(begin):
    # the tokens and log shares of a generation, against the plain draw on the
    # logits of the same steps run one by one (the same bits both times)
    from decode_persistent_sm_gb300 import Engine
    shape = synth.TINY
    g = np.random.default_rng(9)
    B, n = 6, 25
    u = g.random((B, n), dtype=np.float32)
    par = dict(temperature=[0.7, 1.0, 0.0, 1.3, 0.9, 2.0], top_k=[0, 20, 5, 0, 1, 300], top_p=[0.9, 1.0, 0.5, 0.97, 1.0, 0.8],
               min_p=[0.0, 0.02, 0.0, 0.001, 0.0, 0.1])
    first = [3, 900, 17, 4, 4, 0]
    with Engine.from_shape(shape) as eng:
        eng.load_weights(synth.make_weights(shape, 21, gain_std=0.1))
        eng.prefill(synth.make_tokens(21, 50, shape.vocab), logits=False)
        getattr(eng, begin)(B)
        toks, lps = eng.batch_generate_filtered(first, u, **par)
        assert eng.batch_info() == (B, 50 + n)
        getattr(eng, begin)(B)
        feed = list(first)
        for i in range(n):
            z, _ = eng.batch_step(feed)
            for b in range(B):
                want, share = ref.draw(z[b], np.float32(par["temperature"][b]).item(), par["top_k"][b],
                                       np.float32(par["top_p"][b]).item(), np.float32(par["min_p"][b]).item(), float(u[b, i]))
                assert toks[b, i] == want, (b, i)
                assert abs(lps[b, i] - share) <= 2.0 ** -21 * abs(share) + 2.0 ** -40
            feed = [int(t) for t in toks[:, i]]


def test_filtered_generation_defaults_and_greedy():
    from decode_persistent_sm_gb300 import Engine
    shape = synth.TINY
    with Engine.from_shape(shape) as eng:
        eng.load_weights(synth.make_weights(shape, 22, gain_std=0.1))
        eng.prefill(synth.make_tokens(22, 10, shape.vocab), logits=False)
        eng.batch_begin_shared(2)
        greedy, lp = eng.batch_generate_filtered([3, 9], np.zeros((2, 12)), temperature=0.0)
        assert (lp == 0).all()
        eng.batch_begin_shared(2)
        assert np.array_equal(greedy, eng.batch_generate([3, 9], 12, 0.0, 1.0, 0))
        eng.batch_begin_shared(2)
        a, _ = eng.batch_generate_filtered([3, 9], np.full((2, 6), 0.4))
        eng.batch_begin_shared(2)
        b, _ = eng.batch_generate_filtered([3, 9], np.full((2, 6), 0.4), temperature=1.0, top_k=0, top_p=1.0, min_p=0.0)
        assert np.array_equal(a, b)
        eng.batch_begin_shared(2)
        c = [eng.batch_generate_filtered([3, 9] if i == 0 else c0[:, -1], np.full((2, 3), 0.4)) for i, c0 in ((0, None), (1, a[:, :3]))]
        assert np.array_equal(np.concatenate([c[0][0], c[1][0]], 1), a)  # two halves are the whole


def test_rejections():
    from decode_persistent_sm_gb300 import Engine, LaneformerError
    shape = synth.TINY
    u = np.full((2, 2), 0.5)
    with Engine.from_shape(shape) as eng:
        with pytest.raises(LaneformerError, match="NOT_LOADED"):
            eng.batch_begin_shared(2)
        eng.load_weights(synth.make_weights(shape, 1))
        with pytest.raises(LaneformerError, match="NOT_LOADED"):
            eng.batch_generate_filtered([1, 2], u)
        for bad in (0, 17):
            with pytest.raises(LaneformerError, match="INVALID_ARG"):
                eng.batch_begin_shared(bad)
        eng.prefill(synth.make_tokens(1, shape.ctx_cap - 2, shape.vocab), logits=False)
        eng.batch_begin_shared(2)
        for bad in (dict(temperature=-1.0), dict(temperature=1e-31), dict(temperature=np.nan), dict(top_p=0.0), dict(top_p=1.1),
                    dict(min_p=-0.1), dict(min_p=1.5)):
            with pytest.raises(LaneformerError, match="INVALID_ARG"):
                eng.batch_generate_filtered([1, 2], u, **bad)
        for bad_u in (np.full((2, 2), 1.0), np.full((2, 2), -0.1), np.full((2, 2), np.nan)):
            with pytest.raises(LaneformerError, match="INVALID_ARG"):
                eng.batch_generate_filtered([1, 2], bad_u)
        with pytest.raises(LaneformerError, match="INVALID_ARG"):
            eng.batch_generate_filtered([1, shape.vocab], u)
        with pytest.raises(ValueError, match="u must be"):
            eng.batch_generate_filtered([1, 2], np.full((3, 2), 0.5))
        with pytest.raises(LaneformerError, match="CTX_OVERFLOW"):
            eng.batch_generate_filtered([1, 2], np.full((2, 3), 0.5))
        eng.batch_generate_filtered([1, 2], u)  # nothing above ended the batch
        with pytest.raises(LaneformerError, match="CTX_OVERFLOW"):
            eng.batch_step([5, 6])
    with Engine.from_shape(shape.replace(own_lane_immediate=1)) as eng:
        eng.load_weights(synth.make_weights(shape, 1))
        with pytest.raises(LaneformerError, match="UNSUPPORTED"):
            eng.batch_begin_shared(2)


@pytest.mark.slow
def test_full_shape_against_the_oracle():
    rels, agree = run_shared(synth.FULL, 1, 0, 2, 3, gain_std=0.0, kv_fill=300)
    assert_gates(rels, agree, "full shape, shared batch of 3")


@pytest.mark.slow
def test_full_shape_long_prefix_matches_the_separate_caches():
    # beyond the 1024-key windows, 16 samples
    from decode_persistent_sm_gb300 import Engine
    shape = synth.FULL
    with Engine.from_shape(shape) as eng:
        eng.load_weights(synth.make_weights(shape, 2))
        eng.load_kv(synth.make_kv(shape, 2, 2100), 2100)
        toks = np.asarray(synth.make_tokens(2, 16 * 4, shape.vocab)).reshape(4, 16)
        runs = []
        for begin in (eng.batch_begin, eng.batch_begin_shared):
            begin(16)
            runs.append([eng.batch_step([int(t) for t in row])[0] for row in toks])
        for sep, one in zip(*runs):
            for b in range(16):
                assert rel_l2(one[b], sep[b]) <= 5e-3

"""What the batch calls make of the error word that their kernels leave (debug
library: the word is written from the host)."""
import ctypes

import numpy as np
import pytest

import synth

pytestmark = pytest.mark.gpu

# a page, length or position outside the paged cache; a wait of the attention or of the draw, a bad token, a wait of a GEMV
WORDS = [(1, "BOUNDS", True), (2, "TIMEOUT", True), (6, "INVALID_ARG", False), (7, "TIMEOUT", True)]


@pytest.mark.parametrize("word,status,poisons", WORDS)
@pytest.mark.parametrize("call", ["step", "generate", "filtered"])
def test_error_word(call, word, status, poisons):
    from decode_persistent_sm_gb300 import Engine, LaneformerError
    shape = synth.TINY
    with Engine.from_shape(shape, debug=True) as eng:
        eng.load_weights(synth.make_weights(shape, 5))
        prompt = synth.make_tokens(5, 20, shape.vocab)
        eng.prefill(prompt, logits=False)
        eng.batch_begin_shared(2)
        eng.batch_step([1, 2])
        assert eng.raw_call("lf_debug_batch_error", ctypes.c_uint32(word)) == 0
        run = {"step": lambda: eng.batch_step([3, 4]), "generate": lambda: eng.batch_generate([3, 4], 2, 0.0, 1.0, 0),
               "filtered": lambda: eng.batch_generate_filtered([3, 4], np.full((2, 2), 0.5))}[call]
        with pytest.raises(LaneformerError, match=status):
            run()
        assert eng.batch_info() == (0, 0)
        if poisons:
            with pytest.raises(LaneformerError, match=status):
                eng.decode_step(1)
            eng.reset()
            eng.prefill(prompt, logits=False)
        eng.batch_begin_shared(2)
        run()

"""lf_batch_begin and lf_batch_begin_shared without host memory at each of the places
where they allocate some (debug library): LF_ERR_OOM, no batch, no device memory
kept, no capture left open, and the next call as if nothing had happened."""
import numpy as np
import pytest

import synth

pytestmark = pytest.mark.gpu


@pytest.fixture
def lib():
    import decode_persistent_sm_gb300 as lf
    d = lf.load_library(debug=True)
    yield d
    assert d.lf_debug_fail_alloc(0) == 0


@pytest.mark.parametrize("begin", ["batch_begin", "batch_begin_shared"])
def test_no_host_memory_anywhere(lib, begin):
    import torch
    from decode_persistent_sm_gb300 import Engine, LaneformerError
    shape = synth.TINY
    with Engine.from_shape(shape, debug=True) as eng:
        eng.load_weights(synth.make_weights(shape, 31))
        eng.prefill(synth.make_tokens(31, 70, shape.vocab), logits=False)
        getattr(eng, begin)(3)
        want = [eng.batch_step([1, 2, 3])[0], eng.batch_step([4, 5, 6])[0]]
        eng.batch_end()
        torch.cuda.synchronize()
        free, _ = torch.cuda.mem_get_info()
        failed = 0
        for nth in range(1, 200):
            assert lib.lf_debug_fail_alloc(nth) == 0
            try:
                getattr(eng, begin)(3)
                break
            except LaneformerError as e:
                assert "OOM" in str(e)
                failed += 1
            assert eng.batch_info() == (0, 0)
            with pytest.raises(LaneformerError, match="NOT_LOADED"):
                eng.batch_step([1, 2, 3])
        assert failed >= 4 + 2 * shape.n_layers  # before and during the capture, once a sub-block
        assert lib.lf_debug_fail_alloc(0) == 0
        assert np.array_equal(eng.batch_step([1, 2, 3])[0], want[0])
        assert np.array_equal(eng.batch_step([4, 5, 6])[0], want[1])
        eng.batch_end()
        torch.cuda.synchronize()
        assert torch.cuda.mem_get_info()[0] >= free - (4 << 20)
        assert eng.position == 70

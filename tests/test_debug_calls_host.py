"""The debug calls of the batch (no GPU needed): refused by the release library, their
arguments checked, set and put back by the debug library."""
import pytest


@pytest.fixture(scope="module")
def libs():
    from decode_persistent_sm_gb300 import binding, build
    build.build()
    build.build(debug=True)
    return binding.load_library(), binding.load_library(debug=True)


def test_allocation_failure(libs):
    rel, dbg = libs
    assert rel.lf_debug_fail_alloc(1) == 7  # LF_ERR_UNSUPPORTED
    assert rel.lf_debug_fail_alloc(-1) == dbg.lf_debug_fail_alloc(-1) == 1
    assert dbg.lf_debug_fail_alloc(3) == dbg.lf_debug_fail_alloc(0) == 0


def test_batch_error_word(libs):
    # (no engine needed: a null engine is refused first)
    for lib in libs:
        assert lib.lf_debug_batch_error(None, 1) == 1

"""The draw's debug call (no GPU needed): refused by the release library, its
arguments checked, set and put back by the debug library."""


def test_debug_wait_of_the_draw():
    from decode_persistent_sm_gb300 import binding, build
    build.build()
    build.build(debug=True)
    rel, dbg = binding.load_library(), binding.load_library(debug=True)
    assert rel.lf_debug_sample_wait(1000, -1, 1) == 7  # LF_ERR_UNSUPPORTED
    for lib in (rel, dbg):
        assert lib.lf_debug_sample_wait(1000, -2, 1) == 1
        assert lib.lf_debug_sample_wait(1000, 0, -1) == 1
        assert lib.lf_debug_sample_wait(2_000_000_001, 0, 1) == 1
    assert dbg.lf_debug_sample_wait(1000, 3, 2) == 0
    assert dbg.lf_debug_sample_wait(2_000_000_000, -1, 0) == 0

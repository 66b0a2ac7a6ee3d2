"""The chunk attention's debug call (no GPU needed): refused by the release library,
its arguments checked, set and put back by the debug library."""


def test_debug_wait_of_the_chunk_attention():
    from decode_persistent_sm_gb300 import binding, build
    build.build()
    build.build(debug=True)
    rel, dbg = binding.load_library(), binding.load_library(debug=True)
    assert rel.lf_debug_chunk_wait(-1, 0, 1) == 7  # LF_ERR_UNSUPPORTED
    for lib in (rel, dbg):
        for bad in ((-2, 0, 1), (0, -1, 1), (0, 10, 1), (0, 0, -1)):
            assert lib.lf_debug_chunk_wait(*bad) == 1
    assert dbg.lf_debug_chunk_wait(3, 9, 2) == 0
    assert dbg.lf_debug_chunk_wait(-1, 0, 0) == 0

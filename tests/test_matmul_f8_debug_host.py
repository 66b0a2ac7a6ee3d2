"""The 8-bit product's debug call (no GPU needed): refused by the release library,
its argument checked, set and put back by the debug library."""


def test_debug_wait_of_the_8_bit_product():
    from decode_persistent_sm_gb300 import binding, build
    build.build()
    build.build(debug=True)
    rel, dbg = binding.load_library(), binding.load_library(debug=True)
    assert rel.lf_debug_matmul_f8_wait(1000) == 7  # LF_ERR_UNSUPPORTED
    for lib in (rel, dbg):
        assert lib.lf_debug_matmul_f8_wait(2_000_000_001) == 1
    assert dbg.lf_debug_matmul_f8_wait(0) == 0
    assert dbg.lf_debug_matmul_f8_wait(2_000_000_000) == 0

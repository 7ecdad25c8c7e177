"""Child process of test_debug_operators_gpu.py: small cases of the operators around the
attention through the debug library (RA_LIBRARY_VARIANT=debug, every kernel's bounds
checks compiled in), each held to its own test and the error word read behind it.  Exits
non-zero, with the reason on stderr, if a check fires or a result is off; prints "debug
operators ok" otherwise."""
import os
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, ROOT)

import static_sparse_attention_b200 as ra  # noqa: E402
from tests import test_cache8_gpu, test_cache8_kernels_gpu, test_qk_norm_rope_gpu, test_swc_cache8_gpu  # noqa: E402


def run(what, test, *args):
    test(*args)
    st = ra.device_status()
    if st != ra.RA_OK:
        site, block = ra.ctypes.c_int(), ra.ctypes.c_int()
        ra.ra_get_device_error_site(ra.ctypes.byref(site), ra.ctypes.byref(block))
        raise SystemExit(f"{what}: device status {st} (site {site.value}, block {block.value})")


def main():
    assert ra.VARIANT == "debug" and ra.LIB_PATH.endswith("libradattn_debug.so"), ra.LIB_PATH
    for shape in test_qk_norm_rope_gpu.SHAPES:
        for packed, norm, rotated in ((True, True, True), (False, True, False), (False, False, True)):
            run(shape, test_qk_norm_rope_gpu.test_forward_and_backward, shape, packed, not packed, norm, rotated)
    run("packed gradients", test_qk_norm_rope_gpu.test_broadcast_input_and_packed_gradient)
    for case in test_cache8_gpu.APPENDS:
        for norm, rotated, packed in ((True, True, True), (False, False, False)):
            run(case, test_cache8_gpu.test_append, case, norm, rotated, packed)
    for case in test_cache8_gpu.ATTENDS:
        run(case, test_cache8_gpu.test_attention, case)
    for size in test_cache8_kernels_gpu.SIZES:
        for d in (64, 128):
            run(size, test_cache8_kernels_gpu.test_counts, size, d)
            run(size, test_cache8_kernels_gpu.test_large_scales, size, d)
    run("stream", test_swc_cache8_gpu.test_a_refused_step_leaves_the_ring_as_it_was)
    print("debug operators ok")


if __name__ == "__main__":
    main()

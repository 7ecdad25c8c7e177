"""What can be held about the 8-bit ring and the operators beside it without a GPU."""
import ctypes
import os
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "static_sparse_attention_b200", "csrc")


@pytest.fixture(scope="module")
def ra():
    import __graft_entry__
    __graft_entry__.build()
    import static_sparse_attention_b200 as ra
    return ra


def test_the_warp_is_whole_before_the_epilogue_loads_tensor_memory():
    """tcgen05.ld is warp-collective, and a tile's last warp parts where it stores only
    the rows that exist: the loop that does both joins the lanes before each load, and
    the branch around it is taken by a whole warp or not at all."""
    src = open(os.path.join(CSRC, "ra_cache8_tiles.cu")).read()
    epilogue = src[src.index("// ------------------------------------------------------------ epilogue"):]
    entry = epilogue.index("*abort_flag")
    assert re.search(r"__all_sync\(0xFFFFFFFFu, ok && !$", epilogue[:entry])
    parts = epilogue.index("if (!row_valid)")
    body = epilogue[epilogue.rindex("for (int k = 0; k < D / 32; ++k) {", 0, parts):parts]
    assert body.index("__syncwarp();") < body.index("tmem_ld32(")


def test_the_plan_names_a_kernel_and_its_ranges(ra):
    kernel, ranges = ctypes.c_int(-1), ctypes.c_int(-1)

    def plan(B, H, d, nq, s, W, held, kernel=ctypes.byref(kernel), ranges=ctypes.byref(ranges)):
        return ra.ra_cache8_attention_plan(B, H, d, nq, s, W, held, kernel, ranges)

    for args, want in (((1, 12, 64, 1, 37, 8, 7), ra.RA_CACHE8_ROWS_AHEAD), ((30, 40, 64, 1, 64, 8, 8), ra.RA_CACHE8_ROWS),
                       ((1, 40, 128, 100, 1560, 16, 16), ra.RA_CACHE8_ONE_TILE),
                       ((1, 40, 128, 1560, 1560, 16, 16), ra.RA_CACHE8_TWO_TILES)):
        assert plan(*args) == ra.RA_OK and kernel.value == want, args
        need = ctypes.c_size_t()
        assert ra.ra_cache8_attention_workspace_bytes(*args, ctypes.byref(need)) == ra.RA_OK
        assert (need.value > 0) == (ranges.value > 1)
    assert plan(1, 12, 96, 1, 37, 8, 7) == ra.RA_ERR_UNSUPPORTED
    assert plan(1, 12, 64, 1, 37, 8, 9) == ra.RA_ERR_INVALID_ARG
    assert plan(1, 12, 64, 1, 37, 8, 7, kernel=None) == ra.RA_ERR_INVALID_ARG
    assert plan(1, 12, 64, 1, 37, 8, 7, ranges=None) == ra.RA_ERR_INVALID_ARG


def test_the_check_refuses_what_the_attention_refuses(ra):
    MB = 1 << 20
    good = dict(Q=10 * MB, k8=30 * MB, v8=31 * MB, ks=32 * MB, vs=33 * MB, O=40 * MB, B=2, H=1, d=128, nq=3, s=20, W=4,
                held=3, counts=None, scale=0.1, lse=None, ws=50 * MB, ws_bytes=0)
    assert ra.ra_cache8_attention_check(*good.values()) == ra.RA_OK
    for bad in (dict(Q=None), dict(O=None), dict(O=10 * MB), dict(O=30 * MB), dict(lse=40 * MB), dict(held=5),
                dict(scale=0.0), dict(nq=0), dict(counts=60 * MB + 2), dict(d=32), dict(k8=None), dict(vs=33 * MB + 2)):
        args = {**good, **bad}
        st = ra.ra_cache8_attention_check(*args.values())
        assert st != ra.RA_OK and ra.ra_last_error(), bad
        assert ra.ra_cache8_attention(*args.values(), None) == st, bad


@pytest.mark.parametrize("source,checks", [
    ("ra_head_rows.cuh", ["SITE_I_ROPE"]),
    ("ra_qk_norm_rope.cu", ["SITE_I_IN", "SITE_I_OUT", "SITE_I_GRAD_IN", "SITE_I_GRAD_OUT", "SITE_I_PART"]),
    ("ra_cache8.cu", ["SITE_I_IN", "SITE_I_CODE", "SITE_I_SCALE"]),
    ("ra_cache8_attention.cu", ["keys_inside", "scale_inside", "row_inside", "part_inside"]),
    ("ra_cache8_tiles.cu", ["keys_inside", "scale_inside", "row_inside", "part_inside"]),
])
def test_the_debug_build_checks_each_buffer_of_the_operators(source, checks):
    """The debug library's promise, that each global offset is checked before use, for the
    kernels around the attention: their sources hold one for each buffer."""
    src = open(os.path.join(CSRC, source)).read()
    for check in checks:
        assert check in src, check

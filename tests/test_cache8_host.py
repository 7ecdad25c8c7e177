"""What can be held about the 8-bit ring and the operators beside it without a GPU."""
import os
import re

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "static_sparse_attention_b200", "csrc")


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

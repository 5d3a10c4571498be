"""Order of tensor-memory stores and loads in the chunk kernel, by reading its source (no GPU):
a thread's load of columns that it has stored needs the wait for its stores in between."""
import os
import re

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def softmax_loop():
    """The source of a softmax thread's loop over key tiles, without comments."""
    path = os.path.join(ROOT, "quantized_opt_decode_b200", "csrc", "attn_paged_chunk.cu")
    src = re.sub(r"//[^\n]*", "", open(path).read())
    start = src.index("for (int it = 0; it < mine; ++it, lim")
    depth = 0
    for at in range(src.index("{", start), len(src)):
        depth += {"{": 1, "}": -1}.get(src[at], 0)
        if depth == 0:
            return src[start:at]
    raise AssertionError("unbalanced braces")


def test_stored_weights_and_outputs_are_waited_for_before_they_are_read_back():
    """Where the exponent base moves, P of the tile's earlier columns and O are read, scaled and
    stored again; the columns were stored in an earlier turn of the loop over 32-column parts."""
    loop = softmax_loop()
    move = loop[loop.index("top > limit)) {"):]
    first_load = min(move.index("tmem_read_x16(s_col"), move.index("tmem_read_x16(o_col"))
    assert "tmem_st_wait()" in move[:first_load]


def test_masked_scores_and_finished_weights_are_waited_for():
    """Masked scores go back to tensor memory and are read again; P is read by the products."""
    loop = softmax_loop()
    mask = loop[loop.index("tmem_st_x32(s_col"):]
    assert mask.index("tmem_st_wait()") < mask.index("tmem_ld_x32(s_col")
    end = loop[loop.rindex("tmem_st_x16(s_col + 16 * ch"):]
    assert end.index("tmem_st_wait()") < end.index("tc_fence_before()") < end.index("mbar_arrive(&bar.p_full")

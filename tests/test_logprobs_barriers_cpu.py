"""Barriers of csrc/kda_logprobs.cu, by its source: where the lists of candidates overflow, all
threads have read how many pieces there are before one of them starts the count again."""
import os
import re

from linear_attention_serving_gated_gb300 import build


def block_end(text, at):
    """Behind the block whose brace opens first at or after `at`."""
    at = text.index("{", at)
    depth = 0
    for i in range(at, len(text)):
        depth += {"{": 1, "}": -1}.get(text[i], 0)
        if depth == 0:
            return i + 1
    raise AssertionError("no end")


def test_the_count_of_pieces_is_read_before_it_starts_again():
    with open(os.path.join(build.CSRC, "kda_logprobs.cu")) as f:
        text = re.sub(r"//[^\n]*", "", f.read())
    start = text.index("int n = s.piece_count;")
    assert text[:start].rstrip().endswith("__syncthreads();")  # the pieces are all listed
    few = text.index("if (n <= kList)", start)
    many = text.index("if (n > kList)", few)
    again = text.index("s.piece_count = 0", many)
    # with too many pieces nothing of the first branch runs
    path = text[start:few] + text[block_end(text, few):again]
    assert "__syncthreads();" in path, "a late thread may read the new count and take another way through the barriers"
    # with too many candidates its barrier comes behind the read
    assert "__syncthreads();" in text[few:block_end(text, few)]

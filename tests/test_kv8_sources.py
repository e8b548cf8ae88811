"""What cannot be shown on a GPU without risking the race itself, read off the
kernels' sources: memory that a kernel of the same call writes is not read through
the read-only path (__ldg), which supposes that nothing writes it while the reader
runs, and a dependent launch may start before its predecessor has ended."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "sparse_attention_long_tcgen05_b200", "csrc")


@pytest.mark.parametrize("name,written", [
    ("kv8_mqa.cu", ["part.factors", "part.images", "part.ml", "part.o", "part.head_item", "part.tail_item",
                    "part.head_goes_on"]),
    ("kv8_weights.cu", ["factors", "images", "w.w"]),
    ("kv8_evict.cu", ["a.kept", "a.new_lens"])])
def test_results_of_a_kernel_before_are_not_read_as_constants(name, written):
    with open(os.path.join(CSRC, name)) as f:
        text = f.read()
    read_only = re.findall(r"__ldg\(\s*([\w.]+(?:->\w+)*)", text)
    assert not [x for x in read_only if x in written]

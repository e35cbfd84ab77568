"""What the CUDA sources may hold (CPU only)."""
import os
import re

from neighborhood_attention_fwd_gb300 import build as nabuild


def sources():
    for name in sorted(os.listdir(nabuild.CSRC)):
        with open(os.path.join(nabuild.CSRC, name)) as f:
            yield name, f.read()


def test_no_bulk_copy_goes_to_several_blocks():
    """The library also runs as one of several ranks, each on a GPU of its own: its copies into shared memory are each for one
    block.  (The arrival of tcgen05.commit on both barriers of a pair is no copy.)"""
    kind = "multi" + "cast"
    found, copies = [], 0
    for name, text in sources():
        for m in re.finditer(r"cp\.async\.bulk[\w.:]*", text):
            copies += 1
            if kind in m.group():
                found.append((name, text[: m.start()].count("\n") + 1, m.group()))
    assert copies > 5 and not found, found

"""Properties of the 8-bit cache kernels that no run may show failing: what a
bounded wait that gave up leads to, alignment that a toolchain happens to give,
error bounds.  Read from the sources."""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "speculative_decoding_verification_91_b200", "csrc")


def source(name):
    """A kernel file without its comments."""
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


def test_waits_for_an_item_s_slot_are_heeded():
    """A role that writes or reads an item's slot although its wait gave up may tear the item under the
    softmax warps, which then leave their named barriers (those have no time limit) in different numbers."""
    text = source("qattn.cu")
    assert len(re.findall(r"wait\(&it_(full|empty)\[", text)) >= 5
    dropped = re.findall(r"[;{})]\s*wait\(&it_(?:full|empty)\[[^;]*;", text)
    assert not dropped, dropped

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


def test_shared_memory_read_in_16_byte_pieces_is_aligned_to_them():
    """A kernel's dynamic shared memory follows its static one: what is read 16 bytes at a time has to be
    declared so, aligned by hand, or of a 16-byte type."""
    seen = 0
    for name in sorted(os.listdir(CSRC)):
        if not name.endswith(".cu"):
            continue
        text = source(name)
        if not re.search(r"reinterpret_cast<(?:const )?(?:u?int4|float4)\*>", text):
            continue
        for align, kind, var in re.findall(r"extern __shared__\s+(__align__\(\d+\)\s+)?([\w ]+?)\s+(\w+)\[\]", text):
            seen += 1
            by_hand = re.search(r"reinterpret_cast<uintptr_t>\(%s\)\s*\+\s*1023" % var, text)
            only_small = not re.search(r"float4\*>\([^;]*\b%s\b" % var, text) and kind in ("float2", "unsigned long long")
            assert align or by_hand or kind == "uint4" or only_small, (name, var)
    assert seen >= 5


def test_the_error_bound_of_turned_keys_counts_every_rounding():
    """In units of 2^-24 (|x0| + |x1|) magnitude.  Cosine and sine: 1 of the function (one step below 1), half of
    the sum with the angle's tail.  The magnitude: 1/2 step, 1, of its conversion to binary32 (of itself at most
    2^-24), 1 of its product with each.  The entry: 1 of the product that is rounded, 1 of the sum."""
    need = 1.0 + 0.5 + 1.0 + 1.0 + 1.0 + 1.0
    text = source("qcache.cu")
    have = float(re.search(r"kTurnErr = ([\d.]+)f / 16777216\.f;", text).group(1))
    assert have > need
    # the largest entry may be off by twice that bound of itself (its pair's partner is no larger), in steps of
    # binary32 at 1.75 x 2^x: all of those next to the scale's turn are formed again
    steps = 2 * have * 2.0 ** -24 * 1.75 / 2.0 ** -23
    near, least = re.search(r"- 0x600000\) <= (\d+)\)", text), re.search(r"\| 0x600000u\) - (\d+);", text)
    assert steps < int(near.group(1)) and steps < int(least.group(1))

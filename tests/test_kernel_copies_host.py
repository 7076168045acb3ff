"""What asynchronous copies that read nothing are given for an address, from the source (no GPU).

A copy of 16, 8 or 4 bytes asks for an address aligned to as much, also where its source size
is 0.  The rows' numbers lie an odd number of 4-byte words into a layout that is itself aligned
to 4 bytes only, so they can stand in for copies of 4 bytes and no others.
"""
import os
import re

from addmm_implicit_im2col_gb300 import build


def arguments(text, name):
    """The argument lists of all calls of `name`, split at their outer commas."""
    for at in (m.end() for m in re.finditer(re.escape(name) + r"\s*\(", text)):
        depth, parts = 0, [""]
        for ch in text[at:]:
            if ch == "," and depth == 0:
                parts.append("")
                continue
            depth += ch in "([{"
            depth -= ch in ")]}"
            if depth < 0:
                break
            parts[-1] += ch
        yield [p.strip() for p in parts]


def source():
    with open(os.path.join(build.CSRC, "k_adapters.cu")) as f:
        return re.sub(r"//[^\n]*", "", f.read())


def test_stand_ins_of_units_are_the_tensors_themselves():
    calls = [a for a in arguments(source(), "copy_unit") if not a[0].startswith("uint8_t")]
    assert len(calls) >= 4
    for a in calls:
        assert a[-1] in ("p.x", "w"), a  # aligned to the piece that is given before it


def test_row_numbers_stand_in_for_words_only():
    text = source()
    assert "order" not in " ".join(" ".join(a) for a in arguments(text, "ptx::copy_small<8>"))
    assert "order" not in " ".join(" ".join(a) for a in arguments(text, "ptx::copy16"))

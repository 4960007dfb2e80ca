"""Every buffer access leaves its scalar offset at zero.

A raw buffer descriptor's range check holds the lane's offset (register plus immediate) against the record
count; the scalar offset is added to the address unchecked.  A kernel that relies on the check for rows past an
operand's end must therefore keep the scalar offset out of it: no output shows such a read, only an allocation
that ends at an unmapped page would."""
import glob
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "fine_grained_blockwise_amd", "csrc")


def arguments(text, at):
    """The arguments of the call whose opening parenthesis is at text[at]."""
    depth, args, begin = 0, [], at + 1
    for i in range(at, len(text)):
        c = text[i]
        if c in "([{":
            depth += 1
        elif c in ")]}":
            depth -= 1
        if (c == "," and depth == 1) or depth == 0:
            args.append(" ".join(text[begin:i].split()))
            begin = i + 1
        if depth == 0:
            return args
    raise AssertionError("unbalanced call")


def test_scalar_offsets_are_zero():
    seen = 0
    for path in sorted(glob.glob(os.path.join(CSRC, "*.h")) + glob.glob(os.path.join(CSRC, "*.hip"))):
        text = re.sub(r"//[^\n]*", "", open(path).read())
        for m in re.finditer(r"__builtin_amdgcn_raw_buffer_(load|store)_b\d+\(", text):
            args = arguments(text, m.end() - 1)
            scalar = args[3] if m.group(1) == "store" else args[2]  # (data,) descriptor, offset, scalar offset, flags
            assert scalar == "0", (os.path.basename(path), args)
            seen += 1
    assert seen > 5

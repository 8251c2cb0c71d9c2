"""Rules that the HIP sources keep, read from their text: forms that compile and nearly always run right."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "int8_quantized_matmul_rowwise_amd", "csrc")


def arguments(text, at):
    """The arguments of the call whose parenthesis opens at `at`."""
    out, depth, start = [], 0, at + 1
    for i in range(at, len(text)):
        c = text[i]
        if c in "([{":
            depth += 1
        elif c in ")]}":
            depth -= 1
            if depth == 0:
                return out + [text[start:i].strip()]
        elif c == "," and depth == 1:
            out.append(text[start:i].strip())
            start = i + 1
    raise AssertionError("a call without an end")


def wide_stores(text):
    for m in re.finditer(r"__builtin_amdgcn_raw(?:_ptr)?_buffer_store_b(?:96|128)\s*\(", text):
        yield text.count("\n", 0, m.start()) + 1, arguments(text, m.end() - 1)


@pytest.mark.parametrize("path", sorted(glob.glob(os.path.join(CSRC, "*.h*"))), ids=os.path.basename)
def test_wide_buffer_stores_have_no_scalar_offset(path):
    """(data, resource, vector offset, scalar offset, policy): a store of more than 8 bytes with a scalar
    offset can take what a later instruction writes to its data's registers."""
    for line, args in wide_stores(open(path).read()):
        assert len(args) == 5 and args[3] == "0", f"{os.path.basename(path)}:{line}: scalar offset {args[3]}"


def test_the_rule_sees_such_a_store():
    text = "x;\n__builtin_amdgcn_raw_buffer_store_b128(f(a, b[0]), rs, off, piece(i, j), 16);\n__builtin_amdgcn_raw_buffer_store_b64(v, rs, off, at, 0);"
    assert list(wide_stores(text)) == [(2, ["f(a, b[0])", "rs", "off", "piece(i, j)", "16"])]
    assert any(list(wide_stores(open(p).read())) for p in glob.glob(os.path.join(CSRC, "*.h*")))

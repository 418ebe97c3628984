"""Stores to tensor memory are asynchronous, and two of them to the same columns are ordered by a wait
alone.  So whoever stores waits before handing the columns on: a function before it returns, the
softmax's own stores before its next barrier."""
import os
import re

from tests.test_kernel_loads_host import CSRC, code

ROWS = os.path.join(CSRC, "cache_attention_rows.cu")


def body(text, name):
    """What stands between the braces of function `name`."""
    at = text.index("{", re.search(r"\b%s\s*\([^;{]*\)\s*\{" % name, text).start())
    depth = 0
    for i in range(at, len(text)):
        depth += {"{": 1, "}": -1}.get(text[i], 0)
        if depth == 0:
            return text[at + 1:i]
    raise AssertionError(name)


def test_weights_are_there_when_their_function_returns():
    f = body(code(ROWS), "rows_weigh")
    last = f.rindex("tmem_store16(")
    assert "tmem_stored();" in f[last:f.index("return", last)]


def test_rows_of_the_output_are_there_before_the_next_pass():
    f = body(code(ROWS), "cache_attention_rows_kernel")
    for m in re.finditer(r"tmem_store(16|32)\(", f):
        rest = f[m.end():]
        assert 0 < rest.index("tmem_stored();") < min(rest.index("rows_weigh") if "rows_weigh" in rest
                                                      else len(rest), rest.index("mbar_arrive"))

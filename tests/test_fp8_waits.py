"""After a wait has run out, the 8-bit product's CTAs may end only when nothing
of theirs still reads or writes their shared memory.  Such an end cannot be
brought about without a wait that hangs, so the order is read from the source:
what has to happen on every way out stands where no early return can pass it.
"""
import os
import re

SOURCE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "dense_fp32_matrix_10_gb300", "csrc",
                      "fp8_tc.cuh")


def body(name):
    """The text of a function of the source, without comments."""
    with open(SOURCE) as f:
        text = re.sub(r"//[^\n]*", "", f.read())
    at = re.search(r"\b%s\((?:const |__grid)" % name, text).start()
    start = text.index("{", at)
    depth = 0
    for i in range(start, len(text)):
        depth += {"{": 1, "}": -1}.get(text[i], 0)
        if depth == 0:
            return text[start:i + 1]
    raise AssertionError(name)


def test_stores_land_on_every_way_out_of_the_epilogue():
    assert re.search(r"\breturn;", body("fp8_epilogue"))   # it gives up so
    kernel = body("fp8_tc_kernel")
    after = kernel[kernel.index("fp8_epilogue<Cfg>("):]
    wait = after.find("bulk_wait_group_all()")
    assert 0 <= wait < after.index("cluster_sync()") and wait < after.index("__syncthreads()")
    assert "return" not in kernel


def test_tensor_memory_is_read_on_every_way_out_of_the_epilogue():
    kernel = body("fp8_tc_kernel")
    after = kernel[kernel.index("fp8_epilogue<Cfg>("):]
    assert 0 <= after.find("tmem_ld_wait()") < after.index("cluster_sync()")


def test_copies_land_on_every_way_out_of_the_producer():
    text = body("fp8_produce")
    assert not re.search(r"\breturn\b", text)
    last = text[text.rindex("if ("):]
    condition, rest = last[:last.index(")")], last[last.index(")"):]
    assert "ok" not in condition and "bar.full(" in rest

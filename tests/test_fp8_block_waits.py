"""The gradient of the norms around a block exchanges its sums between the CTAs of a cluster, whose waits are limited.  After
one has run out, its warp must send and expect nothing more (an mbarrier's phase takes one arrival), and no CTA may end while
another of its cluster still writes to its shared memory.  Such an end cannot be brought about without a wait that hangs,
so the order is read from the source.
"""
import os
import re

SOURCE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "dense_fp32_matrix_10_gb300", "csrc",
                      "sandwich_backward.cu")


def text():
    with open(SOURCE) as f:
        return re.sub(r"//[^\n]*", "", f.read())


def body(name):
    """The text of a function of the source, without comments."""
    t = text()
    at = re.search(r"\b%s\(" % name, t).start()
    start = t.index("{", t.index(")", at))
    depth = 0
    for i in range(start, len(t)):
        depth += {"{": 1, "}": -1}.get(t[i], 0)
        if depth == 0:
            return t[start:i + 1]
    raise AssertionError(name)


def test_a_warp_that_gave_up_sends_nothing_more():
    t = text()
    sums = t[t.index("operator()(float (&v)[4])"):t.index("void finish()")]
    wait = sums.index("wait_parity_bounded(")
    assert sums.index("mbar_arrive_expect_tx(") < sums.index("st.async") < wait
    assert "__all_sync" in sums[:wait]                                    # the whole warp, or none of it
    assert re.match(r"[^;]*;\s*if \(!ok\) return false;", sums[wait:])
    kernel = body("sandwich_backward_kernel")
    assert kernel.count("row_sums(total)") == 1 and "if (!row_sums(total)) break;" in kernel


def test_every_way_out_meets_the_cluster():
    kernel = body("sandwich_backward_kernel")
    assert "return;" not in re.sub(r"\[&\][^{]*\{", "", kernel)
    after = kernel[kernel.index("if (!row_sums(total)) break;"):]
    assert 0 <= after.index("copies_wait(0);") < after.index("row_sums.finish();")
    assert "cluster_sync();" in body("finish")
    assert "__syncthreads" not in kernel

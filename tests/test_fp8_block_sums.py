"""How the norms' gradient exchanges a row's sums between the CTAs of a cluster, on the host: the scope of the wait, which no
run shows.
"""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "dense_fp32_matrix_10_gb300", "csrc")


def source(name):
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


def test_the_sums_are_waited_for_at_cluster_scope():
    """They are stored by other CTAs, which a wait at a CTA's scope does not order before the reads."""
    waits = re.findall(r"wait_parity_bounded\(([^;]*);", source("sandwich_backward.cu"))
    assert waits and all("SharedOfCluster()" in w for w in waits)
    ptx = source("ptx.cuh")
    wait = ptx[ptx.index("int *status, SharedOfCluster) {"):]
    tries = set(re.findall(r"(mbar_try_wait\w*)\(", wait[:wait.index("return true;\n}")]))
    assert len(tries) == 1
    start = ptx.index("bool %s(" % tries.pop())
    asked = ptx[start:ptx.index("return ok", start)]
    assert ".acquire.cluster." in asked or asked.index(".relaxed.cluster.") < asked.index("fence.acquire.sync_restrict::shared::cluster.cluster")

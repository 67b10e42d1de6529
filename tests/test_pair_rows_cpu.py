"""Rows that the second block of a pair copies to its own shared memory are read by products that
the first block issues: the hand-over needs a release and an acquire of the cluster's scope, and
the order of ordinary before asynchronous accesses. Too late by timing alone it shows nowhere,
so the kernel's source is read for it."""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "fp8_quantized_paged_store_gb300", "csrc")
TEXT = open(os.path.join(CSRC, "fp8_matmul_tiles.cu")).read()


def body(name):
    return re.search(r"\b" + name + r"\([^;{]*\)\s*{(.*?)\n}", TEXT, flags=re.S).group(1)


def test_copied_rows_are_released_to_the_cluster():
    announce = body("announce_rows")
    assert announce.index("kCopied") < announce.index("arrive_rows(") and "arrive_pair(" not in announce
    arrive = body("arrive_rows")
    fence = arrive.index("fence.proxy.async::generic.release.sync_restrict::shared::cta.cluster")
    assert fence < arrive.index("mbarrier.arrive.relaxed.cluster.shared::cluster")


def test_the_issuer_acquires_them_before_its_products():
    wait = body("wait_operands")
    assert wait.index("mbar_test_rows(full") < wait.index("acquire_rows();") < wait.index("return true")
    assert "mbarrier.try_wait.parity.relaxed.cluster" in body("mbar_test_rows")
    assert "fence.proxy.async::generic.acquire.sync_restrict::shared::cluster.cluster" in body("acquire_rows")
    issue = body("issue_tiles")
    assert issue.index("wait_operands<kIndex>(") < issue.index("pair_mma(")

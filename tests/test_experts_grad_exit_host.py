"""The end of the experts' gradient's CTA pairs, by reading the source (no GPU: what this is about
would be a write into shared memory that is another kernel's by then).

A tcgen05.commit arrives on barriers some time after it is issued, in each CTA that its mask names.
Threads that meet at the cluster's barrier do not wait for it, so a CTA may only end once it has
waited, on its own copy, for every commit that is sent to it."""
import os
import re

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "mixture_experts_layer_07_gb300", "csrc")


def source(name):
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


def part(text, start, end):
    a = text.index(start)
    return text[a:text.index(end, a + len(start))]


def kernel():
    return part(source("experts_grad.cu"), "products_kernel(", "\n}\n")


def test_commits_to_both_ctas_are_waited_for_in_both():
    k = kernel()
    commits = re.findall(r"tc_commit2\((\w+)(?:\([^()]*\))?(?:, (\w+))?\)", k)
    assert len(commits) == k.count("tc_commit2(") and commits
    both = {bar for bar, ctas in commits if not ctas}
    assert all(ctas == "kLeader" for _, ctas in commits if ctas)
    # the stages' and the accumulators' go to both; who waits for them is below.  What the leader's
    # issuer alone waits for is sent to the leader alone
    assert both == {"empty_bar", "acc_full"}, both
    assert ("drain_bar", "kLeader") in commits
    producer = part(k, "if (warp == 0) {\n", "else if (warp == 1 && rank == 0)")
    epilogue = k[k.index("setmaxnreg.inc"):]
    # accumulators: the epilogue of either CTA waits for each use
    waits = part(epilogue, "auto wait_acc", "};")
    assert "acc_full(i)" in waits and "rank" not in waits
    # stages: behind its last unit, either producer waits for those that it has filled
    end = producer[producer.index("__syncwarp();\n      }"):]
    loop = part(end, "for (int s = 0; s < kStages && ok; ++s)", "fail();")
    assert re.search(r"mbar_wait_bounded\(empty_bar\(s\), \(armed_parity >> s\) & 1u, abort_flag, kWaitNs\)", loop)
    assert "armed & (1u << s)" in loop
    assert "rank" not in loop and end[:end.index(loop)].rstrip().endswith("}")
    # and they meet behind that
    assert k.index("cluster_sync();", k.index("auto wait_acc")) > k.index(loop)


def test_a_commit_goes_to_the_ctas_that_its_mask_names():
    ptx = source("sm100_ptx.cuh")
    body = part(ptx, "MOE_DEVICE void tc_commit2(", "\n}\n")
    assert '"h"(ctas)' in body and "multicast::cluster" in body
    assert re.search(r"uint16_t ctas = 3", body)
    assert re.search(r"constexpr uint16_t kLeader = 1;", ptx)

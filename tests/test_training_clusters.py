"""Blocks of a cluster that store into each other's shared memory: none leaves before the
others have sent what they send, on any path, and copies in flight land first.  (Shown on
the source, since the paths in question are those of a wait that ran out; on the GPU, the
kernels go through many rows a cluster, in place too.)"""
import os
import re

import pytest
import torch

from lora_rank_adapter_gb300 import _build
from tests.test_training_loss import BF16, DEV, F32, check_policy, make, policy_inputs, run_policy

SOURCE = os.path.join(_build.CSRC, "loss.cu")


def _body(name):
    """The text between the braces of a function of loss.cu, without comments."""
    with open(SOURCE) as f:
        text = re.sub(r"//[^\n]*", "", f.read())
    found = re.search(r"\b%s\([^;{]*\)\s*\{\n(.*?)\n\}\n" % name, text, re.S)
    assert found, name
    return found.group(1)


def _held():
    """The loader's part of the policy kernel up to its return, and the other warps' part."""
    return _body("held_kernel").split("if (warp == kHeldWarps) {")[1].split("    return;\n  }\n", 1)


def test_no_block_leaves_its_cluster_early():
    # the statistics: one way out, behind the barrier at which every block has sent
    stats = _body("stats_kernel")
    assert not re.search(r"\breturn\b", stats)
    sends, arrives, receives = (stats.index(k) for k in ("cluster_send(", "cluster_arrive();\n    if (tid < 32) whole",
                                                         "cluster_merge("))
    assert sends < arrives < receives < stats.rindex("cluster_wait();")
    # the blocks that go through rows: each warp ends by telling all blocks that it has sent its
    # last, on every path, and the loader keeps its block until all have
    loader, work = _held()
    assert loader.index("mbar_wait<true>(&done, 0)") > loader.index("mbar_wait(&full")
    assert "i < kSlots * (kSlots + 1) && !mbar_wait<true>(&done, 0)" in loader      # every wait that may lie ahead
    assert not re.search(r"\breturn\b", work)
    assert re.search(r"\n  \}\s*if \(C > 1 && lane < C\) mbar_arrive_remote\(&done, lane\);\s*$", work)
    assert "mbar_init(&done, C * kHeldWarps);" in _body("held_kernel")
    # only these two send
    with open(SOURCE) as f:
        text = f.read()
    assert len(re.findall(r"\bst_async_f2\(&", text)) == 1 and "st_async_f2(&" in work
    assert len(re.findall(r"\bcluster_send\(", text)) == 2


def test_one_reading_of_the_label_decides_for_a_block():
    """The statistics' blocks pass barriers of the block inside a branch on the label: all of a
    block's threads take the same branch, also where another stream is writing the labels."""
    stats = _body("stats_kernel")
    assert "slots.label = a.labels[t]" in stats and "label = slots.label" in stats


def test_copies_in_flight_land_before_the_block_ends():
    loader, _ = _held()
    assert re.search(r"\}\s*for \(int i = 0; i < kSlots; \+\+i\)\s*if \(again \|\| i < at\.slot\) mbar_wait\(&full", loader)
    assert "if (!ok)\n      for" not in loader


def test_reads_of_a_row_come_before_the_arrival_that_lets_others_write_it():
    """In place, any warp of the block may write the label's element past the exchange: the arrival
    for a warp follows the reads of all its lanes, by a barrier of the warp, or carries the value."""
    _, work = _held()
    assert re.search(r"if \(C == 1\) \{\s*__syncwarp\(\);\s*if \(lane == 0\)", work)
    assert "lane + (__float_as_uint(picked) & h.zero)" in work
    short = _body("short_kernel")
    reads, merge, writes = (short.index(k) for k in ("const float picked", "if (kTeam == 1) __syncwarp();", "g.piece<E>"))
    assert reads < merge < writes and merge < short.index("__syncthreads();") < writes


@pytest.mark.gpu
@pytest.mark.parametrize("T,V,dtype", [(700, 70001, BF16), (2000, 20000, BF16), (900, 40002, F32),
                                       (5000, 300, F32), (3000, 4000, BF16), (3000, 15001, BF16)])
def test_many_rows_a_cluster_in_place(T, V, dtype):
    """Each cluster goes through several rows, some ignored, and the gradient replaces them."""
    torch.cuda.set_device(0)
    full, x, labels = make(T, V, dtype, seed=T)
    old, adv, w, ref = policy_inputs(x, labels, T)
    adv[::7] = 0.0                                # rows without a gradient among them
    want = run_policy(x, labels, old, adv, w)
    for _ in range(3):
        copy = x.clone()
        got = run_policy(copy, labels, old, adv, w, d=copy)
        for k in want:
            assert torch.equal(got[k], want[k]), k
    some = torch.arange(0, T, 41)
    few = run_policy(x[some.to(DEV)], labels[some.to(DEV)], old[some], adv[some], w[some])
    check_policy(few, x[some.to(DEV)], labels[some.to(DEV)], old[some], adv[some], w[some], None)
    rows = some.to(DEV)
    # rows of few and of many: other cuts, so other orders of summation; both coefficients are off by 4e-6 |logp|
    # (below 20) and by 4e-6 of themselves
    assert bool(((want["d"][rows].float() - few["d"].float()).abs()
                 <= 2e-4 * want["d"][rows].float().abs().amax(1, keepdim=True).clamp(min=1e-30)
                 + 2.0 ** -8 * few["d"].float().abs()).all())


@pytest.mark.gpu
def test_few_rows_over_clusters():
    """Rows cut over clusters, ignored ones among them, many times over."""
    from lora_rank_adapter_gb300 import training
    from tests.test_training_loss import check_logps, oracle_logps
    torch.cuda.set_device(0)
    for T in (2, 5, 30, 75):
        _, x, labels = make(T, 50001, BF16, seed=T, ignored=0.4)
        want, _, _ = oracle_logps(x, labels)
        first = None
        for _ in range(50):
            logps = torch.full((T,), 5.0, device=DEV)
            training.lora_token_logps(x, labels, logps)
            first = logps if first is None else first
            assert torch.equal(logps, first)
        check_logps(first, want)

"""No workgroup barrier is reached while the wave's own reads or writes of LDS
may still be under way, in the code that is built for the kernels with barriers
of their own (lds_barrier).  What waves hand each other through LDS is there
only after a wait; a barrier alone does not wait.  The assembly is followed over
every path of its control flow."""

import os
import re
import subprocess

import pytest

from quantized_linear_layers_awq_amd import build

SOURCES = ("gemm.hip", "gemm256.hip", "attn_prefill.hip")


@pytest.fixture(scope="module")
def assembly(tmp_path_factory):
    if not os.path.exists(build.hipcc()):
        pytest.skip("no hipcc")
    folder = tmp_path_factory.mktemp("asm")
    runs = {s: subprocess.Popen([build.hipcc(), *build.compile_flags(), "--cuda-device-only", "-S", os.path.join(build.CSRC, s),
                                 "-o", str(folder / s)], stdout=subprocess.DEVNULL, stderr=subprocess.DEVNULL)
            for s in SOURCES}
    assert all(p.wait() == 0 for p in runs.values())
    return {s: (folder / s).read_text() for s in SOURCES}


def _kernels(text):
    """name -> [(operation, argument)] of each kernel; a block of its own begins at each label and after each branch."""
    name, block, at = None, None, {}
    for line in text.splitlines():
        if m := re.match(r"(_Z\S+):", line):
            name, block = m.group(1), "entry"
            at[name] = {block: []}
            continue
        if name is None:
            continue
        if m := re.match(r"(\.LBB\S+):", line):
            block = m.group(1)
            at[name][block] = []
            continue
        op, _, rest = line.strip().partition(" ")
        op, _, tab = op.partition("\t")
        rest = tab + rest
        ops = at[name][block]
        if op.startswith(("ds_read", "ds_write")):
            ops.append(("lds", None))
        elif op == "s_waitcnt" and (m := re.search(r"lgkmcnt\((\d+)\)", rest)):
            ops.append(("wait", int(m.group(1))))
        elif op == "s_barrier":
            ops.append(("barrier", None))
        elif op == "s_endpgm":
            ops.append(("end", None))
        elif op.startswith(("s_branch", "s_cbranch")):
            ops.append(("go" if op == "s_branch" else "may go", rest.split()[0]))
            block = f"after {block} {len(at[name])}"
            at[name][block] = []
    return at


def _barriers_and_unfinished(blocks):
    """How many barriers there are, and how many of them LDS operations may be outstanding at."""
    order = list(blocks)
    most = {order[0]: 0}  # operations that may be outstanding where a block begins
    work, bad = [order[0]], set()
    while work:
        block = work.pop()
        n, after = most[block], [order[order.index(block) + 1]] if block != order[-1] else []
        for i, (op, arg) in enumerate(blocks[block]):
            if op == "lds":
                n = min(n + 1, 64)
            elif op == "wait":
                n = min(n, arg)
            elif op == "barrier" and n:
                bad.add((block, i))
            elif op == "end":
                after = []
            elif op == "go":
                after = [arg]
            elif op == "may go":
                after = after + [arg]
        for b in after:
            if most.get(b, -1) < n:
                most[b] = n
                work.append(b)
    return sum(op == "barrier" for ops in blocks.values() for op, _ in ops), len(bad)


@pytest.mark.parametrize("source", SOURCES)
def test_lds_operations_are_complete_at_every_barrier(assembly, source):
    counts = {name: _barriers_and_unfinished(blocks) for name, blocks in _kernels(assembly[source]).items()}
    assert sum(n for n, _ in counts.values()) > 0
    assert not {name: c for name, c in counts.items() if c[1]}


def test_the_check_sees_a_missing_wait():
    text = "_Zk:\n\tds_write_b32 v0, v1\n\ts_cbranch_scc1 .LBB0_1\n\ts_waitcnt lgkmcnt(0)\n.LBB0_1:\n\ts_barrier\n\ts_endpgm\n"
    assert _barriers_and_unfinished(_kernels(text)["_Zk"]) == (1, 1)
    assert _barriers_and_unfinished(_kernels(text.replace("\ts_cbranch_scc1 .LBB0_1\n", ""))["_Zk"]) == (1, 0)

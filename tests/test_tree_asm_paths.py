"""What the pair kernel's loops and the products written as inline assembly rely on, read
off the generated code along every path of its control flow: blocks that the compiler
places behind a loop belong to it, and a branch leads to where it leads."""
import os
import re
import subprocess
from collections import namedtuple

import pytest

from sparse_attention_indexer_block_amd import build as B

Ins = namedtuple("Ins", "op args asm text")


@pytest.fixture(scope="module")
def code(tmp_path_factory):
    out = os.path.join(str(tmp_path_factory.mktemp("asm")), "k.s")
    src = "tree_kernels.hip"
    flags = [f for f in B.CFLAGS if f != "-fPIC"]
    subprocess.run([B.HIPCC, *flags, *B.EXTRA.get(src, []), "--cuda-device-only", "-S", os.path.join(B.CSRC, src), "-o", out],
                   check=True, capture_output=True, timeout=600)
    return open(out).read().splitlines()



def graph(code, name):
    """The instructions of a function and, for each, those that may run after it."""
    start = next(i for i, t in enumerate(code) if t.startswith(name))
    end = next(i for i in range(start, len(code)) if code[i].startswith(".Lfunc_end"))
    ins, labels, asm = [], {}, False
    for line in code[start + 1:end]:
        asm = (asm or "ASMSTART" in line) and "ASMEND" not in line
        text = line.split(";")[0].strip()
        if re.fullmatch(r"\.LBB\w+:", text):
            labels[text[:-1]] = len(ins)
        elif text and not text.startswith(".") and not text.endswith(":"):
            op = text.split()[0]
            ins.append(Ins(op, [a.strip() for a in text[len(op):].split(",") if a.strip()], asm, text))
    after = []
    for i, x in enumerate(ins):
        assert not x.op.startswith(("s_setpc", "s_swappc", "s_call", "s_cbranch_i", "s_cbranch_g")), x.text
        to = [labels[x.args[-1]]] if x.op.startswith(("s_branch", "s_cbranch")) else []
        if x.op not in ("s_branch", "s_endpgm"):
            to.append(i + 1)
        after.append([t for t in to if t < len(ins)])
    return ins, after


def loops(after):
    """The sets of instructions that can be reached from each other (more than one each)."""
    n, index, low, stack, on, got, count = len(after), {}, {}, [], set(), [], 0
    for root in range(n):
        if root in index:
            continue
        work = [(root, 0)]
        while work:
            v, k = work.pop()
            if v not in index:
                index[v] = low[v] = count
                count += 1
                stack.append(v)
                on.add(v)
            down = False
            for j in range(k, len(after[v])):
                w = after[v][j]
                if w not in index:
                    work += [(v, j), (w, 0)]
                    down = True
                    break
                if w in on:
                    low[v] = min(low[v], low[w])
            if down:
                continue
            if low[v] == index[v]:
                part = set()
                while True:
                    w = stack.pop()
                    on.discard(w)
                    part.add(w)
                    if w == v:
                        break
                if len(part) > 1:
                    got.append(part)
    return got


@pytest.mark.parametrize("fp8", [0, 1])
def test_the_pair_kernels_two_loops_have_no_wait_of_their_own(code, fp8):
    # one loop of tiles that all rows see, one of tiles that some see; two steps of 68 products each
    ins, after = graph(code, f"_ZN4misa13k_latent_pairILb{fp8}E")
    work = [p for p in loops(after) if any(ins[i].op.startswith("v_mfma") for i in p)]
    assert len(work) == 2
    for part in work:
        assert sum(ins[i].op.startswith("v_mfma") for i in part) == 136
        for i in sorted(part):
            x = ins[i]
            assert not x.op.startswith("scratch_"), x.text
            if x.op == "s_waitcnt" and "vmcnt(" in x.text and not x.asm:
                # next to a load that it waits for, in the rare paths of the walk
                assert any(y.op.startswith("global_load_") and "lds" not in y.op for y in ins[i - 5:i]), [y.text for y in ins[i - 5:i + 1]]


def registers(token):
    m = re.fullmatch(r"([va])\[(\d+):(\d+)\]", token)
    if m:
        return {(m.group(1), i) for i in range(int(m.group(2)), int(m.group(3)) + 1)}
    m = re.fullmatch(r"([va])(\d+)", token)
    return {(m.group(1), int(m.group(2)))} if m else set()


def states(x):
    return int(x.args[0]) + 1 if x.op == "s_nop" else 1


def kernel_names(code):
    return [t.split(":")[0] for t in code if re.match(r"_ZN4misa\d+k_latent\w+:", t)]


def test_products_written_as_asm_wait_for_vector_instructions_on_every_path(code):
    # a product may not read what a vector instruction wrote in the two wait states before it
    checked = 0
    for name in kernel_names(code):
        ins, after = graph(code, name + ":")
        before = [[] for _ in ins]
        for i, to in enumerate(after):
            for t in to:
                before[t].append(i)
        for k, x in enumerate(ins):
            if not (x.op.startswith("v_mfma") and x.asm):
                continue
            checked += 1
            reads = set().union(*[registers(a) for a in x.args[1:]])
            todo = [(p, 0) for p in before[k]]
            while todo:
                i, far = todo.pop()
                y = ins[i]
                if y.op.startswith("v_") and not y.op.startswith(("v_mfma", "v_cmp", "v_readlane", "v_readfirstlane")):
                    wrote = registers(y.args[0]) | (registers(y.args[1]) if "swap" in y.op else set())
                    assert not wrote & reads, (name, y.text, x.text)
                far += states(y)
                if far < 2:
                    todo += [(p, far) for p in before[i]]
    assert checked > 400


def test_results_of_asm_products_are_touched_late_on_every_path(code):
    # a product's result in vector registers needs 12 wait states before another instruction than the product that
    # adds to it may touch it, which the compiler does not know of products that are asm (16 asked for here)
    checked = 0
    for name in kernel_names(code):
        ins, after = graph(code, name + ":")
        for k, x in enumerate(ins):
            if not (x.op.startswith("v_mfma") and x.asm and x.args[0].startswith("v")):
                continue
            checked += 1
            result, best, todo = registers(x.args[0]), {}, [(t, 0) for t in after[k]]
            while todo:
                i, far = todo.pop()
                if best.get(i, 99) <= far:
                    continue
                best[i] = far
                y = ins[i]
                if y.op.startswith("v_mfma") and y.args[0] == x.args[0] and y.args[3] == x.args[0]:
                    continue
                touched = set().union(*[registers(a.split()[0]) for a in y.args if a])
                assert not touched & result, (name, x.text, y.text, far)
                far += states(y)
                if far < 16:
                    todo += [(t, far) for t in after[i]]
    assert checked > 400

"""What the tree kernels' inline copies to LDS rely on, read off the generated code: M0
holds the LDS address of a copy and is set in the copy itself, no other instruction
reads or writes it, and the main loop of the pair kernel waits for copies only where it
says so (a wait of the compiler's own would drain those in flight)."""
import os
import re
import subprocess

import pytest

from sparse_attention_indexer_block_amd import build as B
from test_attention_asm import IMPLICIT

COPY = re.compile(r"((s_mov_b64 s\[\d+:\d+\], \S+\n)?s_mov_b32 m0, s\d+|s_add_u32 m0, s\d+, \S+)\ns_nop 0\nglobal_load_lds_dword(x4)? .*")


@pytest.fixture(scope="module")
def code(tmp_path_factory):
    out = os.path.join(str(tmp_path_factory.mktemp("asm")), "k.s")
    src = "tree_kernels.hip"
    flags = [f for f in B.CFLAGS if f != "-fPIC"]
    subprocess.run([B.HIPCC, *flags, *B.EXTRA.get(src, []), "--cuda-device-only", "-S", os.path.join(B.CSRC, src), "-o", out],
                   check=True, capture_output=True, timeout=600)
    return open(out).read().splitlines()


def test_m0_belongs_to_the_copies(code):
    copies, block = 0, None
    for line in code:
        text = line.strip()
        if text.startswith(";;#ASMSTART"):
            block = []
            continue
        if text.startswith(";;#ASMEND"):
            if any("m0" in t for t in block):
                assert COPY.fullmatch("\n".join(block)), block
                copies += 1
            block = None
            continue
        text = text.split(";")[0].strip()
        if block is not None:
            if text:
                block.append(re.sub(r"\s+", " ", text))
            continue
        if not text or text.startswith("."):
            continue
        assert not re.search(r"\bm0\b", text), line
        assert not IMPLICIT.match(text) or text.startswith("s_sendmsg sendmsg(MSG_DEALLOC_VGPRS)"), line
    assert copies > 0


@pytest.mark.parametrize("fp8", [0, 1])
def test_the_pair_kernels_loop_has_no_wait_of_its_own(code, fp8):
    start = next(i for i, t in enumerate(code) if t.startswith(f"_ZN4misa13k_latent_pairILb{fp8}E"))
    end = next(i for i in range(start, len(code)) if code[i].startswith(".Lfunc_end"))
    body = [t.strip() for t in code[start:end]]
    loop = max(i for i, t in enumerate(body) if "This Loop Header: Depth=1" in t)
    waits = [i for i, t in enumerate(body) if i > loop and t.startswith("s_waitcnt vmcnt(") and "ASMSTART" not in body[i - 1]]
    last = max(i for i, t in enumerate(body) if t.startswith("v_mfma"))
    for i in waits:
        if i < last:  # next to a load that it waits for, in the rare paths of the walk
            assert any(t.startswith("global_load_") and "lds" not in t for t in body[i - 5:i]), body[i - 5:i + 1]
    assert not any(t.startswith("scratch_") for t in body[loop:last])


def _registers(token):
    m = re.fullmatch(r"([va])\[(\d+):(\d+)\]", token)
    if m:
        return {(m.group(1), i) for i in range(int(m.group(2)), int(m.group(3)) + 1)}
    m = re.fullmatch(r"([va])(\d+)", token)
    return {(m.group(1), int(m.group(2)))} if m else set()


def test_products_written_as_asm_wait_for_vector_instructions(code):
    # a product may not read what a vector instruction wrote in the two wait states before it; the compiler does
    # not see that some of these products are asm, so the distance is read off here
    ins = []
    for line in code:
        text = line.split(";")[0].strip()
        if re.match(r"\.LBB", line):
            ins.append(("label", []))
        elif text and not text.startswith("."):
            op = text.split()[0]
            ins.append((op, [a.strip() for a in text[len(op):].split(",")]))
    seen = 0
    for k, (op, args) in enumerate(ins):
        if not op.startswith("v_mfma"):
            continue
        seen += 1
        reads, states = set().union(*[_registers(a) for a in args[1:]]), 0
        for o, a in reversed(ins[max(0, k - 3):k]):
            if states >= 2 or o == "label":
                break
            if o.startswith("v_") and not o.startswith(("v_mfma", "v_cmp", "v_readlane", "v_readfirstlane")):
                wrote = _registers(a[0]) | (_registers(a[1]) if "swap" in o else set())
                assert not wrote & reads, (o, a, op, args)
            states += int(a[0]) + 1 if o == "s_nop" else 1
    assert seen > 100


def test_scores_are_read_long_after_their_last_product(code):
    # a product's result in vector registers needs 12 wait states before any other instruction may touch it (16
    # asked for here), which the compiler does not know of products that are asm
    block, ins = False, []
    for line in code:
        block = (block or "ASMSTART" in line) and "ASMEND" not in line
        text = line.split(";")[0].strip()
        if text and (not text.startswith(".") or line.startswith(".LBB")):
            op = text.split()[0]
            ins.append((op, [a.strip() for a in text[len(op):].split(",")], block))
    checked = 0
    for k, (op, args, asm) in enumerate(ins):
        if not (op.startswith("v_mfma") and asm and args[0].startswith("v")):
            continue
        result, states = _registers(args[0]), 0
        checked += 1
        for o, a, _ in ins[k + 1:k + 40]:
            touched = set().union(*[_registers(x.split()[0]) for x in a if x]) if not o.startswith(".") else set()
            if states >= 16 or (o.startswith("v_mfma") and a[0] == args[0] and a[3] in (args[0], "0")):
                break
            assert not touched & result, (op, args, o, a, states)
            states += int(a[0]) + 1 if o == "s_nop" else 0 if o.startswith(".") else 1
    assert checked > 100

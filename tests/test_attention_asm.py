"""What the attention kernels' inline copies to LDS rely on, read off the
generated code: M0 holds the LDS address of a copy and is set in the copy itself,
and no other instruction of these files reads or writes it, by name or by its
kind (the register is reserved by the compiler, which warns of a clobber of it
instead of honouring one)."""
import os
import re
import subprocess

import pytest

from sparse_attention_indexer_block_amd import build as B

# instructions that take M0 without naming it: other copies to LDS, LDS ones that add the thread's address,
# ordered and global-wave-sync ones, interpolation, messages, relative moves and indexed register modes
IMPLICIT = re.compile(r"^(buffer_load_\w*.*\blds\b|global_load_lds\w*|scratch_load_lds\w*|buffer_load_lds\w*|ds_\w*addtid\w*|ds_gws\w*|"
                      r"ds_ordered\w*|v_interp\w*|s_sendmsg\w*|v_movrel\w*|s_movrel\w*|s_set_gpr_idx\w*|s_ttracedata\w*)")


@pytest.mark.parametrize("src", ["latent_kernels.hip", "expanded_kernels.hip"])
def test_m0_belongs_to_the_copies(src, tmp_path):
    out = os.path.join(str(tmp_path), "k.s")
    flags = [f for f in B.CFLAGS if f != "-fPIC"]
    subprocess.run([B.HIPCC, *flags, *B.EXTRA.get(src, []), "--cuda-device-only", "-S", os.path.join(B.CSRC, src), "-o", out],
                   check=True, capture_output=True, timeout=600)
    copies, block = 0, None
    for line in open(out):
        text = line.strip()
        if text.startswith(";;#ASMSTART"):
            block = []
            continue
        if text.startswith(";;#ASMEND"):
            if any("m0" in t for t in block):
                assert re.fullmatch(r"(s_mov_b64 s\[\d+:\d+\], \S+\n)?s_mov_b32 m0, s\d+\ns_nop 0\nglobal_load_lds_dwordx4 .*", "\n".join(block)), block
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

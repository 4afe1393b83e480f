"""The kernels of drafted tokens copy to LDS as the other attention kernels do: the
same reading of their generated code."""
from test_attention_asm import test_m0_belongs_to_the_copies as _m0_belongs_to_the_copies


def test_m0_belongs_to_the_copies_of_the_tree_kernels(tmp_path):
    _m0_belongs_to_the_copies("tree_kernels.hip", tmp_path)

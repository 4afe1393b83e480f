"""How a call of the attention was cut, by the names that its launches are
profiled under: a kernel and the rows of a workgroup, and whether parts were joined."""
import torch

import sparse_attention_indexer_block_amd as S

LATENT = {16: "k_latent_16", 32: "k_latent_32", 64: "k_latent_wide_64", 128: "k_latent_wide_128"}
EXPANDED = {128: "k_expanded_128", 256: "k_expanded_256"}


def cut_of(call, names):
    """(rows of a workgroup, split or not) of the one attention call that call() makes, and its result."""
    torch.cuda.synchronize()
    S.profile_reset()
    S.profile_enable(True)
    try:
        got = call()
        torch.cuda.synchronize()
    finally:
        S.profile_enable(False)
    ran = [rows for rows, name in names.items() if S.profile_read(name)[1]]
    joined, total = S.profile_read("k_join")[1], S.profile_read("")[1]
    S.profile_reset()
    assert len(ran) == 1 and total == 1 + joined, (ran, joined, total)
    return (ran[0], joined == 1), got

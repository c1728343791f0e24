"""Mask rows of drafts up to the largest, 4096 tokens: chains, stars, random
trees, with positions."""
import numpy as np
import pytest
import torch

import nvfp4_quantized_dense_amd as nv
from serving_reference import family, pack_bits
from test_gpu_kv_attention import dev

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n", [201, 256, 257, 1000, 2049, 4095, 4096])
@pytest.mark.parametrize("kind", ["chain", "star", "random", "near"])
def test_deep(n, kind):
    r, i = np.random.RandomState(n), np.arange(n)
    p = {"chain": i - 1, "star": np.where(i > 0, 0, -1), "random": np.array([r.randint(-1, max(j, 1)) for j in i]),
         "near": i - 1 - np.minimum(r.randint(0, 4, n), i)}[kind].astype(np.int32)
    p[0] = -1
    see = family(p, n)
    words = -(-n // 64)
    lead = 3  # rows of a sequence in front
    tree = torch.full((lead + n, words), 7, dtype=torch.int64, device="cuda")
    pos = torch.full((lead + n,), 50, dtype=torch.int32, device="cuda")
    nv.nvfp4_tree_mask(dev(np.concatenate([[-1, 0, 1], p]), torch.int32), dev([0, lead, lead + n], torch.int32), n, positions=pos, tree=tree)
    assert np.array_equal(tree[lead:].cpu().numpy(), pack_bits(see, words))
    assert np.array_equal(pos[lead:].cpu().numpy(), 50 + see.sum(1) - 1) and pos[:lead].tolist() == [50, 51, 52]
    assert np.array_equal(tree[:lead].cpu().numpy(), pack_bits(np.tril(np.ones((3, 3), bool)), words))

"""The decoder layer example's workspace, on the host."""
import os
import sys
import weakref

import torch

import nvfp4_quantized_dense_amd as nv

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
from decoder_layer import DecoderLayer  # noqa: E402


def test_a_workspace_outlives_its_successor(monkeypatch):
    """Graphs captured before a larger call keep memory of their own."""
    for name in ("nvfp4_calibrate", "nvfp4_quantize"):
        monkeypatch.setattr(nv, name, lambda *a: (torch.ones(1), torch.ones(1)))
    monkeypatch.setattr(nv, "nvfp4_repack_weight", lambda *a: torch.ones(1))
    layer = DecoderLayer(64, 64, 8, 1, 64, pages=4, page_size=16, device="cpu")
    sizes = [(1, 1, 8, 1, 64, 1, n) for n in (600, 5000, 100000)]
    made = []
    for s in sizes:
        ws = layer.workspace(*s)
        assert ws.numel() >= nv.nvfp4_kv_attention_workspace_bytes(*s) and layer.workspace(*s) is ws
        made.append(weakref.ref(ws))
        del ws
    assert len({id(m()) for m in made}) == 3 and all(m() is not None for m in made)

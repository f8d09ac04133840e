"""Arguments of the native calls that no tensor check sees (nothing here
reaches a GPU)."""
import numpy as np
import pytest
import torch

from decode_gemv_tb_b200 import build as tbbuild
from decode_gemv_tb_b200 import tb


def test_a_flag_without_a_truth_value():
    """An exception of the library's kind, raised before anything is launched."""
    tbbuild.build()
    tb.load()
    x = torch.zeros((2, 128), dtype=torch.bfloat16)
    for flag in (np.zeros(2), torch.zeros(2)):
        with pytest.raises(tb.TBError, match="renormalize must be true or false"):
            tb.tb_moe_route(x, x, 1, renormalize=flag)


def test_a_call_without_a_workspace_fills_nothing(monkeypatch):
    """tb_moe's workspace is data that it writes before it reads it: what the call allocates for itself is not filled."""
    tbbuild.build()
    tb.load()
    desc = tb.MoE(*(1 << 40,) * 6, 0, 0, 0, 4, 256, 128)
    layer = tb.MoELayer(desc, (), 0)
    seen = []

    class Calls:
        @staticmethod
        def moe(*args):
            seen.append(args[7])

    monkeypatch.setattr(tb, "_bind", Calls)
    monkeypatch.setattr(torch, "zeros", None)
    monkeypatch.setattr(tb, "workspace", None)
    x, ids = torch.empty((3, 256), dtype=torch.bfloat16), torch.empty((3, 2), dtype=torch.int32)
    tb.tb_moe(layer, x, ids, torch.empty((3, 2)))
    assert seen[0].numel() == tb.moe_workspace_bytes(layer, 3, 2) > 0 and seen[0].dtype == torch.uint8

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

"""The down kernel begins while the up kernel runs and reads ids and weights
ahead of its own wait: layers in a row whose router rewrites the same two
buffers each time, of so few pairs that most SMs run the down kernel only.
The same bits as one by one with fresh buffers."""
import numpy as np
import pytest
import torch

from decode_gemv_tb_b200 import tb
from tests import mx4_ref as R

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.mark.parametrize("T,k", [(1, 1), (1, 4), (3, 2)])
def test_ids_and_weights_rewritten_between_layers(T, k):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    E, H, I, depth = 24, 4096, 128, 16
    rng = np.random.default_rng(T * 10 + k)
    layer = tb.moe_layer(*(R.random_matrix(rows, cols, grid, rng)[1]
                           for rows, cols, grid in ((E * I, H, 0), (E * I, H, 4), (E * H, I, 1))), E, H, I)
    g = torch.Generator().manual_seed(k)
    xs = torch.randn((depth, T, H), generator=g).to(torch.bfloat16).to(DEV)
    rs = torch.randn((depth, E, H), generator=g).to(torch.bfloat16).to(DEV)
    want, taken = [], set()
    for i in range(depth):
        ids, w = tb.tb_moe_route(xs[i], rs[i], k, renormalize=False)
        torch.cuda.synchronize()
        want.append(tb.tb_moe(layer, xs[i], ids, w))
        torch.cuda.synchronize()
        taken.add(tuple(ids.flatten().tolist()))
    assert len(taken) > depth // 2  # the ids do change
    ids, w = torch.empty((T, k), dtype=torch.int32, device=DEV), torch.empty((T, k), device=DEV)
    ws = tb.workspace(tb.moe_workspace_bytes(layer, T, k), DEV)
    ys = torch.empty((depth, T, H), device=DEV)

    def run():
        for i in range(depth):
            tb.tb_moe_route(xs[i], rs[i], k, renormalize=False, ids=ids, weights=w)
            tb.tb_moe(layer, xs[i], ids, w, y=ys[i], ws=ws)

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    for step in (run, graph.replay) * 10:
        ys.fill_(-1.0)
        step()
        assert all(torch.equal(ys[i], want[i]) for i in range(depth))
    assert tb.sync_status() == 0

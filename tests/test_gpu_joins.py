"""Calls whose inputs come from two streams, eager and captured, and a first
call of the process inside a capture."""
import subprocess
import sys

import pytest
import torch

from decode_gemv_tb_b200 import tb
from tests import mx4_ref as R
import numpy as np

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    tb.load()


def setup():
    g = torch.Generator().manual_seed(1)
    E, H, I, T, k, n = 8, 512, 256, 5, 2, 6
    rng = np.random.default_rng(2)
    layer = tb.moe_layer(*(R.random_matrix(r, c, q, rng)[1] for r, c, q in ((E * I, H, 4), (E * I, H, 1), (E * H, I, 2))), E, H, I)
    s = dict(E=E, H=H, T=T, k=k, n=n, layer=layer)
    s["xs"] = torch.randn((n, T, H), generator=g).to(torch.bfloat16).to(DEV)
    s["r"] = torch.randn((E, H), generator=g).to(torch.bfloat16).to(DEV)
    s["W"] = tb.tb_mx4_quantize(torch.randn((640, H), generator=g).to(DEV))
    s["ws"] = [tb.workspace(tb.moe_workspace_bytes(layer, T, k), DEV) for _ in range(2)]
    return s


def want(s):
    out = []
    for x in s["xs"]:
        ids, w = tb.tb_moe_route(x, s["r"], s["k"])
        torch.cuda.synchronize()
        y = tb.tb_moe(s["layer"], x, ids, w)
        q = tb.tb_mx4_quantize(x)
        torch.cuda.synchronize()
        out.append((y, tb.tb_mx4_gemm(*s["W"], *q, s["T"], 640, s["H"])))
        torch.cuda.synchronize()
    return out


def run(s, main, side, bufs, busy):
    """The router and the quantiser on one stream, the expert layer and the product on the other, joined by events: every
    second-stream call waits for the first stream's, and the buffers are written again only behind the reader."""
    x, ids, w, c, t, ys, Ys = bufs
    with torch.cuda.stream(side):
        side.wait_stream(main)
    for i in range(s["n"]):
        with torch.cuda.stream(side):
            busy.mul_(1.0)
            x.copy_(s["xs"][i])
            tb.tb_moe_route(x, s["r"], s["k"], ids=ids, weights=w)
            tb.tb_mx4_quantize(x, codes=c, scales=t)
        with torch.cuda.stream(main):
            tb.tb_mx4_dequantize(*s["W"], 640, s["H"])  # something of its own in front of the join
            main.wait_stream(side)
            tb.tb_moe(s["layer"], x, ids, w, y=ys[i], ws=s["ws"][0])
            tb.tb_mx4_gemm(*s["W"], c, t, s["T"], 640, s["H"], Y=Ys[i])
        side.wait_stream(main)


def test_joins_of_two_streams():
    s = setup()
    ref = want(s)
    n, T, H, k = s["n"], s["T"], s["H"], s["k"]
    bufs = (torch.empty((T, H), dtype=torch.bfloat16, device=DEV), torch.empty((T, k), dtype=torch.int32, device=DEV),
            torch.empty((T, k), device=DEV), torch.empty((T, H // 2), dtype=torch.uint8, device=DEV),
            torch.empty(512 * 4, dtype=torch.uint8, device=DEV), torch.empty((n, T, H), device=DEV), torch.empty((n, T, 640), device=DEV))
    busy = torch.ones(1 << 22, device=DEV)
    main, side = torch.cuda.Stream(), torch.cuda.Stream()

    def check():
        torch.cuda.synchronize()
        for i, (y, Y) in enumerate(ref):
            assert torch.equal(bufs[5][i], y) and torch.equal(bufs[6][i], Y), i
        bufs[5].fill_(-1), bufs[6].fill_(-1)
        torch.cuda.synchronize()
    for _ in range(5):
        run(s, main, side, bufs, busy)
        check()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=main):
        run(s, main, side, bufs, busy)
        main.wait_stream(side)
    for _ in range(5):
        graph.replay()
        check()
    assert tb.sync_status() == 0


FIRST = """
import torch
from decode_gemv_tb_b200 import tb
tb.load()
g = torch.Generator().manual_seed(1)
x = torch.randn((5, 512), generator=g).to(torch.bfloat16).cuda()
r = torch.randn((8, 512), generator=g).to(torch.bfloat16).cuda()
w = torch.randn((8 * 256, 512), generator=g).cuda()
d = torch.randn((8 * 512, 256), generator=g).cuda()
out = {}
def call():
    cw, cd, cx = tb.tb_mx4_quantize(w), tb.tb_mx4_quantize(d), tb.tb_mx4_quantize(x)
    layer = tb.moe_layer((*cw, tb.MX4), (*cw, tb.MX4), (*cd, tb.MX4), 8, 512, 256)
    y = tb.tb_moe(layer, x, *tb.tb_moe_route(x, r, 2))
    return y, tb.tb_mx4_gemm(*cw, *cx, 5, 2048, 512), tb.tb_mx4_dequantize(*cx, 5, 512)
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    out = call()
graph.replay()
torch.cuda.synchronize()
assert all(torch.equal(a, b) for a, b in zip(out, call())) and tb.sync_status() == 0
print("same")
"""


def test_first_calls_inside_a_capture():
    r = subprocess.run([sys.executable, "-c", FIRST], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "same" in r.stdout, r.stderr[-2000:]

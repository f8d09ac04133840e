"""The expert layer's entry points on the host: sizes and every refusal
before anything is launched; the tests' packing against the oracle's."""
import ctypes

import numpy as np
import pytest
import torch

from decode_gemv_tb_b200 import build as tbbuild
from decode_gemv_tb_b200 import tb
from tests import mx4_ref as R

A = 1 << 40  # aligned, never dereferenced
W = 1 << 40  # workspace size, never touched
ARG, SHAPE, ALIGN, UNSUPPORTED = 1, 2, 3, 4


@pytest.fixture(scope="module")
def lib():
    tbbuild.build()
    return tb.load()


def layer(**kw):
    d = dict(gate=A, up=A, down=A, gate_scales=A, up_scales=A, down_scales=A, gate_grid=0, up_grid=1, down_grid=2, E=4,
             H=256, I=128)
    d.update(kw)
    return tb.MoE(*(d[n] for n, _ in tb.MoE._fields_))


def test_workspace(lib):
    for T, k, H, I in ((1, 1, 128, 128), (1, 8, 2048, 768), (64, 16, 4096, 1536), (7, 3, 384, 640)):
        want = 2 * (-(-2 * T * k * I // 256) * 256 + 4 * H * max(T * k, 128))
        assert lib.tb_moe_workspace_bytes(ctypes.addressof(l := layer(H=H, I=I, E=16)), T, k) == want, l
    assert lib.tb_moe_workspace_bytes(0, 1, 1) == 0
    assert lib.tb_moe_workspace_bytes(ctypes.addressof(l := layer()), 65, 1) == 0


def test_moe_refusals(lib):
    def f(l=None, x=A, ldx=256, ids=A, w=A, T=4, k=2, y=A, dt=0, ldy=256, flags=0, ws=A, nws=W, **kw):
        d = layer(**kw)
        return lib.tb_moe(ctypes.addressof(d) if l is None else l, x, ldx, ids, w, T, k, y, dt, ldy, flags, ws, nws, 0)
    assert f(l=0) == ARG and f(x=0) == ARG and f(ids=0) == ARG and f(w=0) == ARG and f(y=0) == ARG and f(ws=0) == ARG
    for n in ("gate", "up", "down", "gate_scales", "up_scales", "down_scales"):
        assert f(**{n: 0}) == ARG and f(**{n: A + 8}) == ALIGN
    for n in ("gate_grid", "up_grid", "down_grid"):
        assert f(**{n: 3}) == UNSUPPORTED and f(**{n: 5}) == ARG and f(**{n: -1}) == ARG
    assert f(k=0) == ARG and f(k=17) == ARG and f(E=0) == ARG and f(E=513) == ARG and f(dt=2) == ARG and f(flags=1) == ARG
    assert f(nws=2 * (2048 + 4 * 256 * 128) - 1) == ARG
    assert f(T=0) == SHAPE and f(T=65) == SHAPE and f(H=200) == SHAPE and f(I=64) == SHAPE and f(I=0) == SHAPE
    assert f(H=(1 << 20) + 128, ldx=1 << 21, ldy=1 << 21) == SHAPE and f(ldx=248) == SHAPE and f(ldy=255) == SHAPE
    assert f(x=A + 8) == ALIGN and f(ldx=260) == ALIGN and f(ids=A + 2) == ALIGN and f(w=A + 1) == ALIGN
    assert f(y=A + 2) == ALIGN and f(ws=A + 64) == ALIGN


def test_route_refusals(lib):
    def f(x=A, ldx=64, r=A, T=3, E=8, H=64, k=2, ids=A, w=A):
        return lib.tb_moe_route(x, ldx, r, T, E, H, k, 1, ids, w, 0)
    assert f(x=0) == ARG and f(r=0) == ARG and f(ids=0) == ARG and f(w=0) == ARG
    assert f(E=0) == ARG and f(E=513) == ARG and f(k=0) == ARG and f(k=9) == ARG and f(k=17, E=32) == ARG
    assert f(T=0) == SHAPE and f(T=65537) == SHAPE and f(H=0) == SHAPE and f(H=60) == SHAPE and f(ldx=56) == SHAPE
    assert f(x=A + 8) == ALIGN and f(ldx=68) == ALIGN and f(r=A + 8) == ALIGN and f(ids=A + 2) == ALIGN
    assert f(H=1 << 17, ldx=1 << 17) == UNSUPPORTED


def test_scalar_entry_points_do_not_take_mx4(lib):
    assert tb.packed_bytes(tb.MX4, 4, 128) == 0
    assert lib.tb_gemv(A, tb.MX4, A, A, A, 0, 16, 128, A, W, 0) == ARG
    assert lib.tb_pack(A, 0, 16, 128, tb.MX4, A, A, 0, 0) == ARG


def test_binding_refusals():
    cpu = torch.zeros(2, 128, dtype=torch.bfloat16)
    with pytest.raises(tb.TBError):
        tb.tb_moe_route(cpu, cpu, 1)
    with pytest.raises(tb.TBError):
        tb.tb_moe_route(cpu.float(), cpu, 1)
    with pytest.raises(tb.TBError):
        tb.moe_layer(*((cpu, cpu, 0),) * 3, 1, 128, 128)


@pytest.mark.parametrize("grid", [0, 1, 2])
def test_packing_matches_the_oracle(oracle, grid):
    rng = np.random.default_rng(grid)
    lo, hi = {0: (-1, 1), 1: (-2, 1), 2: (-4, 3)}[grid]
    codes = rng.integers(lo, hi + 1, (5, 384))
    ones = np.full((5, 3), 0x3F80, dtype=np.uint16)  # scale 1: the weights are the codes
    packed, bad = oracle.pack(codes.astype(np.float32), grid, ones)
    assert bad == 0 and np.array_equal(np.asarray(packed).reshape(5, -1), R.pack_codes(codes, grid))


def test_reference_layer_by_hand():
    """One expert, one token: identity-like matrices give silu(x0) * x1 in every row of the second product."""
    H = I = 128
    wg, wu, wd = torch.zeros(I, H).double(), torch.zeros(I, H).double(), torch.zeros(H, I).double()
    wg[3, 0], wu[3, 1], wd[5, 3] = 1.0, 1.0, 2.0
    x = torch.zeros(1, H)
    x[0, 0], x[0, 1] = 2.0, 3.0
    y, _ = R.moe(wg, wu, wd, 1, x, torch.tensor([[0, -1]]), torch.tensor([[0.5, 9.0]]))
    want = 0.5 * 2.0 * (2.0 / (1 + np.exp(-2.0)) * 3.0)
    assert abs(y[0, 5].item() - want) < 1e-12 and y.abs().sum().item() == y[0, 5].abs().item()

"""Router weights and activations that are infinite or no number: the logits,
the order and the weights that the formulas give in 64-bit IEEE arithmetic."""
import math

import pytest
import torch

from decode_gemv_tb_b200 import tb

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    tb.load()


def reference(x, r, k, renorm):
    """(ids, weights) from products and sums written out (0 times an infinity is no number)."""
    l = (x.double().unsqueeze(1) * r.double().unsqueeze(0)).sum(-1)
    ids, weights = [], []
    for row in l.tolist():
        order = sorted(range(len(row)), key=lambda e: (math.isnan(row[e]), -row[e] if not math.isnan(row[e]) else 0, e))[:k]
        t = torch.tensor(row, dtype=torch.float64)
        p = torch.exp(t - t[order[0]])
        ids.append(order)
        weights.append(p[order] / (p[order] if renorm else p).sum())
    return torch.tensor(ids), torch.stack(weights)


@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("T,E,H,k", [(1, 5, 8, 5), (1, 40, 520, 6), (2, 40, 264, 6), (3, 33, 96, 33 // 2), (64, 256, 512, 8),
                                     (130, 40, 128, 3)])
def test_weights_that_are_no_numbers(T, E, H, k, renorm):
    g = torch.Generator().manual_seed(T * E + k)
    x = torch.randn((T, H), generator=g).to(torch.bfloat16)
    base = (torch.randn((E, H), generator=g) / H ** 0.5).to(torch.bfloat16)
    for what in range(6):
        r, xx = base.clone(), x.clone()
        if what == 0:
            r[E // 2, H // 2] = NAN  # one expert that ranks last
        elif what == 1:
            r[E - 1, 3] = INF  # first for half of the tokens, last for the others
        elif what == 2:
            r[0, H - 1], r[E - 2, 0] = -INF, INF
            r[E - 1, 1], r[E - 1, 2] = INF, -INF
        elif what == 3:
            r[1, 5] = INF
            xx[:, 5] = 0.0  # 0 times an infinity
        elif what == 4:
            r[:, 7] = NAN  # every expert
        else:
            r[2, 4] = INF
            xx[T // 2, 4] = -INF
            xx[0, 6] = NAN
        ids, w = tb.tb_moe_route(xx.to(DEV), r.to(DEV), k, renormalize=renorm)
        rid, rw = reference(xx, r, k, renorm)
        assert torch.equal(ids.long().cpu(), rid), what
        w, tol = w.double().cpu(), (E + 16) * 2.0 ** -22 * rw.nan_to_num(0.0) + 3 * 2.0 ** -149
        assert torch.equal(torch.isnan(w), torch.isnan(rw)), what
        assert torch.all((w.nan_to_num(0.0) - rw.nan_to_num(0.0)).abs() <= tol), what


def test_largest_finite_weights():
    """Next to the infinities, and sums far past fp32."""
    r = torch.zeros(6, 64, dtype=torch.bfloat16)
    big = torch.finfo(torch.bfloat16).max
    for e, v in enumerate((1.0, big, -big, big / 2, 3.0, 0.0)):
        r[e] = v
    x = torch.zeros(3, 64, dtype=torch.bfloat16)
    x[0], x[1, 9], x[2] = big, 2.0 ** -133, -1.0
    for renorm in (True, False):
        ids, w = tb.tb_moe_route(x.to(DEV), r.to(DEV), 6, renormalize=renorm)
        rid, rw = reference(x, r, 6, renorm)
        assert torch.equal(ids.long().cpu(), rid)
        assert torch.all((w.double().cpu() - rw).abs() <= 22 * 2.0 ** -22 * rw + 3 * 2.0 ** -149)

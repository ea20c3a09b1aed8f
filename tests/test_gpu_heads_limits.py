"""Norm and rotation of heads whose squares leave fp32's range, and of heads that have no norm."""
import numpy as np
import pytest
import torch

from oracle import decode as ref
from test_gpu_heads import HALF_STEP, TINY, f64, inputs, rope_table
from test_gpu_paged import DT

pytestmark = pytest.mark.gpu


def close(got, x, odt, weight, eps, rows, interleaved):
    """test_gpu_heads.py's bound, and roundings of 2^-150 where a step's result is subnormal: a product by the factor, times
    a weight of at most 3, and one by the weight, of both elements of a pair; two products and a sum of the rotation: 11."""
    assert np.abs(weight).max() <= 3
    want, size = ref.norm_rope(x, weight, eps, rows, interleaved)
    bound = 15 * 2.0 ** -24 * size + 11 * 2.0 ** -150
    bound = bound + HALF_STEP[odt] * (np.abs(want) + bound) + TINY[odt]
    err = np.abs(f64(got) - want)
    assert np.all(err <= bound), (eps, float((err / bound).max()))


@pytest.mark.parametrize("dt,odt", [("f32", "f32"), ("bf16", "bf16"), ("bf16", "f32"), ("f32", "f16")])
@pytest.mark.parametrize("dim,turn", [(8, 8), (64, 32), (72, 64), (128, 128), (256, 256)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_squares_outside_fp32(qpg, dt, odt, dim, turn, interleaved):
    """Heads of numbers so large that their squares pass fp32, or so small that they vanish in it and eps does not hide them, beside
    ordinary ones in the same warp."""
    n, hq, hk = 6, 9, 3
    q, k, wq, wk = inputs(n, hq, hk, dim, "f32", dim + turn)
    size = torch.tensor([1.0, 1e18, 3e19, 1e25, 1e37, 5e37, 1e-3, 1e-19, 1e-22, 1e-30, 1e-37, 3e-39], device="cuda")
    order = (torch.arange(12, device="cuda") + 5 * torch.arange(n, device="cuda")[:, None]) % 12
    q, k = q * size[order[:, :hq]][..., None], k * size[order[:, hq:]][..., None]
    q, k = q.to(DT[dt]), k.to(DT[dt])
    assert bool(torch.isfinite(q.float()).all()) and bool(torch.isfinite(k.float()).all())
    rope = rope_table(50, turn)
    pos = torch.tensor([0, 49, 3, 3, 17, 1], dtype=torch.int32, device="cuda")
    rows = f64(rope[pos.long()])
    qo, ko = (torch.empty((n, h, dim), dtype=DT[odt], device="cuda") for h in (hq, hk))
    for eps in (0.0, 1e-45, 1e-41, 1e-36, 1e-31, 1e-6, 1.0, 1e38):
        qpg.qpack_qk_norm_rope(q, k, wq, wk, eps=eps, rope=rope, interleaved=interleaved, pos=pos, q_out=qo, k_out=ko)
        for got, x, w in ((qo, q, wq), (ko, k, wk)):
            close(got, f64(x), odt, f64(w), float(np.float32(eps)), rows, interleaved)
    assert qpg.qpack_fetch_fault_flags() == 0


def test_heads_that_have_no_norm(qpg):
    """Zeros with an eps of 0 are 0 / 0; infinities and NaN stay in their heads; neither touches its neighbours in a warp."""
    dim, w = 64, torch.ones(64, device="cuda")
    q = torch.randn((2, 8, dim), device="cuda")
    want, _ = qpg.qpack_qk_norm_rope(q, None, w, eps=0.0)
    bad = q.clone()
    bad[0, 1], bad[0, 3, 5], bad[1, 2, 7], bad[1, 6, 0], bad[1, 6, 1] = 0.0, float("inf"), float("nan"), float("inf"), float("nan")
    got, _ = qpg.qpack_qk_norm_rope(bad, None, w, eps=0.0)
    hit = torch.zeros((2, 8), dtype=torch.bool, device="cuda")
    for at in ((0, 1), (0, 3), (1, 2), (1, 6)):
        hit[at] = True
    assert torch.equal(got[~hit], want[~hit])
    assert torch.isnan(got[0, 1]).all() and torch.isnan(got[1, 2]).all() and torch.isnan(got[1, 6]).all()
    assert torch.isnan(got[0, 3, 5]) and (got[0, 3, :5] == 0).all() and (got[0, 3, 6:] == 0).all()

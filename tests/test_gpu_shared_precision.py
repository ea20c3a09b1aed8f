"""Attention over shared prefixes keeps the bits that attention without sharing keeps: over 8-bit and fp16 caches a weight is off by 2^-22,
whatever the output's type, so that what a 16-bit output shows is its own rounding.

The tolerance is that of attention without sharing (derived in test_gpu_paged.py), with nothing added for a term of 11 bits. Queries
have two elements that are not zero, so of a score's additions two count instead of D."""
import pytest
import torch

from test_gpu_paged import DT, SPLIT, ULP, make_pool
from test_gpu_shared import forked, i32, tables_of
from test_gpu_shared_long import held

pytestmark = pytest.mark.gpu


def check(out, odt, kind, q, pool, tab, lens, prefix, scale):
    D, H = q.shape[2], pool.heads
    ka, va = held(pool, tab[0], prefix)
    for b, L in enumerate(lens):
        kb, vb = held(pool, tab[b], L)
        k, v = torch.cat([ka, kb[:, prefix:]], 1), torch.cat([va, vb[:, prefix:]], 1)
        qr = q[b].double().view(H, -1, D)
        assert int((qr != 0).sum(-1).max()) <= 2
        w = (qr @ k.transpose(1, 2) * scale).softmax(-1)
        want, mean = w @ v, w @ v.abs()
        dx = (qr.abs() @ k.abs().transpose(1, 2)).amax(-1, keepdim=True) * scale * (SPLIT[kind] + (2 + 8) * 2.0 ** -23)
        # second terms of weights below fp16's normal numbers are off by 2^-25 where the largest is 2^7 or more: 2^-32 of it
        tol = mean * (3 * dx + 2.0 ** -22 + 2.0 ** -20 + (L / 8 + 64 + 160) * 2.0 ** -23) + 2.0 ** -32 * v.abs().sum(1)[:, None]
        tol = tol + (want.abs() + tol) * ULP[odt] + 2.0 ** -25
        err = (out[b].double().view_as(want) - want).abs()
        assert (err <= tol).all(), (b, float((err / tol).max()))


@pytest.mark.parametrize("kind", ["i8", "f16"])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("qdt,odt", [("f16", "f16"), ("f32", "f16"), ("f16", "bf16"), ("f32", "f32")])
@pytest.mark.parametrize("rows,G,prefix", [(3, 4, 30), (40, 8, 97)])
def test_weights_keep_their_bits(qpg, kind, D, qdt, odt, rows, G, prefix):
    """Weights of all sizes, of which a few tokens have most."""
    first, pref, lens, tab, pages = forked(qpg, [rows], [prefix], [5, 0, 31], 16, seed=41)
    pool = make_pool(qpg, kind, 1, pages, 2, 16, D, 41)
    q = torch.zeros((rows, 2 * G, D), device="cuda")
    q[:, :, 3], q[:, :, D - 9] = torch.randn((2, rows, 2 * G), device="cuda") * 2
    q = q.to(DT[qdt])
    out = torch.empty(q.shape, dtype=DT[odt], device="cuda")
    qpg.qpack_kv_attend_shared(pool, 0, tables_of(qpg, tab, lens), q, i32(first), i32(pref), scale=1.0, out=out)
    assert qpg.qpack_fetch_fault_flags() == 0
    check(out, odt, kind, q, pool, tab, lens, prefix, 1.0)


@pytest.mark.parametrize("kind", ["i8", "f16"])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_a_token_that_dominates_behind_a_lagging_maximum(qpg, kind, D):
    """One token has nearly all weight and lies up to 2^8 above a maximum that stays where it is: the weight that is multiplied and
    the one that is added up have to be the same. Key heads enough that a block has six tiles or more of one of them, and
    the token is behind the first two of most."""
    rows, G, T, tok = 4, 8, 16, 64 if D == 256 else 128
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    tiles = 16
    H, prefix = -(-6 * sms // tiles), tiles * tok
    first, pref, lens, tab, pages = forked(qpg, [rows], [prefix], [0], T, seed=42)
    pool = make_pool(qpg, kind, 1, pages, H, T, D, 42)
    t = torch.arange(prefix, device="cuda")
    page = torch.from_numpy(tab[0]).cuda().long()[t // T]
    ramp = torch.full((prefix,), -20.0, device="cuda")      # scores, times a query near 1
    ramp[::tok] = 0.0
    ramp[prefix - 2] = 5.0
    if kind == "i8":
        pool.k_scales[0, page, :, t % T, 0] = (ramp.abs() / 127).half()[:, None]
        pool.k[0, page, :, t % T, 5] = (127 * torch.sign(ramp)).to(torch.int8)[:, None]
    else:
        pool.k[0, page, :, t % T, 5] = ramp.half()[:, None]
    q = torch.zeros((rows, H * G, D), device="cuda")
    q[:, :, 5] = torch.linspace(0.9, 1.08, rows * H * G, device="cuda").view(rows, H * G)
    for odt in ("f16", "bf16"):
        out = torch.empty(q.shape, dtype=DT[odt], device="cuda")
        qpg.qpack_kv_attend_shared(pool, 0, tables_of(qpg, tab, lens), q, i32(first), i32(pref), scale=1.0, out=out)
        assert qpg.qpack_fetch_fault_flags() == 0
        check(out, odt, kind, q, pool, tab, lens, prefix, 1.0)

"""GPU: norms of rows whose squares leave fp32's range, in the rotation call and in the cache write."""
import numpy as np
import pytest
import torch

import sparse_attention_07_b200 as sa
from _latent import D_C, D_R, F32_NORM, gen, latent64, make_cache, norm64, pool_rows, rope64, rope_mass, tables

pytestmark = pytest.mark.gpu
DEV = "cuda"

# The arithmetic of the norm is F32_NORM's, and three products more (2^-24 each).
ARITH = F32_NORM + 3 * 2.0 ** -24


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("size,eps", [(1e18, 1e-6), (1e30, 1e-6), (5e37, 1e-6), (1e30, 1e20), (1e-18, 0.0), (1e-25, 0.0),
                                      (1e-37, 0.0), (1e-20, 1e-39)])
@pytest.mark.parametrize("tokens,H,D,inter", [(5, 3, 128, False), (5, 3, 192, True), (700, 33, 128, False), (3, 2, 100, False)])
def test_rows_far_from_one(tokens, H, D, inter, size, eps, dtype):
    """Every third head has values of the given size, and one element far below the others; the rest are ordinary."""
    g = gen(D, DEV)
    q = torch.randn(tokens, H, D, generator=g, device=DEV)
    q.view(-1, D)[::3] *= size
    q.view(-1, D)[::3, 1] *= 2.0 ** -20
    q = q.to(dtype)
    w = 1 + 0.2 * torch.randn(D, generator=g, device=DEV)
    cos, sin = tables(50, D // 2, DEV)  # half of the dims rotate
    rot = D // 2 // 2 * 2
    pos = torch.randint(0, 50, (tokens,), generator=g, device=DEV, dtype=torch.int32)
    got, _ = sa.qk_norm_rope(q, None, cos, sin, pos, q_weight=w, eps=eps, rope_start=0, interleaved=inter)
    y = norm64(q, w, eps)
    mass = torch.cat((rope_mass(y[..., :rot], inter), y[..., rot:].abs()), dim=-1)
    p = pos.long()
    want = torch.cat((rope64(y[..., :rot], cos[p][:, None], sin[p][:, None], inter), y[..., rot:]), dim=-1)
    bound = ARITH * mass + 2.0 ** -126  # (nothing need be kept below fp32's normal range)
    if dtype == torch.bfloat16:
        bound = bound + 2.0 ** -8 * want.abs()
    assert ((got.double() - want).abs() <= bound).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_infinities_and_nans_stay_what_the_formula_makes_of_them(dtype):
    """A row with an infinity: rsqrt(inf) = 0, so its finite values are 0 and the infinity NaN; a NaN spreads over its row."""
    q = torch.ones(3, 2, 128, device=DEV)
    q[0, 0, 5] = torch.inf
    q[1, 1, 7] = torch.nan
    q = q.to(dtype)
    for D in (128, 100):
        got, _ = sa.qk_norm_rope(q[..., :D], None, None, None, None)
        want = norm64(q[..., :D], None, 1e-6)
        assert torch.equal(torch.isnan(got), torch.isnan(want)) and torch.isnan(got[0, 0, 5])
        ok = ~torch.isnan(want)
        assert ((got.double() - want).abs() <= (2.0 ** -8 + F32_NORM) * want.abs())[ok].all()


@pytest.mark.parametrize("q8", [True, False])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("size,eps", [(1e18, 1e-6), (1e30, 1e-6), (5e37, 1e-6), (1e-25, 0.0), (1e-37, 0.0)])
def test_written_rows_far_from_one(q8, dtype, size, eps):
    n = 9
    cache = make_cache((64,), q8, 3, DEV)
    g = gen(n, DEV)
    c = torch.randn(n, D_C, generator=g, device=DEV)
    c[::2] *= size
    c = c.to(dtype)
    kr = torch.zeros(n, D_R, device=DEV, dtype=dtype)
    w = 1 + 0.2 * torch.randn(D_C, generator=g, device=DEV)
    cos, sin = tables(64, D_R, DEV)
    slots = torch.arange(n, device=DEV, dtype=torch.int32)
    sa.mla_cache_write(c, kr, cache["c_cache"], cache["kr_cache"], slots, cache["pps"], cos, sin, weight=w, eps=eps,
                       c_scale=cache["c_scale"], page_table=cache["page_table"], seq_of_row=torch.zeros_like(slots))
    y = norm64(c, w, eps)
    got = latent64(cache, pool_rows(cache, 0, np.arange(n)))
    # a storage rounding is half a step: bf16 2^-8, e4m3 2^-4 of the value or 2^-10 of a scale below max / 224
    block = y.abs().unflatten(-1, (4, 128)).amax(-1).repeat_interleave(128, dim=-1)
    step = 2.0 ** -4 * y.abs() + 2.0 ** -10 / 224 * block * (1 + 2.0 ** -10) if q8 else 2.0 ** -8 * y.abs()
    assert ((got - y).abs() <= step + 2 * ARITH * y.abs()).all()
    assert sa.check_device_error() == 0

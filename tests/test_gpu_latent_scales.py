"""GPU: the smallest scale bytes of the quantised cache, in the read and in attention."""
import numpy as np
import pytest
import torch

import sparse_attention_07_b200 as sa
from _latent import D_C, D_R, SCALE, attend64, gen, latent64, make_cache, pool_rows

pytestmark = pytest.mark.gpu
DEV = "cuda"


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a).astype(np.int32)).to(DEV)


@pytest.mark.parametrize("kind", [t for t in (torch.uint8, getattr(torch, "float8_e8m0fnu", None)) if t])
def test_read_and_attention_agree_on_the_smallest_bytes(kind):
    """Every code under the bytes 0 .. 11 (0 is 2^-127, as float8_e8m0fnu has it): the read is the exact
    value rounded once to bf16, and a row attended to alone comes out as it is read."""
    n = 12
    codes = torch.tensor([b for b in range(256) if b & 127 != 127], dtype=torch.uint8, device=DEV)
    cache = make_cache((n,), True, 1, DEV)
    rows = pool_rows(cache, 0, np.arange(n))
    shift = torch.arange(n, device=DEV)[:, None] * 37
    cache["c_cache"].view(torch.uint8)[rows] = codes[(torch.arange(D_C, device=DEV)[None] + shift) % len(codes)]
    cache["c_scale"][rows] = torch.arange(n, device=DEV).to(torch.uint8)[:, None]
    scale = cache["c_scale"].view(kind)
    got = sa.mla_cache_read(cache["c_cache"], cache["kr_cache"], dev(np.arange(n)[None]), cache["pps"], c_scale=scale,
                            page_table=cache["page_table"])[0][0]
    exact = latent64(cache, rows)
    step = torch.exp2(torch.floor(torch.log2(exact.abs().clamp(min=2.0 ** -126))) - 7)  # of bf16 at the value
    want = torch.round(exact / step) * step
    assert torch.equal(got.double(), want)
    g = gen(2, DEV)
    q = torch.randn(n, 16, D_C, generator=g, device=DEV).bfloat16()
    qr = torch.randn(n, 16, D_R, generator=g, device=DEV).bfloat16()
    out = sa.sparse_mla_decode(q, qr, cache["c_cache"], cache["kr_cache"], dev(np.arange(n)[:, None]), SCALE, cache["pps"],
                               page_table=cache["page_table"], seq_of_row=torch.zeros(n, dtype=torch.int32, device=DEV),
                               c_scale=scale)
    assert torch.equal(out.double(), want[:, None].expand(n, 16, D_C))


@pytest.mark.parametrize("low,high", [(8, 12), (1, 4), (40, 44)])
def test_attention_at_the_smallest_scale_bytes(low, high):
    """Values around 2^-115 (and 2^-122, 2^-83).  The bound is that of the other
    attention tests, with nothing absolute but the formats' own steps: half a step of
    bf16's subnormals (2^-134) per value, and fp32's smallest step for each of the
    n products and their sum.  So an output halved, doubled or zeroed fails."""
    n = 200
    cache = make_cache((n,), True, 4, DEV)
    g = gen(low, DEV)
    cache["c_scale"].copy_(torch.randint(low, high, cache["c_scale"].shape, generator=g, device=DEV))
    q = torch.randn(1, 128, D_C, generator=g, device=DEV).bfloat16()
    qr = torch.randn(1, 128, D_R, generator=g, device=DEV).bfloat16()
    out = sa.sparse_mla_decode(q, qr, cache["c_cache"], cache["kr_cache"], dev(np.arange(n))[None], SCALE, cache["pps"],
                               page_table=cache["page_table"], c_scale=cache["c_scale"])
    want, _, spread, mass = attend64(q[0], qr[0], cache, 0, np.arange(n))
    slack = 2.0 ** -134 + n * 2.0 ** -149
    assert slack < 2.0 ** -6 * want.square().mean().sqrt()
    bound = (2.0 ** -7 + 2.0 ** -16 * mass) * spread + slack
    err = (out[0].double() - want).abs()
    assert (err <= bound).all()
    for wrong in (0.0, 0.5, 2.0):  # such an output would be seen
        assert ((out[0].double() * wrong - want).abs() > bound).float().mean() > 0.5

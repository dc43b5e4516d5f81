"""GPU: drafted rows with infinities and no NaN, and who sees them."""
import numpy as np
import pytest
import torch

import sparse_attention_07_b200 as sa
from _latent import D_C, D_R, SCALE, attend64, check_attention, gen, make_cache, pool_rows

pytestmark = pytest.mark.gpu
DEV = "cuda"


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a).astype(np.int32)).to(DEV)


def spoil(cache, row, dim, sign):
    """An infinite value in one dim of a pool row (e4m3: its 128-dim block overflows bf16), and no NaN."""
    if cache["c_scale"] is None:
        cache["c_cache"][row, dim] = sign * torch.inf
    else:
        codes = cache["c_cache"].view(torch.uint8)
        codes[row, dim // 128 * 128:dim // 128 * 128 + 128] = 0
        codes[row, dim] = 0x7E if sign > 0 else 0xFE  # +-448 at 2^127
        cache["c_scale"][row, dim // 128] = 254


@pytest.mark.parametrize("q8", [True, False])
@pytest.mark.parametrize("H", [128, 16, 3])
@pytest.mark.parametrize("past", [0, 63, 70, 1500])
@pytest.mark.parametrize("dim", [0, 130, 317, 511])
def test_an_infinite_drafted_row_reaches_the_tokens_that_see_it(past, H, q8, dim):
    """Heads whose query has either sign in the infinite dim (scores +inf and
    -inf): all of them are NaN, in output and lse, for the tokens that see the
    row, and the others are as without it."""
    T, bad = 5, 2
    cache = make_cache((past + T,), q8, past + H, DEV)
    spoil(cache, pool_rows(cache, 0, [past + bad]), dim, 1 if dim % 2 else -1)
    g = gen(H + dim, DEV)
    q = torch.randn(1, T, H, D_C, generator=g, device=DEV).bfloat16()
    q[..., dim] = 1.0
    q[:, :, ::2, dim] = -1.0
    qr = torch.randn(1, T, H, D_R, generator=g, device=DEV).bfloat16()
    mask = np.eye(T, dtype=np.uint8)[None]
    mask[0, 4, bad] = 1
    out = torch.zeros(1, T, H, D_C, device=DEV)
    lse = torch.zeros(1, T, H, device=DEV)
    sa.tree_mla_decode(q, qr, cache["c_cache"], cache["kr_cache"], dev([past]), torch.from_numpy(mask).to(DEV), past + T,
                       SCALE, cache["pps"], page_table=cache["page_table"], c_scale=cache["c_scale"], out=out, lse=lse)
    for i in range(T):
        if mask[0, i, bad]:
            assert torch.isnan(out[0, i]).all() and torch.isnan(lse[0, i]).all(), f"token {i} sees the row"
        else:
            pos = np.concatenate((np.arange(past), past + np.flatnonzero(mask[0, i])))
            check_attention(out[0, i], lse[0, i], attend64(q[0, i], qr[0, i], cache, 0, pos), f"token {i}")
    assert sa.check_device_error() == 0


@pytest.mark.parametrize("q8", [True, False])
def test_an_infinite_rope_key_weighs_nothing_or_everything(q8):
    """An infinity among a drafted row's RoPE dims only: the row's values are finite, so a score of -inf is a weight of 0."""
    past, T, H, bad = 90, 3, 32, 1
    cache = make_cache((past + T,), q8, 5, DEV)
    cache["kr_cache"][pool_rows(cache, 0, [past + bad]), 7] = torch.inf
    g = gen(1, DEV)
    q = torch.randn(1, T, H, D_C, generator=g, device=DEV).bfloat16()
    qr = torch.randn(1, T, H, D_R, generator=g, device=DEV).bfloat16()
    qr[..., 7] = -1.0
    qr[:, :, 1::2, 7] = 1.0
    out = sa.tree_mla_decode(q, qr, cache["c_cache"], cache["kr_cache"], dev([past]), None, past + T, SCALE, cache["pps"],
                             page_table=cache["page_table"], c_scale=cache["c_scale"])
    check_attention(out[0, 0], None, attend64(q[0, 0], qr[0, 0], cache, 0, np.arange(past + 1)), "token 0")
    for i in (1, 2):
        pos = np.array([p for p in range(past + i + 1) if p != past + bad])
        check_attention(out[0, i, ::2], None, attend64(q[0, i, ::2], qr[0, i, ::2], cache, 0, pos), f"token {i}, -inf")
        assert torch.isnan(out[0, i, 1::2]).all(), f"token {i}, +inf"
    assert sa.check_device_error() == 0

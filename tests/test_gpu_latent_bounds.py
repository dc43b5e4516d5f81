"""GPU: a length bound far above the rows' lengths, and rows of one call on both sides of a split."""
import numpy as np
import pytest
import torch

import sparse_attention_07_b200 as sa
from _latent import D_C, D_R, SCALE, attend64, check_attention, gen, make_cache

pytestmark = pytest.mark.gpu
DEV = "cuda"


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a).astype(np.int32)).to(DEV)


@pytest.mark.parametrize("bf16_out", [False, True])
@pytest.mark.parametrize("rows,L_max", [(90, 1 << 20), (90, 1 << 23), (3, 1 << 20), (90, 4096)])
def test_dense_rows_of_very_different_lengths(rows, L_max, bf16_out):
    """Lengths from nothing to 2^19 positions of a table whose pages are all the same one: a page's row j stands
    n // 64 times among n positions, once more if j < n % 64."""
    lens = [(0, 1, 63, 64, 65, 1000, 1 << 18, (1 << 18) + 1, (1 << 19) + 5, 300)[r % 10] for r in range(rows)]
    if L_max == 4096:
        lens = [min(n, 4096) for n in lens]
    g = gen(rows, DEV)
    c = torch.randn(64, D_C, generator=g, device=DEV).to(torch.float8_e4m3fn)
    scale = torch.full((64, 4), 127, dtype=torch.uint8, device=DEV)
    kr = torch.randn(64, D_R, generator=g, device=DEV).bfloat16()
    pages = (max(lens) + 63) // 64
    q = torch.randn(rows, 8, D_C, generator=g, device=DEV).bfloat16()
    qr = torch.randn(rows, 8, D_R, generator=g, device=DEV).bfloat16()
    out = torch.full((rows, 8, D_C), torch.nan, device=DEV, dtype=torch.bfloat16 if bf16_out else torch.float32)
    lse = torch.full((rows, 8), torch.nan, device=DEV)
    sa.dense_mla_decode(q, qr, c, kr, dev(lens), L_max, SCALE, pages, page_table=torch.zeros(1, pages, dtype=torch.int32, device=DEV),
                        seq_of_row=torch.zeros(rows, dtype=torch.int32, device=DEV), out=out, lse=lse, c_scale=scale)
    v, k64 = c.double(), kr.double()
    for r, n in enumerate(lens):
        if n == 0:
            assert (out[r] == 0).all() and torch.isneginf(lse[r]).all()
            continue
        count = torch.full((64,), n // 64, device=DEV) + (torch.arange(64, device=DEV) < n % 64)
        z = (q[r].double() @ v.T + qr[r].double() @ k64.T) * SCALE
        mass = ((q[r].double().abs() @ v.abs().T + qr[r].double().abs() @ k64.abs().T) * SCALE).max().item()
        z = z + torch.log(count.double())
        p = torch.softmax(z, dim=1)
        check_attention(out[r], lse[r], (p @ v, torch.logsumexp(z, dim=1), p @ v.abs(), mass), f"row {r} of {n}")
    assert sa.check_device_error() == 0


@pytest.mark.parametrize("q8", [True, False])
@pytest.mark.parametrize("B,T,H", [(80, 2, 64), (1, 3, 128), (5, 40, 16)])
def test_trees_under_a_generous_bound(B, T, H, q8):
    rng = np.random.Generator(np.random.PCG64(B))
    past, draft = rng.integers(0, 900, B), rng.integers(0, T + 1, B)
    cache = make_cache(past + draft, q8, B, DEV, extra_pages=1, junk_nan=True)
    g = gen(B, DEV)
    q = torch.randn(B, T, H, D_C, generator=g, device=DEV).bfloat16()
    qr = torch.randn(B, T, H, D_R, generator=g, device=DEV).bfloat16()
    out = torch.full((B, T, H, D_C), -7.0, device=DEV)
    lse = torch.full((B, T, H), -7.0, device=DEV)
    sa.tree_mla_decode(q, qr, cache["c_cache"], cache["kr_cache"], dev(past), None, 1 << 21, SCALE, cache["pps"],
                       n_draft=dev(draft), c_scale=cache["c_scale"], page_table=cache["page_table"], out=out, lse=lse)
    for b in range(B):
        for i in range(draft[b]):
            check_attention(out[b, i], lse[b, i], attend64(q[b, i], qr[b, i], cache, b, np.arange(past[b] + i + 1)), f"{b},{i}")
        assert (out[b, draft[b]:] == -7).all() and (lse[b, draft[b]:] == -7).all()
    assert sa.check_device_error() == 0

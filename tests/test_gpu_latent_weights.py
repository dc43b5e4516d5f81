"""GPU: the weights that the latent-cache attention applies sum to 1."""
import numpy as np
import pytest
import torch

import sparse_attention_07_b200 as sa
from _latent import D_C, D_R, SCALE, gen

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("rows,H,n", [(1, 16, 2), (1, 128, 100), (2, 64, 5000), (80, 128, 200), (160, 32, 64)])
@pytest.mark.parametrize("call", ["sparse", "dense", "tree", "tree_bf16"])
def test_equal_values_come_out_as_they_are(call, rows, H, n):
    """Every latent row holds one value: whatever the scores (they differ by the RoPE keys), the output is that
    value.  The weights are rounded to bf16, but so is their sum: what is left are fp32 sums of n terms (n 2^-24
    each, the tensor cores' truncated 2^-27 of it), and a few roundings of the division and the merge."""
    g = gen(n, DEV)
    pages = -(-n // 64)
    c = torch.full((rows * pages * 64, D_C), 1.375, device=DEV)
    c = c.bfloat16() if call == "tree_bf16" else c.to(torch.float8_e4m3fn)
    scale = None if call == "tree_bf16" else torch.full((len(c), 4), 127, dtype=torch.uint8, device=DEV)
    kr = torch.randn(len(c), D_R, generator=g, device=DEV).bfloat16()
    q = torch.randn(rows, H, D_C, generator=g, device=DEV).bfloat16()
    qr = torch.randn(rows, H, D_R, generator=g, device=DEV).bfloat16()
    kw = dict(c_scale=scale)
    length = torch.full((rows,), n, dtype=torch.int32, device=DEV)
    if call == "sparse":
        idx = torch.from_numpy(np.random.default_rng(n).permutation(n).astype(np.int32)).to(DEV).expand(rows, n).contiguous()
        out = sa.sparse_mla_decode(q, qr, c, kr, idx, SCALE, pages, **kw)
    elif call == "dense":
        out = sa.dense_mla_decode(q, qr, c, kr, length, n, SCALE, pages, **kw)
    else:
        out = sa.tree_mla_decode(q[:, None], qr[:, None], c, kr, length - 1, None, n, SCALE, pages, **kw)[:, 0]
    assert ((out - 1.375).abs() <= 1.375 * (n * 2.0 ** -24 + 2.0 ** -20)).all()

"""GPU: calls of the latent-cache attention that take long or have very many rows."""
import math

import pytest
import torch

import sparse_attention_07_b200 as sa
from _latent import D_C, D_R, SCALE, check_attention, gen

pytestmark = pytest.mark.gpu
DEV = "cuda"


def one_page():
    """A quantised cache of one page whose row j is 1 + j % 2 in every dim, RoPE keys 0."""
    c = torch.ones(64, D_C, device=DEV)
    c[1::2] = 2
    return dict(c=c.to(torch.float8_e4m3fn), s=torch.full((64, 4), 127, dtype=torch.uint8, device=DEV),
                kr=torch.zeros(64, D_R, device=DEV, dtype=torch.bfloat16))


def test_an_sm_pair_at_work_for_seconds():
    """One row per SM pair over 205 million positions (every page of the table is the same one) and an L_max
    that asks for no split: some five seconds in one pair, longer than any time limit of a wait.  All weights
    are 1, and each thread's sum of them, a multiple of 16 below 2^28, is exact in fp32, so the lse is the
    logarithm of the length (2^-16 as in the other tests).  The aggregation of so many keys outruns the tensor
    cores' fp32 accumulation: of the output, that it is between the values."""
    tiles = 3_200_000
    n = 64 * tiles
    rows = torch.cuda.get_device_properties(0).multi_processor_count // 2
    cache = one_page()
    table = torch.zeros(1, tiles, dtype=torch.int32, device=DEV)
    seq = torch.zeros(rows, dtype=torch.int32, device=DEV)
    q = torch.zeros(rows, 1, D_C, device=DEV, dtype=torch.bfloat16)
    qr = torch.zeros(rows, 1, D_R, device=DEV, dtype=torch.bfloat16)
    lse = torch.zeros(rows, 1, device=DEV)
    out = sa.dense_mla_decode(q, qr, cache["c"], cache["kr"], torch.full((rows,), n, dtype=torch.int32, device=DEV), 100,
                              SCALE, tiles, page_table=table, seq_of_row=seq, lse=lse, c_scale=cache["s"])
    assert sa.check_device_error() == 0
    assert (lse - math.log(n)).abs().max() <= 2.0 ** -16 * (1 + math.log(n))
    assert (out > 0).all() and (out <= 2).all()


def test_very_many_rows_of_one_key():
    """Thousands of rows per SM pair, one slot each: every output is its key's row."""
    rows = 320_000
    cache = one_page()
    idx = (torch.arange(rows, device=DEV, dtype=torch.int32) % 65 - 1)[:, None].contiguous()  # -1: nothing
    q = torch.ones(rows, 1, D_C, device=DEV, dtype=torch.bfloat16)
    qr = torch.zeros(rows, 1, D_R, device=DEV, dtype=torch.bfloat16)
    out = torch.empty(rows, 1, D_C, device=DEV, dtype=torch.bfloat16)
    sa.sparse_mla_prefill(q, qr, cache["c"], cache["kr"], idx, SCALE, 1, seq_of_row=torch.zeros_like(idx[:, 0]), out=out,
                          c_scale=cache["s"])
    assert sa.check_device_error() == 0
    want = torch.where(idx < 0, 0, 1 + idx % 2)
    assert (out[:, 0] == want).all()


@pytest.mark.parametrize("call", ["dense", "tree", "tree_bf16"])
@pytest.mark.parametrize("n", [1 << 18, (1 << 20) + 64, 1 << 22])
def test_long_sums_of_one_sign(call, n):
    """A row for every SM pair over a million and more positions (every page the same) whose values are all
    positive: within the bound of the short rows."""
    rows = torch.cuda.get_device_properties(0).multi_processor_count // 2
    g = gen(n % 1000, DEV)
    v = torch.rand(64, D_C, generator=g, device=DEV) + 0.5
    c = v.bfloat16() if call == "tree_bf16" else v.to(torch.float8_e4m3fn)
    scale = None if call == "tree_bf16" else torch.full((64, 4), 127, dtype=torch.uint8, device=DEV)
    kr = torch.randn(64, D_R, generator=g, device=DEV).bfloat16()
    table = torch.zeros(1, n // 64, dtype=torch.int32, device=DEV)
    seq = torch.zeros(rows, dtype=torch.int32, device=DEV)
    q = (torch.randn(rows, 1, D_C, generator=g, device=DEV) * 0.1).bfloat16()
    qr = (torch.randn(rows, 1, D_R, generator=g, device=DEV) * 0.3).bfloat16()
    length = torch.full((rows,), n, dtype=torch.int32, device=DEV)
    lse = torch.zeros(rows, 1, device=DEV)
    kw = dict(page_table=table, seq_of_row=seq, c_scale=scale)
    if call == "dense":
        out = sa.dense_mla_decode(q, qr, c, kr, length, n, SCALE, n // 64, lse=lse, **kw)
    else:  # a chain of one drafted token, the last position
        out = sa.tree_mla_decode(q[:, None], qr[:, None], c, kr, length - 1, None, n, SCALE, n // 64,
                                 lse=lse.view(rows, 1, 1), **kw)[:, 0]
    # every position j stands n / 64 times: the softmax over the page, and log(n / 64) more
    v, q, qr = c.double(), q[:, 0].double(), qr[:, 0].double()
    z = (q @ v.T + qr @ kr.double().T) * SCALE
    mass = ((q.abs() @ v.abs().T + qr.abs() @ kr.double().abs().T) * SCALE).max().item()
    p = torch.softmax(z, dim=1)
    want = (p @ v, torch.logsumexp(z, dim=1) + math.log(n // 64), p @ v.abs(), mass)
    check_attention(out[:, 0], lse[:, 0], want, f"{call} over {n}")
    assert sa.check_device_error() == 0

"""GPU: per-head norm and rotation of queries and keys against the definition in fp64."""
import pytest
import torch

import sparse_attention_07_b200 as sa
from _latent import F32_NORM, gen, norm64, rope64, rope_mass, tables

pytestmark = pytest.mark.gpu
DEV = "cuda"


def check(got, x, w, cos, sin, pos, eps, norm, start, interleaved):
    y = norm64(x, w, eps) if norm else (x.double() if w is None else x.double() * w.double())
    mass = y.abs()
    if cos is not None:
        a, b = start, start + 2 * cos.shape[1]
        p = pos.long()
        part = y[..., a:b]
        mass = torch.cat((mass[..., :a], rope_mass(part, interleaved), mass[..., b:]), dim=-1)
        y = torch.cat((y[..., :a], rope64(part, cos[p][:, None], sin[p][:, None], interleaved), y[..., b:]), dim=-1)
    bound = F32_NORM * mass + 2.0 ** -120
    if got.dtype == torch.bfloat16:
        bound = bound + 2.0 ** -8 * y.abs()
    err = (got.double() - y).abs()
    assert (err <= bound).all(), f"error {(err - bound).max().item():.3e} over its bound"


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("tokens,Hq,Hk,D,rot,start,inter,weight,norm", [
    (1, 1, 0, 64, 64, 0, False, True, True),
    (8, 32, 4, 128, 128, 0, False, True, True),
    (8, 32, 4, 128, 128, 0, True, False, True),
    (33, 128, 1, 192, 64, 128, True, True, True),
    (33, 7, 3, 96, 48, 48, False, True, True),
    (5, 3, 3, 256, 32, 224, False, True, True),
    (700, 33, 5, 128, 64, 0, False, True, True),     # several heads per thread, a ragged last group
    (700, 33, 5, 128, 64, 0, True, True, True),
    (9, 5, 2, 64, 64, 0, True, False, False),        # rotation only
    (9, 5, 2, 128, 0, 0, False, True, True),         # norm only
    (6, 4, 2, 100, 20, 40, False, True, True),       # pieces of eight dims straddle the halves
    (6, 4, 2, 30, 6, 3, True, True, True),
    (3, 2, 1, 512, 512, 0, False, True, True),
    (3, 2, 1, 2, 2, 0, False, True, True),
    (3, 2, 1, 1, 0, 0, False, True, True),
])
def test_norm_rope(dtype, tokens, Hq, Hk, D, rot, start, inter, weight, norm):
    g = gen(tokens * 7 + D + rot, DEV)
    q = (torch.randn(tokens, Hq, D, generator=g, device=DEV) * 3).to(dtype)
    k = (torch.randn(tokens, Hk, D, generator=g, device=DEV) * 0.2).to(dtype) if Hk else None
    qw = 1 + 0.2 * torch.randn(D, generator=g, device=DEV) if weight else None
    kw = 1 + 0.2 * torch.randn(D, generator=g, device=DEV) if weight else None
    cos, sin = tables(1000, rot, DEV) if rot else (None, None)
    pos = torch.randint(0, 1000, (tokens,), generator=g, device=DEV, dtype=torch.int32) if rot else None
    qo, ko = sa.qk_norm_rope(q, k, cos, sin, pos, q_weight=qw, k_weight=kw, eps=1e-6, norm=norm, rope_start=start,
                             interleaved=inter)
    check(qo, q, qw, cos, sin, pos, 1e-6, norm, start, inter)
    assert qo.dtype == dtype
    if Hk:
        check(ko, k, kw, cos, sin, pos, 1e-6, norm, start, inter)
    else:
        assert ko is None
    assert sa.check_device_error() == 0


@pytest.mark.parametrize("tokens", [4, 900])
@pytest.mark.parametrize("shift", [0, 1])
def test_views_and_in_place(tokens, shift):
    """q and k as views of one projection (shift: not 16-byte aligned), rotated
    in place; the dims between and behind them stay as they were."""
    D, Hq, Hk = 128, 12, 2
    g = gen(tokens, DEV)
    buf = torch.randn(tokens, (Hq + Hk) * D + 40, generator=g, device=DEV).bfloat16()
    before = buf.clone()
    at = 8 + shift
    q = buf[:, at:at + Hq * D].unflatten(1, (Hq, D))
    k = buf[:, at + Hq * D + 8:at + Hq * D + 8 + Hk * D].unflatten(1, (Hk, D))
    q0, k0 = q.clone(), k.clone()
    cos, sin = tables(tokens, D, DEV)
    pos = torch.arange(tokens, device=DEV, dtype=torch.int32)
    want = sa.qk_norm_rope(q0, k0, cos, sin, pos)
    sa.qk_norm_rope(q, k, cos, sin, pos, q_out=q, k_out=k)
    check(q, q0, None, cos, sin, pos, 1e-6, True, 0, False)
    check(k, k0, None, cos, sin, pos, 1e-6, True, 0, False)
    if not shift:
        assert torch.equal(q, want[0]) and torch.equal(k, want[1])
    touched = torch.zeros_like(buf, dtype=torch.bool)
    touched[:, at:at + Hq * D] = True
    touched[:, at + Hq * D + 8:at + Hq * D + 8 + Hk * D] = True
    assert torch.equal(buf[~touched], before[~touched])


def test_head_major_and_broadcast_inputs():
    """Heads before tokens in memory, and one key row shared by every token."""
    g = gen(3, DEV)
    q = torch.randn(6, 50, 64, generator=g, device=DEV).bfloat16().transpose(0, 1)
    k = torch.randn(1, 2, 64, generator=g, device=DEV).bfloat16().expand(50, 2, 64)
    cos, sin = tables(64, 64, DEV)
    pos = torch.arange(50, device=DEV, dtype=torch.int32)
    qo, ko = sa.qk_norm_rope(q, k, cos, sin, pos)
    check(qo, q, None, cos, sin, pos, 1e-6, True, 0, False)
    check(ko, k, None, cos, sin, pos, 1e-6, True, 0, False)


def test_zero_rows_large_values_and_no_tokens():
    q = torch.zeros(2, 3, 128, device=DEV)
    q[1] = 1e15
    qo, _ = sa.qk_norm_rope(q, None, None, None, None)
    assert (qo[0] == 0).all()
    check(qo, q, None, None, None, None, 1e-6, True, 0, False)
    e = torch.empty(0, 3, 128, device=DEV)
    assert sa.qk_norm_rope(e, None, None, None, None)[0].shape == e.shape


def test_bad_position_is_reported():
    q = torch.randn(3, 2, 64, device=DEV)
    cos, sin = tables(10, 64, DEV)
    pos = torch.tensor([0, 10, -1], device=DEV, dtype=torch.int32)
    qo, _ = sa.qk_norm_rope(q, None, cos, sin, pos)
    assert sa.check_device_error() == 0x900
    check(qo, q, None, cos, sin, torch.zeros(3, device=DEV, dtype=torch.int32), 1e-6, True, 0, False)
    assert sa.check_device_error() == 0


def test_refusals():
    q = torch.randn(3, 2, 64, device=DEV)
    cos, sin = tables(10, 64, DEV)
    pos = torch.zeros(3, device=DEV, dtype=torch.int32)
    with pytest.raises(TypeError):
        sa.qk_norm_rope(q.half(), None, cos, sin, pos)
    with pytest.raises(TypeError):
        sa.qk_norm_rope(q, q.bfloat16(), cos, sin, pos)
    with pytest.raises(ValueError):
        sa.qk_norm_rope(q, None, cos, sin, pos[:2])
    with pytest.raises(ValueError):
        sa.qk_norm_rope(q.transpose(1, 2), None, cos, sin, pos)
    with pytest.raises(ValueError):
        sa.qk_norm_rope(q, None, cos, sin, pos, q_out=q.new_empty(3, 1, 64).expand(3, 2, 64))
    with pytest.raises(sa.SparseAttnError):
        sa.qk_norm_rope(q[..., :32], None, cos, sin, pos)  # more rotated dims than the head has
    with pytest.raises(sa.SparseAttnError):
        sa.qk_norm_rope(q, None, cos, sin, pos, rope_start=2)
    with pytest.raises(sa.SparseAttnError):
        sa.qk_norm_rope(q, None, cos, sin, pos, eps=-1.0)

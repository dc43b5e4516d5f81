"""GPU: the latent cache written (normalised, rotated, quantised) and read back, against fp64."""
import numpy as np
import pytest
import torch

import sparse_attention_07_b200 as sa
from _latent import (D_C, D_R, F32_NORM, gen, latent64, make_cache, norm64, pool_rows, rope64, rope_mass, tables)

pytestmark = pytest.mark.gpu
DEV = "cuda"


def inputs(tokens, dtype, seed, spread=False):
    g = gen(seed, DEV)
    c = torch.randn(tokens, D_C, generator=g, device=DEV) * 3
    if spread:  # blocks of very different magnitudes, one of zeros
        c = c * torch.exp2(torch.randint(-20, 20, (tokens, 4), generator=g, device=DEV).float()).repeat_interleave(128, 1)
        c[0, 128:256] = 0
    kr = torch.randn(tokens, D_R, generator=g, device=DEV)
    return c.to(dtype), kr.to(dtype), 1 + 0.2 * torch.randn(D_C, generator=g, device=DEV)


def check_rows(cache, rows, c, kr, w, norm, cos, sin, pos, inter):
    y = norm64(c, w, 1e-6) if norm else (c.double() if w is None else c.double() * w.double())
    got = latent64(cache, rows)
    f32 = F32_NORM * y.abs()
    if cache["c_scale"] is None:
        bound = 2.0 ** -8 * y.abs() + f32
    else:
        scale = torch.exp2(cache["c_scale"][rows].double() - 127)
        amax = y.abs().unflatten(-1, (4, 128)).amax(-1)
        live = amax > 0
        assert (448 * scale >= amax * (1 - 2.0 ** -18))[live].all(), "a value does not fit its scale"
        assert (224 * scale <= amax * (1 + 2.0 ** -18))[live].all(), "the scale is not the smallest"
        # half an e4m3 step: 2^-4 of the value, or of the smallest normal 2^-6 below it
        step = torch.maximum(y.abs() * 2.0 ** -4, scale.repeat_interleave(128, 1) * 2.0 ** -10)
        bound = step * (1 + 2.0 ** -10) + f32
    err = (got - y).abs()
    assert (err <= bound).all(), f"latent error {(err - bound).max().item():.3e} over its bound"
    want = rope64(kr, cos[pos], sin[pos], inter)
    err = (cache["kr_cache"][rows].double() - want).abs()
    assert (err <= 2.0 ** -8 * want.abs() + F32_NORM * rope_mass(kr, inter)).all(), "RoPE key"


@pytest.mark.parametrize("q8", [True, False])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("tokens,inter,norm,weight,pad", [
    (1, True, True, True, 0), (5, False, True, True, 16), (130, True, True, False, 0), (66, False, False, True, 32),
    (3, True, False, False, 0)])
def test_write(q8, dtype, tokens, inter, norm, weight, pad):
    """Tokens of three sequences at scattered slots; every other row of the pool stays as it was."""
    lens = (200, 64, 130)
    cache = make_cache(lens, q8, tokens, DEV, c_pad=pad)
    rng = np.random.Generator(np.random.PCG64(tokens))
    every = [(b, p) for b, n in enumerate(lens) for p in range(n)]
    pick = rng.permutation(len(every))[:tokens]
    seq, slot = np.array([every[i][0] for i in pick]), np.array([every[i][1] for i in pick])
    rows = pool_rows(cache, seq, slot)
    c, kr, w = inputs(tokens, dtype, tokens + q8, spread=not norm)
    w = w if weight else None
    cos, sin = tables(500, D_R, DEV)
    pos = torch.from_numpy(rng.integers(0, 500, size=tokens)).to(DEV)
    before = {k: cache[k].clone() for k in ("c_cache", "kr_cache", "c_scale") if cache[k] is not None}
    dev = lambda a: torch.from_numpy(a.astype(np.int32)).to(DEV)  # noqa: E731
    sa.mla_cache_write(c, kr, cache["c_cache"], cache["kr_cache"], dev(slot), cache["pps"], cos, sin,
                       positions=pos.to(torch.int32), weight=w, norm=norm, interleaved=inter,
                       c_scale=cache["c_scale"], page_table=cache["page_table"], seq_of_row=dev(seq))
    check_rows(cache, rows, c, kr, w, norm, cos, sin, pos, inter)
    others = torch.ones(len(cache["kr_cache"]), dtype=torch.bool, device=DEV)
    others[rows] = False
    for k, was in before.items():
        assert torch.equal(cache[k][others].view(torch.uint8), was[others].view(torch.uint8)), k
    # read back: exactly the cached values, as bf16
    want = latent64(cache, rows)
    got, gkr = sa.mla_cache_read(cache["c_cache"], cache["kr_cache"], dev(slot)[:, None], cache["pps"],
                                 c_scale=cache["c_scale"], page_table=cache["page_table"], seq_of_row=dev(seq))
    assert torch.equal(got[:, 0].double(), want) and torch.equal(gkr[:, 0], cache["kr_cache"][rows])
    assert sa.check_device_error() == 0


def test_write_defaults_padding_and_fused_view():
    """One token per sequence at its own slot (positions = slots, contiguous
    pages), c and kr as views of one projection, padded tokens skipped, scales
    as float8_e8m0fnu."""
    lens = (65, 3, 128, 64)
    cache = make_cache(lens, True, 5, DEV, paged=False)
    buf = torch.randn(4, D_C + D_R, device=DEV).bfloat16()
    c, kr = buf[:, :D_C], buf[:, D_C:]
    slots = torch.tensor([64, -1, 127, 0], device=DEV, dtype=torch.int32)
    cos, sin = tables(200, D_R, DEV)
    before = cache["c_cache"].clone()
    sa.mla_cache_write(c, kr, cache["c_cache"], cache["kr_cache"], slots, cache["pps"], cos, sin,
                       c_scale=cache["c_scale"].view(torch.float8_e8m0fnu))
    live = [0, 2, 3]
    rows = pool_rows(cache, np.array(live), np.array([64, 127, 0]))
    check_rows(cache, rows, c[live], kr[live], None, True, cos, sin, slots[live].long(), False)
    same = torch.ones(len(before), dtype=torch.bool, device=DEV)
    same[rows] = False
    assert torch.equal(before[same].view(torch.uint8), cache["c_cache"][same].view(torch.uint8))
    assert sa.check_device_error() == 0


def test_scale_borders_ties_and_non_finite_blocks():
    """Maxima on and next to 448 * 2^n, values on the ties of e4m3, and blocks
    with NaN or infinity (byte 255, read back as NaN, their neighbours whole)."""
    c = torch.zeros(1, D_C, device=DEV)
    c[0, 0], c[0, 1] = 448.0, 17.0            # scale 1; 17 lies between 16 and 18: ties to 16
    c[0, 128] = float(np.nextafter(np.float32(448), np.float32(1e9)))  # scale 2
    c[0, 129] = 38.0                          # 38 / 2 = 19: between 18 and 20, ties to 20
    c[0, 256], c[0, 257] = 1e-30, float("nan")
    c[0, 384], c[0, 385] = float("inf"), 1.0
    cache = make_cache((64,), True, 1, DEV)
    cos, sin = tables(64, D_R, DEV)
    slots = torch.zeros(1, dtype=torch.int32, device=DEV)
    sa.mla_cache_write(c, torch.zeros(1, D_R, device=DEV), cache["c_cache"], cache["kr_cache"], slots, 1, cos, sin,
                       norm=False, c_scale=cache["c_scale"], page_table=cache["page_table"])
    row = pool_rows(cache, 0, [0])
    assert cache["c_scale"][row].tolist() == [[127, 128, 255, 255]]
    got = sa.mla_cache_read(cache["c_cache"], cache["kr_cache"], slots[:, None], 1, c_scale=cache["c_scale"],
                            page_table=cache["page_table"])[0][0, 0]
    assert got[0] == 448 and got[1] == 16 and got[128] == 448 and got[129] == 40
    assert (got[2:128] == 0).all() and (got[130:256] == 0).all() and torch.isnan(got[256:]).all()


@pytest.mark.parametrize("q8", [True, False])
@pytest.mark.parametrize("rows,k", [(1, 1), (3, 5), (2, 64), (5, 131)])
def test_read(q8, rows, k):
    lens = [100 + 37 * r for r in range(rows)]
    cache = make_cache(lens, q8, k, DEV, junk_nan=True, c_pad=16)
    rng = np.random.Generator(np.random.PCG64(k))
    idx = np.stack([rng.integers(0, n, size=k) for n in lens]).astype(np.int32)
    idx[rng.random(idx.shape) < 0.2] = -1
    idx[0, 0] = lens[0] - 1
    got, kr = sa.mla_cache_read(cache["c_cache"], cache["kr_cache"], torch.from_numpy(idx).to(DEV), cache["pps"],
                                c_scale=cache["c_scale"], page_table=cache["page_table"])
    for r in range(rows):
        live = torch.from_numpy(idx[r] >= 0).to(DEV)
        at = pool_rows(cache, r, np.maximum(idx[r], 0))
        want = torch.where(live[:, None], latent64(cache, at), 0.0)
        assert torch.equal(got[r].double(), want)
        assert torch.equal(kr[r], torch.where(live[:, None], cache["kr_cache"][at], torch.zeros((), device=DEV).bfloat16()))
    assert sa.check_device_error() == 0


def test_every_code_and_scale_reads_exactly():
    """All e4m3 codes but the two NaNs under every scale a written block can have."""
    codes = torch.tensor([b for b in range(256) if b & 127 != 127], dtype=torch.uint8, device=DEV)
    c = torch.zeros(4 * 64, D_C, dtype=torch.uint8, device=DEV)
    c[:, :] = codes[torch.arange(D_C, device=DEV) % len(codes)]
    scale = torch.arange(1, 255, device=DEV).to(torch.uint8)
    s = scale[torch.arange(4 * 64, device=DEV) % 247]  # bytes 1 .. 247
    cache = dict(c_cache=c.view(torch.float8_e4m3fn), c_scale=s[:, None].expand(-1, 4).contiguous(),
                 kr_cache=torch.zeros(256, D_R, device=DEV).bfloat16())
    idx = torch.arange(256, device=DEV, dtype=torch.int32)[None]
    got = sa.mla_cache_read(cache["c_cache"], cache["kr_cache"], idx, 4, c_scale=cache["c_scale"])[0][0]
    want = latent64(cache, idx[0].long())
    # rounded to bf16's range: 8 significant bits hold every product, subnormals and overflow aside
    assert torch.equal(got.double(), want.float().bfloat16().double())


def test_bad_slots_and_indices_are_reported():
    cache = make_cache((64, 64), True, 2, DEV)
    cache["page_table"][1, 0] = 99  # a page outside the pool
    cos, sin = tables(64, D_R, DEV)
    before = cache["c_cache"].clone()
    c, kr, w = inputs(2, torch.bfloat16, 1)
    for slots in ([64, -1], [-1, 0]):  # past the page table; on the bad page
        sa.mla_cache_write(c, kr, cache["c_cache"], cache["kr_cache"],
                           torch.tensor(slots, device=DEV, dtype=torch.int32), 1, cos, sin,
                           positions=torch.zeros(2, dtype=torch.int32, device=DEV), c_scale=cache["c_scale"],
                           page_table=cache["page_table"])
        assert sa.check_device_error() == 0x700
        assert torch.equal(before.view(torch.uint8), cache["c_cache"].view(torch.uint8))
        got = sa.mla_cache_read(cache["c_cache"], cache["kr_cache"],
                                torch.tensor(slots, device=DEV, dtype=torch.int32)[:, None], 1,
                                c_scale=cache["c_scale"], page_table=cache["page_table"])[0]
        assert sa.check_device_error() == 0x700
        bad = slots.index(max(slots))
        assert torch.equal(got[bad, 0].double(), latent64(cache, torch.zeros(1, dtype=torch.long, device=DEV))[0])
    sa.mla_cache_write(c, kr, cache["c_cache"], cache["kr_cache"], torch.tensor([3, -1], device=DEV, dtype=torch.int32),
                       1, cos, sin, positions=torch.tensor([64, 0], dtype=torch.int32, device=DEV),
                       c_scale=cache["c_scale"], page_table=cache["page_table"])
    assert sa.check_device_error() == 0x900


def test_refusals():
    cache = make_cache((64, 64), True, 2, DEV)
    c, kr, w = inputs(2, torch.bfloat16, 1)
    cos, sin = tables(64, D_R, DEV)
    slots = torch.zeros(2, dtype=torch.int32, device=DEV)

    def write(**kw):
        a = dict(c=c, kr=kr, c_cache=cache["c_cache"], kr_cache=cache["kr_cache"], slots=slots, pages_per_seq=1,
                 cos=cos, sin=sin, c_scale=cache["c_scale"], page_table=cache["page_table"])
        a.update(kw)
        sa.mla_cache_write(**a)

    for kw in (dict(c_scale=None), dict(c_cache=cache["c_cache"].bfloat16()), dict(slots=slots[:1]),
               dict(kr=kr[:, :32]), dict(cos=cos[:, :16]), dict(page_table=cache["page_table"][:1]),
               dict(c_cache=cache["c_cache"][:100], kr_cache=cache["kr_cache"][:100], c_scale=cache["c_scale"][:100])):
        with pytest.raises(ValueError):
            write(**kw)
    for kw in (dict(slots=slots.long()), dict(c=c.half(), kr=kr.half()), dict(weight=w.bfloat16()),
               dict(kr_cache=cache["kr_cache"].float())):
        with pytest.raises(TypeError):
            write(**kw)
    with pytest.raises(sa.SparseAttnError):
        write(c=torch.randn(2, D_C + 1, device=DEV).bfloat16()[:, 1:])  # rows not 16-byte aligned
    with pytest.raises(sa.SparseAttnError):
        write(eps=-1.0)
    with pytest.raises(ValueError):
        sa.mla_cache_read(cache["c_cache"], cache["kr_cache"], slots[:, None], 1, page_table=cache["page_table"])

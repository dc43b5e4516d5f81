"""Helpers of the latent-cache tests: seeded caches, and the definitions in
fp64 (plain torch on whatever device the tensors are on)."""
import numpy as np
import torch

PAGE, D_C, D_R, BLK = 64, 512, 64, 128
SCALE = 1.0 / 192 ** 0.5


def gen(seed, device):
    g = torch.Generator(device=device)
    g.manual_seed(seed)
    return g


def decode_e4m3(codes):
    """The value of e4m3 codes (uint8) from their fields, in fp64."""
    b = codes.long()
    e, m = (b >> 3) & 15, b & 7
    mag = torch.where(e > 0, (8 + m).double() * torch.exp2((e - 10).double()), m.double() * 2.0 ** -9)
    return torch.where(b >= 128, -mag, mag)


def latent64(cache, rows):
    """fp64 latent rows of the given pool rows."""
    if cache["c_scale"] is None:
        return cache["c_cache"][rows].double()
    s = cache["c_scale"].view(torch.uint8)[rows].long()
    scale = torch.where(s == 255, torch.nan, torch.exp2((s - 127).double()))
    return decode_e4m3(cache["c_cache"].view(torch.uint8)[rows]) * scale.repeat_interleave(BLK, dim=-1)


def make_cache(lens, q8, seed, device, extra_pages=0, junk_nan=False, c_pad=0, paged=True):
    """Pools for sequences of the given lengths behind a shuffled page table.
    junk_nan: every pool row that is not a position of a sequence holds NaN.
    c_pad: extra elements between latent rows (a strided pool)."""
    g = gen(seed, device)
    rng = np.random.Generator(np.random.PCG64(seed))
    need = [max(1, -(-int(n) // PAGE)) + extra_pages for n in lens]
    total, most = sum(need), max(need)
    if paged:
        perm = rng.permutation(total)
        table = np.full((len(lens), most), -1, dtype=np.int32)
        at = 0
        for b, n in enumerate(need):
            table[b, :n] = perm[at:at + n]
            at += n
        page_table = torch.from_numpy(table).to(device)
    else:
        total = len(lens) * most
        table = np.arange(total).reshape(len(lens), most)
        page_table = None
    rows = total * PAGE
    wide = torch.randn((rows, D_C + c_pad), generator=g, device=device)
    scale = None
    if q8:
        c = (wide * 96).clamp(-448, 448).to(torch.float8_e4m3fn)
        scale = torch.randint(118, 122, (rows, 4), generator=g, device=device, dtype=torch.int32).to(torch.uint8)
    else:
        c = wide.bfloat16()
    c = c[:, :D_C]
    kr = torch.randn((rows, D_R), generator=g, device=device).bfloat16()
    if junk_nan:
        used = torch.zeros(rows, dtype=torch.bool)
        for b, n in enumerate(lens):
            p = np.arange(n)
            used[torch.from_numpy(table[b, p // PAGE].astype(np.int64) * PAGE + p % PAGE)] = True
        junk = (~used).to(device)
        kr[junk] = torch.nan
        if q8:
            scale[junk] = 255
        else:
            c[junk] = torch.nan
    return dict(c_cache=c, c_scale=scale, kr_cache=kr, page_table=page_table, table=table, pps=most)


def pool_rows(cache, seq, pos):
    pos = np.asarray(pos, dtype=np.int64)
    rows = cache["table"][seq, pos // PAGE].astype(np.int64) * PAGE + pos % PAGE
    return torch.from_numpy(rows).to(cache["kr_cache"].device)


def attend64(q, qr, cache, seq, pos, scale=SCALE):
    """softmax attention of q [H, 512], qr [H, 64] over positions `pos`, in fp64:
    (out, lse, sum_j p_j |c_j|, the largest sum_i |q_i c_i| scale)."""
    q, qr = q.double(), qr.double()
    if len(pos) == 0:
        z = torch.zeros_like(q)
        return z, torch.full((q.shape[0],), -torch.inf, dtype=torch.float64, device=q.device), z, 0.0
    rows = pool_rows(cache, seq, pos)
    c, kr = latent64(cache, rows), cache["kr_cache"][rows].double()
    s = (q @ c.T + qr @ kr.T) * scale
    mass = ((q.abs() @ c.abs().T + qr.abs() @ kr.abs().T) * abs(scale)).max().item()
    p = torch.softmax(s, dim=1)
    return p @ c, torch.logsumexp(s, dim=1), p @ c.abs(), mass


def check_attention(got, lse, want, what):
    """Element bound against fp64.  The probabilities may be rounded to bf16
    (half a step, 2^-8 relative) in numerator and normaliser alike, so the
    output is off by at most 2 * 2^-8 * sum_j p_j |c_j|; the 576-term scores
    are accumulated in fp32 (at most 2^-17 of their absolute mass), which moves
    each probability by that in relative terms, twice; a bf16 output adds half
    a step of the result.  lse: the score error, plus 2^-16 for its own
    exponentials, sum and logarithm."""
    out64, lse64, spread, mass = want
    eps_z = mass * 2.0 ** -17
    bound = (2.0 ** -7 + 2 * eps_z) * spread + 2.0 ** -30
    if got.dtype == torch.bfloat16:
        bound = bound * (1 + 2.0 ** -8) + 2.0 ** -8 * out64.abs()
    err = (got.double() - out64).abs()
    assert torch.isfinite(got).all(), f"{what}: non-finite output"
    assert (err <= bound).all(), f"{what}: error {(err - bound).max().item():.3e} over its bound"
    if lse is not None:
        empty = torch.isneginf(lse64)
        assert torch.equal(torch.isneginf(lse), empty), f"{what}: empty rows differ"
        if not empty.all():
            d = (lse.double() - lse64)[~empty].abs().max().item()
            assert d <= eps_z + 2.0 ** -16 * (1 + lse64[~empty].abs().max().item()), f"{what}: lse off by {d:.3e}"


def rope64(x, cos, sin, interleaved):
    x, cos, sin = x.double(), cos.double(), sin.double()
    out = torch.empty_like(x)
    half = x.shape[-1] // 2
    for i in range(half):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        out[..., a] = x[..., a] * cos[..., i] - x[..., b] * sin[..., i]
        out[..., b] = x[..., b] * cos[..., i] + x[..., a] * sin[..., i]
    return out


def rope_mass(x, interleaved):
    """|x_a| + |x_b| of every rotated pair: what the two products of an output can reach."""
    x = x.double().abs()
    half = x.shape[-1] // 2
    if interleaved:
        return x.unflatten(-1, (half, 2)).sum(-1).repeat_interleave(2, dim=-1)
    s = x[..., :half] + x[..., half:]
    return torch.cat((s, s), dim=-1)


def norm64(x, w, eps):
    x = x.double()
    y = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
    return y if w is None else y * w.double()


def tables(n_pos, rot, device, base=10000.0):
    inv = base ** (-torch.arange(0, rot, 2, device=device, dtype=torch.float64) / rot)
    a = torch.arange(n_pos, device=device, dtype=torch.float64)[:, None] * inv
    return a.cos().float(), a.sin().float()


# fp32 arithmetic of norm and rotation: at most 32 roundings of 2^-24 (the sum
# of squares 16 + 5 adds, halved by the root; 4 for rsqrt's 2 ulp; the products)
F32_NORM = 2.0 ** -19
EMPTY_POS = np.empty(0, dtype=np.int64)

"""GPU: the latent-cache operators used together, captured, far into a large
pool, at the ends of the scale range, and when a wait runs out."""
import numpy as np
import pytest
import torch

import sparse_attention_07_b200 as sa
from _latent import (D_C, D_R, F32_NORM, SCALE, attend64, check_attention, gen, latent64, make_cache, norm64, pool_rows,
                     rope64, rope_mass, tables)

pytestmark = pytest.mark.gpu
DEV = "cuda"


def ints(a):
    return torch.from_numpy(np.ascontiguousarray(a).astype(np.int32)).to(DEV)


class Step:
    """Two sequences: prefixes written, one decode step over a selection, five drafted tokens verified."""

    LENS, H, K, T = (600, 130), 32, 128, 5
    H_I, D_I = 4, 64

    def __init__(self, q8):
        self.q8 = q8
        self.pages = [(n + 1 + self.T + 63) // 64 for n in self.LENS]
        total = sum(self.pages)
        perm = np.random.Generator(np.random.PCG64(1)).permutation(total)
        self.table = np.full((2, max(self.pages)), -1, dtype=np.int32)
        self.table[0, :self.pages[0]] = perm[:self.pages[0]]
        self.table[1, :self.pages[1]] = perm[self.pages[0]:]
        self.pps = max(self.pages)
        rows = total * 64
        self.cache = dict(
            c_cache=torch.zeros(rows, D_C, device=DEV, dtype=torch.float8_e4m3fn if q8 else torch.bfloat16),
            c_scale=torch.zeros(rows, 4, device=DEV, dtype=torch.uint8) if q8 else None,
            kr_cache=torch.zeros(rows, D_R, device=DEV, dtype=torch.bfloat16), page_table=ints(self.table),
            table=self.table, pps=self.pps)
        self.cos, self.sin = tables(700, D_R, DEV)
        # slots, rotary positions and sequences of the prefix, of the step's tokens and of the drafts
        self.seq = np.repeat([0, 1], self.LENS)
        self.slot = np.concatenate([np.arange(n) for n in self.LENS])
        depth = np.array([0, 1, 1, 2, 2])
        parent = (-1, 0, 0, 1, 2)
        self.mask = np.zeros((2, self.T, self.T), dtype=np.uint8)
        for i, p in enumerate(parent):
            if p >= 0:
                self.mask[:, i] = self.mask[:, p]
            self.mask[:, i, i] = 1
        n = np.array(self.LENS)
        self.plan = dict(
            seq=ints(self.seq), slot=ints(self.slot), now=ints(n), past=ints(n + 1), seq_d=ints(np.repeat([0, 1], self.T)),
            slot_d=ints((n[:, None] + 1 + np.arange(self.T)).ravel()), pos_d=ints((n[:, None] + 1 + depth).ravel()),
            mask=torch.from_numpy(self.mask).to(DEV))
        self.pos_d = n[:, None] + 1 + depth
        self.x = {}
        tokens = sum(self.LENS)
        for name, shape in dict(c=(tokens, D_C), kr=(tokens, D_R), c1=(2, D_C), kr1=(2, D_R), cd=(2 * self.T, D_C),
                                krd=(2 * self.T, D_R), q=(2, self.H, D_C), qr=(2, self.H, D_R),
                                qd=(2, self.T, self.H, D_C), qrd=(2 * self.T, self.H, D_R)).items():
            self.x[name] = torch.empty(*shape, device=DEV, dtype=torch.bfloat16)
        self.x["q_idx"] = torch.empty(2, self.H_I, self.D_I, device=DEV)
        self.x["k_idx"] = torch.empty(rows, self.D_I, device=DEV)
        self.w_idx = torch.rand(2, self.H_I, generator=gen(7, DEV), device=DEV)
        self.weight = torch.rand(D_C, generator=gen(8, DEV), device=DEV) + 0.5

    def fill(self, seed):
        g = gen(seed, DEV)
        for t in self.x.values():
            t.copy_(torch.randn(t.shape, generator=g, device=DEV))

    def write(self, c, kr, slots, positions, seq):
        sa.mla_cache_write(c, kr, self.cache["c_cache"], self.cache["kr_cache"], slots, self.pps, self.cos, self.sin,
                           positions=positions, weight=self.weight, interleaved=True, c_scale=self.cache["c_scale"],
                           page_table=self.cache["page_table"], seq_of_row=seq)

    def run(self):
        x, p, cache = self.x, self.plan, self.cache
        kw = dict(page_table=cache["page_table"], c_scale=cache["c_scale"])
        self.write(x["c"], x["kr"], p["slot"], None, p["seq"])
        self.write(x["c1"], x["kr1"], p["now"], None, None)
        qr, _ = sa.qk_norm_rope(x["qr"], None, self.cos, self.sin, p["now"], norm=False, interleaved=True)
        scores = sa.index_scores(x["q_idx"], self.w_idx, x["k_idx"], p["past"], self.pps, page_table=cache["page_table"])
        idx = sa.topk_select(scores, p["past"], self.K)
        if self.q8:
            out = sa.sparse_mla_decode(x["q"], qr, cache["c_cache"], cache["kr_cache"], idx, SCALE, self.pps, **kw)
        else:
            out = sa.sparse_mla_decode(x["q"], qr, cache["c_cache"], cache["kr_cache"], idx, SCALE, self.pps,
                                       page_table=cache["page_table"])
        self.write(x["cd"], x["krd"], p["slot_d"], p["pos_d"], p["seq_d"])
        qrd, _ = sa.qk_norm_rope(x["qrd"], None, self.cos, self.sin, p["pos_d"], norm=False, interleaved=True)
        tree = sa.tree_mla_decode(x["qd"], qrd.view(2, self.T, self.H, D_R), cache["c_cache"], cache["kr_cache"],
                                  p["past"], p["mask"], 640, SCALE, self.pps, **kw)
        return dict(qr=qr, idx=idx, out=out, qrd=qrd, tree=tree)


def check_rotated(got, x, cos, sin, what):
    """One rounding to bf16 (2^-8 of the value), and fp32 arithmetic (F32_NORM of what the products reach)."""
    want, mass = rope64(x, cos, sin, True), rope_mass(x, True)
    err = (got.double() - want).abs()
    assert (err <= 2.0 ** -8 * want.abs() + 2 * F32_NORM * mass + 2.0 ** -130).all(), what


@pytest.mark.parametrize("q8", [True, False])
def test_a_decode_step_and_its_drafts(q8):
    s = Step(q8)
    s.fill(3)
    got = s.run()
    x, cache = s.x, s.cache
    assert sa.check_device_error() == 0
    # the cache: latent rows within the quantiser's half step, RoPE keys within bf16's
    for c, kr, seq, slot, pos in ((x["c"], x["kr"], s.seq, s.slot, s.slot),
                                  (x["c1"], x["kr1"], np.arange(2), np.array(s.LENS), np.array(s.LENS)),
                                  (x["cd"], x["krd"], np.repeat([0, 1], s.T),
                                   (np.array(s.LENS)[:, None] + 1 + np.arange(s.T)).ravel(), s.pos_d.ravel())):
        rows = torch.from_numpy(s.table[seq, slot // 64].astype(np.int64) * 64 + slot % 64).to(DEV)
        want = norm64(c, s.weight, 1e-6)
        have = latent64(cache, rows)
        # e4m3: 2^-4 of the value, or 2^-10 of the scale, which is below max / 224 (a power of two, 448 s / 2 < max)
        block = want.abs().unflatten(-1, (4, 128)).amax(-1).repeat_interleave(128, dim=-1)
        step = 2.0 ** -4 * want.abs() + 2.0 ** -10 / 224 * block * (1 + 2.0 ** -10) if q8 else 2.0 ** -8 * want.abs()
        assert ((have - want).abs() <= step + 2 * F32_NORM * want.abs()).all(), "latent rows"
        at = torch.from_numpy(pos).to(DEV)
        check_rotated(cache["kr_cache"][rows], kr, s.cos[at], s.sin[at], "RoPE keys")
    n = torch.tensor(s.LENS, device=DEV)
    check_rotated(got["qr"], x["qr"], s.cos[n][:, None], s.sin[n][:, None], "queries")
    for b, length in enumerate(s.LENS):
        idx = got["idx"][b].cpu().numpy()
        assert (np.diff(idx) > 0).all() and idx[0] >= 0 and idx[-1] <= length and len(idx) == s.K
        check_attention(got["out"][b], None, attend64(x["q"][b], got["qr"][b], cache, b, idx), f"step {b}")
        for i in range(s.T):
            pos = np.concatenate((np.arange(length + 1), length + 1 + np.flatnonzero(s.mask[b, i])))
            check_attention(got["tree"][b, i], None,
                            attend64(x["qd"][b, i], got["qrd"].view(2, s.T, s.H, D_R)[b, i], cache, b, pos), f"draft {b},{i}")


@pytest.mark.parametrize("q8", [True, False])
def test_the_step_captured_and_on_another_stream(q8):
    """The whole run captured in one graph and replayed on new contents, and
    run on a stream of its own, gives the eager run's bits."""
    s = Step(q8)
    want = {}
    for seed in (1, 2):
        s.fill(seed)
        want[seed] = {k: v.clone() for k, v in s.run().items()}
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        s.fill(1)
        got = s.run()
    side.synchronize()
    assert all(torch.equal(got[k], want[1][k]) for k in got)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = s.run()
    for seed in (2, 1, 2):
        s.fill(seed)
        graph.replay()
        torch.cuda.synchronize()
        for k in got:
            assert torch.equal(got[k], want[seed][k]), k
    assert sa.check_device_error() == 0


def test_offsets_past_32_bits():
    """Rows whose byte offsets pass 2^32 in the codes and in the RoPE keys, and
    heads whose element offsets pass 2^31."""
    n = 200
    pages = (1 << 23) // 64 + 4  # 512-byte codes: the last four pages lie past 2^32
    c = torch.empty(pages * 64, D_C, device=DEV, dtype=torch.float8_e4m3fn)
    scale = torch.empty(pages * 64, 4, device=DEV, dtype=torch.uint8)
    kr = torch.empty(pages * 64, 512, device=DEV, dtype=torch.bfloat16)[:, :D_R]  # rows of 1024 bytes
    table = np.arange(pages - 1, pages - 5, -1, dtype=np.int32)[None]
    cache = dict(c_cache=c, c_scale=scale, kr_cache=kr, page_table=ints(table), table=table, pps=4)
    cos, sin = tables(n, D_R, DEV)
    g = gen(5, DEV)
    x = torch.randn(n, D_C, generator=g, device=DEV).bfloat16()
    xr = torch.randn(n, D_R, generator=g, device=DEV).bfloat16()
    pos = np.arange(n)
    sa.mla_cache_write(x, xr, c, kr, ints(pos), 4, cos, sin, c_scale=scale, page_table=cache["page_table"],
                       seq_of_row=ints(pos * 0))
    back, kr_back = sa.mla_cache_read(c, kr, ints(pos)[None], 4, c_scale=scale, page_table=cache["page_table"])
    rows = pool_rows(cache, 0, pos)
    assert torch.equal(back[0].double(), latent64(cache, rows)) and torch.equal(kr_back[0], kr[rows])
    want = norm64(x, None, 1e-6)
    assert ((back[0].double() - want).abs() <= 2.0 ** -4 * want.abs() + 2.0 ** -16 * want.abs().max()).all()
    q = torch.randn(1, 64, D_C, generator=g, device=DEV).bfloat16()
    qr = torch.randn(1, 64, D_R, generator=g, device=DEV).bfloat16()
    out = sa.sparse_mla_decode(q, qr, c, kr, ints(pos)[None], SCALE, 4, page_table=cache["page_table"], c_scale=scale)
    check_attention(out[0], None, attend64(q[0], qr[0], cache, 0, pos), "far rows")
    tree = sa.tree_mla_decode(q[:, None], qr[:, None], c, kr, ints([n - 1]), None, n, SCALE, 4,
                              page_table=cache["page_table"], c_scale=scale)
    check_attention(tree[0, 0], None, attend64(q[0], qr[0], cache, 0, pos), "far rows of a tree")
    assert sa.check_device_error() == 0
    del c, scale, kr, cache, back, kr_back
    far = torch.empty((1 << 31) + 4 * 64, device=DEV, dtype=torch.bfloat16)
    heads = far.as_strided((2, 4, 64), (1 << 31, 64, 1))
    heads.copy_(torch.randn(2, 4, 64, generator=g, device=DEV))
    near = heads.clone()
    at = ints([3, 7])
    a, b = sa.qk_norm_rope(heads, heads[:, :1], cos, sin, at)
    c2, d = sa.qk_norm_rope(near, near[:, :1], cos, sin, at)
    assert torch.equal(a, c2) and torch.equal(b, d)


@pytest.mark.parametrize("scale", [-SCALE, 0.0, 1e-30])
def test_scales_of_the_scores(scale):
    """Negative, zero and vanishing factors of the scores."""
    cache = make_cache((300,), True, 4, DEV, junk_nan=True)
    g = gen(4, DEV)
    q = torch.randn(1, 100, D_C, generator=g, device=DEV).bfloat16()
    qr = torch.randn(1, 100, D_R, generator=g, device=DEV).bfloat16()
    idx = np.full((1, 320), -1)
    idx[0, 10:310] = np.arange(300)
    lse = torch.empty(1, 100, device=DEV)
    out = sa.sparse_mla_decode(q, qr, cache["c_cache"], cache["kr_cache"], ints(idx), scale, cache["pps"],
                               page_table=cache["page_table"], lse=lse, c_scale=cache["c_scale"])
    check_attention(out[0], lse[0], attend64(q[0], qr[0], cache, 0, np.arange(300), scale), f"scale {scale}")


@pytest.mark.parametrize("low,high,gain", [(133, 138, 2.0 ** -17), (126, 131, 2.0 ** -8), (1, 4, 1.0), (231, 235, 2.0 ** -110)])
def test_scale_bytes_at_the_ends(low, high, gain):
    """Latent rows far from 1 in size, both sides of where one bf16 factor
    stops reaching (byte 134), and at the smallest and largest scales.  The
    bound's absolute term scales with the values."""
    n = 200
    cache = make_cache((n,), True, 4, DEV)
    g = gen(low, DEV)
    cache["c_scale"].copy_(torch.randint(low, high, cache["c_scale"].shape, generator=g, device=DEV))
    q = (torch.randn(1, 128, D_C, generator=g, device=DEV) * gain).bfloat16()
    qr = torch.randn(1, 128, D_R, generator=g, device=DEV).bfloat16()
    out = sa.sparse_mla_decode(q, qr, cache["c_cache"], cache["kr_cache"], ints(np.arange(n))[None], SCALE,
                               cache["pps"], page_table=cache["page_table"], c_scale=cache["c_scale"])
    want, _, spread, mass = attend64(q[0], qr[0], cache, 0, np.arange(n))
    # as check_attention; of values below bf16's normal range (2^-126) nothing need be kept
    bound = (2.0 ** -7 + 2.0 ** -16 * mass) * spread + 2.0 ** -120
    assert torch.isfinite(out).all() and ((out[0].double() - want).abs() <= bound).all()


def test_an_overflowing_drafted_row_stays_with_its_tokens():
    """A drafted row that overflows bf16 (codes 448 at the byte 254) reaches no token that does not see it."""
    past, T, H = 100, 4, 16
    cache = make_cache((past + T,), True, 6, DEV)
    bad = pool_rows(cache, 0, [past + 2])
    cache["c_cache"].view(torch.uint8)[bad] = 0x7E
    cache["c_scale"][bad] = 254
    g = gen(4, DEV)
    q = torch.randn(1, T, H, D_C, generator=g, device=DEV).bfloat16()
    qr = torch.randn(1, T, H, D_R, generator=g, device=DEV).bfloat16()
    mask = np.eye(T, dtype=np.uint8)[None]
    out = sa.tree_mla_decode(q, qr, cache["c_cache"], cache["kr_cache"], ints([past]), torch.from_numpy(mask).to(DEV),
                             past + T, SCALE, cache["pps"], page_table=cache["page_table"], c_scale=cache["c_scale"])
    for i in (0, 1, 3):
        pos = np.concatenate((np.arange(past), [past + i]))
        check_attention(out[0, i], None, attend64(q[0, i], qr[0, i], cache, 0, pos), f"token {i}")


def many(rows, H, k, seed):
    """`rows` selections of up to k positions of five sequences, with empty slots and empty rows."""
    lens = (900, 64, 333, 1, 2000)
    cache = make_cache(lens, True, seed, DEV, junk_nan=True)
    rng = np.random.Generator(np.random.PCG64(seed))
    seq = rng.integers(0, 5, rows)
    idx = np.full((rows, k), -1, dtype=np.int64)
    for r in range(rows):
        m = min(k, lens[seq[r]])
        idx[r, :m] = rng.permutation(lens[seq[r]])[:m]
        idx[r, rng.random(k) < 0.1] = -1
    idx[::7] = -1
    g = gen(seed, DEV)
    q = torch.randn(rows, H, D_C, generator=g, device=DEV).bfloat16()
    qr = torch.randn(rows, H, D_R, generator=g, device=DEV).bfloat16()
    return cache, seq, idx, q, qr


@pytest.mark.parametrize("bf16_out", [False, True])
@pytest.mark.parametrize("rows,H,k", [(75, 128, 1), (149, 64, 200), (400, 33, 130), (1000, 8, 512), (230, 128, 513)])
def test_more_short_selections_than_the_gpu_has_sms(rows, H, k, bf16_out):
    """Rows that share an SM pair one after the other (and, with 513 slots, do not), each against fp64."""
    cache, seq, idx, q, qr = many(rows, H, k, rows)
    out = torch.full((rows, H, D_C), torch.nan, device=DEV, dtype=torch.bfloat16 if bf16_out else torch.float32)
    lse = torch.full((rows, H), torch.nan, device=DEV)

    def call():
        sa.sparse_mla_prefill(q, qr, cache["c_cache"], cache["kr_cache"], ints(idx), SCALE, cache["pps"],
                              page_table=cache["page_table"], seq_of_row=ints(seq), out=out, lse=lse,
                              c_scale=cache["c_scale"])

    call()
    for r in range(rows):
        check_attention(out[r], lse[r], attend64(q[r], qr[r], cache, seq[r], idx[r][idx[r] >= 0]), f"row {r}")
    first = out.clone(), lse.clone()
    for _ in range(10):
        call()
    assert torch.equal(out, first[0]) and torch.equal(lse, first[1])
    assert sa.check_device_error() == 0


def test_wait_limit_runs_out_between_rows_of_a_pair():
    """As below, where several rows share an SM pair."""
    cache, seq, idx, q, qr = many(300, 64, 100, 3)

    def call():
        return sa.sparse_mla_decode(q, qr, cache["c_cache"], cache["kr_cache"], ints(idx), SCALE, cache["pps"],
                                    page_table=cache["page_table"], seq_of_row=ints(seq), c_scale=cache["c_scale"])

    call()
    assert sa.check_device_error() == 0
    sa.set_wait_limit_ns(200)
    try:
        call()
        torch.cuda.synchronize()
        code = sa.check_device_error()
    finally:
        sa.set_wait_limit_ns(0)
    assert code & 0xF00 == 0xA00, f"expected a latent-attention wait site, got 0x{code:x}"
    out = call()
    assert sa.check_device_error() == 0
    for r in range(0, 300, 11):
        check_attention(out[r], None, attend64(q[r], qr[r], cache, seq[r], idx[r][idx[r] >= 0]), f"row {r}")


def test_broadcast_token_rows_are_refused():
    """Rows of the written tokens that overlap (stride 0) are not a layout the write reads."""
    cache = make_cache((64, 64), True, 2, DEV)
    cos, sin = tables(8, D_R, DEV)
    c, kr = torch.zeros(1, D_C, device=DEV).bfloat16(), torch.zeros(1, D_R, device=DEV).bfloat16()
    for a, b in ((c.expand(2, D_C), kr.repeat(2, 1)), (c.repeat(2, 1), kr.expand(2, D_R))):
        with pytest.raises(sa.SparseAttnError):
            sa.mla_cache_write(a, b, cache["c_cache"], cache["kr_cache"], ints([0, 0]), cache["pps"], cos, sin,
                               c_scale=cache["c_scale"], page_table=cache["page_table"])


@pytest.mark.parametrize("q8", [True, False])
def test_a_length_past_the_page_table_is_reported(q8):
    """A length no page table holds is recorded and costs no more than the table's own positions."""
    cache = make_cache((128,), q8, 2, DEV)
    g = gen(4, DEV)
    q = torch.randn(1, 1, 16, D_C, generator=g, device=DEV).bfloat16()
    qr = torch.randn(1, 1, 16, D_R, generator=g, device=DEV).bfloat16()
    sa.tree_mla_decode(q, qr, cache["c_cache"], cache["kr_cache"], ints([2 ** 31 - 1]), None, 200, SCALE, cache["pps"],
                       page_table=cache["page_table"], c_scale=cache["c_scale"])
    assert sa.check_device_error() == 0x700


def test_wait_limit_runs_out_and_the_next_call_is_correct():
    """With a limit of 200 ns the wait for the first converted operand (some 2
    us) runs out: the kernel records a code of its own and returns, and with
    the default limit the same call is right.  (The time is looked at between
    tries, and a try of the hardware's may itself last a microsecond or two, as
    long as any wait of the bf16 cache's.)"""
    past, T, H = 3000, 2, 64
    cache = make_cache((past + T,), True, 6, DEV)
    g = gen(4, DEV)
    q = torch.randn(1, T, H, D_C, generator=g, device=DEV).bfloat16()
    qr = torch.randn(1, T, H, D_R, generator=g, device=DEV).bfloat16()

    def call():
        return sa.tree_mla_decode(q, qr, cache["c_cache"], cache["kr_cache"], ints([past]), None, past + T, SCALE,
                                  cache["pps"], page_table=cache["page_table"], c_scale=cache["c_scale"])

    call()
    assert sa.check_device_error() == 0
    sa.set_wait_limit_ns(200)
    try:
        call()
        torch.cuda.synchronize()
        code = sa.check_device_error()
    finally:
        sa.set_wait_limit_ns(0)
    assert code & 0xF00 == 0xA00, f"expected a latent-attention wait site, got 0x{code:x}"
    out = call()
    assert sa.check_device_error() == 0
    for i in range(T):
        check_attention(out[0, i], None, attend64(q[0, i], qr[0, i], cache, 0, np.arange(past + i + 1)), f"token {i}")

"""Measured cases of the operators around the latent cache, each with its plain form.

  norm_rope  per-head RMS norm of queries and keys with the rotary rotation in the same pass
  cache      latent rows normalised, rotated, quantised and written to the paged cache, and read back
  read       a prefix of the quantised cache read back as bf16 rows
  sparse     attention over the selected rows of the quantised cache
  tree       attention of a tree of drafted tokens over the cached prefix and their own ancestors

``own`` chooses between the plain form (elementary torch operations in fp32,
rounded once at the end) and the library's calls.  ``exact`` is the definition
in fp64.  A quantised latent row is 512 e4m3 codes and four scale bytes, one
per 128 dims; byte e stands for 2^(e-127), and a value is code * scale.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
D_C, D_R, PAGE, BLK = 512, 64, 64, 128
SCALE = 1.0 / math.sqrt(128 + D_R)
EPS = 1e-6
E4M3_MAX = 448.0


# ---------------------------------------------------------------- cases
def listed():
    return [
        # one decode step of the NSA workload's heads (8 sequences, 32 query and 4 key heads of 128): latency
        dict(name="norm_rope_decode", op="norm_rope", tokens=8, hq=32, hk=4, d=128, rot=128, start=0,
             interleaved=False, weight=True, dtype="bf16", max_pos=131072, strided=False),
        # a prefill chunk of 4096 tokens, the same heads, q and k views of one fused projection
        dict(name="norm_rope_chunk", op="norm_rope", tokens=4096, hq=32, hk=4, d=128, rot=128, start=0,
             interleaved=False, weight=True, dtype="bf16", max_pos=65536, strided=True),
        # MLA queries of a ragged batch in fp32: 128 content dims and 64 rotated ones per head, pairs interleaved
        dict(name="norm_rope_mla_f32", op="norm_rope", tokens=1021, hq=128, hk=1, d=192, rot=64, start=128,
             interleaved=True, weight=False, dtype="f32", max_pos=65536, strided=False),
        # one decode step appends a token to each of 32 sequences: latency
        dict(name="cache_decode", op="cache", tokens=32, seqs=32, pages=64, q8=True, dtype="bf16",
             interleaved=True),
        # a prefill chunk appended to one sequence and read back for the chunk's own attention
        dict(name="cache_chunk", op="cache", tokens=4096, seqs=1, pages=1024, q8=True, dtype="bf16",
             interleaved=True),
        # the prefix of a 64K sequence read back
        dict(name="read_prefix", op="read", rows=1, k=61440, pages=1024),
        # the rows a ragged batch selected, with padded slots
        dict(name="read_selected", op="read", rows=31, k=777, pages=100),
        # one sequence, 16 heads, 128 selected positions: the smallest decode
        dict(name="sparse_tiny", op="sparse", rows=1, seqs=1, H=16, k=128, lo=2048, hi=2048),
        # ragged long-context decode: 64 sequences of 8K to 128K, top-2048, 128 heads
        dict(name="sparse_ragged", op="sparse", rows=64, seqs=64, H=128, k=2048, lo=8192, hi=131072),
        # 1024 queries of a prefill chunk over 64K tokens
        dict(name="sparse_prefill", op="sparse", rows=1024, seqs=1, H=128, k=2048, lo=65536, hi=65536),
        # one sequence verifies a chain-like draft of 7 tokens over a short bf16 prefix, 128 heads
        dict(name="tree_one", op="tree", B=1, T=7, H=128, lo=1900, hi=1900, q8=False, ragged=False),
        # a ragged batch verifies trees of 48 tokens over the quantised cache, heads sharded to 16 per GPU
        dict(name="tree_batch", op="tree", B=32, T=48, H=16, lo=512, hi=4096, q8=True, ragged=True),
    ]


def _logint(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm_rope", "cache", "read", "sparse", "tree"])
    if op == "norm_rope":
        d = rng.choice([64, 96, 128, 192, 256])
        rot = rng.choice([d, d // 2, 32])
        return dict(op=op, tokens=_logint(rng, 1, 4096), hq=_logint(rng, 1, 48), hk=rng.choice([0, 1, 2, 4, 8]), d=d,
                    rot=rot, start=rng.choice([0, d - rot]), interleaved=rng.random() < 0.5,
                    weight=rng.random() < 0.5, dtype=rng.choice(["bf16", "f32"]), max_pos=_logint(rng, 64, 131072),
                    strided=rng.random() < 0.5)
    if op == "cache":
        seqs = _logint(rng, 1, 64)
        per = _logint(rng, 1, 4096 // seqs)
        return dict(op=op, tokens=seqs * per, seqs=seqs, pages=(per + 63) // 64 + rng.randint(0, 20),
                    q8=rng.random() < 0.7, dtype=rng.choice(["bf16", "f32"]), interleaved=rng.random() < 0.5)
    if op == "read":
        rows = _logint(rng, 1, 64)
        k = _logint(rng, 1, 61440 // rows)
        return dict(op=op, rows=rows, k=k, pages=(k + 63) // 64 + rng.randint(0, 50))
    if op == "sparse":
        one = rng.random() < 0.5
        rows = _logint(rng, 1, 1000 if one else 64)
        lo = _logint(rng, 1, 65536 if one else 32768)
        hi = lo if one else _logint(rng, lo, 65536)
        return dict(op=op, rows=rows, seqs=1 if one else rows, H=_logint(rng, 1, 128), k=_logint(rng, 1, 2048),
                    lo=lo, hi=hi)
    lo = _logint(rng, 1, 4096)
    return dict(op=op, B=_logint(rng, 1, 7), T=_logint(rng, 1, 64), H=_logint(rng, 1, 128), lo=lo,
                hi=_logint(rng, lo, 4096), q8=rng.random() < 0.5, ragged=rng.random() < 0.5)


# ---------------------------------------------------------------- inputs
def _dtype(name):
    return torch.float32 if name == "f32" else torch.bfloat16


def _tables(max_pos, rot):
    inv = 10000.0 ** (-torch.arange(0, rot, 2, device=DEV, dtype=torch.float64) / rot)
    ang = torch.arange(max_pos, device=DEV, dtype=torch.float64)[:, None] * inv
    return ang.cos().float(), ang.sin().float()


def _page_table(g, need):
    """[seqs, max] int32: every sequence's pages drawn from one shuffled pool, -1 past its end."""
    total, most = int(sum(need)), int(max(need))
    perm = torch.randperm(total, generator=g, device=DEV).to(torch.int32)
    table = torch.full((len(need), most), -1, dtype=torch.int32, device=DEV)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = perm[at:at + n]
        at += n
    return table, total


def _pool(g, pages, q8):
    """Latent and RoPE-key rows of a filled cache (values around N(0,1))."""
    n = pages * PAGE
    c = torch.randn((n, D_C), generator=g, device=DEV, dtype=torch.bfloat16)
    scale = None
    if q8:
        c = c.mul_(96).clamp_(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
        scale = torch.randint(119, 122, (n, D_C // BLK), generator=g, device=DEV, dtype=torch.int32).to(torch.uint8)
    kr = torch.randn((n, D_R), generator=g, device=DEV, dtype=torch.bfloat16)
    return c, scale, kr


def _lens(case, n, seed):
    rng = np.random.Generator(np.random.PCG64(seed))
    return rng.integers(case["lo"], case["hi"] + 1, size=n).astype(np.int64)


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    randn = lambda *s: torch.randn(s, generator=g, device=DEV)  # noqa: E731
    op, s = case["op"], dict(case=dict(case))
    if op == "norm_rope":
        t, hq, hk, d = case["tokens"], case["hq"], case["hk"], case["d"]
        x = (randn(t, hq + hk, d) * 2).to(_dtype(case["dtype"]))
        s["q"], s["k"] = x[:, :hq], (x[:, hq:] if hk else None)
        if not case["strided"]:
            s["q"], s["k"] = s["q"].contiguous(), (s["k"].contiguous() if hk else None)
        s["qw"], s["kw"] = (1 + 0.1 * randn(d), 1 + 0.1 * randn(d)) if case["weight"] else (None, None)
        s["cos"], s["sin"] = _tables(case["max_pos"], case["rot"])
        s["pos"] = torch.randint(0, case["max_pos"], (t,), generator=g, device=DEV, dtype=torch.int32)
    elif op == "cache":
        t, n, pages = case["tokens"], case["seqs"], case["pages"]
        per = t // n
        s["c"] = (randn(t, D_C) * 3).to(_dtype(case["dtype"]))
        s["kr"] = randn(t, D_R).to(_dtype(case["dtype"]))
        s["w"] = 1 + 0.1 * randn(D_C)
        s["table"], total = _page_table(g, [pages] * n)
        s["c_cache"], s["c_scale"], s["kr_cache"] = _pool(g, total, case["q8"])
        first = torch.randint(0, pages * PAGE - per + 1, (n,), generator=g, device=DEV)
        s["idx"] = (first[:, None] + torch.arange(per, device=DEV)).to(torch.int32)  # [seqs, per]
        s["slots"] = s["idx"].reshape(-1)
        s["seq"] = torch.arange(n, device=DEV, dtype=torch.int32).repeat_interleave(per)
        s["cos"], s["sin"] = _tables(pages * PAGE, D_R)
    elif op == "read":
        n, k, pages = case["rows"], case["k"], case["pages"]
        s["table"], total = _page_table(g, [pages] * n)
        s["c_cache"], s["c_scale"], s["kr_cache"] = _pool(g, total, True)
        if n == 1:
            s["idx"] = torch.arange(k, device=DEV, dtype=torch.int32)[None]
        else:
            u = torch.rand((n, pages * PAGE), generator=g, device=DEV)
            s["idx"] = u.topk(k, dim=1)[1].sort(dim=1)[0].to(torch.int32)
            s["idx"][:, k - k // 16:] = -1
    elif op == "sparse":
        n, rows, H, k = case["seqs"], case["rows"], case["H"], case["k"]
        lens = _lens(case, n, seed)
        s["table"], total = _page_table(g, [int(v + PAGE - 1) // PAGE for v in lens])
        s["c_cache"], s["c_scale"], s["kr_cache"] = _pool(g, total, True)
        s["q_lat"], s["q_rope"] = randn(rows, H, D_C).bfloat16(), randn(rows, H, D_R).bfloat16()
        s["seq"] = torch.arange(rows, device=DEV, dtype=torch.int32) if n == rows else \
            torch.zeros(rows, device=DEV, dtype=torch.int32)
        vis = torch.from_numpy(lens).to(DEV)[s["seq"].long()]
        u = torch.rand((rows, int(lens.max())), generator=g, device=DEV)
        u = torch.where(torch.arange(u.shape[1], device=DEV) < vis[:, None], u, -1.0)
        have = min(k, u.shape[1])
        v, i = u.topk(have, dim=1)
        i = torch.where(v >= 0, i, 1 << 30).sort(dim=1)[0]
        s["idx"] = torch.full((rows, k), -1, dtype=torch.int32, device=DEV)
        s["idx"][:, :have] = torch.where(i < (1 << 30), i, -1).to(torch.int32)
        s["out"] = torch.empty(rows, H, D_C, dtype=torch.bfloat16, device=DEV)
        if own:
            import sparse_attention_07_b200 as sa
            s["ws"] = torch.empty(sa.sparse_mla_q8_workspace_size(rows, H, k), dtype=torch.uint8, device=DEV)
    else:
        B, T, H = case["B"], case["T"], case["H"]
        past = _lens(case, B, seed)
        rng = np.random.Generator(np.random.PCG64(seed + 1))
        nd = rng.integers(1, T + 1, size=B) if case["ragged"] else np.full(B, T)
        m = np.zeros((B, T, T), dtype=np.uint8)  # token i sees itself and its ancestors
        for i in range(T):
            parent = rng.integers(max(-1, i - 4), i, size=B)
            up = np.maximum(parent, 0)
            m[:, i] = np.where((parent >= 0)[:, None], m[np.arange(B), up], 0)
            m[:, i, i] = 1
        s["mask"] = torch.from_numpy(m).to(DEV)
        s["past"] = torch.from_numpy(past.astype(np.int32)).to(DEV)
        s["nd"] = torch.from_numpy(nd.astype(np.int32)).to(DEV)
        s["L_max"] = int(case["hi"]) + T
        s["table"], total = _page_table(g, [int(v + T + PAGE - 1) // PAGE for v in past])
        s["c_cache"], s["c_scale"], s["kr_cache"] = _pool(g, total, case["q8"])
        s["q_lat"], s["q_rope"] = randn(B, T, H, D_C).bfloat16(), randn(B, T, H, D_R).bfloat16()
        s["out"] = torch.zeros(B, T, H, D_C, dtype=torch.bfloat16, device=DEV)
        if own:
            import sparse_attention_07_b200 as sa
            s["ws"] = torch.empty(sa.tree_mla_workspace_size(B, T, H, s["L_max"]), dtype=torch.uint8, device=DEV)
    return s


# ---------------------------------------------------------------- plain forms
def _plain_norm(x, w):
    y = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
    return y if w is None else y * w


def _plain_rope(x, cos, sin, interleaved):
    """Rotate the last dim of x: pairs (2i, 2i+1) if interleaved, else (i, i + half)."""
    if interleaved:
        a, b = x[..., 0::2], x[..., 1::2]
        return torch.stack((a * cos - b * sin, b * cos + a * sin), dim=-1).flatten(-2)
    a, b = x.chunk(2, dim=-1)
    return torch.cat((a * cos - b * sin, b * cos + a * sin), dim=-1)


def _plain_quantise(y):
    """fp32 rows -> (e4m3 codes, scale bytes): the smallest power of two with amax / scale <= 448."""
    v = y.view(*y.shape[:-1], D_C // BLK, BLK)
    amax = v.abs().amax(-1)
    m, e = torch.frexp(amax / E4M3_MAX)  # amax / 448 = m * 2^e, m in [0.5, 1)
    e = torch.where(m == 0.5, e - 1, e)
    byte = torch.where(amax > 0, (e + 127).clamp(1, 254), 127)
    codes = torch.ldexp(v, (127 - byte)[..., None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
    return codes.flatten(-2), byte.to(torch.uint8)


def _plain_rows(s, pool):
    """fp32 latent and RoPE rows of the given pool rows."""
    kr = s["kr_cache"][pool].float()
    if s["c_scale"] is None:
        return s["c_cache"][pool].float(), kr
    c = s["c_cache"].view(torch.uint8)[pool].view(torch.float8_e4m3fn).float()
    sc = torch.exp2(s["c_scale"][pool].float() - 127.0)
    return (c.view(*c.shape[:-1], D_C // BLK, BLK) * sc[..., None]).flatten(-2), kr


def _pool_rows(s, seq, pos):
    """Pool row of each position (positions < 0: row 0, masked by the caller)."""
    p = pos.clamp(min=0).long()
    return s["table"][seq, p // PAGE].long() * PAGE + p % PAGE


def _plain_attend(ql, qr, c, kr, seen):
    """ql [n, m, 512], qr [n, m, 64], c [n, L, 512], kr [n, L, 64], seen [n, m or 1, L] -> [n, m, 512] fp32."""
    z = (ql.float() @ c.transpose(1, 2) + qr.float() @ kr.transpose(1, 2)) * SCALE
    z = torch.where(seen, z, float("-inf"))
    top = z.amax(-1, keepdim=True)
    p = torch.exp(z - torch.where(top == float("-inf"), 0.0, top))
    total = p.sum(-1, keepdim=True)
    return (p / torch.where(total > 0, total, 1.0)) @ c


def _plain(s):
    case = s["case"]
    op = case["op"]
    if op == "norm_rope":
        cos, sin = s["cos"][s["pos"].long()][:, None], s["sin"][s["pos"].long()][:, None]
        a, b = case["start"], case["start"] + case["rot"]

        def one(x, w):
            y = _plain_norm(x.float(), w)
            return torch.cat((y[..., :a], _plain_rope(y[..., a:b], cos, sin, case["interleaved"]), y[..., b:]),
                             dim=-1).to(x.dtype)

        return {"q": one(s["q"], s["qw"]), "k": None if s["k"] is None else one(s["k"], s["kw"])}
    if op == "cache":
        at = _pool_rows(s, s["seq"].long(), s["slots"])
        y = _plain_norm(s["c"].float(), s["w"])
        p = s["slots"].long()
        s["kr_cache"][at] = _plain_rope(s["kr"].float(), s["cos"][p], s["sin"][p], case["interleaved"]).bfloat16()
        if case["q8"]:
            codes, byte = _plain_quantise(y)
            s["c_cache"].view(torch.uint8)[at] = codes.view(torch.uint8)
            s["c_scale"][at] = byte
        else:
            s["c_cache"][at] = y.bfloat16()
        c, kr = _plain_rows(s, at.view(s["idx"].shape))
        return {"c": c.bfloat16(), "kr": kr.bfloat16()}
    if op == "read":
        n = s["idx"].shape[0]
        c, kr = _plain_rows(s, _pool_rows(s, torch.arange(n, device=DEV)[:, None], s["idx"]))
        live = (s["idx"] >= 0)[..., None]
        return {"c": torch.where(live, c, 0.0).bfloat16(), "kr": torch.where(live, kr, 0.0).bfloat16()}
    if op == "sparse":
        c, kr = _plain_rows(s, _pool_rows(s, s["seq"].long()[:, None], s["idx"]))
        return {"out": _plain_attend(s["q_lat"], s["q_rope"], c, kr, (s["idx"] >= 0)[:, None]).bfloat16()}
    B, T, H = case["B"], case["T"], case["H"]
    pos = torch.arange(s["L_max"], device=DEV)[None].expand(B, -1)
    past, nd = s["past"].long()[:, None], s["nd"].long()[:, None]
    held = pos < past + nd
    c, kr = _plain_rows(s, _pool_rows(s, torch.arange(B, device=DEV)[:, None], torch.where(held, pos, 0)))
    j = (pos - past).clamp(0, T - 1)
    drafted = torch.gather(s["mask"], 2, j[:, None].expand(B, T, -1)).bool()
    seen = held[:, None] & ((pos < past)[:, None] | drafted)
    o = _plain_attend(s["q_lat"].view(B, T * H, D_C), s["q_rope"].view(B, T * H, D_R), c, kr,
                      seen.repeat_interleave(H, dim=1)).view(B, T, H, D_C)
    live = torch.arange(T, device=DEV)[None] < nd
    return {"out": torch.where(live[..., None, None], o, 0.0).bfloat16()}


# ---------------------------------------------------------------- one pass
def run(state):
    if not own:
        return _plain(state)
    import sparse_attention_07_b200 as sa
    s, case = state, state["case"]
    op = case["op"]
    if op == "norm_rope":
        q, k = sa.qk_norm_rope(s["q"], s["k"], s["cos"], s["sin"], s["pos"], q_weight=s["qw"], k_weight=s["kw"],
                               eps=EPS, rope_start=case["start"], interleaved=case["interleaved"])
        return {"q": q, "k": k}
    pps = s["table"].shape[1]
    if op == "cache":
        sa.mla_cache_write(s["c"], s["kr"], s["c_cache"], s["kr_cache"], s["slots"], pps, s["cos"], s["sin"],
                           weight=s["w"], eps=EPS, interleaved=case["interleaved"], c_scale=s["c_scale"],
                           page_table=s["table"], seq_of_row=s["seq"])
        c, kr = sa.mla_cache_read(s["c_cache"], s["kr_cache"], s["idx"], pps, c_scale=s["c_scale"],
                                  page_table=s["table"])
        return {"c": c, "kr": kr}
    if op == "read":
        c, kr = sa.mla_cache_read(s["c_cache"], s["kr_cache"], s["idx"], pps, c_scale=s["c_scale"],
                                  page_table=s["table"])
        return {"c": c, "kr": kr}
    if op == "sparse":
        out = sa.sparse_mla_decode(s["q_lat"], s["q_rope"], s["c_cache"], s["kr_cache"], s["idx"], SCALE, pps,
                                   page_table=s["table"], seq_of_row=s["seq"], out=s["out"], workspace=s["ws"],
                                   c_scale=s["c_scale"])
        return {"out": out}
    out = sa.tree_mla_decode(s["q_lat"], s["q_rope"], s["c_cache"], s["kr_cache"], s["past"], s["mask"], s["L_max"],
                             SCALE, pps, n_draft=s["nd"], c_scale=s["c_scale"], page_table=s["table"], out=s["out"],
                             workspace=s["ws"])
    return {"out": out}


# ---------------------------------------------------------------- bytes and operations
def work(case):
    op = case["op"]
    row = lambda q8: (D_C + D_C // BLK if q8 else 2 * D_C) + 2 * D_R  # noqa: E731  bytes of one cached token
    if op == "norm_rope":
        t, e = case["tokens"], 4 if case["dtype"] == "f32" else 2
        n = t * (case["hq"] + case["hk"]) * case["d"]
        angles = min(t, case["max_pos"]) * case["rot"] * 4
        return {"bytes": 2 * n * e + angles + 4 * t, "flops": 6 * n}
    if op == "cache":
        t, e = case["tokens"], 4 if case["dtype"] == "f32" else 2
        angles = t // case["seqs"] * D_R * 4
        return {"bytes": t * ((D_C + D_R) * (e + 2) + 2 * row(case["q8"]) + 8) + angles, "flops": 8 * t * (D_C + D_R)}
    if op == "read":
        n = case["rows"] * case["k"]
        return {"bytes": n * (row(True) + 2 * (D_C + D_R) + 4), "flops": n * D_C}
    if op == "sparse":
        rows, H = case["rows"], case["H"]
        k = min(case["k"], (case["lo"] + case["hi"]) // 2)
        # every selected row once: rows of one sequence share its cache
        cached = min(rows * k, case["hi"]) if case["seqs"] == 1 else rows * k
        return {"bytes": cached * row(True) + 4 * rows * case["k"] + rows * H * (2 * D_C + D_R) * 2,
                "flops": 2.0 * rows * H * k * (2 * D_C + D_R)}
    B, T, H = case["B"], case["T"], case["H"]
    L = (case["lo"] + case["hi"]) / 2
    t = (T + 1) / 2 if case["ragged"] else T
    return {"bytes": B * ((L + t) * row(case["q8"]) + t * H * (2 * D_C + D_R) * 2 + T * T),
            "flops": 2.0 * B * t * H * (L + min(t, 8)) * (2 * D_C + D_R)}


# ---------------------------------------------------------------- the definition in 64 bits
def _exact_rotate(x, ang_cos, ang_sin, interleaved):
    """The rotation as a product of complex numbers (x1 + i x2) * (cos + i sin)."""
    half = x.shape[-1] // 2
    pairs = x.unflatten(-1, (half, 2)) if interleaved else x.unflatten(-1, (2, half)).transpose(-1, -2)
    y = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * torch.complex(ang_cos, ang_sin))
    return y.flatten(-2) if interleaved else y.transpose(-1, -2).flatten(-2)


def _exact_latent(s, rows):
    c = s["c_cache"]
    if s["c_scale"] is None:
        return c[rows].double()
    b = c.view(torch.uint8)[rows].long()
    e, m = (b >> 3) & 15, b & 7
    mag = torch.where(e > 0, (8 + m).double() * torch.exp2((e - 10).double()), m.double() * 2.0 ** -9)
    val = torch.where(b >= 128, -mag, mag)
    return val * torch.exp2(s["c_scale"][rows].double() - 127).repeat_interleave(BLK, dim=-1)


def _exact_head_rows(q, qr, c, kr):
    """softmax attention of every query of one row: q [m, 512], c [n, 512]; n may be 0."""
    if c.shape[0] == 0:
        return torch.zeros_like(q)
    z = (torch.cat((q, qr), 1) @ torch.cat((c, kr), 1).T) * SCALE
    return torch.softmax(z, dim=1) @ c


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "norm_rope":
        def one(x, w):
            x = x.double()
            x = x / torch.sqrt(x.square().sum(-1, keepdim=True) / x.shape[-1] + EPS)
            x = x if w is None else x * w.double()
            p, a, r = s["pos"].long(), case["start"], case["rot"]
            x = x.clone()
            x[..., a:a + r] = _exact_rotate(x[..., a:a + r], s["cos"].double()[p][:, None],
                                            s["sin"].double()[p][:, None], case["interleaved"])
            return x
        return {"q": one(s["q"], s["qw"]), "k": None if s["k"] is None else one(s["k"], s["kw"])}
    if op == "cache":
        x = s["c"].double()
        x = x / torch.sqrt(x.square().sum(-1, keepdim=True) / D_C + EPS) * s["w"].double()
        if case["q8"]:
            v = x.unflatten(-1, (D_C // BLK, BLK))
            amax = v.abs().amax(-1, keepdim=True)
            sc = torch.exp2(torch.ceil(torch.log2(amax / E4M3_MAX)).clamp(-126, 127))
            u = v / sc
            step = torch.exp2(torch.floor(torch.log2(u.abs().clamp(min=2.0 ** -6))) - 3)
            x = (torch.round(u / step) * step * sc).flatten(-2)
        p = s["slots"].long()
        kr = _exact_rotate(s["kr"].double(), s["cos"].double()[p], s["sin"].double()[p], case["interleaved"])
        return {"c": x.view(*s["idx"].shape, D_C), "kr": kr.view(*s["idx"].shape, D_R)}
    if op == "read":
        seq = torch.arange(case["rows"], device=DEV)[:, None]
        rows = _pool_rows(s, seq, s["idx"])
        live = (s["idx"] >= 0)[..., None]
        return {"c": _exact_latent(s, rows) * live, "kr": s["kr_cache"][rows].double() * live}
    if op == "sparse":
        out = torch.zeros(case["rows"], case["H"], D_C, dtype=torch.float64, device=DEV)
        for r in range(case["rows"]):
            pos = s["idx"][r][s["idx"][r] >= 0]
            rows = _pool_rows(s, s["seq"][r].long(), pos)
            out[r] = _exact_head_rows(s["q_lat"][r].double(), s["q_rope"][r].double(), _exact_latent(s, rows),
                                      s["kr_cache"][rows].double())
        return {"out": out}
    out = torch.zeros(case["B"], case["T"], case["H"], D_C, dtype=torch.float64, device=DEV)
    past, nd, mask = s["past"].tolist(), s["nd"].tolist(), s["mask"].cpu().numpy()
    for b in range(case["B"]):
        for i in range(nd[b]):
            pos = np.concatenate((np.arange(past[b]), past[b] + np.flatnonzero(mask[b, i, :nd[b]])))
            rows = _pool_rows(s, torch.tensor(b, device=DEV), torch.from_numpy(pos).to(DEV))
            out[b, i] = _exact_head_rows(s["q_lat"][b, i].double(), s["q_rope"][b, i].double(),
                                         _exact_latent(s, rows), s["kr_cache"][rows].double())
    return {"out": out}

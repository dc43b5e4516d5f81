"""GPU: MLA attention over the quantised latent cache, and of drafted trees
over either cache, against the definition in fp64."""
import numpy as np
import pytest
import torch

import sparse_attention_07_b200 as sa
from _latent import D_C, D_R, EMPTY_POS, SCALE, attend64, check_attention, gen, make_cache

pytestmark = pytest.mark.gpu
DEV = "cuda"


def queries(shape, seed, gain=1.0):
    g = gen(seed, DEV)
    q = torch.randn(*shape, D_C, generator=g, device=DEV) * gain
    return q.bfloat16(), torch.randn(*shape, D_R, generator=g, device=DEV).bfloat16()


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a).astype(np.int32)).to(DEV)


def selection(lens, k, seed, drop=0.1):
    """[rows, k] distinct positions, some slots -1 (at any place), the last row all -1 if there are several."""
    rng = np.random.Generator(np.random.PCG64(seed))
    idx = np.full((len(lens), k), -1, dtype=np.int64)
    for r, n in enumerate(lens):
        m = min(k, n)
        idx[r, :m] = rng.permutation(n)[:m]
        idx[r, rng.random(k) < drop] = -1
    if len(lens) > 1:
        idx[-1] = -1
    return idx


def check_rows(out, lse, q, qr, cache, seq_of, pos_of, what):
    for r in range(out.shape[0]):
        want = attend64(q[r], qr[r], cache, seq_of(r), pos_of(r))
        check_attention(out[r], None if lse is None else lse[r], want, f"{what} row {r}")


@pytest.mark.parametrize("bf16_out", [False, True])
@pytest.mark.parametrize("lens,H,k", [
    ((100,), 16, 1), ((100, 70), 128, 63), ((300, 1, 64), 77, 64), ((300, 129), 1, 65), ((500,) * 5, 64, 200),
    ((1500, 2000), 128, 1000), ((5000,), 128, 2048), ((90,) * 90, 65, 80), ((3, 9000), 100, 4100)])
def test_sparse_q8(lens, H, k, bf16_out):
    cache = make_cache(lens, True, H + k, DEV, junk_nan=True, c_pad=16 * (k % 2))
    idx = selection(lens, k, k)
    q, qr = queries((len(lens), H), H * k)
    out = torch.full((len(lens), H, D_C), torch.nan, device=DEV, dtype=torch.bfloat16 if bf16_out else torch.float32)
    lse = torch.full((len(lens), H), torch.nan, device=DEV)
    got = sa.sparse_mla_decode(q, qr, cache["c_cache"], cache["kr_cache"], dev(idx), SCALE, cache["pps"],
                               page_table=cache["page_table"], out=out, lse=lse, c_scale=cache["c_scale"])
    assert got is out
    check_rows(out, lse, q, qr, cache, lambda r: r, lambda r: idx[r][idx[r] >= 0], f"H={H} k={k}")
    assert sa.check_device_error() == 0


def test_sparse_q8_prefill_rows_share_a_sequence():
    """Many rows of one sequence, unpaged, through the prefill call."""
    n, rows, k, H = 700, 160, 100, 32
    cache = make_cache((n,), True, 1, DEV, paged=False)
    idx = np.full((rows, k), -1, dtype=np.int64)
    rng = np.random.Generator(np.random.PCG64(4))
    for r in range(rows):
        m = min(k, r + 1)
        idx[r, :m] = np.sort(rng.permutation(r + 1)[:m])
    q, qr = queries((rows, H), 9)
    seq = torch.zeros(rows, dtype=torch.int32, device=DEV)
    out = sa.sparse_mla_prefill(q, qr, cache["c_cache"], cache["kr_cache"], dev(idx), SCALE, cache["pps"],
                                seq_of_row=seq, c_scale=cache["c_scale"])
    assert out.dtype == torch.float32
    check_rows(out, None, q, qr, cache, lambda r: 0, lambda r: idx[r][idx[r] >= 0], "prefill")


def test_sparse_q8_large_scores_and_scale_bytes():
    """Scores that grow along the row (the running maximum moves many times)
    and differ by thousands, and blocks with tiny and large scales."""
    n, H, k = 640, 128, 640
    cache = make_cache((n,), True, 2, DEV)
    from _latent import pool_rows
    rows = pool_rows(cache, 0, np.arange(n))
    cache["c_scale"][rows] = (110 + torch.arange(n, device=DEV) * 14 // n).to(torch.uint8)[:, None]
    cache["c_scale"][rows[5]] = 1
    q, qr = queries((1, H), 5, gain=8.0)
    idx = np.arange(n)[None]
    lse = torch.empty(1, H, device=DEV)
    out = sa.sparse_mla_decode(q, qr, cache["c_cache"], cache["kr_cache"], dev(idx), SCALE, cache["pps"],
                               page_table=cache["page_table"], lse=lse, c_scale=cache["c_scale"])
    check_rows(out, lse, q, qr, cache, lambda r: 0, lambda r: idx[0], "growing scores")


def test_sparse_q8_nan_in_a_selected_row_shows():
    """A selected block with byte 255 makes the output NaN; the same block unselected does not."""
    cache = make_cache((128,), True, 2, DEV)
    from _latent import pool_rows
    cache["c_scale"][pool_rows(cache, 0, [70]), 1] = 255
    q, qr = queries((2, 16), 5)
    idx = np.stack([np.arange(0, 70), np.arange(1, 71)])
    out = sa.sparse_mla_decode(q, qr, cache["c_cache"], cache["kr_cache"], dev(idx), SCALE, cache["pps"],
                               page_table=cache["page_table"], seq_of_row=torch.zeros(2, dtype=torch.int32, device=DEV),
                               c_scale=cache["c_scale"])
    assert torch.isfinite(out[0]).all() and torch.isnan(out[1]).all()


@pytest.mark.parametrize("lens,H", [((100, 2048, 0), 128), ((1, 5000), 16), ((64, 63, 65, 128), 77)])
def test_dense_q8(lens, H):
    cache = make_cache(lens, True, H, DEV, junk_nan=True)
    q, qr = queries((len(lens), H), H)
    lse = torch.empty(len(lens), H, device=DEV)
    out = sa.dense_mla_decode(q, qr, cache["c_cache"], cache["kr_cache"], dev(np.array(lens)), max(lens), SCALE,
                              cache["pps"], page_table=cache["page_table"], lse=lse, c_scale=cache["c_scale"])
    check_rows(out, lse, q, qr, cache, lambda r: r, lambda r: np.arange(lens[r]), f"dense H={H}")
    assert sa.check_device_error() == 0


def tree_masks(B, T, seed):
    """Ancestor masks of random trees (a token sees itself and its ancestors)."""
    rng = np.random.Generator(np.random.PCG64(seed))
    m = np.zeros((B, T, T), dtype=np.uint8)
    for b in range(B):
        for i in range(T):
            p = int(rng.integers(max(-1, i - 5), i)) if i else -1
            if p >= 0:
                m[b, i] = m[b, p]
            m[b, i, i] = 1
    return m


def run_tree(past, draft, T, H, q8, mask, seed, bf16_out=False, L_max=None, **kw):
    lens = [p + T for p in past]
    held = [p + d for p, d in zip(past, draft)]
    cache = make_cache(held, q8, seed, DEV, extra_pages=-(-T // 64) + 1, junk_nan=True)
    B = len(past)
    q, qr = queries((B, T, H), seed)
    out = torch.full((B, T, H, D_C), -7.0, device=DEV, dtype=torch.bfloat16 if bf16_out else torch.float32)
    lse = torch.full((B, T, H), -7.0, device=DEV)
    sa.tree_mla_decode(q, qr, cache["c_cache"], cache["kr_cache"], dev(np.array(past)),
                       None if mask is None else torch.from_numpy(mask).to(DEV), L_max or max(lens), SCALE,
                       cache["pps"], n_draft=dev(np.array(draft)), c_scale=cache["c_scale"],
                       page_table=cache["page_table"], out=out, lse=lse, **kw)
    return cache, q, qr, out, lse


def check_tree(cache, q, qr, out, lse, past, draft, mask, what):
    B, T = out.shape[:2]
    m = np.tril(np.ones((T, T), dtype=np.uint8))[None].repeat(B, 0) if mask is None else mask
    for b in range(B):
        for i in range(draft[b]):
            pos = np.concatenate((np.arange(past[b]), past[b] + np.flatnonzero(m[b, i, :draft[b]])))
            check_attention(out[b, i], lse[b, i], attend64(q[b, i], qr[b, i], cache, b, pos), f"{what} {b},{i}")
        assert (out[b, draft[b]:] == -7).all() and (lse[b, draft[b]:] == -7).all(), "rows past n_draft were written"
    assert sa.check_device_error() == 0


@pytest.mark.parametrize("q8", [True, False])
@pytest.mark.parametrize("past,draft,T,H", [
    ((40,), (1,), 1, 128), ((1900,), (7,), 7, 128), ((0, 1, 63), (5, 3, 0), 5, 16), ((64, 127, 500), (9, 9, 2), 9, 1),
    ((200, 17), (65, 64), 65, 24), ((300, 129, 1000), (33, 20, 1), 33, 64), ((100, 0), (6, 4), 6, 77),
    ((10,), (130,), 130, 3)])
def test_tree(past, draft, T, H, q8):
    mask = tree_masks(len(past), T, T + H)
    got = run_tree(past, draft, T, H, q8, mask, T * 3 + H)
    check_tree(*got, past, draft, mask, f"T={T} H={H}")


@pytest.mark.parametrize("q8", [True, False])
def test_tree_chain_bf16_output_and_short_L_max(q8):
    """No mask (a chain), bf16 output, and an L_max below the true length (it only sets the split)."""
    past, draft = (777, 30), (12, 5)
    got = run_tree(past, draft, 12, 40, q8, None, 3, bf16_out=True, L_max=100)
    check_tree(*got, past, draft, None, "chain")


@pytest.mark.parametrize("q8", [True, False])
@pytest.mark.parametrize("H", [128, 8])
def test_tree_empty_rows_and_nan_siblings(q8, H):
    """A token whose mask is empty over no prefix gives zeros; a drafted row
    that holds NaN (or, in bf16, infinity) reaches only the tokens that see it."""
    T = 6
    past, draft = (0, 70), (6, 6)
    mask = np.zeros((2, T, T), dtype=np.uint8)
    mask[:, np.arange(T), np.arange(T)] = 1
    mask[0, 2] = 0                    # sees nothing at all
    mask[:, 5, 1] = 1                 # token 5 sees token 1
    cache, q, qr, out, lse = run_tree(past, draft, T, H, q8, mask, 11)
    from _latent import pool_rows
    for b in range(2):
        at = pool_rows(cache, b, [past[b] + 1, past[b] + 3])
        if q8:
            cache["c_scale"][at, 2] = 255
        else:
            cache["c_cache"][at[0], 300] = torch.nan
            cache["c_cache"][at[1], 10] = torch.inf
        cache["kr_cache"][at[1], 5] = torch.nan
    sa.tree_mla_decode(q, qr, cache["c_cache"], cache["kr_cache"], dev(np.array(past)), torch.from_numpy(mask).to(DEV),
                       76, SCALE, cache["pps"], n_draft=dev(np.array(draft)), c_scale=cache["c_scale"],
                       page_table=cache["page_table"], out=out, lse=lse)
    for b in range(2):
        for i in range(T):
            if i in (1, 3, 5):
                assert torch.isnan(out[b, i]).any(-1).all(), f"token {b},{i} sees a NaN row"
            else:
                pos = np.concatenate((np.arange(past[b]), past[b] + np.flatnonzero(mask[b, i])))
                check_attention(out[b, i], lse[b, i], attend64(q[b, i], qr[b, i], cache, b, pos), f"{b},{i}")
    assert (out[0, 2] == 0).all() and torch.isneginf(lse[0, 2]).all()


def test_tree_of_one_token_equals_dense():
    """A chain of one token over n - 1 positions sees what dense attention over n sees."""
    lens = (500, 65)
    cache = make_cache(lens, True, 3, DEV)
    q, qr = queries((2, 48), 3)
    dense = sa.dense_mla_decode(q, qr, cache["c_cache"], cache["kr_cache"], dev(np.array(lens)), 500, SCALE,
                                cache["pps"], page_table=cache["page_table"], c_scale=cache["c_scale"])
    tree = sa.tree_mla_decode(q[:, None], qr[:, None], cache["c_cache"], cache["kr_cache"], dev(np.array(lens) - 1),
                              None, 500, SCALE, cache["pps"], c_scale=cache["c_scale"],
                              page_table=cache["page_table"])
    assert torch.equal(dense, tree[:, 0])


def test_seq_of_row_maps_trees():
    past, T, H = (200, 90), 4, 16
    cache = make_cache([p + T for p in past], False, 3, DEV)
    q, qr = queries((3, T, H), 3)
    order = (1, 0, 1)
    out = sa.tree_mla_decode(q, qr, cache["c_cache"], cache["kr_cache"], dev(np.array([past[s] for s in order])), None,
                             204, SCALE, cache["pps"], page_table=cache["page_table"], seq_of_row=dev(np.array(order)))
    for b, s in enumerate(order):
        for i in range(T):
            check_attention(out[b, i], None, attend64(q[b, i], qr[b, i], cache, s, np.arange(past[s] + i + 1)), f"{b}")


def test_bad_pages_are_reported():
    cache = make_cache((128, 128), True, 2, DEV)
    cache["page_table"][1, 1] = 1 << 20
    q, qr = queries((2, 16), 5)
    idx = dev(np.stack([np.arange(128), np.arange(128)]))
    sa.sparse_mla_decode(q, qr, cache["c_cache"], cache["kr_cache"], idx, SCALE, cache["pps"],
                         page_table=cache["page_table"], c_scale=cache["c_scale"])
    assert sa.check_device_error() == 0x700
    sa.tree_mla_decode(q[:, None], qr[:, None], cache["c_cache"], cache["kr_cache"], dev(np.array([100, 128])), None,
                       300, SCALE, cache["pps"], page_table=cache["page_table"], c_scale=cache["c_scale"])
    assert sa.check_device_error() == 0x700  # sequence 1: the bad page, and a position past the table
    sa.tree_mla_decode(q[:, None], qr[:, None], cache["c_cache"], cache["kr_cache"], dev(np.array([100, 10])), None,
                       300, SCALE, cache["pps"], page_table=cache["page_table"], c_scale=cache["c_scale"])
    assert sa.check_device_error() == 0


def test_two_streams_and_a_replayed_graph():
    """Calls on two streams with workspaces of their own, and a captured call
    replayed on new contents, agree with plain calls bit for bit."""
    lens = (3000, 2500)
    cache = make_cache(lens, True, 8, DEV)
    idx = dev(selection(lens + (1,), 2048, 3)[:2])
    qs = [queries((2, 128), s) for s in (1, 2)]

    def call(q, ws, out):
        return sa.sparse_mla_decode(q[0], q[1], cache["c_cache"], cache["kr_cache"], idx, SCALE, cache["pps"],
                                    page_table=cache["page_table"], c_scale=cache["c_scale"], out=out, workspace=ws)

    n = max(256, sa.sparse_mla_q8_workspace_size(2, 128, 2048))
    ws = [torch.empty(n, dtype=torch.uint8, device=DEV) for _ in range(2)]
    plain = [call(q, ws[0], None).clone() for q in qs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [torch.empty(2, 128, D_C, device=DEV) for _ in range(2)]
    for _ in range(20):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                call(qs[i], ws[i], outs[i])
    torch.cuda.synchronize()
    for o, p in zip(outs, plain):
        assert torch.equal(o, p)
    q = [t.clone() for t in qs[0]]
    out = torch.empty(2, 128, D_C, device=DEV)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(q, ws[0], out)
    for i in (1, 0, 1):
        for t, src in zip(q, qs[i]):
            t.copy_(src)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, plain[i])
    assert sa.check_device_error() == 0


def test_repeats_bit_identical():
    past, draft, T, H = (1500, 3000, 2222), (16, 9, 16), 16, 128
    mask = tree_masks(3, T, 1)
    cache, q, qr, out, lse = run_tree(past, draft, T, H, True, mask, 5)
    first = out.clone()
    for _ in range(30):
        sa.tree_mla_decode(q, qr, cache["c_cache"], cache["kr_cache"], dev(np.array(past)),
                           torch.from_numpy(mask).to(DEV), 3016, SCALE, cache["pps"], n_draft=dev(np.array(draft)),
                           c_scale=cache["c_scale"], page_table=cache["page_table"], out=out, lse=lse)
    assert torch.equal(out, first)
    assert sa.check_device_error() == 0


def test_refusals():
    cache = make_cache((64, 64), True, 2, DEV)
    q, qr = queries((2, 16), 5)
    idx = dev(np.zeros((2, 8)))

    def sparse(**kw):
        a = dict(q_lat=q, q_rope=qr, c_cache=cache["c_cache"], kr_cache=cache["kr_cache"], idx=idx, scale=SCALE,
                 pages_per_seq=1, page_table=cache["page_table"], c_scale=cache["c_scale"])
        a.update(kw)
        return sa.sparse_mla_decode(**a)

    for kw in (dict(q_lat=q[..., :256]), dict(q_lat=q.transpose(0, 1)), dict(idx=idx[:1]), dict(q_rope=qr[:1]),
               dict(c_scale=cache["c_scale"][:, :2]), dict(c_cache=cache["c_cache"].bfloat16()),
               dict(q_lat=q.cpu()), dict(out=torch.empty(2, 16, 64, device=DEV))):
        with pytest.raises(ValueError):
            sparse(**kw)
    for kw in (dict(q_lat=q.float()), dict(idx=idx.long()), dict(out=torch.empty(2, 16, D_C, device=DEV).half()),
               dict(c_scale=cache["c_scale"].float())):
        with pytest.raises(TypeError):
            sparse(**kw)
    with pytest.raises(sa.SparseAttnError):
        sparse(scale=float("inf"))
    with pytest.raises(sa.SparseAttnError):
        wide = queries((2, 129), 1)
        sparse(q_lat=wide[0], q_rope=wide[1])
    past = dev(np.array([3, 3]))

    def tree(**kw):
        a = dict(q_lat=q[:, None], q_rope=qr[:, None], c_cache=cache["c_cache"], kr_cache=cache["kr_cache"],
                 n_past=past, tree_mask=None, L_max=64, scale=SCALE, pages_per_seq=1, c_scale=cache["c_scale"],
                 page_table=cache["page_table"])
        a.update(kw)
        return sa.tree_mla_decode(**a)

    for kw in (dict(n_past=past[:1]), dict(tree_mask=torch.ones(2, 2, 2, dtype=torch.uint8, device=DEV)),
               dict(c_scale=None), dict(n_draft=past[:1])):
        with pytest.raises(ValueError):
            tree(**kw)
    with pytest.raises(TypeError):
        tree(tree_mask=torch.ones(2, 1, 1, device=DEV))
    with pytest.raises(sa.SparseAttnError):
        tree(L_max=0)


def test_no_rows():
    cache = make_cache((64,), True, 2, DEV)
    q, qr = queries((0, 16), 5)
    out = sa.sparse_mla_decode(q, qr, cache["c_cache"], cache["kr_cache"], dev(np.zeros((0, 8))), SCALE, 1,
                               page_table=cache["page_table"], c_scale=cache["c_scale"])
    assert out.shape == (0, 16, D_C)
    assert len(EMPTY_POS) == 0

"""C-ABI checks of the latent-cache operators that need no GPU: bad arguments
are refused on the host, before any launch (no pointer is dereferenced)."""
import ctypes

import pytest
import torch

import sparse_attention_07_b200 as sa

FAKE = ctypes.c_void_p(0x1000)
ODD = ctypes.c_void_p(0x1004)
ODDER = ctypes.c_void_p(0x1001)


@pytest.fixture(scope="module")
def L():
    from sparse_attention_07_b200 import build
    build.build()
    return sa.lib()


def caller(fn, **good):
    def call(**kw):
        assert set(kw) <= set(good)
        return fn(*{**good, **kw}.values())
    return call


def test_norm_rope(L):
    call = caller(L.sa_qk_norm_rope, q=FAKE, qts=4096, qhs=128, qo=FAKE, qots=4096, qohs=128, Hq=32, k=FAKE, kts=512,
                  khs=128, ko=FAKE, kots=512, kohs=128, Hk=4, dt=sa.SA_BF16, qw=None, kw=None, norm=1, eps=1e-6,
                  cos=FAKE, sin=FAKE, n_pos=10, pos=FAKE, tokens=4, D=128, start=0, rot=128, inter=0, st=None)
    assert call(tokens=0) == sa.SA_OK
    assert call(Hq=0, Hk=0) == sa.SA_OK
    for kw in (dict(tokens=-1), dict(Hq=-1), dict(D=0), dict(rot=130), dict(rot=3), dict(start=2), dict(eps=-1.0),
               dict(eps=float("nan")), dict(q=None), dict(qo=None), dict(k=None), dict(cos=None), dict(pos=None),
               dict(n_pos=0), dict(q=ODDER), dict(ko=ODDER), dict(sin=ODDER), dict(qw=ODDER)):
        assert call(**kw) == sa.SA_EINVAL, kw
    for kw in (dict(dt=sa.SA_E4M3), dict(D=513, rot=0), dict(tokens=1 << 30)):
        assert call(**kw) == sa.SA_EUNSUPPORTED, kw


def test_cache_write(L):
    call = caller(L.sa_mla_cache_write, c=FAKE, cin=512, kr=FAKE, krin=64, dt=sa.SA_BF16, w=None, norm=1, eps=1e-6,
                  cos=FAKE, sin=FAKE, n_pos=10, pos=None, inter=0, cc=FAKE, cdt=sa.SA_E4M3, cld=512, cs=FAKE, sld=4,
                  krc=FAKE, krld=64, pool=4, pt=None, pps=4, sor=None, slots=FAKE, tokens=2, dc=512, dR=64, st=None)
    assert call(tokens=0) == sa.SA_OK
    for kw in (dict(tokens=-1), dict(c=None), dict(kr=None), dict(cos=None), dict(slots=None), dict(cc=None),
               dict(krc=None), dict(cs=None), dict(cdt=sa.SA_BF16), dict(cin=511), dict(cin=516), dict(cld=520),
               dict(sld=3), dict(sld=6), dict(krld=60), dict(krld=68), dict(c=ODD), dict(cc=ODD), dict(w=ODD),
               dict(kr=ODDER), dict(cs=ODDER), dict(eps=-1.0), dict(n_pos=0), dict(pool=0), dict(pps=0)):
        assert call(**kw) == sa.SA_EINVAL, kw
    for kw in (dict(dt=sa.SA_E4M3), dict(cdt=sa.SA_F32), dict(dc=256), dict(dR=32), dict(pool=1 << 40)):
        assert call(**kw) == sa.SA_EUNSUPPORTED, kw


def test_cache_read(L):
    call = caller(L.sa_mla_cache_read, cc=FAKE, cdt=sa.SA_E4M3, cld=512, cs=FAKE, sld=4, krc=FAKE, krld=64, pool=4,
                  pt=None, pps=4, sor=None, idx=FAKE, rows=2, k=8, dc=512, dR=64, co=FAKE, kro=FAKE, st=None)
    assert call(rows=0) == sa.SA_OK
    assert call(k=0) == sa.SA_OK
    for kw in (dict(rows=-1), dict(idx=None), dict(co=None), dict(co=ODD), dict(kro=ODD), dict(cs=None), dict(cld=8)):
        assert call(**kw) == sa.SA_EINVAL, kw
    assert call(dc=576) == sa.SA_EUNSUPPORTED


@pytest.mark.parametrize("dense", [False, True])
def test_q8_attention(L, dense):
    call = caller(L.sa_dense_mla_q8 if dense else L.sa_sparse_mla_q8, ql=FAKE, qr=FAKE, cc=FAKE, cld=512, cs=FAKE,
                  sld=4, krc=FAKE, krld=64, pool=4, pt=None, pps=4, sor=None, idx=FAKE, rows=400, H=128, k=64, dc=512,
                  dR=64, scale=0.07, out=FAKE, odt=sa.SA_F32, lse=None, ws=None, wsb=0, st=None)
    assert call(rows=0) == sa.SA_OK
    for kw in (dict(rows=-1), dict(H=0), dict(k=0), dict(idx=None), dict(ql=None), dict(out=None), dict(cs=None),
               dict(scale=float("nan")), dict(cld=500), dict(ql=ODD), dict(qr=ODD), dict(out=ODD), dict(krc=ODD),
               dict(lse=ODDER), dict(idx=ODDER)):
        assert call(**kw) == sa.SA_EINVAL, kw
    for kw in (dict(H=129), dict(dc=576), dict(odt=sa.SA_E4M3), dict(rows=(1 << 24) + 1)):
        assert call(**kw) == sa.SA_EUNSUPPORTED, kw


def test_tree(L):
    call = caller(L.sa_tree_mla_decode, ql=FAKE, qr=FAKE, cc=FAKE, cdt=sa.SA_BF16, cld=512, cs=None, sld=0, krc=FAKE,
                  krld=64, pool=4, pt=None, pps=4, sor=None, past=FAKE, nd=None, mask=None, B=40, T=16, H=128, L=64,
                  dc=512, dR=64, scale=0.07, out=FAKE, odt=sa.SA_BF16, lse=None, ws=None, wsb=0, st=None)
    assert call(B=0) == sa.SA_OK
    for kw in (dict(B=-1), dict(T=0), dict(L=0), dict(past=None), dict(past=ODDER), dict(nd=ODDER), dict(cs=FAKE),
               dict(cdt=sa.SA_E4M3), dict(cld=516), dict(scale=float("inf"))):
        assert call(**kw) == sa.SA_EINVAL, kw
    for kw in (dict(T=1025), dict(H=200), dict(cdt=sa.SA_F32)):
        assert call(**kw) == sa.SA_EUNSUPPORTED, kw


def test_workspace_sizes(L):
    """Sizes of impossible calls are 0; a workspace that a size asks for is refused when missing."""
    assert L.sa_sparse_mla_q8_workspace_size(0, 128, 64) == 0
    assert L.sa_tree_mla_workspace_size(1, 0, 128, 64) == 0
    need = L.sa_sparse_mla_q8_workspace_size(1, 128, 2048)
    if need:
        a = (FAKE, FAKE, FAKE, 512, FAKE, 4, FAKE, 64, 64, None, 64, None, FAKE, 1, 128, 2048, 512, 64, 0.07, FAKE,
             sa.SA_F32, None)
        assert L.sa_sparse_mla_q8(*a, None, need, None) == sa.SA_EINVAL
        assert L.sa_sparse_mla_q8(*a, FAKE, need - 1, None) == sa.SA_EINVAL


def test_more_keys_than_32_bits_of_tiles_hold(L):
    assert L.sa_sparse_mla_q8_workspace_size(1, 128, 2 ** 31 - 1) == 0
    assert L.sa_tree_mla_workspace_size(1, 1, 128, 2 ** 31 - 1) == 0
    call = caller(L.sa_sparse_mla_q8, ql=FAKE, qr=FAKE, cc=FAKE, cld=512, cs=FAKE, sld=4, krc=FAKE, krld=64, pool=4,
                  pt=None, pps=4, sor=None, idx=FAKE, rows=1, H=128, k=2 ** 30 + 1, dc=512, dR=64, scale=0.07, out=FAKE,
                  odt=sa.SA_F32, lse=None, ws=None, wsb=0, st=None)
    assert call() == sa.SA_EUNSUPPORTED
    assert call(k=64, cld=2 ** 31) == sa.SA_EUNSUPPORTED
    assert call(k=64, krld=2 ** 31) == sa.SA_EUNSUPPORTED


def test_a_quantised_cache_without_its_scales_is_refused():
    """Without c_scale the calls read a bf16 cache, twice an e4m3 one's bytes."""
    q, qr = torch.zeros(1, 2, 512).bfloat16(), torch.zeros(1, 2, 64).bfloat16()
    c, kr = torch.zeros(64, 512).to(torch.float8_e4m3fn), torch.zeros(64, 64).bfloat16()
    one = torch.zeros(1, 1, dtype=torch.int32)
    for call in (sa.sparse_mla_decode, sa.sparse_mla_prefill):
        with pytest.raises(ValueError):
            call(q, qr, c, kr, one, 0.07, 1)
    with pytest.raises(ValueError):
        sa.sparse_mla_decode_static(q, qr, c, kr, one, 0.07, 1)
    with pytest.raises(ValueError):
        sa.dense_mla_decode(q, qr, c, kr, one[0], 1, 0.07, 1)


def test_cpu_tensors_are_refused():
    q = torch.zeros(1, 2, 64)
    with pytest.raises(ValueError):
        sa.qk_norm_rope(q, None, None, None, None)


def test_page_tables_of_more_positions_than_32_bits_count(L):
    """A row's keys (up to the table's positions, and drafted ones) are counted in 32 bits."""
    call = caller(L.sa_dense_mla_q8, ql=FAKE, qr=FAKE, cc=FAKE, cld=512, cs=FAKE, sld=4, krc=FAKE, krld=64, pool=4, pt=FAKE,
                  pps=2 ** 24 + 1, sor=None, n=FAKE, rows=1, H=128, L_max=64, dc=512, dR=64, scale=0.07, out=FAKE,
                  odt=sa.SA_F32, lse=None, ws=None, wsb=0, st=None)
    assert call() == sa.SA_EUNSUPPORTED
    assert call(pps=2 ** 31 - 1) == sa.SA_EUNSUPPORTED

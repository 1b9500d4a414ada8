"""What the 8-bit paged cache's calls refuse before any launch, their
workspace sizes and empty calls (no GPU)."""
import ctypes

import pytest
import torch

import compressed_sparse_attention_topk_b200 as csa2
from compressed_sparse_attention_topk_b200 import build as csa2_build

P = ctypes.c_void_p
FAKE = P(256)  # never dereferenced: validation fails first
OK, INVALID, UNSUPPORTED, WORKSPACE = (csa2.CSA2_OK, csa2.CSA2_ERR_INVALID_ARG,
                                       csa2.CSA2_ERR_UNSUPPORTED, csa2.CSA2_ERR_WORKSPACE)


@pytest.fixture(scope="module")
def lib():
    csa2_build.build()
    return csa2.lib()


def cache(**kw):
    f = dict(k=256, v=256, k_scale=256, v_scale=256, k_sum=256, pages=8, Hk=2, block=64, D=128)
    f.update(kw)
    return ctypes.byref(csa2.KV8(*(f[n] for n, _ in csa2.KV8._fields_)))


BAD_CACHES = [(dict(k=None), INVALID), (dict(v=264), INVALID), (dict(k_scale=None), INVALID),
              (dict(k_sum=258), INVALID), (dict(pages=0), INVALID), (dict(Hk=0), INVALID),
              (dict(block=0), INVALID), (dict(D=0), INVALID), (dict(block=48), UNSUPPORTED),
              (dict(block=256), UNSUPPORTED), (dict(D=96), UNSUPPORTED),
              (dict(D=256), UNSUPPORTED), (dict(Hk=129), UNSUPPORTED),
              (dict(pages=1 << 24), UNSUPPORTED)]


@pytest.mark.parametrize("kw,rc", BAD_CACHES)
def test_every_call_checks_the_cache(lib, kw, rc):
    c = cache(**kw)
    H = 4
    assert lib.csa2_kv8_append(c, FAKE, 256, FAKE, 256, FAKE, 1, None) == rc
    assert lib.csa2_kv8_unpack(c, FAKE, 1, FAKE, FAKE, None) == rc
    assert lib.csa2_kv8_select(FAKE, 512, c, FAKE, 4, FAKE, FAKE, 1, 1, H, 4, 1, 1, FAKE, FAKE,
                               1 << 20, None) == rc
    assert lib.csa2_kv8_attn(FAKE, 512, c, FAKE, 4, FAKE, FAKE, 1, 1, H, None, 0, 0.1, FAKE, FAKE,
                             FAKE, 1 << 30, None) == rc
    assert lib.csa2_kv8_append(None, FAKE, 256, FAKE, 256, FAKE, 1, None) == INVALID


def tables(lib, **kw):
    a = dict(lens=FAKE, add=P(512), B=2, block=64, table=FAKE, width=4, free=FAKE, n_free=3,
             lens_out=P(1024), cu=FAKE, slots=FAKE, pos=FAKE, cap=8, used=FAKE)
    a.update(kw)
    return lib.csa2_block_tables(*a.values(), None)


@pytest.mark.parametrize("kw,rc", [
    (dict(lens=None), INVALID), (dict(add=None), INVALID), (dict(table=None), INVALID),
    (dict(free=None), INVALID), (dict(lens_out=None), INVALID), (dict(cu=None), INVALID),
    (dict(slots=None), INVALID), (dict(pos=None), INVALID), (dict(used=None), INVALID),
    (dict(lens_out=FAKE), INVALID),          # in place: other CTAs still read lens
    (dict(lens_out=P(512)), INVALID),        # or add
    (dict(slots=P(260)), INVALID), (dict(B=-1), INVALID), (dict(width=0), INVALID),
    (dict(cap=-1), INVALID), (dict(n_free=-1), INVALID), (dict(block=0), INVALID),
    (dict(block=24), UNSUPPORTED), (dict(B=4097), UNSUPPORTED),
    (dict(width=1 << 25), UNSUPPORTED), (dict(cap=1 << 31), UNSUPPORTED)])
def test_block_tables_refuses(lib, kw, rc):
    assert tables(lib, **kw) == rc


def test_append_and_unpack_refuse(lib):
    c = cache()

    def append(k=FAKE, ks=256, v=FAKE, vs=256, slots=FAKE, n=1):
        return lib.csa2_kv8_append(c, k, ks, v, vs, slots, n, None)

    assert append(n=0, k=None, v=None, slots=None) == OK
    assert append(n=-1) == INVALID
    assert append(k=None) == INVALID and append(v=None) == INVALID
    assert append(slots=None) == INVALID and append(slots=P(260)) == INVALID
    assert append(k=P(264)) == INVALID                      # misaligned rows
    assert append(ks=260) == INVALID and append(vs=248) == INVALID   # stride
    assert lib.csa2_kv8_unpack(c, FAKE, 0, FAKE, FAKE, None) == OK
    assert lib.csa2_kv8_unpack(c, FAKE, 4, None, None, None) == OK   # nothing asked for
    assert lib.csa2_kv8_unpack(c, None, 4, FAKE, None, None) == INVALID
    assert lib.csa2_kv8_unpack(c, FAKE, -1, FAKE, None, None) == INVALID
    assert lib.csa2_kv8_unpack(c, FAKE, 4, P(264), None, None) == INVALID


def select(lib, **kw):
    a = dict(q=FAKE, stride=512, c=cache(), table=FAKE, width=4, cu=FAKE, lens=FAKE, B=1, n=1,
             H=4, n_sel=4, n_first=1, n_last=1, sel=FAKE, ws=FAKE, bytes=1 << 20)
    a.update(kw)
    return lib.csa2_kv8_select(*a.values(), None)


@pytest.mark.parametrize("kw,rc", [
    (dict(n=0, q=None), OK), (dict(B=0, q=None), OK), (dict(n=-1), INVALID),
    (dict(B=-1), INVALID), (dict(q=None), INVALID), (dict(table=None), INVALID),
    (dict(cu=None), INVALID), (dict(lens=None), INVALID), (dict(sel=None), INVALID),
    (dict(width=0), INVALID), (dict(H=3), INVALID), (dict(stride=508), INVALID),
    (dict(stride=504), INVALID), (dict(q=P(264)), INVALID), (dict(n_sel=0), INVALID),
    (dict(n_first=-1), INVALID), (dict(n_last=0), INVALID),
    (dict(n_first=4, n_last=1), INVALID), (dict(n_sel=1), INVALID),
    (dict(H=130, stride=1 << 16), UNSUPPORTED),
    (dict(n_sel=4097), UNSUPPORTED), (dict(width=65537, bytes=1 << 40), UNSUPPORTED),
    (dict(B=4097), UNSUPPORTED), (dict(ws=None), WORKSPACE), (dict(ws=P(264)), WORKSPACE),
    (dict(bytes=8), WORKSPACE)])
def test_select_refuses(lib, kw, rc):
    assert select(lib, **kw) == rc


def attn(lib, **kw):
    a = dict(q=FAKE, stride=512, c=cache(), table=FAKE, width=4, cu=FAKE, lens=FAKE, B=1, n=1,
             H=4, sel=None, n_sel=0, scale=0.1, out=FAKE, lse=FAKE, ws=FAKE, bytes=1 << 30)
    a.update(kw)
    return lib.csa2_kv8_attn(*a.values(), None)


@pytest.mark.parametrize("kw,rc", [
    (dict(n=0, q=None), OK), (dict(B=0, q=None), OK), (dict(n=-1), INVALID),
    (dict(q=None), INVALID), (dict(out=None), INVALID), (dict(out=P(264)), INVALID),
    (dict(lse=P(258)), INVALID), (dict(H=3), INVALID), (dict(stride=504), INVALID),
    (dict(sel=FAKE), INVALID), (dict(n_sel=4), INVALID), (dict(sel=P(258), n_sel=4), INVALID),
    (dict(scale=float("nan")), INVALID), (dict(scale=float("inf")), INVALID),
    (dict(H=130, stride=1 << 16), UNSUPPORTED), (dict(sel=FAKE, n_sel=65537), UNSUPPORTED),
    (dict(B=4097), UNSUPPORTED), (dict(width=(1 << 24) + 1), UNSUPPORTED),
    (dict(ws=None), WORKSPACE), (dict(ws=P(264)), WORKSPACE),
    (dict(bytes=8), WORKSPACE)])
def test_attn_refuses(lib, kw, rc):
    assert attn(lib, **kw) == rc


def test_workspace_queries(lib):
    assert csa2.kv8_select_workspace_size(5, 2, 100) >= 256
    assert csa2.kv8_select_workspace_size(0, 2, 100) >= 256
    for bad in ((-1, 2, 100), (5, 0, 100), (5, 2, 0), (5, 2, 65537), (5, 129, 100)):
        assert csa2.kv8_select_workspace_size(*bad) == 0
    assert csa2.kv8_attn_workspace_size(32, 32, 16, 2, 128) >= 256
    for bad in ((-1, 1, 16, 2, 128, 0), (1, -1, 16, 2, 128, 0), (1, 1, 15, 2, 128, 0),
                (1, 1, 16, 2, 96, 0), (1, 1, 16, 0, 128, 0), (1, 1, 16, 2, 128, -1)):
        assert csa2.kv8_attn_workspace_size(*bad) == 0


def test_bindings_refuse_host_tensors():
    x = torch.zeros(2, dtype=torch.int32)
    csa2._kv8_types()
    with pytest.raises(TypeError):
        csa2._check_dense(x, "x", torch.int32, 0)
    with pytest.raises(TypeError):
        csa2.KV8Cache(*[torch.zeros(1)] * 5)
    with pytest.raises(TypeError):
        csa2._check_tokens(torch.zeros(2, 4, 64, dtype=torch.bfloat16), "q", 64, None, 0)
    if torch.cuda.is_available():
        with pytest.raises(TypeError):
            csa2.block_tables(x, x, torch.zeros(2, 4, dtype=torch.int32), x, 64, 8)

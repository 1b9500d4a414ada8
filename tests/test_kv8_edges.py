"""Calls at the edge of what the 8-bit paged cache accepts, answered before
any launch (no GPU)."""
import ctypes

import pytest

import compressed_sparse_attention_topk_b200 as csa2
from compressed_sparse_attention_topk_b200 import build as csa2_build

P = ctypes.c_void_p
FAKE = P(256)  # never dereferenced
OK, INVALID = csa2.CSA2_OK, csa2.CSA2_ERR_INVALID_ARG


@pytest.fixture(scope="module")
def lib():
    csa2_build.build()
    return csa2.lib()


def cache():
    return ctypes.byref(csa2.KV8(256, 256, 256, 256, 256, 8, 2, 64, 128))


def attn(lib, **kw):
    a = dict(q=FAKE, stride=512, c=cache(), table=FAKE, width=4, cu=FAKE, lens=FAKE, B=1, n=1,
             H=4, sel=None, n_sel=0, scale=0.1, out=FAKE, lse=FAKE, ws=FAKE, bytes=1 << 30)
    a.update(kw)
    return lib.csa2_kv8_attn(*a.values(), None)


@pytest.mark.parametrize("kw,rc", [
    (dict(n=0, n_sel=4), OK),             # the lists of no token: a null pointer
    (dict(B=0, n_sel=4), OK), (dict(n=0, n_sel=-1), INVALID),
    (dict(n_sel=4), INVALID), (dict(sel=FAKE), INVALID)])
def test_lists_of_no_token(lib, kw, rc):
    assert attn(lib, **kw) == rc

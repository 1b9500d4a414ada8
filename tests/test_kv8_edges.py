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


# places 1 KiB apart or more: B = 3, width 4, 5 free pages, cap 8
PLACES = dict(lens=(1024, 12), add=(2048, 12), table=(10240, 48), free=(4096, 20),
              lens_out=(5120, 12), cu=(6144, 16), slots=(7168, 64), pos=(8192, 32),
              used=(9216, 4))
WRITTEN = ("table", "lens_out", "cu", "slots", "pos", "used")


def tables(lib, moved, **kw):
    at = {k: v[0] for k, v in PLACES.items()}
    at.update(moved)
    a = dict(B=3, block=64, width=4, n_free=5, cap=8)
    a.update(kw)
    return lib.csa2_block_tables(at["lens"], at["add"], a["B"], a["block"], at["table"],
                                 a["width"], at["free"], a["n_free"], at["lens_out"], at["cu"],
                                 at["slots"], at["pos"], a["cap"], at["used"], None)


@pytest.mark.parametrize("one", WRITTEN)
@pytest.mark.parametrize("other", PLACES)
def test_block_tables_refuses_outputs_that_overlap(lib, one, other):
    """What is written shares no byte with anything else: other blocks of the
    launch read the lengths, the lists and the tables again."""
    if one == other:
        return
    (at, size), own = PLACES[other], PLACES[one][1]
    for off in (0, size - 4, 4 - own):
        where = at + off
        if one == "slots" and where % 8:
            continue
        assert tables(lib, {one: where}) == INVALID, off

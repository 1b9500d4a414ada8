"""Calls at the edge of what the 8-bit paged cache's documentation allows, on
the GPU."""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import compressed_sparse_attention_topk_b200 as csa2
from compressed_sparse_attention_topk_b200 import build as csa2_build
from tests import _kv8 as ref
from tests.test_gpu_kv8 import check_attn, dev, dev_bf16, gpu_cache, make_step

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    csa2_build.build()
    csa2.lib()
    csa2.get_device_status()


def small_step(rng, lens, adds, H, Hk, D, bs, **kw):
    """(q, cache, table, cu, lens) of a step as host arrays and as the calls
    take them."""
    table, cu, P = make_step(rng, lens, adds, bs, **kw)
    c = ref.new_cache(rng, P, Hk, bs, D)
    q = ref.bf16(rng.standard_normal((int(cu[-1]), H, D)).astype(np.float32))
    host = (q, c, table, cu, np.array(lens, np.int32))
    return host, (dev_bf16(q), gpu_cache(c), dev(table), dev(cu), dev(host[4]))


def test_lists_without_a_place_are_refused():
    """They must not mean every block, which a list tensor's null pointer does."""
    _, args = small_step(np.random.default_rng(1), [70, 9], [2, 1], 4, 2, 64, 32)
    sel = torch.empty((3, 2, 0), dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError):
        csa2.kv8_attn(*args, sel=sel)
    out, lse = csa2.kv8_attn(*args, sel=torch.full((3, 2, 1), -1, dtype=torch.int32,
                                                   device="cuda"))
    assert (out == 0).all() and torch.isneginf(lse).all()
    assert csa2.get_device_status() == 0


def test_a_step_without_tokens():
    _, (q, c, table, cu, lens) = small_step(np.random.default_rng(2), [70, 9], [1, 0], 4, 2, 64,
                                            32)
    q, cu = q[:0], torch.zeros_like(cu)
    sel = csa2.kv8_select(q, c, table, cu, lens, 3)
    assert sel.shape == (0, 2, 3)
    for s in (None, sel):
        out, lse = csa2.kv8_attn(q, c, table, cu, lens, sel=s)
        assert out.shape == (0, 4, 64) and lse.shape == (0, 4)
    none = torch.empty((0, 2, 64), dtype=torch.bfloat16, device="cuda")
    slots = torch.empty(0, dtype=torch.int64, device="cuda")
    csa2.kv8_append(c, none, none, slots)
    assert csa2.kv8_unpack(c, slots)[0].shape == (0, 2, 64)
    assert csa2.get_device_status() == 0


def test_strides_that_address_nothing_are_not_looked_at():
    """One token of a projection of odd width, no token with strides of its
    own: the same results as from dense tensors."""
    (q, c, table, cu, lens), args = small_step(np.random.default_rng(3), [150], [1], 4, 2, 64, 32)
    want = csa2.kv8_attn(*args)
    wide = torch.zeros((1, 4 * 64 + 2 * 2 * 64 + 1), dtype=torch.bfloat16, device="cuda")
    wide[:, :256] = args[0].view(1, 256)
    one = wide.as_strided((1, 4, 64), (wide.shape[1], 64, 1))
    assert one.stride(0) % 8 != 0
    got = csa2.kv8_attn(one, *args[1:])
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    sel = csa2.kv8_select(one, *args[1:], 3)
    assert torch.equal(sel, csa2.kv8_select(*args, 3))
    new = wide[:, 256:].as_strided((1, 2, 64), (wide.shape[1], 64, 1))
    csa2.kv8_append(args[1], new, new, dev(np.array([3], np.int64)))
    none = torch.empty_strided((0, 4, 64), (1, 1, 1), dtype=torch.bfloat16, device="cuda")
    assert csa2.kv8_attn(none, *args[1:])[0].shape == (0, 4, 64)
    assert csa2.kv8_select(none, *args[1:], 3).shape == (0, 2, 3)
    two = torch.zeros((2, 4 * 64 + 1), dtype=torch.bfloat16, device="cuda")[:, :256].view(2, 4, 64)
    with pytest.raises(csa2.CSA2Error):
        csa2.kv8_attn(two, *args[1:])
    assert csa2.get_device_status() == 0


# --- device status ------------------------------------------------------------

STATUS = """
import torch
import compressed_sparse_attention_topk_b200 as csa2

def copies():
    with torch.profiler.profile(activities=[torch.profiler.ProfilerActivity.CUDA]) as p:
        code = csa2.get_device_status()
        torch.cuda.synchronize()
    return code, sum(1 for e in p.events() if "memcpy" in e.name.lower() and "dtoh" in e.name.lower())

x = torch.tensor([-1], dtype=torch.int32, device="cuda")
csa2.get_device_status()
print(*copies())
csa2.block_tables(x, x, x.view(1, 1).clone(), x.clone(), 16, 1)
print(*copies())
print(*copies())
"""


def test_status_is_one_copy_for_those_who_never_use_the_cache():
    """And the cache's own word is read once it was used."""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", STATUS], cwd=root, capture_output=True, text=True,
                       timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
    lines = [tuple(map(int, x.split())) for x in r.stdout.split("\n") if x[:1].isdigit()]
    if lines[-1][1] == 0:
        pytest.skip("the profiler reports no copies here")
    assert lines == [(0, 1), (4, 2), (0, 2)]


# --- the handle ---------------------------------------------------------------

@pytest.mark.parametrize("name", ["k", "v", "k_scale", "v_scale", "k_sum", "pages", "D"])
def test_a_cache_keeps_the_tensors_that_it_was_made_of(name):
    """Its calls go by their pointers."""
    c = csa2.KV8Cache.empty(3, 2, 16, 64)
    old = getattr(c, name)
    with pytest.raises(AttributeError):
        setattr(c, name, old.clone() if torch.is_tensor(old) else old + 1)
    assert getattr(c, name) is old


# --- block tables -------------------------------------------------------------

@pytest.mark.parametrize("B,cap", [(3, 9), (0, 2), (2, 0)])
def test_block_tables_on_buffers_side_by_side(B, cap):
    """Parts of one buffer, with nothing between them."""
    rng = np.random.default_rng(8)
    lens, add = rng.integers(0, 40, B).astype(np.int32), rng.integers(0, 3, B).astype(np.int32)
    table = rng.integers(0, 50, (B, 4)).astype(np.int32)
    free = np.arange(60, 70, dtype=np.int32)
    want = ref.block_tables(lens, add, table, free, 16, cap)
    buf = torch.zeros(2 * cap + cap + 8 * B + 12, dtype=torch.int32, device="cuda")
    s, p, a, b, t, f, o, u, n = buf.split((2 * cap, cap, B, B, 4 * B, 10, B, B + 1, 1)
                                          if B else (2 * cap, cap, 0, 0, 0, 10, 0, 1, 1))
    for x, y in ((a, lens), (b, add), (t, table.reshape(-1)), (f, free)):
        x.copy_(dev(y))
    out = (o, u, s.view(torch.int64), p, n)
    csa2.block_tables(a, b, t.view(B, 4), f, 16, cap, out=out)
    for x, y in zip(out + (t,), want):
        assert np.array_equal(x.cpu().numpy(), np.reshape(y, -1))
    assert csa2.get_device_status() == (4 if cap < int(add.sum()) else 0)
    if B:
        with pytest.raises(csa2.CSA2Error):
            csa2.block_tables(a, b, t.view(B, 4), f, 16, cap, out=(buf[3 * cap:3 * cap + B],
                                                                   *out[1:]))


def test_block_tables_records_tokens_of_a_page_that_was_never_there():
    """A request whose last page is missing (a free list too short the step
    before): its tokens have no slot, and the status word says so each time."""
    lens, add = np.array([20, 16, 5], np.int32), np.array([3, 2, 1], np.int32)
    table = np.array([[7, -1, 9], [3, 4, 9], [6, 9, 9]], np.int32)
    free = np.array([11, 12], np.int32)
    for t, a, status in ((table, add, 4), (table, np.array([0, 2, 1], np.int32), 0),
                         (np.abs(table), add, 0)):
        want = ref.block_tables(lens, a, t, free, 16, 8)
        g = dev(t)
        got = csa2.block_tables(dev(lens), dev(a), g, dev(free), 16, 8)
        for x, y in zip(got + (g,), want):
            assert np.array_equal(x.cpu().numpy().reshape(-1), np.reshape(y, -1))
        assert csa2.get_device_status() == status
    # a page that the free list lends is none either
    got = csa2.block_tables(dev(lens), dev(add), dev(np.abs(table)), dev(np.array([-5], np.int32)),
                            16, 8)
    assert (got[2][3:5] == -1).all() and got[4].item() == 1
    assert csa2.get_device_status() == 4


# --- choice of blocks ---------------------------------------------------------

def check_select(host, args, n_sel, n_first=1, n_last=1):
    q, c, table, cu, lens = host
    want = np.full((len(q), c["k"].shape[1], n_sel), -7, np.int32)
    ref.select(q, c, table, cu, lens, n_sel, n_first, n_last, want)
    got = torch.full(want.shape, -7, dtype=torch.int32, device="cuda")
    csa2.kv8_select(*args, n_sel, n_first, n_last, out=got)
    got = got.cpu().numpy()
    assert np.array_equal(got, want), np.argwhere((got != want).any(-1))[:5]


@pytest.mark.parametrize("lens,adds,width", [([500], [1], 9), ([40, 700, 16], [2, 300, 1], 12),
                                             ([289], [1], 9)])
def test_select_records_a_table_narrower_than_the_sequence(lens, adds, width):
    """Blocks past the table's width do not exist; that is recorded."""
    (q, c, table, cu, lens), args = small_step(np.random.default_rng(4), lens, adds, 4, 2, 64, 32)
    table = np.ascontiguousarray(table[:, :width])
    check_select((q, c, table, cu, lens), (*args[:2], dev(table), *args[3:]), 5)
    assert csa2.get_device_status() == 1
    # of the same width, no longer than the table: nothing to record
    lens = np.minimum(lens, width * 32)
    check_select((q, c, table, cu, lens), (*args[:2], dev(table), *args[3:4], dev(lens)), 5)
    assert csa2.get_device_status() == 0


@pytest.mark.parametrize("lens,adds,extra_width", [([900, 20], [3, 1], 41000),
                                                   ([41500 * 16 - 3], [2], 3)])
def test_select_of_rows_wider_than_shared_memory(lens, adds, extra_width):
    host, args = small_step(np.random.default_rng(5), lens, adds, 2, 1, 64, 16,
                            extra_width=extra_width)
    assert host[2].shape[1] > 40960
    check_select(host, args, 40, 2, 3)
    assert csa2.get_device_status() == 0


@pytest.mark.parametrize("extra_width", [1, 3000])
def test_select_of_padding_alone_with_calls_behind_it(extra_width):
    """Steps whose tokens all belong to nobody write nothing, and the calls
    behind them find their inputs as they left them."""
    host, args = small_step(np.random.default_rng(6), [900, 20], [3, 1], 4, 2, 64, 16,
                            extra_width=extra_width)
    none = torch.zeros_like(args[3])
    for _ in range(20):
        out = torch.full((4, 2, 8), -7, dtype=torch.int32, device="cuda")
        csa2.kv8_select(*args[:3], none, args[4], 8, out=out)
        args[3].copy_(args[3].clone())
        check_select(host, args, 8)
        assert (out == -7).all()
    assert csa2.get_device_status() == 0


# --- attention ----------------------------------------------------------------

@pytest.mark.parametrize("H,D,T", [(4, 64, 1), (8, 128, 1), (16, 128, 2)])
def test_attn_a_missing_page_of_16_under_a_position_past_2_to_the_30(H, D, T):
    """Lengths past every table's reach: the missing half of a unit of two
    pages (a bad page, or the end of a list) is not seen."""
    rng = np.random.default_rng(7)
    (q, c, table, cu, _), args = small_step(rng, [16], [T], H, 2, D, 16)
    table = np.array([[table[0, 0], -1]], np.int32)
    lens = dev(np.array([(1 << 30) + 100], np.int32))
    # every token sees the page whole, as a single one at its last position does
    want = [np.zeros((T, H, D)), np.zeros((T, H))]
    info = [np.zeros((T, H, D))] + [np.zeros((T, H)) for _ in range(3)]
    for i in range(T):
        out, lse, more = ref.attn(q[i:i + 1], c, table, np.array([0, 1]), [16])
        for x, y in zip(want + info, (out, lse) + more):
            x[i] = y[0]
    args = (*args[:2], dev(table), args[3], lens)
    check_attn(*csa2.kv8_attn(*args), *want, info, T)
    assert csa2.get_device_status() == 1
    sel = torch.zeros((T, 2, 1), dtype=torch.int32, device="cuda")
    check_attn(*csa2.kv8_attn(*args, sel=sel), *want, info, T)
    assert csa2.get_device_status() == 0


@pytest.mark.parametrize("H,T", [(2, 1), (4, 2), (8, 1), (16, 1), (8, 40)])
@pytest.mark.parametrize("D,bs", [(64, 16), (128, 64)])
def test_attn_queries_with_one_large_element(H, T, D, bs):
    """A large element that meets zero codes: the logits are all the small ones'.

    Beside the bounds of ref.attn_bounds a query element is held to 2^-29 of its
    row's largest (sequences whose tiles have at most 4 rows) or 2^-25 (fp16,
    the largest in [1, 2): the half step of an fp16 subnormal), so a logit may
    be off by q_err max|q| sum_d |k_d| |sm_scale| more, and a weight and the sum
    of weights by a factor of exp of that each."""
    rng = np.random.default_rng(9)
    Hk, lens, sm_scale = 2, [700, 90], 1e5
    (q, c, table, cu, lens), _ = small_step(rng, lens, [T, 1], H, Hk, D, bs)
    q = q * np.exp2(-rng.uniform(16, 22, q.shape))
    q[:, :, 5] = 1.0
    q = ref.bf16(q.astype(np.float32))
    c["k"][..., 5] = 0
    out, lse, info = ref.attn(q, c, table, cu, lens, None, sm_scale)
    q_err = 2.0 ** -29 if T * H // Hk <= 4 else 2.0 ** -25
    sums = np.abs(c["k"].astype(np.float64)).sum(-1).max(-1) * c["k_scale"]
    logit = q_err * sums.max() * sm_scale
    tol, tol_lse = ref.attn_bounds(out, lse, info)
    tol = tol + np.expm1(2 * logit) * info[0]
    got, got_lse = csa2.kv8_attn(dev_bf16(q), gpu_cache(c), dev(table), dev(cu), dev(lens),
                                 sm_scale=sm_scale)
    off = np.abs(got.float().cpu().numpy() - out) / tol
    assert off.max() <= 1, off.max()
    off = np.abs(got_lse.cpu().numpy() - lse) / (tol_lse + logit)
    assert off.max() <= 1, off.max()
    assert csa2.get_device_status() == 0


@pytest.mark.parametrize("H,T", [(4, 1), (8, 1), (4, 64)])
def test_attn_queries_next_to_the_largest_number(H, T):
    """Query elements of 2^127 and more, up to the largest bf16."""
    rng = np.random.default_rng(10)
    (q, c, table, cu, lens), _ = small_step(rng, [300], [T], H, 2, 128, 64)
    big = ref.bf16(np.full(1, 3.3895313892515355e38, np.float32))[0]
    q = ref.bf16(np.clip(q, -1, 1) * big)
    q[..., ::7] = big
    q[..., 1::7] = -big
    sm_scale = 2.0 ** -126
    out, lse, info = ref.attn(q, c, table, cu, lens, None, sm_scale)
    got, got_lse = csa2.kv8_attn(dev_bf16(q), gpu_cache(c), dev(table), dev(cu), dev(lens),
                                 sm_scale=sm_scale)
    check_attn(got, got_lse, out, lse, info, T)
    assert csa2.get_device_status() == 0


@pytest.mark.parametrize("T", [1, 5, 200])
@pytest.mark.parametrize("scale", [2.0 ** -75, 2.0 ** 75])
def test_attn_value_scales_at_the_ends_of_their_range(T, scale):
    """Pages of the smallest or the largest value scale, flat weights over
    thousands of positions: nothing overflows or loses bits."""
    rng = np.random.default_rng(11)
    (q, c, table, cu, lens), args = small_step(rng, [5000, 300], [T, 1], 8, 2, 64, 64)
    c["v_scale"][:] = np.float32(scale)
    c["v"][:] = np.where(c["v"] >= 20, 127, c["v"])
    out, lse, info = ref.attn(q, c, table, cu, lens, None, 0.01)
    got, got_lse = csa2.kv8_attn(args[0], gpu_cache(c), *args[2:], sm_scale=0.01)
    # (the bounds' absolute 1e-30 is 1e-8 of the smallest scale)
    check_attn(got, got_lse, out, lse, info, len(q))
    assert np.abs(out).max() > 8 * scale
    assert csa2.get_device_status() == 0


@pytest.mark.parametrize("G,rows", [(1, 33), (4, 9)])
def test_attn_value_scales_far_apart_beside_a_long_sequence(G, rows):
    """What the header says of one token beside a sequence of more than 32 query
    rows: scales down to 2^-80 of the largest count."""
    rng = np.random.default_rng(12)
    (q, c, table, cu, lens), args = small_step(rng, [200, 150], [2 * rows, 1], 2 * G, 2, 64, 16)
    c["v_scale"][:] = 1.0
    c["v_scale"][table[1, 1:4]] = np.float32(2.0 ** -79)
    c["k"][table[1, 1]] = 127          # a page that takes nearly all the weight
    q[-1] = 0.5
    out, lse, info = ref.attn(q, c, table, cu, lens, None, 1.0)
    got, got_lse = csa2.kv8_attn(dev_bf16(q), gpu_cache(c), *args[2:], sm_scale=1.0)
    check_attn(got, got_lse, out, lse, info, len(q))
    assert csa2.get_device_status() == 0

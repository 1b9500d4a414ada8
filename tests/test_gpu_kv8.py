"""The 8-bit paged key/value cache on the GPU against plain implementations on
the host (tests/_kv8.py): tables, slots, codes, scales and chosen blocks
equal, attention within bounds derived from its roundings."""
import numpy as np
import pytest
import torch

import compressed_sparse_attention_topk_b200 as csa2
from compressed_sparse_attention_topk_b200 import build as csa2_build
from tests import _kv8 as ref
from tests._kv8 import cdiv

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    csa2_build.build()
    csa2.lib()
    csa2.get_device_status()


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def dev_bf16(a):
    """fp32 values that are bf16 values -> a bf16 tensor of those bits."""
    return dev(a).to(torch.bfloat16)


def gpu_cache(c):
    return csa2.KV8Cache(*(dev(c[n]) for n in ("k", "v", "k_scale", "v_scale", "k_sum")))


def same_cache(g, c, what=""):
    torch.cuda.synchronize()
    for n in ("k_scale", "v_scale", "k_sum", "k", "v"):
        a, b = getattr(g, n).cpu().numpy(), c[n]
        assert np.array_equal(a, b), f"{what} {n}: {int((a != b).sum())} of {a.size} differ"


def make_step(rng, lens, adds, bs, spare=0, extra_width=1):
    """(table, cu, pages): every sequence's blocks on distinct pages, in a
    random order; -1 past its last block."""
    blocks = [cdiv(max(n, 0), bs) for n in lens]
    P = sum(blocks) + spare
    P = max(P, 1)
    order = rng.permutation(P).astype(np.int32)
    table = np.full((len(lens), max(blocks + [1]) + extra_width), -1, np.int32)
    at = 0
    for b, m in enumerate(blocks):
        table[b, :m] = order[at:at + m]
        at += m
    cu = np.concatenate([[0], np.cumsum(adds)]).astype(np.int32)
    return table, cu, P


# --- block tables -------------------------------------------------------------

@pytest.mark.parametrize("B,bs,longest,adds", [
    (1, 16, 0, 1), (1, 64, 63, 2), (2, 16, 16, 16), (7, 32, 100, 40), (33, 64, 1000, 1),
    (100, 128, 500, 300), (700, 16, 200, 5), (4096, 16, 30, 3)])
def test_block_tables(B, bs, longest, adds):
    rng = np.random.default_rng(B + bs)
    lens = rng.integers(0, longest + 1, B).astype(np.int32)
    add = rng.integers(0, adds + 1, B).astype(np.int32)
    add[0] = adds
    if B > 2:
        add[1] = 0
        lens[2] = 0
    width = cdiv(longest + adds, bs) + 1
    table = rng.integers(1000, 2000, (B, width)).astype(np.int32)
    free = rng.permutation(int(sum(cdiv(int(a), bs) + 1 for a in add))).astype(np.int32)
    cap = int(add.sum()) + 13
    want = ref.block_tables(lens, add, table, free, bs, cap)
    g = dev(table)
    for _ in range(2):  # a second call on the same lengths changes nothing
        got = csa2.block_tables(dev(lens), dev(add), g, dev(free), bs, cap)
    names = ("lens", "cu", "slots", "pos", "used")
    for x, y, name in zip(got, want[:5], names):
        assert np.array_equal(x.cpu().numpy().reshape(-1), np.reshape(y, -1)), name
    assert np.array_equal(g.cpu().numpy(), want[5])
    assert csa2.get_device_status() == 0


def test_block_tables_out_of_pages_room_and_cap():
    """Too few free pages, a request past its row, negative lengths, too many
    tokens: -1 where there is no page, everything recorded, nothing written
    outside."""
    lens = np.array([5, 60, -3, 10], np.int32)
    add = np.array([30, 10, 20, -7], np.int32)
    table = np.full((5, 4), 77, np.int32)           # one guard row
    free = np.array([9, 8, 7], np.int32)
    want = ref.block_tables(lens, add, table[:4], free, 16, 50)
    g = dev(table)
    out = (torch.empty(4, dtype=torch.int32, device="cuda"),
           torch.empty(5, dtype=torch.int32, device="cuda"),
           torch.full((50,), 5, dtype=torch.int64, device="cuda"),
           torch.full((50,), 5, dtype=torch.int32, device="cuda"),
           torch.empty(1, dtype=torch.int32, device="cuda"))
    got = csa2.block_tables(dev(lens), dev(add), g[:4], dev(free), 16, 50, out=out)
    for x, y, name in zip(got, want[:5], ("lens", "cu", "slots", "pos", "used")):
        assert np.array_equal(x.cpu().numpy().reshape(-1), np.reshape(y, -1)), name
    assert np.array_equal(g[:4].cpu().numpy(), want[5])
    assert (g[4] == 77).all()
    assert csa2.get_device_status() == 4
    # no requests at all
    empty = torch.empty(0, dtype=torch.int32, device="cuda")
    lens_out, cu, slots, pos, used = csa2.block_tables(
        empty, empty, torch.empty((0, 4), dtype=torch.int32, device="cuda"), dev(free), 16, 3)
    assert cu.tolist() == [0] and slots.tolist() == [-1] * 3 and used.tolist() == [0]
    assert csa2.get_device_status() == 0


# --- append and read back -----------------------------------------------------

@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("bs", [16, 32, 64, 128])
@pytest.mark.parametrize("Hk", [1, 3])
def test_append_over_steps(D, bs, Hk):
    """Prompts, then single tokens, then drafts that are partly overwritten."""
    rng = np.random.default_rng(D + bs + Hk)
    lens = np.array([0, 1, bs - 1, bs, 3 * bs + 5], np.int32)
    B = len(lens)
    width = 12
    table = rng.permutation(B * width).astype(np.int32).reshape(B, width)
    c = ref.new_cache(rng, B * width, Hk, bs, D)
    g = gpu_cache(c)
    for step, add in enumerate(([2 * bs + 3, 0, 1, bs, 1], [1] * B, [5] * B, [3] * B)):
        slots = []
        for b in range(B):
            p = np.arange(lens[b], lens[b] + add[b])
            slots.append(table[b, p // bs].astype(np.int64) * bs + p % bs)
        slots = np.concatenate(slots + [np.array([-1, -1])])
        n = len(slots)
        x = rng.standard_normal((n, 2 * Hk + 1, D)) * np.exp(rng.uniform(-3, 3, (n, 1, 1)))
        if step == 1:
            x[0] = 0.0
        x = ref.bf16(x.astype(np.float32))
        ref.append(c, x[:, 1:Hk + 1], x[:, Hk + 1:], slots)
        t = dev_bf16(x)
        csa2.kv8_append(g, t[:, 1:Hk + 1], t[:, Hk + 1:], dev(slots))
        same_cache(g, c, f"step {step}")
        keep = 2 if step == 2 else None  # of five drafts two stay
        lens = lens + (np.array(add, np.int32) if keep is None else keep)
    rows = np.concatenate([rng.integers(0, B * width * bs, 40), [-1, 0, B * width * bs - 1]])
    k, v = csa2.kv8_unpack(g, dev(rows))
    for got, name in ((k, "k"), (v, "v")):
        want = (c[name].astype(np.float32) * c[name + "_scale"][:, :, None, None]).transpose(
            0, 2, 1, 3).reshape(-1, Hk, D)[rows]
        want[rows < 0] = 0
        assert np.array_equal(got.cpu().numpy(), want), name
    assert csa2.get_device_status() == 0


def test_append_many_tokens_and_a_page_ending_inside_a_group():
    rng = np.random.default_rng(5)
    bs, Hk, D, n = 64, 2, 128, 1500            # several tokens per CTA
    P = cdiv(n + 40, bs)
    order = rng.permutation(P)
    p = np.arange(n) + 37
    slots = order[p // bs].astype(np.int64) * bs + p % bs
    slots[700:705] = -1                        # a gap inside a page
    c = ref.new_cache(rng, P, Hk, bs, D)
    # the gap splits a page into two runs: leave the second one out
    again = (p // bs == p[705] // bs) & (np.arange(n) >= 705)
    slots[again] = -1
    g = gpu_cache(c)
    x = ref.bf16(rng.standard_normal((n, 2 * Hk, D)).astype(np.float32))
    ref.append(c, x[:, :Hk], x[:, Hk:], slots)
    t = dev_bf16(x)
    csa2.kv8_append(g, t[:, :Hk], t[:, Hk:], dev(slots))
    same_cache(g, c)
    assert csa2.get_device_status() == 0


def test_append_edge_values():
    """Zero rows, the largest bf16, subnormals, a page whose scale stays."""
    rng = np.random.default_rng(6)
    bs, Hk, D = 16, 1, 64
    c = ref.new_cache(rng, 4, Hk, bs, D)
    c["k_scale"][1], c["v_scale"][1] = 100.0, 100.0   # far above the new rows
    c["k_scale"][2], c["v_scale"][2] = 0.0, 0.0
    g = gpu_cache(c)
    slots = np.array([0, 1, 16 + 7, 32 + 3, 48, 49], np.int64)
    x = np.zeros((6, 2, D), np.float32)
    x[2] = ref.bf16(rng.standard_normal((2, D)).astype(np.float32))
    x[3] = np.float32(3.3895313892515355e38)           # the largest finite bf16
    x[4] = 1e-40
    x[5] = -2e-40
    x = ref.bf16(x)
    ref.append(c, x[:, :1], x[:, 1:], slots)
    csa2.kv8_append(g, dev_bf16(x)[:, :1], dev_bf16(x)[:, 1:], dev(slots))
    same_cache(g, c)
    assert csa2.get_device_status() == 0


def test_slots_past_the_cache_are_skipped_and_recorded():
    rng = np.random.default_rng(7)
    c = ref.new_cache(rng, 2, 2, 16, 64)
    g = gpu_cache(c)
    slots = np.array([3, 32, 1 << 40, -5], np.int64)
    x = ref.bf16(rng.standard_normal((4, 4, 64)).astype(np.float32))
    ref.append(c, x[:, :2], x[:, 2:], slots)
    csa2.kv8_append(g, dev_bf16(x)[:, :2], dev_bf16(x)[:, 2:], dev(slots))
    same_cache(g, c)
    assert csa2.get_device_status() == 1
    k, _ = csa2.kv8_unpack(g, dev(slots))
    assert (k[1:] == 0).all() and (k[0] != 0).any()
    assert csa2.get_device_status() == 1


# --- choice of blocks ---------------------------------------------------------

def run_select(rng, lens, adds, H, Hk, D, bs, n_sel, n_first=1, n_last=1, pad=0, edit=None):
    table, cu, P = make_step(rng, lens, adds, bs)
    c = ref.new_cache(rng, P, Hk, bs, D)
    n = int(cu[-1]) + pad
    q = ref.bf16(rng.standard_normal((n, H + 1, D)).astype(np.float32))
    if edit:
        edit(c, table, q)
    want = np.full((n, Hk, n_sel), -7, np.int32)
    ref.select(q[:, 1:], c, table, cu, lens, n_sel, n_first, n_last, want)
    out = torch.full((n, Hk, n_sel), -7, dtype=torch.int32, device="cuda")
    csa2.kv8_select(dev_bf16(q)[:, 1:], gpu_cache(c), dev(table), dev(cu),
                    dev(np.array(lens, np.int32)), n_sel, n_first, n_last, out=out)
    got = out.cpu().numpy()
    assert np.array_equal(got, want), np.argwhere((got != want).any(-1))[:5]


@pytest.mark.parametrize("lens,adds,H,Hk,D,bs,n_sel", [
    ([1], [1], 1, 1, 64, 16, 2), ([40], [1], 4, 2, 64, 16, 2), ([1000], [1], 8, 1, 128, 16, 9),
    ([5000, 17, 800], [1, 1, 1], 16, 4, 128, 16, 32), ([2000, 2000], [5, 0], 6, 2, 64, 32, 20),
    ([3000], [150], 8, 2, 128, 64, 7), ([700, 64, 129], [70, 64, 1], 4, 4, 64, 64, 4),
    ([20000], [3], 2, 1, 128, 16, 64), ([9000, 300], [9, 40], 16, 1, 128, 128, 5),
    ([70000], [2], 4, 1, 64, 16, 128), ([5, 0, 33], [5, 0, 33], 2, 2, 128, 32, 3)])
def test_select(lens, adds, H, Hk, D, bs, n_sel):
    run_select(np.random.default_rng(sum(lens) + n_sel), lens, adds, H, Hk, D, bs, n_sel)
    assert csa2.get_device_status() == 0


@pytest.mark.parametrize("n_first,n_last,n_sel", [(0, 1, 1), (0, 1, 6), (3, 4, 7), (3, 4, 12),
                                                  (2, 30, 40), (0, 1, 4096)])
def test_select_forced_blocks_and_padding(n_first, n_last, n_sel):
    run_select(np.random.default_rng(n_sel), [900, 20], [20, 20], 4, 2, 64, 16, n_sel, n_first,
               n_last, pad=3)
    assert csa2.get_device_status() == 0


def test_select_ties_zero_and_non_finite_queries():
    def edit(c, table, q):
        c["k_sum"][:] = c["k_sum"][0]              # every block of a head ties up to its scale
        c["k_scale"][:] = np.float32(0.5)
        c["k_scale"][::3] = np.float32(0.25)
        q[0] = 0.0
        q[1, :, 3] = np.inf
        q[2, :, 5] = np.nan
        q[3, :, 0] = 3.0e38                        # a group sum beyond fp32

    run_select(np.random.default_rng(3), [1500], [6], 4, 2, 64, 16, 11, edit=edit)
    assert csa2.get_device_status() == 0


def test_select_extreme_sums_and_a_bad_page():
    def edit(c, table, q):
        c["k_sum"][:, :, :] = np.where(np.arange(c["k_sum"].shape[2]) % 2, 16256, -16256)
        c["k_sum"][::2] *= -1
        q[:] = np.where(np.arange(q.shape[2]) % 2, 2.0, -2.0)
        table[0, 4], table[0, 9] = -1, 10 ** 6

    run_select(np.random.default_rng(4), [128 * 40], [3], 2, 1, 128, 128, 12, edit=edit)
    assert csa2.get_device_status() == 1


# --- attention ----------------------------------------------------------------

def run_attn(rng, lens, adds, H, Hk, D, bs, sel=None, pad=0, edit=None, sm_scale=None, peak=1.0,
             extra_width=1):
    """sel: None, or a function (rng, n, Hk, blocks of each token) -> lists."""
    table, cu, P = make_step(rng, lens, adds, bs, extra_width=extra_width)
    c = ref.new_cache(rng, P, Hk, bs, D)
    n = int(cu[-1]) + pad
    q = ref.bf16((peak * rng.standard_normal((n, H + 1, D))).astype(np.float32))
    if edit:
        edit(c, table, q)
    lists = None
    if sel is not None:
        blocks = [pos // bs + 1 if b >= 0 and pos >= 0 else 0
                  for _, b, pos in ref.positions(cu, lens, n)]
        lists = sel(rng, n, Hk, blocks).astype(np.int32)
    out = torch.full((n, H, D), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((n, H), 7.0, device="cuda")
    csa2.kv8_attn(dev_bf16(q)[:, 1:], gpu_cache(c), dev(table), dev(cu),
                  dev(np.array(lens, np.int32)), sel=None if lists is None else dev(lists),
                  sm_scale=sm_scale, out=out, lse=lse)
    want, want_lse, info = ref.attn(q[:, 1:], c, table, cu, lens, lists, sm_scale)
    check_attn(out, lse, want, want_lse, info, int(cu[-1]))


def check_attn(out, lse, want, want_lse, info, n):
    got, got_lse = out.float().cpu().numpy(), lse.cpu().numpy()
    assert (got[n:] == 7).all() and (got_lse[n:] == 7).all(), "padding rows were written"
    got, got_lse, want, want_lse = got[:n], got_lse[:n], want[:n], want_lse[:n]
    tol, tol_lse = ref.attn_bounds(want, want_lse, [x[:n] for x in info])
    assert np.array_equal(np.isneginf(got_lse), np.isneginf(want_lse))
    empty = np.isneginf(want_lse)
    assert (got[empty] == 0).all()
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), (f"out: {bad.sum()} of {bad.size} off, worst "
                           f"{np.nanmax(np.abs(got - want) / tol)} of its bound, first "
                           f"{np.argwhere(bad)[0]}")
    d = np.abs(got_lse[~empty] - want_lse[~empty])
    assert (d <= tol_lse[~empty]).all(), (d / tol_lse[~empty]).max()


SHAPES = [
    ([1], [1], 1, 1, 64, 16), ([1], [1], 1, 1, 128, 128), ([2], [2], 2, 2, 64, 32),
    ([17], [1], 8, 2, 64, 16), ([64], [1], 4, 4, 128, 64), ([65], [1], 16, 1, 128, 64),
    ([1000], [1], 8, 2, 64, 32), ([300, 1, 0, 77], [1, 1, 0, 1], 16, 2, 128, 64),
    ([5000, 31, 2049], [1, 1, 1], 16, 4, 128, 128), ([700, 700], [5, 5], 16, 4, 128, 64),
    ([333, 90], [3, 8], 6, 2, 64, 16), ([400], [7], 32, 1, 64, 32), ([260], [2], 96, 2, 128, 16),
    ([200], [200], 4, 2, 64, 64), ([500, 40], [129, 40], 8, 2, 128, 32),
    ([1300], [300], 16, 4, 128, 64), ([150, 600, 20], [150, 77, 1], 4, 4, 64, 128),
    ([130], [130], 16, 1, 128, 16), ([257], [100], 5, 1, 128, 64), ([90, 35], [64, 33], 24, 8, 64, 16),
    # long and short sequences in one step
    ([700, 300, 40, 9, 1200], [90, 1, 1, 0, 1], 16, 4, 128, 64),
    ([33, 800, 260], [1, 200, 6], 8, 2, 64, 16), ([400, 64, 700, 5], [1, 64, 8, 2], 16, 2, 128, 32),
    ([50, 60], [8, 9], 8, 2, 64, 64), ([300, 500, 100], [32, 33, 2], 3, 3, 128, 128),
]


@pytest.mark.parametrize("lens,adds,H,Hk,D,bs", SHAPES)
def test_attn_all_blocks(lens, adds, H, Hk, D, bs):
    run_attn(np.random.default_rng(sum(lens) + H), lens, adds, H, Hk, D, bs, pad=2)
    assert csa2.get_device_status() == 0


@pytest.mark.parametrize("lens,adds,H,Hk,D,bs", [
    ([700, 300, 40, 9, 1200], [90, 1, 1, 0, 1], 16, 4, 128, 64),
    ([33, 800, 260], [1, 200, 6], 8, 2, 64, 16), ([400, 64, 700, 5], [1, 64, 8, 2], 16, 2, 128, 32),
    ([300, 500, 100], [32, 133, 2], 3, 3, 128, 128), ([900, 50, 0], [300, 50, 0], 4, 2, 64, 64),
    ([64, 64, 64, 64], [33, 32, 31, 64], 8, 8, 128, 32), ([1, 2, 2000], [1, 2, 600], 32, 1, 64, 32)])
def test_attn_long_and_short_sequences_under_a_wide_table(lens, adds, H, Hk, D, bs):
    """Tables that reach far: both attention kernels, each on its own sequences."""
    run_attn(np.random.default_rng(sum(lens) + D), lens, adds, H, Hk, D, bs, pad=3,
             extra_width=(1 << 17) // bs)
    assert csa2.get_device_status() == 0


def some_blocks(n_sel):
    def make(rng, n, Hk, blocks):
        s = np.full((n, Hk, n_sel), -1)
        for i in range(n):
            for h in range(Hk):
                m = min(blocks[i], n_sel)
                s[i, h, :m] = np.sort(rng.permutation(blocks[i])[:m])
        return s
    return make


@pytest.mark.parametrize("lens,adds,H,Hk,D,bs", SHAPES)
@pytest.mark.parametrize("n_sel", [1, 6, 40])
def test_attn_listed_blocks(lens, adds, H, Hk, D, bs, n_sel):
    run_attn(np.random.default_rng(sum(lens) + H + n_sel), lens, adds, H, Hk, D, bs,
             sel=some_blocks(n_sel), pad=1)
    assert csa2.get_device_status() == 0


def test_attn_lists_in_any_order_with_gaps_and_empty_ones():
    def make(rng, n, Hk, blocks):
        s = np.full((n, Hk, 9), -1)
        for i in range(n):
            for h in range(Hk):
                m = (i + h) % 8
                s[i, h, rng.permutation(9)[:m]] = rng.permutation(blocks[i])[:m]
        s[3] = -1                     # sees nothing
        s[4, 0] = 10 ** 6             # blocks that the token does not see
        return s

    run_attn(np.random.default_rng(8), [900], [40], 8, 2, 128, 32, sel=make)
    assert csa2.get_device_status() == 0


@pytest.mark.parametrize("T", [1, 40])
def test_attn_bad_pages_are_skipped_and_recorded(T):
    def edit(c, table, q):
        table[0, 1], table[0, 3], table[1, :] = -1, 10 ** 6, -1

    run_attn(np.random.default_rng(9), [300, 50], [T, T], 8, 2, 64, 32, edit=edit)
    assert csa2.get_device_status() == 1


@pytest.mark.parametrize("T", [2, 70])
def test_attn_more_new_tokens_than_length(T):
    """Tokens at negative positions see nothing."""
    run_attn(np.random.default_rng(10), [T - 1, 1, 0], [T, 2, 1], 4, 2, 64, 16)
    assert csa2.get_device_status() == 0


@pytest.mark.parametrize("T", [1, 100])
def test_attn_table_narrower_than_the_sequence(T):
    """Blocks past the table's width are skipped and recorded."""
    rng = np.random.default_rng(11)
    lens, bs = [500], 32
    table, cu, P = make_step(rng, lens, [T], bs)
    table = np.ascontiguousarray(table[:, :9])
    c = ref.new_cache(rng, P, 2, bs, 128)
    q = ref.bf16(rng.standard_normal((T, 4, 128)).astype(np.float32))
    out, lse = csa2.kv8_attn(dev_bf16(q), gpu_cache(c), dev(table), dev(cu), dev(np.int32(lens)))
    check_attn(out, lse, *ref.attn(q, c, table, cu, lens), T)
    assert csa2.get_device_status() == 1


@pytest.mark.parametrize("T", [1, 64])
@pytest.mark.parametrize("peak,sm_scale", [(30.0, None), (1e-3, None), (1.0, -0.2), (1.0, 0.0),
                                           (1e4, 1e-5), (1e30, 1e-31)])
def test_attn_peaked_flat_and_scaled_logits(T, peak, sm_scale):
    run_attn(np.random.default_rng(12), [700, 90], [T, 1], 8, 2, 128, 64, peak=peak,
             sm_scale=sm_scale)
    assert csa2.get_device_status() == 0


@pytest.mark.parametrize("T", [1, 70])
@pytest.mark.parametrize("first", [None, 1e-39, 1e30])
def test_attn_scales_far_apart(T, first):
    """Pages of zeros, tiny and large value scales beside one another; a first
    page whose scale is far from all others."""
    def edit(c, table, q):
        c["v_scale"][:] = np.float32(10.0) ** np.random.default_rng(1).integers(
            -9, 4, c["v_scale"].shape).astype(np.float32)
        c["v_scale"][::3] = 0.0
        c["k_scale"][::4] = 0.0
        if first is not None:
            c["v_scale"][table[:, 0]] = np.float32(first)

    run_attn(np.random.default_rng(13), [600, 200], [T, 1], 8, 2, 64, 16, edit=edit)
    assert csa2.get_device_status() == 0


@pytest.mark.parametrize("T", [1, 70])
def test_attn_extreme_codes(T):
    def edit(c, table, q):
        c["k"][:] = np.where(c["k"] >= 0, 127, -127)
        c["v"][:] = np.where(c["v"] >= 0, 127, -128)

    run_attn(np.random.default_rng(14), [400], [T], 8, 2, 128, 64, edit=edit)
    assert csa2.get_device_status() == 0


def test_attn_rows_of_unwritten_pages_do_not_leak():
    """NaN scales of pages that no token sees, and codes behind the last
    token, change nothing."""
    rng = np.random.default_rng(15)
    lens, bs, Hk, D = [70, 33], 32, 2, 64
    table, cu, P = make_step(rng, lens, [1, 1], bs, spare=4)
    c = ref.new_cache(rng, P, Hk, bs, D)
    q = dev_bf16(ref.bf16(rng.standard_normal((2, 4, D)).astype(np.float32)))
    args = (dev(table), dev(cu), dev(np.int32(lens)))
    a = csa2.kv8_attn(q, gpu_cache(c), *args)
    for b, n in enumerate(lens):
        c["k"][table[b, n // bs], :, n % bs:] = 127
        c["v"][table[b, n // bs], :, n % bs:] = -128
    unused = np.setdiff1d(np.arange(P), table[table >= 0])
    c["k_scale"][unused], c["v_scale"][unused] = np.nan, np.nan
    b = csa2.kv8_attn(q, gpu_cache(c), *args)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("T", [2, 3, 90])
@pytest.mark.parametrize("H", [4, 8])
def test_attn_non_finite_queries_stay_in_their_rows(T, H):
    rng = np.random.default_rng(16)
    table, cu, P = make_step(rng, [200], [T], 64)
    c = ref.new_cache(rng, P, 2, 64, 128)
    q = ref.bf16(rng.standard_normal((T, H, 128)).astype(np.float32))
    args = (gpu_cache(c), dev(table), dev(cu), dev(np.int32([200])))
    a = csa2.kv8_attn(dev_bf16(q), *args)[0]
    q[1, 2, 5], q[1, 3, 5] = np.nan, np.inf
    b = csa2.kv8_attn(dev_bf16(q), *args)[0]
    ok = torch.ones(T, H, dtype=torch.bool)
    ok[1, 2:4] = False
    assert torch.equal(a[ok], b[ok])
    assert b[1, 2].isnan().all()


def test_attn_without_lse_and_on_another_stream():
    rng = np.random.default_rng(17)
    table, cu, P = make_step(rng, [900, 400], [1, 1], 64)
    c = ref.new_cache(rng, P, 2, 64, 128)
    q = dev_bf16(ref.bf16(rng.standard_normal((2, 16, 128)).astype(np.float32)))
    g, t, u, n = gpu_cache(c), dev(table), dev(cu), dev(np.int32([900, 400]))
    a, _ = csa2.kv8_attn(q, g, t, u, n)
    out = torch.empty_like(a)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        ws = torch.empty(csa2.kv8_attn_workspace_size(2, 2, 16, 2, 128), dtype=torch.uint8,
                         device="cuda")
        rc = csa2.lib().csa2_kv8_attn(q.data_ptr(), q.stride(0), g._ref, t.data_ptr(),
                                      t.shape[1], u.data_ptr(), n.data_ptr(), 2, 2, 16, None, 0,
                                      128 ** -0.5, out.data_ptr(), None, ws.data_ptr(),
                                      ws.numel(), st.cuda_stream)
    assert rc == csa2.CSA2_OK
    torch.cuda.synchronize()
    assert torch.equal(a, out)


def test_attn_results_do_not_depend_on_the_batch_order_of_runs():
    """The same call twice gives the same bits (no atomics in the sums)."""
    rng = np.random.default_rng(18)
    lens = [4000, 30, 900, 2500]
    table, cu, P = make_step(rng, lens, [1] * 4, 32)
    c = ref.new_cache(rng, P, 4, 32, 128)
    q = dev_bf16(ref.bf16(rng.standard_normal((4, 16, 128)).astype(np.float32)))
    args = (q, gpu_cache(c), dev(table), dev(cu), dev(np.int32(lens)))
    a = csa2.kv8_attn(*args)
    for _ in range(5):
        b = csa2.kv8_attn(*args)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def attn_on_gpu(q, c, table, cu, lens, sm_scale):
    """tests._kv8.attn in float64 on the GPU, a head at a time, for lengths that
    the host takes long for; no lists."""
    P, Hk, bs, D = c["k"].shape
    n, H = q.shape[:2]
    G = H // Hk
    x = {k: dev(v).double() for k, v in c.items() if k in ("k", "v", "k_scale", "v_scale")}
    qd = dev(q).double()
    out = torch.zeros((n, H, D), dtype=torch.float64, device="cuda")
    lse = torch.full((n, H), -np.inf, dtype=torch.float64, device="cuda")
    A, S = torch.zeros_like(out), torch.zeros_like(lse)
    N, M = torch.zeros_like(lse), torch.zeros_like(lse)
    for b, m in enumerate(lens):
        t0, t1 = int(cu[b]), int(cu[b + 1])
        if t1 == t0 or m == 0:
            continue
        pages = dev(table[b, :cdiv(m, bs)].astype(np.int64))
        pos = torch.arange(m - (t1 - t0), m, device="cuda")
        hidden = torch.arange(m, device="cuda")[None] > pos[:, None]
        for h in range(Hk):
            k = (x["k"][pages, h] * x["k_scale"][pages, h][:, None, None]).reshape(-1, D)[:m]
            v = (x["v"][pages, h] * x["v_scale"][pages, h][:, None, None]).reshape(-1, D)[:m]
            for a in range(h * G, (h + 1) * G):
                y = (qd[t0:t1, a] @ k.T * sm_scale).masked_fill(hidden, -np.inf)
                lse[t0:t1, a] = torch.logsumexp(y, -1)
                w = (y - lse[t0:t1, a][:, None]).exp()
                out[t0:t1, a] = w @ v
                A[t0:t1, a] = w @ v.abs()
                S[t0:t1, a] = (qd[t0:t1, a].abs() @ k.abs().T).amax(-1) * abs(sm_scale)
                N[t0:t1, a] = (pos + 1).double()
                M[t0:t1, a] = 127 * x["v_scale"][pages, h].max()
    return [y.cpu().numpy() for y in (out, lse)] + [[y.cpu().numpy() for y in (A, S, N, M)]]


@pytest.mark.parametrize("lens,adds,H,Hk,D,bs", [
    ([50000, 3000, 1], [1, 1, 1], 16, 2, 128, 64), ([30000, 9000], [1, 1], 4, 1, 64, 16),
    ([20000], [1], 8, 8, 128, 128), ([25000, 700], [5, 5], 16, 4, 128, 64),
    ([18000, 18000], [4, 7], 16, 4, 64, 32), ([6000, 4000], [700, 300], 16, 4, 128, 64),
    ([5000], [1500], 8, 2, 64, 16), ([9000, 100, 3000], [33, 100, 257], 32, 2, 128, 32),
    ([2500], [2500], 4, 4, 128, 128), ([7000], [900], 12, 4, 64, 64),
    ([20000, 9000, 3000, 40], [1, 500, 1, 40], 16, 4, 128, 64)])
def test_attn_long(lens, adds, H, Hk, D, bs):
    rng = np.random.default_rng(sum(lens) + D)
    table, cu, P = make_step(rng, lens, adds, bs)
    c = ref.new_cache(rng, P, Hk, bs, D)
    n = int(cu[-1])
    q = ref.bf16(rng.standard_normal((n, H, D)).astype(np.float32))
    g, args = gpu_cache(c), (dev(table), dev(cu), dev(np.int32(lens)))
    want = attn_on_gpu(q, c, table, cu, lens, D ** -0.5)
    first = None
    for _ in range(3):  # the same bits every time
        out, lse = csa2.kv8_attn(dev_bf16(q), g, *args)
        check_attn(out, lse, *want, n)
        first = first or (out, lse)
        assert torch.equal(out, first[0]) and torch.equal(lse, first[1])
    if n <= 20:  # every block listed: the same rows through the lists
        width = max(cdiv(m, bs) for m in lens)
        sel = np.broadcast_to(np.arange(width, dtype=np.int32), (n, Hk, width))
        out, lse = csa2.kv8_attn(dev_bf16(q), g, *args, sel=dev(sel))
        check_attn(out, lse, *want, n)
    assert csa2.get_device_status() == 0


def test_cache_beyond_32_bit_offsets():
    """Pages whose codes lie past 4 GiB: write, read back, choose, attend."""
    rng = np.random.default_rng(21)
    Hk, bs, D, H = 4, 128, 128, 8
    P = (1 << 32) // (Hk * bs * D) + 12
    assert (P - 1) * Hk * bs * D > 1 << 32
    if torch.cuda.mem_get_info()[0] < 12 << 30:
        pytest.skip("needs 12 GB of device memory")
    g = csa2.KV8Cache(*(torch.empty(s, dtype=d, device="cuda") for s, d in (
        ((P, Hk, bs, D), torch.int8), ((P, Hk, bs, D), torch.int8), ((P, Hk), torch.float32),
        ((P, Hk), torch.float32), ((P, Hk, D), torch.int16))))
    used = np.array([P - 1, 3, P - 2, P - 7, 0, P - 3], np.int32)
    small = ref.new_cache(rng, len(used), Hk, bs, D)   # those pages alone
    at = dev(used.astype(np.int64))
    for name in ("k", "v", "k_scale", "v_scale", "k_sum"):
        getattr(g, name)[at] = dev(small[name])
    # three pages for each of two sequences; one decode token and 30 tokens
    for adds, lens in (([1, 1], [300, 384]), ([30, 30], [330, 380])):
        cu = np.concatenate([[0], np.cumsum(adds)]).astype(np.int32)
        n = int(cu[-1])
        local = np.arange(6, dtype=np.int32).reshape(2, 3)
        pos = np.concatenate([np.arange(m - a, m) for m, a in zip(lens, adds)])
        seq = np.repeat([0, 1], adds)
        slots = local[seq, pos // bs].astype(np.int64) * bs + pos % bs
        x = ref.bf16(rng.standard_normal((n, H + 2 * Hk, D)).astype(np.float32))
        ref.append(small, x[:, H:H + Hk], x[:, H + Hk:], slots)
        far = used[local[seq, pos // bs]].astype(np.int64) * bs + pos % bs
        xs = dev_bf16(x)
        csa2.kv8_append(g, xs[:, H:H + Hk], xs[:, H + Hk:], dev(far))
        for name in ("k_scale", "v_scale", "k_sum", "k", "v"):
            assert np.array_equal(getattr(g, name)[at].cpu().numpy(), small[name]), name
        k, v = csa2.kv8_unpack(g, dev(far))
        assert np.array_equal(k.cpu().numpy(), (
            small["k"].astype(np.float32) * small["k_scale"][:, :, None, None]).transpose(
                0, 2, 1, 3).reshape(-1, Hk, D)[slots])
        args = (dev(used[local]), dev(cu), dev(np.int32(lens)))
        lists = np.zeros((n, Hk, 2), np.int32)
        ref.select(x[:, :H], small, local, cu, lens, 2, 0, 1, lists)
        got = csa2.kv8_select(xs[:, :H], g, *args, 2, 0, 1)
        assert np.array_equal(got.cpu().numpy(), lists)
        for sel in (None, lists):
            out, lse = csa2.kv8_attn(xs[:, :H], g, *args, sel=None if sel is None else got)
            check_attn(out, lse, *ref.attn(x[:, :H], small, local, cu, lens, sel), n)
    assert csa2.get_device_status() == 0


def test_calls_on_two_streams_at_once():
    """Calls with scratch of their own run side by side; each keeps its bits."""
    rng = np.random.default_rng(22)
    jobs = []
    for lens, adds, H, Hk in (([6000, 900], [1, 1], 16, 2), ([1500], [200], 8, 2),
                              ([4000, 4000], [5, 5], 16, 4)):
        table, cu, P = make_step(rng, lens, adds, 32)
        c = ref.new_cache(rng, P, Hk, 32, 128)
        q = dev_bf16(ref.bf16(rng.standard_normal((int(cu[-1]), H, 128)).astype(np.float32)))
        args = (q, gpu_cache(c), dev(table), dev(cu), dev(np.int32(lens)))
        sel = csa2.kv8_select(*args, 6)
        jobs.append((args, sel, csa2.kv8_attn(*args), csa2.kv8_attn(*args, sel=sel)))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in jobs]
    got = [[] for _ in jobs]
    for _ in range(8):
        for (args, sel, _, _), st, res in zip(jobs, streams, got):
            with torch.cuda.stream(st):
                s = csa2.kv8_select(*args, 6)
                res.append((s, csa2.kv8_attn(*args), csa2.kv8_attn(*args, sel=s)))
    torch.cuda.synchronize()
    for (args, sel, dense, listed), res in zip(jobs, got):
        for s, a, b in res:
            assert torch.equal(s, sel)
            assert all(torch.equal(x, y) for x, y in zip(a + b, dense + listed))
    assert csa2.get_device_status() == 0


# --- together -----------------------------------------------------------------

def test_a_serving_run_prompt_decode_drafts_then_a_captured_step():
    """Tables, append, choice of blocks and attention as a server runs them:
    prompts in one step, decode steps, drafts; then a decode step captured into
    a graph and replayed on changed inputs."""
    rng = np.random.default_rng(19)
    B, H, Hk, D, bs, width, n_sel = 3, 8, 2, 128, 16, 24, 6
    P = B * width
    c = ref.new_cache(rng, P, Hk, bs, D)
    g = gpu_cache(c)
    lens, table = np.zeros(B, np.int32), np.full((B, width), -1, np.int32)
    free = rng.permutation(P).astype(np.int32)
    g_table = dev(table)

    def host_step(add, x, sel):
        nonlocal lens, table, free
        n = int(sum(add))
        new_lens, cu, slots, pos, used, table = ref.block_tables(lens, add, table, free, bs, n)
        ref.append(c, x[:n, H:H + Hk], x[:n, H + Hk:], slots)
        lists = None
        if sel:
            lists = np.zeros((n, Hk, n_sel), np.int32)
            ref.select(x[:n, :H], c, table, cu, new_lens, n_sel, 1, 1, lists)
        res = ref.attn(x[:n, :H], c, table, cu, new_lens, lists)
        lens, free = new_lens, free[used:]
        return res, lists

    def gpu_step(g_lens, g_add, g_free, x, cap, sel):
        lens_out, cu, slots, pos, used = csa2.block_tables(g_lens, g_add, g_table, g_free, bs, cap)
        csa2.kv8_append(g, x[:, H:H + Hk], x[:, H + Hk:], slots)
        lists = csa2.kv8_select(x[:, :H], g, g_table, cu, lens_out, n_sel) if sel else None
        out, lse = csa2.kv8_attn(x[:, :H], g, g_table, cu, lens_out, sel=lists)
        return out, lse, lists

    def inputs(n):
        return ref.bf16(rng.standard_normal((n, H + 2 * Hk, D)).astype(np.float32))

    for add, sel in (([150, 7, 64], False), ([1, 1, 1], False), ([1, 1, 1], True),
                     ([5, 5, 5], True)):
        n = sum(add)
        x = inputs(n)
        out, lse, lists = gpu_step(dev(lens), dev(np.int32(add)), dev(free), dev_bf16(x), n, sel)
        want, want_lists = host_step(add, x, sel)
        if sel:
            assert np.array_equal(lists.cpu().numpy(), want_lists)
        check_attn(out, lse, *want, n)
        same_cache(g, c)

    # one decode step as a graph, inputs in fixed buffers
    s_lens, s_add, s_free = dev(lens), dev(np.int32([1] * B)), dev(free)
    s_x = dev_bf16(inputs(B))
    saved = [t.clone() for t in (g.k, g.v, g.k_scale, g.v_scale, g.k_sum, g_table)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        gpu_step(s_lens, s_add, s_free, s_x, B, True)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        res = gpu_step(s_lens, s_add, s_free, s_x, B, True)
    for t, old in zip((g.k, g.v, g.k_scale, g.v_scale, g.k_sum, g_table), saved):
        t.copy_(old)
    for _ in range(3):
        x = inputs(B)
        s_x.copy_(dev_bf16(x))
        s_lens.copy_(dev(lens))
        s_free[:len(free)].copy_(dev(free))
        graph.replay()
        torch.cuda.synchronize()
        want, want_lists = host_step([1] * B, x, True)
        assert np.array_equal(res[2].cpu().numpy(), want_lists)
        check_attn(res[0], res[1], *want, B)
        same_cache(g, c)
    assert csa2.get_device_status() == 0

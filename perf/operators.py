"""The 8-bit paged key/value cache and the attention over it: what is measured of them.

Five operators: block tables and slot maps from request lengths (``block_tables``), the cache's
writer and reader (``kv8_append``, ``kv8_unpack``), the choice of blocks by a cheap score
(``kv8_select``) and the attention over all or the chosen blocks (``kv8_attn``).

The cache: P pages of ``bs`` tokens; int8 codes k, v [P, Hk, bs, D], fp32 scales k_scale, v_scale
[P, Hk], int16 k_sum [P, Hk, D] (the sum of the page's key codes).  Sequence b owns the tokens
cu[b] .. cu[b+1]-1 of the step and has lens[b] tokens in the cache once they are written.

Where ``own`` is false ``run`` computes the operators from elementary torch operations.
"""
import math
import random

import numpy as np
import torch

own = False


# --- cases ------------------------------------------------------------------------------------

def listed():
    """Head counts, dims, batch sizes and context lengths are those of the repository's own
    workloads (8 or 16 query heads of 64 or 128; batches 1, 4, 8, 32; 4,096 to 262,144 positions;
    2,048 selected positions; 5 draft tokens; 4,096-token chunks)."""
    return [
        # a decode step's bookkeeping: every request adds one token
        {"name": "tables_decode_b32", "op": "tables", "B": 32, "T": 1, "N": 4096, "bs": 64,
         "ragged": True},
        # admission of many requests at once, ragged prompts
        {"name": "tables_chunks_b512", "op": "tables", "B": 512, "T": 256, "N": 32768, "bs": 32,
         "ragged": True},
        # the per-token write of a decode step, in the middle of a page
        {"name": "append_decode_b32", "op": "append", "B": 32, "T": 1, "N": 4096, "Hk": 4,
         "D": 128, "bs": 64, "ragged": True},
        # a prefill chunk's write, ragged, over many pages
        {"name": "append_chunk_t4096", "op": "append", "B": 4, "T": 4096, "N": 16384, "Hk": 4,
         "D": 128, "bs": 64, "ragged": True},
        # 2,048 positions of 262,144 for one decode token: 32 blocks of 64
        {"name": "select_decode_n262144", "op": "select", "B": 4, "T": 1, "N": 262144, "H": 16,
         "Hk": 4, "D": 128, "bs": 64, "n_sel": 32, "ragged": False},
        # every token of a prefill chunk chooses its own blocks
        {"name": "select_chunk_t4096", "op": "select", "B": 1, "T": 4096, "N": 65536, "H": 16,
         "Hk": 4, "D": 128, "bs": 64, "n_sel": 32, "ragged": False},
        # one short request alone: latency
        {"name": "attn_tiny_n1024", "op": "attn", "B": 1, "T": 1, "N": 1024, "H": 8, "Hk": 2,
         "D": 64, "bs": 32, "n_sel": 0, "ragged": False},
        # a full decode batch over long ragged contexts
        {"name": "attn_decode_b32_n131072", "op": "attn", "B": 32, "T": 1, "N": 131072, "H": 16,
         "Hk": 2, "D": 128, "bs": 64, "n_sel": 0, "ragged": True},
        # five draft tokens verified together over the longest context
        {"name": "attn_drafts_t5_n262144", "op": "attn", "B": 4, "T": 5, "N": 262144, "H": 16,
         "Hk": 4, "D": 128, "bs": 64, "n_sel": 0, "ragged": False},
        # a prefill chunk over its own tokens and a cached prefix
        {"name": "attn_chunk_t2048_n16384", "op": "attn", "B": 1, "T": 2048, "N": 16384, "H": 16,
         "Hk": 4, "D": 128, "bs": 64, "n_sel": 0, "ragged": False},
        # decode over the chosen blocks only
        {"name": "sel_decode_b32_n131072", "op": "attn", "B": 32, "T": 1, "N": 131072, "H": 16,
         "Hk": 2, "D": 128, "bs": 64, "n_sel": 32, "ragged": True},
        # every token of a chunk over its own chosen blocks
        {"name": "sel_chunk_t1024_n32768", "op": "attn", "B": 1, "T": 1024, "N": 32768, "H": 16,
         "Hk": 4, "D": 128, "bs": 64, "n_sel": 32, "ragged": False},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    """Any operator, page size, head layout and length of the listed ranges, at most the largest
    listed case's cache, scores and gathers."""
    op = rng.choice(["tables", "append", "select", "attn", "attn", "attn"])
    bs = rng.choice([16, 32, 64, 128])
    if op == "tables":
        return {"op": op, "B": _log(rng, 1, 512), "T": _log(rng, 1, 256),
                "N": _log(rng, 256, 32768), "bs": bs, "ragged": rng.random() < 0.8}
    D = rng.choice([64, 128])
    Hk = rng.choice([1, 2, 4, 8])
    if op == "append":
        B, T = _log(rng, 1, 64), rng.choice([1, rng.randint(2, 8), _log(rng, 16, 4096)])
        while B * T > 16384:
            B = max(1, B // 2)
        return {"op": op, "B": B, "T": T, "N": T + _log(rng, 1, 8192), "Hk": Hk, "D": D, "bs": bs,
                "ragged": rng.random() < 0.7}
    G = rng.choice([1, 2, 4, 8, 16])
    H = Hk * G if Hk * G <= 32 else 16
    Hk = min(Hk, H)
    if op == "select":
        B, T = _log(rng, 1, 16), rng.choice([1, rng.randint(2, 8), _log(rng, 64, 4096)])
        N = T + _log(rng, 64 * bs, 262144)  # blocks enough for a choice
        while B * (N // bs) * Hk * T > 1 << 24 or B * (N // bs) * Hk > 65536:
            B, T = max(1, B // 2), max(1, (T * 3) // 4)
            N = max(T + 64 * bs, (N * 3) // 4)
        return {"op": op, "B": B, "T": T, "N": N, "H": H, "Hk": Hk, "D": D, "bs": bs,
                "n_sel": rng.randint(4, min(64, N // (8 * bs))), "ragged": rng.random() < 0.5}
    n_sel = rng.choice([0, 0, rng.randint(4, 2048 // bs + 4)])
    B, T = _log(rng, 1, 64), rng.choice([1, 1, rng.randint(2, 8), _log(rng, 16, 2048)])
    N = T + _log(rng, 1, 262144)
    while (B * N * Hk * D * 2 > 1 << 30 or B * T * H * N > 1 << 29
           or B * T * Hk * n_sel * bs * D > 1 << 30):
        if B > 1:
            B = max(1, B // 2)
        elif n_sel:
            n_sel, T = (n_sel + 1) // 2, (T + 1) // 2
        else:
            N = max(T, (N * 3) // 4)
            T = min(T, N)
    return {"op": op, "B": B, "T": T, "N": N, "H": H, "Hk": Hk, "D": D, "bs": bs, "n_sel": n_sel,
            "ragged": rng.random() < 0.6}


def _lengths(case):
    """(tokens in the cache after the step, new tokens) per sequence.  Ragged: lengths from N / 3
    to N, new tokens from T / 4 to T, and in a batch of eight or more some sequences that add
    nothing."""
    B, T, N = case["B"], case["T"], case["N"]
    total, new = [], []
    for b in range(B):
        t, n = T, N
        if case["ragged"]:
            t = max(1, T - T * ((b * 13) % 16) // 20)
            n = N - N * ((b * 29) % 32) // 48
            if B >= 8 and b % 8 == 5:
                t = 0
        total.append(max(n, t))
        new.append(t)
    return total, new


def _pages(tokens, bs):
    return -(-tokens // bs)


# --- inputs -----------------------------------------------------------------------------------

def _ints(values, dtype=torch.int32):
    return torch.tensor(values, dtype=dtype, device="cuda")


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    host = random.Random(seed)
    op, B, bs = case["op"], case["B"], case["bs"]
    total, new = _lengths(case)
    cu = [0]
    for t in new:
        cu.append(cu[-1] + t)
    s = {"case": case, "n": cu[-1]}

    if op == "tables":
        before = [max(0, n - t - host.randint(0, bs)) for n, t in zip(total, new)]
        have = [_pages(x, bs) for x in before]
        pool = sum(have) + sum(_pages(x + t, bs) for x, t in zip(before, new))
        order = torch.randperm(pool, generator=g, device="cuda", dtype=torch.int32)
        width = max(_pages(n, bs) for n in total) + 1
        table = torch.full((B, width), -1, dtype=torch.int32, device="cuda")
        held = torch.arange(width, device="cuda")[None] < _ints(have)[:, None]
        table[held] = order[:sum(have)]
        s.update(lens=_ints(before), add=_ints(new), table=table,
                 free=order[sum(have):].contiguous(), cap=cu[-1] + 7)
        return s

    Hk, D = case["Hk"], case["D"]
    if op == "append":
        # the pages that the step touches, in a random order
        first = [(n - t) // bs for n, t in zip(total, new)]
        count = [_pages(n, bs) - f if t else 0 for n, t, f in zip(total, new, first)]
        P = max(1, sum(count))
        order = torch.randperm(P, generator=g, device="cuda")
        base = [0]
        for c in count:
            base.append(base[-1] + c)
        pos = np.concatenate([np.arange(n - t, n) - f * bs + b0 * bs
                              for n, t, f, b0 in zip(total, new, first, base)])
        pos = torch.from_numpy(pos).cuda()
        s["slots"] = order[pos // bs] * bs + pos % bs
        qkv = torch.randn((s["n"], 2 * Hk, D), generator=g, device="cuda")
        qkv *= 1 + 3 * (torch.rand((2 * Hk, D), generator=g, device="cuda") < 0.05)
        qkv = qkv.to(torch.bfloat16)
        s["k_new"], s["v_new"] = qkv[:, :Hk], qkv[:, Hk:]
        s["read"] = torch.arange(P * bs, device="cuda")
        s.update(_cache(g, P, Hk, bs, D, True))
        return s

    H = case["H"]
    blocks = [_pages(n, bs) for n in total]
    P = sum(blocks)
    order = torch.randperm(P, generator=g, device="cuda", dtype=torch.int32)
    width = max(blocks)
    held = torch.arange(width, device="cuda")[None] < _ints(blocks)[:, None]
    table = torch.full((B, width), -1, dtype=torch.int32, device="cuda")
    table[held] = order
    qkv = 2 * torch.randn((s["n"], H + 2 * Hk, D), generator=g, device="cuda")
    s.update(q=qkv.to(torch.bfloat16)[:, :H], table=table, cu=_ints(cu), lens=_ints(total))
    s.update(_cache(g, P, Hk, bs, D, op == "attn"))
    s["max_new"] = max(new)
    if op == "attn" and case["n_sel"]:
        # block 0, the token's own block and a random choice of the others
        _, seq, at = _token_rows(s)
        last = (at // bs)[:, None, None]
        j = torch.arange(width, device="cuda")
        key = torch.rand((s["n"], Hk, width), generator=g, device="cuda")
        key = torch.where((j == 0) | (j == last), 2.0, torch.where(j <= last, key, -1.0))
        val, idx = key.topk(min(case["n_sel"], width), dim=-1)
        idx = torch.where(val >= 0, idx, width).sort(dim=-1).values
        sel = torch.full((s["n"], Hk, case["n_sel"]), -1, dtype=torch.int32, device="cuda")
        sel[..., :idx.shape[-1]] = torch.where(idx < width, idx, -1).to(torch.int32)
        s["sel"] = sel
    return s


def _cache(g, P, Hk, bs, D, codes):
    """A cache in use: normal codes with a few strong key channels, scales of a page and head."""
    dev = "cuda"
    strong = 1 + 2 * (torch.rand((Hk, 1, D), generator=g, device=dev) < 0.04)
    s = {"k_scale": 0.03 * torch.exp(0.2 * torch.randn((P, Hk), generator=g, device=dev)),
         "v_scale": 0.02 * torch.exp(0.2 * torch.randn((P, Hk), generator=g, device=dev))}
    if not codes:  # the choice of blocks reads the sums alone
        x = torch.randn((P, Hk, D), generator=g, device=dev) * 400 * strong[:, 0]
        s["k_sum"] = x.round().clamp(-127 * bs, 127 * bs).to(torch.int16)
        s["k"] = torch.zeros((P, Hk, bs, D), dtype=torch.int8, device=dev)
        s["v"] = torch.zeros((P, Hk, bs, D), dtype=torch.int8, device=dev)
        return s
    for name, by in (("k", strong), ("v", 1)):
        s[name] = torch.empty((P, Hk, bs, D), dtype=torch.int8, device=dev)
        for part in s[name].split(max(1, (1 << 27) // (Hk * bs * D))):
            x = torch.randn(part.shape, generator=g, device=dev) * 28 * by
            part.copy_(x.round_().clamp_(-127, 127))
    s["k_sum"] = s["k"].sum(dim=2, dtype=torch.int32).to(torch.int16)
    return s


def _token_rows(s):
    """(token, its sequence, its position) of every token of the step."""
    cu, lens = s["cu"].long(), s["lens"].long()
    tok = torch.arange(s["n"], device=cu.device)
    seq = torch.searchsorted(cu[1:], tok, right=True)
    return tok, seq, lens[seq] - cu[seq + 1] + tok


# --- one pass ---------------------------------------------------------------------------------

def run(state):
    op = state["case"]["op"]
    if own:
        import compressed_sparse_attention_topk_b200 as csa2
        if op == "tables":
            names = ("lens", "cu", "slots", "pos", "used")
            out = csa2.block_tables(state["lens"], state["add"], state["table"], state["free"],
                                    state["case"]["bs"], state["cap"])
            return dict(zip(names, out), table=state["table"])
        if "cache" not in state:  # the handle that a program keeps beside its tensors
            state["cache"] = csa2.KV8Cache(state["k"], state["v"], state["k_scale"],
                                           state["v_scale"], state["k_sum"])
        cache = state["cache"]
        if op == "append":
            csa2.kv8_append(cache, state["k_new"], state["v_new"], state["slots"])
            k, v = csa2.kv8_unpack(cache, state["read"])
            return {"k": k, "v": v, "k_scale": state["k_scale"], "v_scale": state["v_scale"],
                    "k_sum": state["k_sum"]}
        if op == "select":
            return csa2.kv8_select(state["q"], cache, state["table"], state["cu"], state["lens"],
                                   state["case"]["n_sel"])
        out, lse = csa2.kv8_attn(state["q"], cache, state["table"], state["cu"], state["lens"],
                                 sel=state.get("sel"))
        return {"out": out, "lse": lse}
    if op == "tables":
        return _tables(state)
    if op == "append":
        return _append(state)
    if op == "select":
        return _select(state)
    return _attend_selected(state) if "sel" in state else _attend(state)


def _tables(s):
    bs, lens, add, table, free = s["case"]["bs"], s["lens"], s["add"], s["table"], s["free"]
    have, need = (lens + bs - 1) // bs, (lens + add + bs - 1) // bs
    taken = torch.cumsum(need - have, 0)
    j = torch.arange(table.shape[1], device=table.device)[None]
    at = (taken - (need - have) - have)[:, None] + j
    fresh = (j >= have[:, None]) & (j < need[:, None])
    page = free[at.clamp(0, free.numel() - 1)]
    table = torch.where(fresh, torch.where(at < free.numel(), page, -1), table)
    cu = torch.cat([torch.zeros_like(add[:1]), torch.cumsum(add, 0)]).to(torch.int32)
    tok = torch.arange(s["cap"], device=table.device)
    seq = torch.searchsorted(cu[1:].long(), tok, right=True)
    real = seq < lens.numel()
    seq = seq.clamp(max=lens.numel() - 1)
    pos = lens[seq] + tok - cu[seq]
    page = table[seq, torch.where(real, pos // bs, 0)].long()
    slots = torch.where(real & (page >= 0), page * bs + pos % bs, -1)
    return {"lens": lens + add, "cu": cu, "slots": slots,
            "pos": torch.where(real, pos, -1).to(torch.int32),
            "used": taken[-1:].to(torch.int32), "table": table}


def _append(s):
    bs = s["case"]["bs"]
    P, Hk, _, D = s["k"].shape
    page, row = s["slots"] // bs, s["slots"] % bs
    start = torch.full((P,), bs, device=row.device).scatter_reduce(0, page, row, "amin")
    end = torch.zeros((P,), dtype=row.dtype, device=row.device).scatter_reduce(0, page, row + 1,
                                                                               "amax")
    touched = (start < bs)[:, None]
    r = torch.arange(bs, device=row.device)
    old = (r < start[:, None])[:, None, :, None] & touched[:, :, None, None]
    q127 = torch.full((1,), 127.0, device=row.device)
    out = {}
    for name in ("k", "v"):
        x = s[name + "_new"].float()
        big = torch.zeros((P, Hk), device=row.device).scatter_reduce(
            0, page[:, None].expand(-1, Hk), x.abs().amax(-1), "amax")
        had = s[name + "_scale"]
        before = torch.where((start == 0)[:, None], 0.0, had)
        scale = torch.where(touched, torch.maximum(before, big / q127), had)
        ratio = torch.where(scale > 0, before / scale, 1.0)
        codes = s[name].float()
        codes = torch.where(old & (scale > before)[:, :, None, None],
                            torch.round(codes * ratio[:, :, None, None]), codes)
        of = scale[page][:, :, None]
        fresh = torch.where(of > 0, torch.round(x / of), 0.0).clamp(-127, 127)
        codes[page, :, row] = fresh
        out[name] = (codes * scale[:, :, None, None]).transpose(1, 2).reshape(P * bs, Hk, D)
        out[name + "_scale"] = scale
        if name == "k":
            held = (r < end[:, None])[:, None, :, None]
            total = torch.where(held, codes, 0.0).sum(2)
            out["k_sum"] = torch.where(touched[:, :, None], total, s["k_sum"].float()).to(
                torch.int16)
    return out


def _select(s):
    case = s["case"]
    bs, n_sel, Hk, D = case["bs"], case["n_sel"], case["Hk"], case["D"]
    tok, seq, at = _token_rows(s)
    n = s["n"]
    qs = s["q"].double().reshape(n, Hk, -1, D).sum(2).float()
    big = qs.abs().amax(-1, keepdim=True)
    q8 = torch.where(big > 0, torch.round(qs * (torch.full_like(big, 127.0) / big)), 0.0)
    # the dots reach 2^28: exact in 64 bits, over every sequence's blocks
    page = s["table"].clamp(min=0).long()
    q8p = torch.zeros((page.shape[0], s["max_new"], Hk, D), dtype=torch.float64, device=page.device)
    q8p[seq, tok - s["cu"].long()[seq]] = q8.double()
    dots = torch.einsum("bthd,bjhd->bthj", q8p, s["k_sum"][page].double())
    score = dots[seq, tok - s["cu"].long()[seq]].float() * s["k_scale"][page][seq].transpose(1, 2)
    j = torch.arange(page.shape[1], device=page.device)
    last = (at // bs)[:, None, None]
    score = torch.where((j == 0) | (j == last), math.inf, torch.where(j < last, score, -math.inf))
    val, idx = score.sort(dim=-1, descending=True, stable=True)
    val, idx = val[..., :n_sel], idx[..., :n_sel]
    none = page.shape[1]
    idx = torch.where(val > -math.inf, idx, none).sort(dim=-1).values
    out = torch.full((n, Hk, n_sel), -1, dtype=torch.int32, device=page.device)
    out[..., :idx.shape[-1]] = torch.where(idx < none, idx, -1).to(torch.int32)
    return out


def _softmax_rows(x, v):
    """Rows of logits x [..., q, s] (-inf: not seen) and values v [..., s, d] -> (out, lse)."""
    m = x.amax(-1, keepdim=True)
    m = torch.where(m > -math.inf, m, 0.0)
    p = (x - m).exp_()
    total = p.sum(-1, keepdim=True)
    out = torch.where(total > 0, (p @ v) / total, 0.0)
    return out, (m + total.log()).squeeze(-1)


def _attend(s):
    case = s["case"]
    bs, Hk, D, H = case["bs"], case["Hk"], case["D"], case["H"]
    G, T = H // Hk, s["max_new"]
    tok, seq, at = _token_rows(s)
    t = tok - s["cu"].long()[seq]
    page = s["table"].clamp(min=0).long()
    B, width = page.shape
    k = (s["k"][page] * s["k_scale"][page][..., None, None]).transpose(1, 2)
    k = k.reshape(B, Hk, width * bs, D)
    q = torch.zeros((B, T, H, D), device=page.device)
    q[seq, t] = s["q"].float()
    q = q.reshape(B, T, Hk, G, D).transpose(1, 2).reshape(B, Hk, T * G, D)
    x = (q @ k.transpose(2, 3)) * (1.0 / math.sqrt(D))
    del k
    seen = torch.zeros((B, T), dtype=torch.long, device=page.device)
    seen[seq, t] = at + 1
    seen = seen.repeat_interleave(G, 1)[:, None, :, None]
    x.masked_fill_(torch.arange(width * bs, device=page.device) >= seen, -math.inf)
    v = (s["v"][page] * s["v_scale"][page][..., None, None]).transpose(1, 2)
    out, lse = _softmax_rows(x, v.reshape(B, Hk, width * bs, D))
    out = out.reshape(B, Hk, T, G, D).transpose(1, 2).reshape(B, T, H, D)
    lse = lse.reshape(B, Hk, T, G).transpose(1, 2).reshape(B, T, H)
    return {"out": out[seq, t].to(torch.bfloat16), "lse": lse[seq, t]}


def _attend_selected(s):
    case = s["case"]
    bs, Hk, D, H = case["bs"], case["Hk"], case["D"], case["H"]
    n, sel = s["n"], s["sel"].long()
    _, seq, at = _token_rows(s)
    page = s["table"].long()[seq[:, None, None], sel.clamp(min=0)]
    h = torch.arange(Hk, device=page.device)[None, :, None]
    S = sel.shape[-1] * bs
    k = s["k"][page, h] * s["k_scale"][page, h][..., None, None]
    x = s["q"].float().reshape(n, Hk, -1, D) @ k.reshape(n, Hk, S, D).transpose(2, 3)
    del k
    key = sel[..., None] * bs + torch.arange(bs, device=page.device)
    hidden = (sel < 0)[..., None] | (key > at[:, None, None, None])
    x = (x * (1.0 / math.sqrt(D))).masked_fill_(hidden.reshape(n, Hk, 1, S), -math.inf)
    v = s["v"][page, h] * s["v_scale"][page, h][..., None, None]
    out, lse = _softmax_rows(x, v.reshape(n, Hk, S, D))
    return {"out": out.reshape(n, H, D).to(torch.bfloat16), "lse": lse.reshape(n, H)}


# --- the definition in 64 bits ----------------------------------------------------------------

def exact(case, seed):
    if case["op"] in ("tables", "select"):  # whole numbers
        return None
    s = prepare(case, seed)
    return _exact_append(s) if case["op"] == "append" else _exact_attn(s)


def _exact_append(s):
    """Page by page on the host.  The format's own fp32 roundings (scale, ratio, code) are part of
    the definition; the values that the codes stand for are products in 64 bits."""
    bs, f32 = s["case"]["bs"], np.float32
    slots = s["slots"].cpu().numpy()
    res = {}
    for name in ("k", "v"):
        codes = s[name].cpu().numpy().copy()
        scale = s[name + "_scale"].cpu().numpy().copy()
        x = s[name + "_new"].float().cpu().numpy()
        for p in np.unique(slots // bs):
            who = np.nonzero(slots // bs == p)[0]
            r0 = int(slots[who[0]] % bs)
            rows = x[who].transpose(1, 0, 2)                              # [Hk, m, D]
            old = scale[p] if r0 else np.zeros_like(scale[p])
            new = np.maximum(old, np.abs(rows).max((1, 2)).astype(f32) / f32(127))
            for h in np.nonzero(new > old)[0]:
                ratio = f32(old[h] / new[h])
                codes[p, h, :r0] = np.rint(codes[p, h, :r0].astype(f32) * ratio)
            with np.errstate(divide="ignore", invalid="ignore"):
                c = np.rint(rows / new[:, None, None])
            c = np.where(new[:, None, None] > 0, c, 0)
            codes[p, :, r0:r0 + len(who)] = np.clip(c, -127, 127)
            scale[p] = new
        P, Hk, _, D = codes.shape
        value = codes.astype(np.float64) * scale.astype(np.float64)[:, :, None, None]
        res[name] = value.transpose(0, 2, 1, 3).reshape(P * bs, Hk, D)
        res[name + "_scale"] = scale.astype(np.float64)
    res["k_sum"] = None
    return res


def _exact_attn(s):
    """Sequence by sequence, head by head, dense over the sequence's keys in float64."""
    case = s["case"]
    bs, Hk, D, H = case["bs"], case["Hk"], case["D"], case["H"]
    G = H // Hk
    total, new = _lengths(case)
    out = torch.zeros((s["n"], H, D), dtype=torch.float64, device="cuda")
    lse = torch.full((s["n"], H), -math.inf, dtype=torch.float64, device="cuda")
    t0 = 0
    for b, (n, t) in enumerate(zip(total, new)):
        if t == 0:
            continue
        pages = s["table"][b, :_pages(n, bs)].long()
        at = torch.arange(n - t, n, device="cuda")
        for h in range(Hk):
            k = s["k"][pages, h].double() * s["k_scale"][pages, h].double()[:, None, None]
            v = s["v"][pages, h].double() * s["v_scale"][pages, h].double()[:, None, None]
            k, v = k.reshape(-1, D)[:n], v.reshape(-1, D)[:n]
            see = torch.arange(n, device="cuda")[None] <= at[:, None]
            if "sel" in s:
                listed_blocks = torch.zeros((t, len(pages) + 1), dtype=torch.bool, device="cuda")
                chosen = s["sel"][t0:t0 + t, h].long()
                listed_blocks.scatter_(1, torch.where(chosen < 0, len(pages), chosen), True)
                see = see & listed_blocks[:, :-1].repeat_interleave(bs, 1)[:, :n]
            q = s["q"][t0:t0 + t, h * G:(h + 1) * G].double()
            for part in range(G):
                x = (q[:, part] @ k.T) / math.sqrt(D)
                x = x.masked_fill_(~see, -math.inf)
                norm = torch.logsumexp(x, -1)
                lse[t0:t0 + t, h * G + part] = norm
                out[t0:t0 + t, h * G + part] = (x - norm[:, None]).exp_() @ v
        t0 += t
    return {"out": out, "lse": lse}


# --- what a pass cannot do without ------------------------------------------------------------

def work(case):
    op, bs = case["op"], case["bs"]
    total, new = _lengths(case)
    n = sum(new)
    if op == "tables":
        # lengths in and out, the page of each block touched, the new pages, slots and positions
        return {"bytes": 16 * case["B"] + 12 * n + 12 * sum(_pages(t, bs) for t in new),
                "flops": 0}
    Hk, D = case["Hk"], case["D"]
    if op == "append":
        pages = sum(_pages(m, bs) - (m - t) // bs for m, t in zip(total, new) if t)
        earlier = sum((m - t) % bs for m, t in zip(total, new) if t)
        write = (4 * D + 2 * D) * Hk * n + D * Hk * earlier + (16 + 2 * D) * Hk * pages + 8 * n
        return {"bytes": write + (2 * D + 8 * D) * Hk * pages * bs, "flops": 0}
    H = case["H"]
    # keys that the tokens of a sequence see, and the cache that it reads
    sees = [t * m - t * (t - 1) // 2 for m, t in zip(total, new)]
    if op == "select":
        blocks = sum(_pages(m, bs) for m, t in zip(total, new) if t)
        return {"bytes": (2 * D + 8) * Hk * blocks + 2 * D * H * n + 4 * n * Hk * case["n_sel"],
                "flops": 2 * D * Hk * sum(sees) / bs}
    rows = 2 * D * H * n + 2 * D * H * n + 4 * H * n
    if case["n_sel"]:
        # each sequence's chosen blocks, at most its whole cache
        kept = [min(m, case["n_sel"] * bs) for m in total]
        read = sum(min(m, t * c) for m, t, c in zip(total, new, kept))
        return {"bytes": 2 * D * Hk * read + rows + 4 * n * Hk * case["n_sel"],
                "flops": 4 * D * H * sum(t * c for t, c in zip(new, kept))}
    read = sum(m for m, t in zip(total, new) if t)
    return {"bytes": (2 * D + 12 / bs) * Hk * read + rows, "flops": 4 * D * H * sum(sees)}

"""Operators over a paged key/value cache: appending rotated keys and values,
selecting pages by a cheap score, and attention over all or the selected pages.

Conventions (those of include/dsa.h).  Token i of sequence b has position
start[b] + i; its query row sees the positions s <= start[b] + i here (the
row's own token included: `inclusive`).  The cache is a pool of pages of `page`
tokens, [n_pages, n_kv, page, D]; block_table[b, j] is the pool page that holds
positions j * page .. j * page + page - 1 of sequence b.  An 8-bit cache holds
E4M3 codes with one power-of-two scale for each page and key/value head (for K
and for V).  A complete page has a summary: the mean of its cached keys in 8
bits (127 / amax), which the page selection scores.

Three operators, `op`:
  append  rotates q and the new keys by their positions (pairs i, i + rot/2 of
          the first rot columns), writes keys and values to their pages
          (quantised, rescaling the older tokens of a page whose scale grows),
          and the summaries of the pages that become complete.
  select  page scores (8-bit pooled query . 8-bit page summary, exact in whole
          numbers, times the page's scale), the best n_sel pages per row and
          key/value head; the first page and the last are always among them.
  attn    softmax attention of each query head over its key/value head's pages:
          all of them (sel = 0), or the selected ones.
"""
import math

import torch

own = False

PAGE_SCALE_MIN = 2.0 ** -100
ROT_BASE = 10000.0


# ---------------------------------------------------------------- the cases
def listed():
    return [
        # one token of one conversation joins a 16-bit cache: latency
        dict(name="append_decode_b1", op="append", B=1, lq=1, ctx=5000, n_h=32, n_kv=8, D=128, page=64, fmt="bf16", rot=128),
        # a decode step of 64 conversations, 8-bit cache, pages partly filled
        dict(name="append_decode_b64_8bit", op="append", B=64, lq=1, ctx=9001, n_h=64, n_kv=8, D=128, page=64, fmt="e4m3", rot=128),
        # the prompts of a prefill batch, ragged, part of the columns rotated
        dict(name="append_prompts_16k_8bit", op="append", B=5, lq=4096, ctx=5003, n_h=64, n_kv=8, D=128, page=64, fmt="e4m3", rot=64),
        # page choice of a decode step at 200,000 cached tokens
        dict(name="select_decode_b8_200k", op="select", B=8, lq=1, ctx=200000, n_h=64, n_kv=8, D=128, page=64, fmt="e4m3", n_sel=32),
        # page choice of every row of a prompt chunk, smaller heads
        dict(name="select_chunk_4k_at_32k", op="select", B=1, lq=4096, ctx=32768, n_h=28, n_kv=4, D=64, page=32, fmt="bf16", n_sel=64),
        # decode of one short conversation: latency
        dict(name="attn_decode_b1_1k", op="attn", B=1, lq=1, ctx=1001, n_h=32, n_kv=8, D=64, page=16, fmt="bf16", sel=0),
        # decode of 32 ragged conversations, 16-bit cache, an odd group of 7
        dict(name="attn_decode_b32_16k", op="attn", B=32, lq=1, ctx=16384, n_h=28, n_kv=4, D=128, page=64, fmt="bf16", sel=0),
        # decode over the whole 8-bit cache at 200,000 tokens: bytes
        dict(name="attn_decode_b8_200k_8bit", op="attn", B=8, lq=1, ctx=200000, n_h=64, n_kv=8, D=128, page=64, fmt="e4m3", sel=0),
        # the same step over 32 selected pages of each row and head
        dict(name="attn_decode_b8_200k_sel32", op="attn", B=8, lq=1, ctx=200000, n_h=64, n_kv=8, D=128, page=64, fmt="e4m3", sel=32),
        # a chunk of a long prompt over the whole 8-bit cache: arithmetic
        dict(name="attn_chunk_4k_at_16k_8bit", op="attn", B=1, lq=4096, ctx=16384, n_h=64, n_kv=8, D=128, page=64, fmt="e4m3", sel=0),
        # ragged prompts in one 16-bit batch, smaller heads, small pages
        dict(name="attn_prompts_b4_2k", op="attn", B=4, lq=2111, ctx=2111, n_h=28, n_kv=4, D=64, page=16, fmt="bf16", sel=0),
        # the chunk over 32 selected pages (2,048 tokens) of each row and head
        dict(name="attn_chunk_2k_at_32k_sel32", op="attn", B=1, lq=2048, ctx=32768, n_h=64, n_kv=8, D=128, page=64, fmt="e4m3", sel=32),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "select", "attn", "attn"])
    n_kv = rng.choice([1, 2, 4, 8])
    G = rng.choice([1, 2, 4, 5, 7, 8, 12, 16])
    c = dict(op=op, n_kv=n_kv, n_h=n_kv * G, D=rng.choice([64, 128]), page=rng.choice([16, 32, 64, 128]), fmt=rng.choice(["bf16", "e4m3"]))
    if rng.random() < 0.5:  # decode steps, now and then a few tokens for each sequence
        c["B"] = _log(rng, 1, 64)
        c["lq"] = rng.choice([1, 1, 1, 2, 5])
        c["ctx"] = _log(rng, 40, min(200000, 1600000 // c["B"]))
        c["lq"] = min(c["lq"], c["ctx"])
    else:  # prompts and chunks of prompts
        c["B"] = rng.choice([1, 1, 2, 3, 4])
        c["lq"] = _log(rng, 17, 4096 // c["B"])
        c["ctx"] = max(c["lq"], _log(rng, 17, 16384))
    if op == "append":
        c["rot"] = rng.choice([c["D"], c["D"] // 2])
    elif op == "select":
        c["n_sel"] = rng.choice([3, 8, 16, 32, 64])
    else:
        c["sel"] = 0 if rng.random() < 0.6 else max(2, rng.choice([512, 1024, 2048]) // c["page"])
    return c


def _lens(c):
    """Rows and first positions of each sequence: ragged downwards from lq and ctx."""
    q, start = [], []
    for b in range(c["B"]):
        lq = c["lq"] if b == 0 else max(1, c["lq"] - (b * c["lq"]) // (c["B"] + 1) - b % 2 * (c["lq"] > 9))
        ctx = c["ctx"] if b == 0 else max(lq, c["ctx"] - (b * 7919) % max(1, c["ctx"] // 2))
        q.append(lq)
        start.append(ctx - lq)
    return q, start


# ---------------------------------------------------------------- the inputs
def _pow2_scale(amax):
    """The smallest power of two X with amax <= 448 X, at least 2^-100."""
    m, e = torch.frexp(amax.float())
    return torch.ldexp(torch.ones_like(m), e - 9 + (m > 0.875).to(e.dtype)).clamp_min(PAGE_SCALE_MIN)


def _tree_sum(x):
    """Sum over dim 2 (a power of two long) by halving."""
    while x.shape[2] > 1:
        h = x.shape[2] // 2
        x = x[:, :, :h] + x[:, :, h:]
    return x[:, :, 0]


def _summary(k, scale):
    """8-bit summaries of pages k [n, n_kv, page, D] with scales [n, n_kv]."""
    total = _tree_sum(k.float()) * (1.0 if scale is None else scale[..., None])
    amax = total.abs().amax(-1, keepdim=True)
    ok = torch.isfinite(amax) & (amax > 0)
    codes = torch.where(ok, (total * (127.0 / amax)).round(), 0).to(torch.int8)
    return codes, torch.where(ok, amax / 127.0 * (1.0 / k.shape[2]), 0)[..., 0]


def prepare(case, seed):
    c = dict(case)
    dev = "cuda"
    g = torch.Generator(device=dev).manual_seed(seed)
    q_lens, start = _lens(c)
    B, page, n_kv, n_h, D = c["B"], c["page"], c["n_kv"], c["n_h"], c["D"]
    need = [-(-(s + n) // page) for s, n in zip(start, q_lens)]
    n_pages, max_pages = sum(need), max(need)
    order = torch.randperm(n_pages, generator=g, device=dev).to(torch.int32)
    bt = torch.zeros((B, max_pages), dtype=torch.int32, device=dev)
    at = 0
    for b, n in enumerate(need):
        bt[b, :n] = order[at:at + n]
        at += n
    cu = [0]
    for n in q_lens:
        cu.append(cu[-1] + n)
    total = cu[-1]
    st = dict(case=c, q_lens=q_lens, start=start, total=total, n_pages=n_pages, max_Lq=max(q_lens), max_Lk=max(s + n for s, n in zip(start, q_lens)),
              bt=bt, cu_q=torch.tensor(cu, dtype=torch.int32, device=dev), start_pos=torch.tensor(start, dtype=torch.int32, device=dev))
    st["seq"] = torch.repeat_interleave(torch.arange(B, device=dev), torch.tensor(q_lens, device=dev))
    st["pos"] = torch.arange(total, device=dev) - st["cu_q"].long()[st["seq"]] + st["start_pos"].long()[st["seq"]]

    def values(*shape, spread=1.0):
        return torch.randn(shape, generator=g, device=dev, dtype=torch.bfloat16) * spread

    # keys: a few channels with a constant part, as trained keys have; values:
    # tokens of different sizes
    k = values(n_pages, n_kv, page, D)
    k += 1.5 * (torch.rand((n_kv, 1, D), generator=g, device=dev) < 0.06).to(torch.bfloat16)
    v = values(n_pages, n_kv, page, D) * (0.25 + torch.rand((n_pages, n_kv, page, 1), generator=g, device=dev, dtype=torch.bfloat16))
    if c["op"] == "append":  # what is not yet in the cache is whatever was there
        st["k_new"], st["v_new"], st["q"] = values(total, n_kv, D, spread=1.5), values(total, n_kv, D), values(total, n_h, D, spread=2.0)
        half = c["rot"] // 2
        # angles of far positions: 64 bits until the sine and cosine
        inv = ROT_BASE ** (-torch.arange(half, device=dev, dtype=torch.float64) / half)
        ang = torch.arange(st["max_Lk"], device=dev, dtype=torch.float64)[:, None] * inv
        st["cos"], st["sin"] = ang.cos().float(), ang.sin().float()
    else:
        st["q"] = values(total, n_h, D, spread=2.0)
    if c["fmt"] == "e4m3":
        for name, x in (("k", k), ("v", v)):
            s = _pow2_scale(x.abs().amax((2, 3)))
            st[name + "_scale"] = s
            st[name] = (x / s[..., None, None].to(x.dtype)).to(torch.float8_e4m3fn)
    else:
        st["k"], st["v"], st["k_scale"], st["v_scale"] = k, v, None, None
    del k, v
    if c["op"] != "attn":
        st["sum"] = torch.empty((n_pages, n_kv, D), dtype=torch.int8, device=dev)
        st["sum_scale"] = torch.empty((n_pages, n_kv), dtype=torch.float32, device=dev)
        step = max(1, (1 << 26) // (n_kv * page * D))
        for a in range(0, n_pages, step):
            s = None if st["k_scale"] is None else st["k_scale"][a:a + step]
            st["sum"][a:a + step], st["sum_scale"][a:a + step] = _summary(st["k"][a:a + step], s)
    if c["op"] == "attn" and c["sel"]:
        # chosen pages: the first, the last, and others at random, ascending
        n = st["pos"] // page + 1
        score = torch.rand((total, n_kv, max_pages), generator=g, device=dev)
        p = torch.arange(max_pages, device=dev)
        score = score.masked_fill(p >= n[:, None, None], -1.0)
        score = score.masked_fill((p == 0) | (p == n[:, None, None] - 1), 2.0)
        top = score.topk(min(c["sel"], max_pages), dim=-1)
        sel = torch.where(top.values >= 0, top.indices, max_pages).sort(-1).values
        sel = torch.nn.functional.pad(sel, (0, c["sel"] - sel.shape[-1]), value=max_pages)
        st["sel"] = torch.where(sel < max_pages, sel, -1).to(torch.int32)
        del score, top, sel
    st["scale"] = 1.0 / math.sqrt(D)
    if own:
        from sparse_attention_13_b200 import dsa
        st["kv"] = dsa.PagedKV(st["k"], st["v"], st["k_scale"], st["v_scale"], st.get("sum"), st.get("sum_scale"))
        st["batch"] = dsa.PagedBatch(st["cu_q"], st["start_pos"], st["bt"], total_q=total, max_Lq=st["max_Lq"], max_Lk=st["max_Lk"])
    return st


# ---------------------------------------------------------------- one pass
def run(st):
    c = st["case"]
    if own:
        return _run_own(st, c)
    return {"append": _plain_append, "select": _plain_select, "attn": _plain_attn}[c["op"]](st, c)


def _run_own(st, c):
    from sparse_attention_13_b200 import dsa
    if c["op"] == "append":
        q = dsa.paged_append(st["kv"], st["batch"], st["k_new"], st["v_new"], st["cos"], st["sin"], q=st["q"])
        return _append_outputs(st, q)
    if c["op"] == "select":
        return {"sel": dsa.page_topk(st["q"], st["kv"], st["batch"], c["n_sel"], inclusive=True)}
    lse = torch.empty(st["q"].shape[:2], dtype=torch.float32, device="cuda")
    out = dsa.paged_attn(st["q"], st["kv"], st["batch"], st["scale"], sel=st.get("sel"), inclusive=True, lse=lse)
    return {"out": out, "lse": lse}


def _append_outputs(st, q):
    r = {"q": q, "k": st["k"], "v": st["v"], "sum": st["sum"], "sum_scale": st["sum_scale"]}
    if st["k_scale"] is not None:
        r["k_scale"], r["v_scale"] = st["k_scale"], st["v_scale"]
    return r


def _rotate(x, cos, sin, rot):
    """x [n, heads, D] f32 (or f64) by the angles of its rows, cos and sin [n, rot/2]."""
    a, b, rest = x[..., :rot // 2], x[..., rot // 2:rot], x[..., rot:]
    c, s = cos[:, None], sin[:, None]
    return torch.cat([a * c - b * s, b * c + a * s, rest], -1)


def _plain_append(st, c):
    page = c["page"]
    cos, sin = st["cos"][st["pos"]], st["sin"][st["pos"]]
    q = _rotate(st["q"].float(), cos, sin, c["rot"]).to(torch.bfloat16)
    k, v = _rotate(st["k_new"].float(), cos, sin, c["rot"]), st["v_new"].float()
    pid = st["bt"][st["seq"], st["pos"] // page].long()
    slot = st["pos"] % page
    # the pages that this call writes to, and the first new slot of each
    touched, inv = torch.unique(pid, return_inverse=True)
    first = torch.full((touched.numel(),), page, device="cuda", dtype=torch.long).scatter_reduce(0, inv, slot, "amin")
    last = torch.zeros((touched.numel(),), device="cuda", dtype=torch.long).scatter_reduce(0, inv, slot, "amax")
    for name, x in (("k", k), ("v", v)):
        pool = st[name]
        if c["fmt"] == "bf16":
            pool[pid, :, slot] = x.to(torch.bfloat16)
            continue
        scale = st[name + "_scale"]
        amax = torch.where(torch.isfinite(x), x.abs(), 0).amax(-1)
        amax = torch.zeros((touched.numel(), c["n_kv"]), device="cuda").index_reduce(0, inv, amax, "amax")
        old = torch.where(first[:, None] > 0, scale[touched], 0)
        new = torch.maximum(old, _pow2_scale(amax))
        codes = pool.view(torch.uint8)[touched].view(torch.float8_e4m3fn)
        again = (codes.float() * (old / new)[..., None, None]).to(torch.float8_e4m3fn)
        keep = torch.arange(page, device="cuda")[None, None, :, None] < first[:, None, None, None]
        pool.view(torch.uint8)[touched] = torch.where(keep, again.view(torch.uint8), codes.view(torch.uint8))
        x = (x / new[inv][..., None]).clamp(-448, 448).to(torch.float8_e4m3fn)
        pool.view(torch.uint8)[pid, :, slot] = x.view(torch.uint8)
        scale[touched] = new
    whole = touched[last == page - 1]
    k_pages = st["k"][whole] if c["fmt"] == "bf16" else st["k"].view(torch.uint8)[whole].view(torch.float8_e4m3fn)
    st["sum"][whole], st["sum_scale"][whole] = _summary(k_pages, None if st["k_scale"] is None else st["k_scale"][whole])
    return _append_outputs(st, q)


def _plain_select(st, c):
    n_kv, page, n_sel = c["n_kv"], c["page"], c["n_sel"]
    rows = st["total"]
    pooled = st["q"].view(rows, n_kv, -1, c["D"]).double().sum(2).float()
    amax = pooled.abs().amax(-1, keepdim=True)
    codes = torch.where(amax > 0, (pooled * (127.0 / amax)).round(), 0)
    n = (st["pos"] // page + 1)[:, None, None]
    p = torch.arange(st["bt"].shape[1], device="cuda")
    top_v, top_i = [], []
    for b in range(c["B"]):  # each sequence has pages of its own
        at = slice(sum(st["q_lens"][:b]), sum(st["q_lens"][:b + 1]))
        ids = st["bt"][b].long()
        # whole numbers below 2^24: exact in 32 bits whatever the order
        dot = torch.einsum("rkd,pkd->rkp", codes[at], st["sum"][ids].float())
        score = dot * st["sum_scale"][ids].t()
        score = score.masked_fill((p == 0) | (p == n[at] - 1), math.inf).masked_fill(p >= n[at], -math.inf)
        # equal scores: the lower page first
        val, idx = score.sort(dim=-1, descending=True, stable=True)
        val = torch.nn.functional.pad(val, (0, n_sel), value=-math.inf)[..., :n_sel]
        top_v.append(val), top_i.append(torch.nn.functional.pad(idx, (0, n_sel))[..., :n_sel])
    none = st["bt"].shape[1]
    idx = torch.where(torch.cat(top_v) > -math.inf, torch.cat(top_i), none).sort(-1).values
    return {"sel": torch.where(idx < none, idx, -1).to(torch.int32)}


def _pages(st, name, ids, dtype):
    """The cached values of pages `ids`, [n_kv, n * page, D], dequantised."""
    pool, scale = st[name], st[name + "_scale"]
    if scale is None:
        x = pool[ids].to(dtype)
    else:
        x = pool.view(torch.uint8)[ids].view(torch.float8_e4m3fn).to(dtype) * scale[ids][..., None, None].to(dtype)
    return x.transpose(0, 1).reshape(pool.shape[1], -1, pool.shape[3])


def _attend(q, k, v, scale, seen):
    """q [n_kv, G, rows, D] over k, v [n_kv, L, D]; seen [n_kv or 1, rows, L]."""
    s = torch.einsum("hgrd,hld->hgrl", q, k) * scale
    s.masked_fill_(~seen[:, None], -math.inf)
    m = s.amax(-1, keepdim=True)
    s = s.sub_(m).exp_()
    total = s.sum(-1, keepdim=True)
    return torch.einsum("hgrl,hld->hgrd", s, v) / total, (m + total.log())[..., 0]


def _plain_attn(st, c, dtype=torch.float32):
    n_kv, page = c["n_kv"], c["page"]
    G = c["n_h"] // n_kv
    outs, lses = [], []
    at = 0
    for b, lq in enumerate(st["q_lens"]):
        L = st["start"][b] + lq
        ids = st["bt"][b, :-(-L // page)].long()
        k, v = _pages(st, "k", ids, dtype), _pages(st, "v", ids, dtype)
        pos = torch.arange(k.shape[1], device="cuda")
        rows_at_once = max(1, (1 << 30) // (c["n_h"] * k.shape[1]))
        for r in range(0, lq, rows_at_once):
            rows = slice(at + r, at + min(lq, r + rows_at_once))
            seen = (pos <= st["pos"][rows, None])[None]
            if c["sel"]:
                chosen = torch.zeros((rows.stop - rows.start, n_kv, st["bt"].shape[1] + 1), dtype=torch.bool, device="cuda")
                chosen.scatter_(2, st["sel"][rows].long() % chosen.shape[2], True)  # -1: the last, which is no page
                seen = seen & chosen.transpose(0, 1)[..., pos // page]
            q = st["q"][rows].to(dtype).view(-1, n_kv, G, c["D"]).permute(1, 2, 0, 3)
            o, lse = _attend(q, k, v, st["scale"], seen)
            outs.append(o.permute(2, 0, 1, 3).reshape(-1, c["n_h"], c["D"]).to(torch.bfloat16 if dtype is torch.float32 else dtype))
            lses.append(lse.permute(2, 0, 1).reshape(-1, c["n_h"]))
        at += lq
    return {"out": torch.cat(outs), "lse": torch.cat(lses)}


# ---------------------------------------------------------------- the floor
def work(case):
    c = case
    q_lens, start = _lens(c)
    rows = sum(q_lens)
    e = 1 if c["fmt"] == "e4m3" else 2
    n_kv, n_h, D, page = c["n_kv"], c["n_h"], c["D"], c["page"]
    if c["op"] == "append":
        # new keys, values and queries in, rotated queries and the cache's
        # rows out; the angles; the other keys of pages that become complete
        older = sum(s % page for s, n in zip(start, q_lens) if (s + n) // page > s // page)
        pages = sum((s + n - 1) // page - s // page + 1 for s, n in zip(start, q_lens))
        whole = sum((s + n) // page - s // page for s, n in zip(start, q_lens))
        b = rows * (2 * n_kv * D * (2 + e) + 4 * n_h * D + 4 * c["rot"]) + older * n_kv * D * e + whole * n_kv * (D + 4)
        b += pages * n_kv * 8 * (e == 1)
        return {"bytes": b, "flops": rows * (n_h + n_kv) * c["rot"] * 3 + rows * n_kv * D * 2}
    seen = [[s + i + 1 for i in range(n)] for s, n in zip(start, q_lens)]
    if c["op"] == "select":
        pages = [[-(-t // page) for t in x] for x in seen]
        b = rows * (n_h * D * 2 + n_kv * c["n_sel"] * 4) + sum(max(x) for x in pages) * (n_kv * (D + 4) + 4)
        return {"bytes": b, "flops": sum(map(sum, pages)) * n_kv * D * 2}
    io = rows * n_h * (4 * D + 4)
    if not c["sel"]:
        keys = sum(max(x) for x in seen)
        pairs = sum(map(sum, seen))
        return {"bytes": io + keys * n_kv * D * e * 2 + 4 * (keys // page), "flops": pairs * n_h * D * 4}
    each = [[min(t, (c["sel"] - 1) * page + (t - 1) % page + 1) for t in x] for x in seen]
    # a page is read once for each sequence at the least
    keys = sum(min(max(x), sum(y)) for x, y in zip(seen, each))
    return {"bytes": io + keys * n_kv * D * e * 2 + rows * n_kv * c["sel"] * 4, "flops": sum(map(sum, each)) * n_h * D * 4}


# ---------------------------------------------------------------- the definition in 64 bits
def _to_e4m3(x):
    """Nearest E4M3 values of x in 64 bits: 4 significant bits, ties to even, saturated; steps of 2^-9 below 2^-6."""
    _, e = torch.frexp(x)
    step = torch.ldexp(torch.ones_like(x), (e - 4).clamp_min(-9))
    return ((x / step).round() * step).clamp(-448, 448)


def exact(case, seed):
    if case["op"] == "select":  # whole numbers
        return None
    st = prepare(case, seed)
    c = st["case"]
    f8 = c["fmt"] == "e4m3"
    if c["op"] == "append":
        return _exact_append(st, c, f8)
    n_kv, page, D = c["n_kv"], c["page"], c["D"]
    G = c["n_h"] // n_kv
    out = torch.empty((st["total"], n_kv, G, D), dtype=torch.float64, device="cuda")
    lse = torch.empty((st["total"], n_kv, G), dtype=torch.float64, device="cuda")
    at = 0
    for b, lq in enumerate(st["q_lens"]):
        L = st["start"][b] + lq
        tok = torch.arange(L, device="cuda")
        ids, slots = st["bt"][b].long()[tok // page], tok % page
        for h in range(n_kv):
            K = (st["k"].view(torch.uint8)[ids, h, slots].view(torch.float8_e4m3fn) if f8 else st["k"][ids, h, slots]).double()
            V = (st["v"].view(torch.uint8)[ids, h, slots].view(torch.float8_e4m3fn) if f8 else st["v"][ids, h, slots]).double()
            if f8:
                K, V = K * st["k_scale"].double()[ids, h, None], V * st["v_scale"].double()[ids, h, None]
            step = max(1, (1 << 27) // (G * L))
            for r in range(0, lq, step):
                n = min(step, lq - r)
                x = st["q"][at + r:at + r + n, h * G:(h + 1) * G].double().reshape(n * G, D) @ K.t() / math.sqrt(D)
                x = x.view(n, G, L)
                gone = tok[None, :] > (st["start"][b] + r + torch.arange(n, device="cuda"))[:, None]
                if c["sel"]:
                    chosen = (st["sel"][at + r:at + r + n, h, :, None] == torch.arange(st["bt"].shape[1], device="cuda")).any(1)
                    gone = gone | ~chosen[:, tok // page]
                x = x.masked_fill(gone[:, None], -math.inf)
                z = torch.logsumexp(x, -1)
                lse[at + r:at + r + n, h] = z
                out[at + r:at + r + n, h] = ((x - z[..., None]).exp().view(n * G, L) @ V).view(n, G, D)
        at += lq
    return {"out": out.view(-1, c["n_h"], D), "lse": lse.view(-1, c["n_h"])}


def _exact_append(st, c, f8):
    page, half = c["page"], c["rot"] // 2
    cos, sin = st["cos"].double()[st["pos"]], st["sin"].double()[st["pos"]]

    def turned(x):
        z = torch.complex(x[..., :half], x[..., half:2 * half]) * torch.complex(cos, sin)[:, None]
        return torch.cat([z.real, z.imag, x[..., 2 * half:]], -1)

    q = turned(st["q"].double())
    new = {"k": turned(st["k_new"].double()), "v": st["v_new"].double()}
    pools, scales = {}, {}
    summ, summ_scale = st["sum"].clone(), st["sum_scale"].double()
    for name in ("k", "v"):
        pools[name] = st[name].double()
        if f8:
            scales[name] = st[name + "_scale"].double()
    at = 0
    for b, lq in enumerate(st["q_lens"]):  # page by page, token by token's page
        p0, end = st["start"][b], st["start"][b] + lq
        for j in range(p0 // page, (end - 1) // page + 1):
            lo, hi = max(p0, j * page), min(end, (j + 1) * page)
            pg = int(st["bt"][b, j])
            a, n = lo - j * page, hi - lo
            for name in ("k", "v"):
                x = new[name][at + lo - p0:at + hi - p0].transpose(0, 1)  # [n_kv, n, D]
                if not f8:
                    pools[name][pg, :, a:a + n] = x
                    continue
                r = x.abs().amax((1, 2))
                X = torch.exp2(torch.ceil(torch.log2((r / 448).clamp_min(PAGE_SCALE_MIN))))
                X = torch.where(r <= 448 * X / 2, X / 2, X)  # log2 may have been a rounding above
                if a:
                    old = scales[name][pg]
                    X = torch.maximum(X, old)
                    pools[name][pg, :, :a] = _to_e4m3(pools[name][pg, :, :a] * (old / X)[:, None, None])
                scales[name][pg] = X
                pools[name][pg, :, a:a + n] = _to_e4m3(x / X[:, None, None])
            if hi == (j + 1) * page:
                mean = (pools["k"][pg] if f8 else pools["k"][pg].to(torch.bfloat16).double()).mean(1)
                if f8:
                    mean = mean * scales["k"][pg][:, None]
                summ_scale[pg] = mean.abs().amax(-1) / 127
        at += lq
    r = {"q": q, "k": pools["k"], "v": pools["v"], "sum": None, "sum_scale": summ_scale}
    if f8:
        r["k_scale"], r["v_scale"] = scales["k"], scales["v"]
    return r

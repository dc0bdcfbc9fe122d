"""GPU parity of the paged-cache operators (dsa_paged_append, dsa_page_topk,
dsa_paged_attn) against plain 64-bit forms, at the sizes and masks where they
can go wrong."""
import math

import pytest
import torch

import paged_ref as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dsa():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from sparse_attention_13_b200 import dsa as _dsa
    _dsa.lib()
    return _dsa


def _gen(seed):
    return torch.Generator().manual_seed(seed)


def _angles(n_pos, rot):
    inv = 10000.0 ** (-torch.arange(rot // 2, dtype=torch.float64) / max(1, rot // 2))
    a = torch.arange(n_pos, dtype=torch.float64)[:, None] * inv
    return a.cos().float(), a.sin().float()


def _table(q_lens, starts, page, g, spare=3):
    """Pool pages of each sequence in random order, and the pool's size."""
    need = [-(-(s + n) // page) for s, n in zip(starts, q_lens)]
    order = torch.randperm(sum(need) + spare, generator=g).tolist()
    table, at = [], 0
    for n in need:
        table.append(order[at:at + n])
        at += n
    width = max(max(need), 1)
    t = torch.full((len(need), width), -1, dtype=torch.int32)
    for b, row in enumerate(table):
        t[b, :len(row)] = torch.tensor(row, dtype=torch.int32)
    return table, t.cuda(), sum(need) + spare


def _pool(dsa, n_pages, page, n_kv, D, fmt, fill_nan=True, summaries=True):
    """A pool whose every byte is NaN (and NaN scales): what no call has
    written must not matter."""
    kv = dsa.PagedKV.empty(n_pages, page, n_kv, D, fmt=fmt, summaries=summaries)
    if fill_nan:
        for t in (kv.k, kv.v):
            t.view(torch.uint8).fill_(0xFF)
        for t in (kv.k_scale, kv.v_scale, kv.sum_scale):
            if t is not None:
                t.fill_(float("nan"))
        if kv.sum is not None:
            kv.sum.fill_(77)
    return kv


def _bf16(g, *shape, std=1.0):
    return (torch.randn(shape, generator=g) * std).to(torch.bfloat16)


def _filled(dsa, q_lens, starts, n_kv, D, page, fmt, seed, std=1.0, hook=None):
    """A cache that holds every position below start + rows of each sequence
    (appended as one prompt), its float64 mirror, and the batch of the rows."""
    g = _gen(seed)
    ends = [s + n for s, n in zip(starts, q_lens)]
    table, t, n_pages = _table(ends, [0] * len(ends), page, g)
    kv = _pool(dsa, n_pages, page, n_kv, D, fmt)
    total = sum(ends)
    k, v = _bf16(g, max(total, 1), n_kv, D, std=std), _bf16(g, max(total, 1), n_kv, D, std=std)
    if hook:
        hook(k, v)
    if total:
        fill = dsa.PagedBatch.from_lens(ends, [0] * len(ends), t)
        dsa.paged_append(kv, fill, k[:total].cuda(), v[:total].cuda())
    batch = dsa.PagedBatch.from_lens(q_lens, starts, t)
    return kv, ref.Cache(kv), batch, table, g


# ---------------------------------------------------------------- append
def _check_cache(kv, mirror, touched, before):
    """Touched pages equal the mirror (codes within one rounding of the f32
    rotation), all others are bit for bit what they were."""
    f8 = kv.k_scale is not None
    for name, scale in (("k", "ks"), ("v", "vs")):
        got = getattr(kv, name).cpu()
        want = getattr(mirror, name)
        if f8:
            assert torch.equal(getattr(kv, name + "_scale").cpu().double()[sorted(touched)], getattr(mirror, scale)[sorted(touched)])
        for pg in range(got.shape[0]):
            if pg not in touched:
                assert torch.equal(got[pg].view(torch.uint8), before[name][pg].view(torch.uint8)), f"{name} page {pg} was touched"
                continue
            x, y = got[pg].float().double(), want[pg]
            nan = torch.isnan(y)
            assert torch.equal(torch.isnan(x), nan)
            # a rotation in f32 moves a value by at most 3 * 2^-24 of its pair;
            # next to a border that is one step of the format
            step = y.abs().clamp_min(2.0 ** -6) * 2.0 ** -3 if f8 else y.abs().clamp_min(1e-30) * 2.0 ** -7
            assert ((x == y) | ((x - y).abs() <= step))[~nan].all()
            assert (x != y)[~nan].double().mean() <= 1e-3 + 8.0 / x.numel()


APPEND = [
    # q_lens, starts, n_h, n_kv, D, page, rot, interleaved
    ([1], [0], 8, 2, 64, 16, 64, False),
    ([1], [15], 8, 2, 128, 16, 128, False),           # completes a page
    ([1, 1, 0, 1], [63, 64, 10, 5], 12, 4, 128, 64, 64, True),
    ([33, 130, 1], [31, 0, 127], 6, 2, 64, 32, 32, False),
    ([300], [77], 7, 1, 128, 128, 128, True),
    ([2, 5], [127, 126], 16, 8, 64, 128, 16, False),
    ([17, 16, 15], [16, 0, 1], 4, 4, 64, 16, 0, False),
]


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("case", range(len(APPEND)))
def test_append(dsa, case, fmt):
    q_lens, starts, n_h, n_kv, D, page, rot, inter = APPEND[case]
    kv, mirror, batch, table, g = _filled(dsa, [0] * len(starts), starts, n_kv, D, page, fmt, 100 + case, std=0.3)
    # the rows of the call need pages of their own beyond those of the filled part
    ends = [s + n for s, n in zip(starts, q_lens)]
    need = [-(-e // page) for e in ends]
    extra = kv.k.shape[0]
    n_pages = extra + sum(need)
    big = _pool(dsa, n_pages, page, n_kv, D, fmt)
    for name in ("k", "v", "k_scale", "v_scale", "sum", "sum_scale"):
        if getattr(kv, name) is not None:
            getattr(big, name).view(torch.uint8)[:extra] = getattr(kv, name).view(torch.uint8)
    t = torch.full((len(need), max(max(need), 1)), -1, dtype=torch.int32)
    for b, n in enumerate(need):
        table[b] = table[b] + list(range(extra, extra + n - len(table[b])))
        extra += max(0, n - len(table[b]))
        extra = max(extra, max(table[b], default=0) + 1)
        t[b, :n] = torch.tensor(table[b][:n], dtype=torch.int32)
    kv, mirror = big, ref.Cache(big)
    batch = dsa.PagedBatch.from_lens(q_lens, starts, t.cuda())
    assert dsa.check_paged(kv, batch) == 0
    total = sum(q_lens)
    # a fused projection: q, k and v are slices of one row
    fused = _bf16(g, total, (n_h + 2 * n_kv) * D, std=1.5).cuda()
    q = fused[:, :n_h * D].unflatten(1, (n_h, D))
    k = fused[:, n_h * D:(n_h + n_kv) * D].unflatten(1, (n_kv, D))
    v = fused[:, (n_h + n_kv) * D:].unflatten(1, (n_kv, D))
    cos, sin = _angles(max(ends), rot) if rot else (None, None)
    dev = lambda x: None if x is None else x.cuda()  # noqa: E731
    before = {n: getattr(kv, n).cpu().clone() for n in ("k", "v")}
    before_sum = kv.sum.cpu().clone()
    q_out = dsa.paged_append(kv, batch, k, v, dev(cos), dev(sin), q=q, interleaved=inter)
    touched = set()
    mirror.append(q_lens, starts, table, k.cpu(), v.cpu(), cos, sin, inter, touched)
    _check_cache(kv, mirror, touched, before)
    pos = torch.cat([torch.arange(s, s + n) for s, n in zip(starts, q_lens)])
    want = ref.rotate(q.cpu().double(), cos, sin, pos, inter)
    x = q.cpu().double().abs()
    pair = x + (0 if not rot else x.amax(-1, keepdim=True))
    assert ((q_out.cpu().double() - want).abs() <= 2.0 ** -8 * want.abs() + 4 * 2.0 ** -24 * pair).all()
    # summaries: complete pages only
    done = {table[b][j] for b in range(len(ends)) for j in range(starts[b] // page, ends[b] // page) if q_lens[b]}
    for pg in range(kv.sum.shape[0]):
        if pg in done:
            assert (kv.sum[pg].cpu().int() - mirror.sum[pg].int()).abs().max() <= 2
            torch.testing.assert_close(kv.sum_scale[pg].cpu().double(), mirror.sum_scale[pg].double(), rtol=1e-2, atol=0)
        else:
            assert torch.equal(kv.sum[pg].cpu(), before_sum[pg])


def test_append_in_place_queries(dsa):
    g = _gen(5)
    table, t, n = _table([40], [0], 16, g)
    kv = _pool(dsa, n, 16, 2, 64, "bf16")
    batch = dsa.PagedBatch.from_lens([40], [0], t)
    cos, sin = (x.cuda() for x in _angles(40, 64))
    k, q = _bf16(g, 40, 2, 64).cuda(), _bf16(g, 40, 6, 64).cuda()
    want = dsa.paged_append(kv, batch, k, k, cos, sin, q=q)
    got = dsa.paged_append(kv, batch, k, k, cos, sin, q=q, q_out=q)
    assert got.data_ptr() == q.data_ptr() and torch.equal(got, want)


@pytest.mark.parametrize("D", [64, 128])
def test_append_token_by_token_equals_the_rule(dsa, D):
    # sizes grow along the page, so its scale grows again and again and the
    # older codes are rescaled each time
    page, n_kv, n = 32, 2, 70
    g = _gen(6)
    table, t, n_pages = _table([n], [0], page, g)
    kv = _pool(dsa, n_pages, page, n_kv, D, "e4m3")
    mirror = ref.Cache(kv)
    grow = 2.0 ** (torch.arange(n) * 0.4 % 9)[:, None, None]
    k, v = ((_bf16(g, n, n_kv, D).float() * grow).to(torch.bfloat16) for _ in range(2))
    batch = dsa.PagedBatch.from_lens([1], [0], t)
    batch = dsa.PagedBatch(batch.cu_q, batch.start_pos, t, total_q=1, max_Lq=1, max_Lk=n)
    for i in range(n):
        batch.start_pos.fill_(i)
        dsa.paged_append(kv, batch, k[i:i + 1].cuda(), v[i:i + 1].cuda())
        mirror.append([1], [i], table, k[i:i + 1], v[i:i + 1], None, None, False)
    for name, scale in (("k", "ks"), ("v", "vs")):
        got, want = getattr(kv, name).cpu().float().double(), getattr(mirror, name)
        for j in range(-(-n // page)):
            used = min(page, n - j * page)
            assert torch.equal(got[table[0][j], :, :used], want[table[0][j], :, :used])
        pages = table[0][:-(-n // page)]
        assert torch.equal(getattr(kv, name + "_scale").cpu().double()[pages], getattr(mirror, scale)[pages])
    whole = table[0][:n // page]
    assert torch.equal(kv.sum.cpu()[whole], mirror.sum[whole])


def test_append_special_values(dsa):
    # zeros, infinities, NaN, the largest and the smallest bf16 values
    page, n_kv, D = 16, 1, 64
    g = _gen(7)
    for fmt in ("e4m3", "bf16"):
        table, t, n_pages = _table([48], [0], page, g)
        kv = _pool(dsa, n_pages, page, n_kv, D, fmt)
        k = torch.zeros(48, 1, D, dtype=torch.bfloat16)
        k[16, 0, 0], k[17, 0, 1], k[18, 0, 2], k[19, 0, 3] = float("inf"), -float("inf"), float("nan"), 3.0
        k[32, 0, 0], k[33, 0, 1] = 3.3895314e38, 1e-38
        mirror = ref.Cache(kv)
        touched = set()
        before = {n: getattr(kv, n).cpu().clone() for n in ("k", "v")}
        dsa.paged_append(kv, dsa.PagedBatch.from_lens([48], [0], t), k.cuda(), k.cuda())
        mirror.append([48], [0], table, k, k, None, None, False, touched)
        _check_cache(kv, mirror, touched, before)
        assert (kv.sum[table[0][0]] == 0).all() and (kv.sum_scale[table[0][0]] == 0).all()
        assert (kv.sum[table[0][1]] == 0).all() and (kv.sum_scale[table[0][1]] == 0).all()


# ---------------------------------------------------------------- selection
SELECT = [
    # q_lens, starts, n_h, n_kv, D, page, n_sel, n_first, n_last, inclusive
    ([1], [0], 4, 2, 64, 16, 4, 1, 1, False),          # nothing visible
    ([1, 1, 1], [640, 639, 641], 8, 2, 128, 16, 8, 1, 1, True),
    ([40], [600], 14, 2, 64, 16, 5, 0, 1, False),
    ([7, 0, 130], [1000, 3, 0], 6, 6, 128, 32, 3, 1, 2, True),
    ([3], [5000], 128, 1, 64, 16, 100, 4, 9, True),
    ([1], [20000], 16, 8, 128, 16, 1024, 1, 1, False),
    ([2], [700], 2, 2, 64, 128, 1, 0, 1, True),
]


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("case", range(len(SELECT)))
def test_page_topk(dsa, case, fmt):
    q_lens, starts, n_h, n_kv, D, page, n_sel, n_first, n_last, inc = SELECT[case]
    kv, mirror, batch, table, g = _filled(dsa, q_lens, starts, n_kv, D, page, fmt, 200 + case)
    total = sum(q_lens)
    q = _bf16(g, total, n_h, D)
    got = dsa.page_topk(q.cuda(), kv, batch, n_sel, n_first=n_first, n_last=n_last, inclusive=inc).cpu()
    r = 0
    G = n_h // n_kv
    for b, n in enumerate(q_lens):
        for i in range(n):
            vis = -(-(starts[b] + i + inc) // page)
            for h in range(n_kv):
                pages = table[b][:vis]
                want = ref.select_row(q[r, h * G:(h + 1) * G].double(), mirror.sum[pages, h] if vis else mirror.sum[:0, h],
                                      mirror.sum_scale[pages, h] if vis else mirror.sum_scale[:0, h], vis, n_sel, n_first, n_last)
                assert got[r, h].tolist() == want, (b, i, h)
            r += 1


def test_page_topk_ties_and_signs(dsa):
    # few distinct summaries and scales, zero queries, negative scores: equal
    # scores go to the lower page
    g = _gen(8)
    page, n_kv, D, n = 16, 2, 64, 300
    kv = _pool(dsa, n, page, n_kv, D, "bf16")
    kv.sum.copy_(torch.randint(-1, 2, (n, n_kv, 1), generator=g).to(torch.int8).expand(n, n_kv, D))
    kv.sum_scale.copy_(2.0 ** torch.randint(-1, 1, (n, n_kv), generator=g).float())
    t = torch.randperm(n, generator=g).to(torch.int32)[None].cuda()
    batch = dsa.PagedBatch.from_lens([4], [n * page - 4], t)
    q = _bf16(g, 4, 4, D)
    q[1] = 0
    q[2] = float("inf")
    q[3] = -q[0]
    sel = dsa.page_topk(q.cuda(), kv, batch, 37, inclusive=True).cpu()
    pages = t[0].cpu().long()
    for r in range(4):
        for h in range(n_kv):
            vis = -(-(n * page - 4 + r + 1) // page)
            want = ref.select_row(q[r, 2 * h:2 * h + 2].double(), kv.sum.cpu()[pages[:vis], h], kv.sum_scale.cpu()[pages[:vis], h], vis, 37, 1, 1)
            assert sel[r, h].tolist() == want


# ---------------------------------------------------------------- attention
def _check_attn(dsa, kv, mirror, batch, table, q_lens, starts, q, scale, inc, sel=None, rows=None):
    total, n_h, D = q.shape
    n_kv, page = kv.k.shape[1], kv.k.shape[2]
    G = n_h // n_kv
    lse = torch.full((total + 1, n_h), 123.0, device="cuda")
    out = torch.full((total + 1, n_h, D), 55.0, dtype=torch.bfloat16, device="cuda")
    got = dsa.paged_attn(q.cuda(), kv, batch, scale, sel=None if sel is None else sel.cuda(), inclusive=inc, out=out[:total], lse=lse[:total])
    dsa.check_device_errors()
    assert (out[total] == 55.0).all() and (lse[total] == 123.0).all()  # behind the last row
    got, lse = got.cpu().double(), lse.cpu().double()
    r = 0
    for b, n in enumerate(q_lens):
        pages = table[b]
        for i in range(n):
            t = starts[b] + i + inc
            if rows is None or r in rows:
                for h in range(n_kv):
                    K, V = mirror.rows(pages, h)
                    seen = torch.arange(K.shape[0]) < t
                    if sel is not None:
                        chosen = torch.zeros(len(pages) + 1, dtype=torch.bool)
                        for e in sel[r, h].tolist():
                            if 0 <= e < len(pages):
                                chosen[e] = True
                        seen &= chosen[torch.arange(K.shape[0]) // page]
                    vmax = float(mirror.vs[pages, h][torch.isfinite(mirror.vs[pages, h])].max()) if mirror.f8 and pages else 0.0
                    for j in range(G):
                        o, z, tol, ztol = ref.attend_row(q[r, h * G + j].double(), K, V, seen, scale, vmax)
                        err = (got[r, h * G + j] - o).abs()
                        assert (err <= tol).all(), (b, i, h, j, float((err - tol).max()))
                        if z == -math.inf:
                            assert lse[r, h * G + j] == -math.inf
                        else:
                            assert abs(lse[r, h * G + j] - z) <= ztol, (b, i, h, j)
            r += 1


ATTN = [
    # q_lens, starts, n_h, n_kv, D, page, inclusive
    ([1], [0], 4, 2, 64, 16, False),                    # sees nothing
    ([1], [0], 4, 2, 128, 64, True),                    # sees itself
    ([1, 1, 1, 1], [127, 128, 129, 1000], 8, 1, 128, 64, False),
    ([1, 1], [3000, 77], 7, 1, 64, 32, True),
    ([1] * 5, [1, 16, 500, 2049, 33], 24, 2, 128, 16, True),
    ([1], [4100], 128, 4, 128, 128, True),              # groups of 32
    ([2], [515], 128, 1, 64, 64, True),                 # one head for all
    ([4, 1, 0, 2], [900, 30, 5, 0], 16, 2, 128, 64, True),   # a few rows each, an empty sequence
    ([9], [120], 6, 6, 64, 16, False),                  # a group of one
    ([70], [0], 8, 2, 128, 64, True),
    ([150, 3, 260], [0, 500, 133], 10, 2, 128, 64, True),
    ([300], [1000], 28, 4, 64, 32, False),
    ([129], [1], 5, 1, 128, 128, True),
    ([40, 257], [4000, 0], 32, 2, 64, 16, True),
]


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("case", range(len(ATTN)))
def test_attention_all_pages(dsa, case, fmt):
    q_lens, starts, n_h, n_kv, D, page, inc = ATTN[case]
    kv, mirror, batch, table, g = _filled(dsa, q_lens, starts, n_kv, D, page, fmt, 300 + case)
    total = sum(q_lens)
    q = _bf16(g, total, n_h, D, std=1.5)
    rows = None if total <= 80 else set(torch.randperm(total, generator=g)[:24].tolist()) | {0, total - 1}
    _check_attn(dsa, kv, mirror, batch, table, q_lens, starts, q, 1 / math.sqrt(D), inc, rows=rows)


SPARSE = [
    # q_lens, starts, n_h, n_kv, D, page, n_sel, inclusive
    ([1], [0], 4, 2, 64, 16, 3, False),
    ([1, 1, 1], [1000, 5, 64], 8, 2, 128, 64, 4, True),
    ([1], [9000], 16, 2, 128, 16, 65, True),
    ([20], [600], 14, 2, 64, 32, 7, False),
    ([130, 0, 5], [0, 9, 700], 8, 1, 128, 64, 5, True),
    ([33], [100], 40, 2, 128, 128, 1, True),
    ([300], [200], 4, 4, 64, 64, 3, True),
]


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("case", range(len(SPARSE)))
def test_attention_selected_pages(dsa, case, fmt):
    q_lens, starts, n_h, n_kv, D, page, n_sel, inc = SPARSE[case]
    kv, mirror, batch, table, g = _filled(dsa, q_lens, starts, n_kv, D, page, fmt, 400 + case)
    total = sum(q_lens)
    q = _bf16(g, total, n_h, D, std=1.5)
    sel = torch.full((total, n_kv, n_sel), -1, dtype=torch.int32)
    r = 0
    for b, n in enumerate(q_lens):
        for i in range(n):
            vis = -(-(starts[b] + i + inc) // page)
            for h in range(n_kv):
                pick = torch.randperm(vis, generator=g)[:n_sel]
                if (r + h) % 4 == 1:  # any order, holes, and pages that the row does not see
                    sel[r, h, n_sel - len(pick):] = pick.int()
                    sel[r, h, 0] = [-1, vis, 1 << 30, -5][r % 4]
                elif (r + h) % 7 != 6:  # (now and then a row with no page at all)
                    sel[r, h, :len(pick)] = pick.int().sort().values
            r += 1
    rows = None if total <= 40 else set(torch.randperm(total, generator=g)[:40].tolist()) | {0, total - 1}
    _check_attn(dsa, kv, mirror, batch, table, q_lens, starts, q, 1 / math.sqrt(D), inc, sel=sel, rows=rows)


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("lq", [1, 3, 140])
def test_attention_large_scores_and_unequal_scales(dsa, fmt, lq):
    # scores of hundreds (the softmax is nearly one-hot) and values whose size
    # differs by 2^30 between pages and heads
    def hook(k, v):
        k.mul_(8)
        v.mul_((2.0 ** (torch.arange(v.shape[0]) // 64 * 5 % 31 - 15))[:, None, None].to(v.dtype))
    kv, mirror, batch, table, g = _filled(dsa, [lq], [1500], 2, 128, 64, fmt, 500 + lq, hook=hook)
    q = _bf16(g, lq, 8, 128, std=4)
    rows = None if lq < 10 else {0, 1, 50, 138, 139}
    _check_attn(dsa, kv, mirror, batch, table, [lq], [1500], q, 1 / math.sqrt(128), True, rows=rows)


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("lq,sparse", [(1, False), (4, False), (150, False), (4, True)])
def test_nan_tokens_reach_only_the_rows_that_see_them(dsa, fmt, lq, sparse):
    # token 700 + lq - 1 (the last row's own) has NaN keys and values; only the
    # last row sees it.  All unused slots hold NaN throughout these tests.
    def hook(k, v):
        k[700 + lq - 1] = float("nan")
        v[700 + lq - 1] = float("nan")
    kv, mirror, batch, table, g = _filled(dsa, [lq], [700], 2, 64, 32, fmt, 600 + lq, hook=hook)
    q = _bf16(g, lq, 8, 64)
    sel = None
    if sparse:
        sel = torch.arange(17, 23, dtype=torch.int32).expand(lq, 2, 6).contiguous().cuda()
    out = dsa.paged_attn(q.cuda(), kv, batch, 0.125, sel=sel, inclusive=True)
    assert torch.isnan(out[lq - 1]).all()
    assert torch.isfinite(out[:lq - 1]).all()


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
def test_infinite_values_reach_only_the_rows_that_see_them(dsa, fmt):
    # V = inf in one column of token 650 and of token 705: rows from 705 on see
    # both, the others the first alone (an 8-bit cache holds 448 X instead)
    def hook(k, v):
        v[705, :, 3] = float("inf")
    kv, mirror, batch, table, g = _filled(dsa, [20], [695], 2, 64, 32, fmt, 620, hook=hook)
    out = dsa.paged_attn(_bf16(g, 20, 8, 64).cuda(), kv, batch, 0.125, inclusive=True)
    assert torch.isfinite(out[:10]).all()
    if fmt == "bf16":
        assert (out[10:, :, 3] == float("inf")).all()
        assert torch.isfinite(out[10:, :, :3]).all() and torch.isfinite(out[10:, :, 4:]).all()


def test_selecting_every_page_equals_all_pages(dsa):
    kv, mirror, batch, table, g = _filled(dsa, [3, 1], [500, 900], 2, 128, 64, "e4m3", 700)
    q = _bf16(g, 4, 8, 128).cuda()
    sel = dsa.page_topk(q, kv, batch, 20, inclusive=True)
    a = dsa.paged_attn(q, kv, batch, 0.09, inclusive=True)
    b = dsa.paged_attn(q, kv, batch, 0.09, sel=sel, inclusive=True)
    # the same weights and values, in another order of summation
    torch.testing.assert_close(a.float(), b.float(), rtol=2 * 2.0 ** -8, atol=2.0 ** -7)


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("lq", [1, 100])
def test_graph_replay_second_stream_and_shared_pages(dsa, fmt, lq):
    # two sequences share their first pages; the captured call follows changes
    # of the batch arrays; a call on another stream gives the same bits
    kv, mirror, batch, table, g = _filled(dsa, [lq], [640], 2, 128, 64, fmt, 800 + lq)
    t = batch.block_table.repeat(2, 1).contiguous()
    both = dsa.PagedBatch.from_lens([lq, lq], [640, 640], t)
    q = _bf16(g, 2 * lq, 8, 128).cuda()
    q[lq:] = q[:lq]
    a = dsa.paged_attn(q, kv, both, 0.09, inclusive=True)
    # the two may be cut into parts at different tiles: another order of the
    # f32 sums, and weights rounded to 8 bits under another maximum, each
    # within 2^-8 sum p|v| <= 2^-8 max|V| of the exact value, then one rounding
    most = 2 * 2.0 ** -8 * float(mirror.rows(table[0], 0)[1].nan_to_num().abs().max())

    def near(x, y):
        torch.testing.assert_close(x.float(), y.float(), rtol=2 * 2.0 ** -8, atol=most)

    near(a[:lq], a[lq:])
    ws = torch.empty(max(16, dsa.paged_attn_workspace(kv, both, 8)), dtype=torch.uint8, device="cuda")
    out = torch.zeros_like(a)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            dsa.paged_attn(q, kv, both, 0.09, inclusive=True, out=out, ws=ws)
        graph.replay()
        s.synchronize()
        assert torch.equal(out, a)
        both.start_pos[1] = 100
        graph.replay()
        s.synchronize()
    near(out[:lq], a[:lq])
    assert not torch.equal(out[lq:], a[lq:])
    assert torch.equal(out, dsa.paged_attn(q, kv, both, 0.09, inclusive=True))


def test_broken_contracts_are_counted_and_harmless(dsa):
    kv, mirror, batch, table, g = _filled(dsa, [2, 3], [100, 40], 2, 64, 16, "e4m3", 900)
    assert dsa.check_paged(kv, batch) == 0
    t = batch.block_table
    keep = t.clone()
    t[0, 3] = kv.k.shape[0]
    assert dsa.check_paged(kv, batch) == 1
    q = _bf16(g, 5, 4, 64).cuda()
    good = dsa.paged_attn(q, kv, dsa.PagedBatch.from_lens([2, 3], [100, 40], keep), 0.1)
    out = dsa.paged_attn(q, kv, batch, 0.1)
    dsa.page_topk(q, kv, batch, 3)
    dsa.check_device_errors()
    assert torch.equal(out[2:], good[2:])
    t.copy_(keep)
    batch.start_pos[1] = -1
    assert dsa.check_paged(kv, batch) == 1
    batch.start_pos[1] = 1 << 20
    assert dsa.check_paged(kv, batch) == 1
    before = kv.k.view(torch.uint8).clone()
    k = _bf16(g, 5, 2, 64).cuda()
    batch.start_pos[0] = -7
    dsa.paged_append(kv, batch, k, k)
    assert torch.equal(kv.k.view(torch.uint8), before)
    dsa.paged_attn(q, kv, batch, 0.1)
    dsa.check_device_errors()


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
def test_serving_loop(dsa, fmt):
    # a prompt, then decode steps, as a layer runs them: append and rotate,
    # choose pages, attend over them (and over all pages), each step checked
    # against the plain forms on the cache's contents
    page, n_kv, n_h, D, n_sel = 16, 2, 6, 64, 5
    prompts, steps = [75, 130, 3], 6
    g = _gen(11)
    room = [p + steps for p in prompts]
    table, t, n_pages = _table(room, [0] * 3, page, g)
    kv = _pool(dsa, n_pages, page, n_kv, D, fmt)
    cos, sin = (x.cuda() for x in _angles(max(room), D))
    mirror = ref.Cache(kv)
    lens, starts = prompts, [0, 0, 0]
    for step in range(steps + 1):
        batch = dsa.PagedBatch.from_lens(lens, starts, t)
        total = sum(lens)
        q, k, v = _bf16(g, total, n_h, D, std=1.5).cuda(), _bf16(g, total, n_kv, D).cuda(), _bf16(g, total, n_kv, D).cuda()
        qr = dsa.paged_append(kv, batch, k, v, cos, sin, q=q)
        mirror.append(lens, starts, table, k.cpu(), v.cpu(), cos.cpu(), sin.cpu(), False)
        seen = ref.Cache(kv)
        for name in ("k", "v"):  # up to roundings next to a border, the mirror's cache
            for b in range(3):
                for p in range(starts[b] + lens[b]):
                    x, y = getattr(seen, name)[table[b][p // page], :, p % page], getattr(mirror, name)[table[b][p // page], :, p % page]
                    assert (x - y).abs().max() <= 0.13 * y.abs().max()
        sel = dsa.page_topk(qr, kv, batch, n_sel, inclusive=True)
        rows = set(torch.randperm(total, generator=g)[:12].tolist()) | {total - 1}
        _check_attn(dsa, kv, seen, batch, table, lens, starts, qr.cpu(), 1 / 8, True, sel=sel.cpu(), rows=rows)
        _check_attn(dsa, kv, seen, batch, table, lens, starts, qr.cpu(), 1 / 8, True, rows=rows)
        starts, lens = [s + n for s, n in zip(starts, lens)], [1, 1, 1]


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
def test_one_long_chunk_among_many_short_sequences(dsa, fmt):
    # 70 sequences (more than a warp looks at in one go), most with one row or
    # none, one with 300: every operator finds its rows
    g = _gen(21)
    q_lens = [1] * 70
    q_lens[41], q_lens[3], q_lens[69], q_lens[33] = 300, 0, 0, 17
    starts = [int(x) for x in torch.randint(0, 200, (70,), generator=g)]
    starts[0], starts[41] = 0, 90
    page, n_kv, n_h, D = 16, 2, 8, 64
    ends = [s + n for s, n in zip(starts, q_lens)]
    table, t, n_pages = _table(ends, [0] * 70, page, g)
    kv = _pool(dsa, n_pages, page, n_kv, D, fmt)
    mirror = ref.Cache(kv)
    for lens, begin in ((starts, [0] * 70), (q_lens, starts)):
        batch = dsa.PagedBatch.from_lens(lens, begin, t)
        k, v = _bf16(g, sum(lens), n_kv, D), _bf16(g, sum(lens), n_kv, D)
        before = {n: getattr(kv, n).cpu().clone() for n in ("k", "v")}
        dsa.paged_append(kv, batch, k.cuda(), v.cuda())
        touched = set()
        mirror.append(lens, begin, table, k, v, None, None, False, touched)
        _check_cache(kv, mirror, touched, before)
    assert dsa.check_paged(kv, batch) == 0
    seen = ref.Cache(kv)
    q = _bf16(g, sum(q_lens), n_h, D)
    sel = dsa.page_topk(q.cuda(), kv, batch, 4, inclusive=True).cpu()
    r = 0
    for b, n in enumerate(q_lens):
        for i in range(n):
            vis = -(-(starts[b] + i + 1) // page)
            for h in range(n_kv):
                pages = table[b][:vis]
                assert sel[r, h].tolist() == ref.select_row(q[r, 4 * h:4 * h + 4].double(), seen.sum[pages, h], seen.sum_scale[pages, h], vis, 4, 1, 1)
            r += 1
    rows = set(torch.randperm(sum(q_lens), generator=g)[:60].tolist()) | {0, sum(q_lens) - 1}
    _check_attn(dsa, kv, seen, batch, table, q_lens, starts, q, 0.125, True, rows=rows)
    _check_attn(dsa, kv, seen, batch, table, q_lens, starts, q, 0.125, True, sel=sel, rows=rows)


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
def test_decode_of_many_sequences(dsa, fmt):
    # 300 sequences with a row each, lengths from nothing to 700 tokens
    g = _gen(22)
    B, page, n_kv, n_h, D = 300, 32, 2, 6, 64
    starts = [int(x) for x in torch.randint(0, 700, (B,), generator=g)]
    starts[0] = starts[129] = starts[299] = 0
    kv, mirror, batch, table, g = _filled(dsa, [1] * B, starts, n_kv, D, page, fmt, 23)
    q = _bf16(g, B, n_h, D, std=1.5)
    rows = set(torch.randperm(B, generator=g)[:60].tolist()) | {0, 1, 127, 128, 129, 298, 299}
    for inc in (False, True):
        _check_attn(dsa, kv, mirror, batch, table, [1] * B, starts, q, 0.125, inc, rows=rows)


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
def test_pool_beyond_32_bit_offsets(dsa, fmt):
    # the same pages at the start of a small pool and at the end of one whose K
    # and V pass 2^32 bytes each: bit-identical results and cache contents
    g = _gen(31)
    page, n_kv, n_h, D, lens = 128, 16, 32, 128, [300, 1, 140]
    n = sum(-(-x // page) for x in lens)
    big = (1 << 32) // (page * n_kv * D * (2 if fmt == "bf16" else 1)) + 2 * n
    k, v, q = (_bf16(g, sum(lens), h, D).cuda() for h in (n_kv, n_kv, n_h))
    kept = []
    for n_pages, first in ((n, 0), (big, big - n)):
        kv = dsa.PagedKV.empty(n_pages, page, n_kv, D, fmt=fmt)
        t = torch.full((3, 3), -1, dtype=torch.int32)
        at = first
        for b, x in enumerate(lens):
            t[b, :-(-x // page)] = torch.arange(at, at + -(-x // page))
            at += -(-x // page)
        batch = dsa.PagedBatch.from_lens(lens, [0] * 3, t.cuda())
        for name in ("k", "v"):
            getattr(kv, name).view(torch.uint8)[first:first + n].zero_()
        dsa.paged_append(kv, batch, k, v)
        assert dsa.check_paged(kv, batch) == 0
        rows = dsa.PagedBatch.from_lens([1, 1, 1], [299, 0, 139], t.cuda())
        sel = dsa.page_topk(q[:3], kv, rows, 2, inclusive=True)
        kept.append([dsa.paged_attn(q, kv, batch, 0.09, inclusive=True), dsa.paged_attn(q[:3], kv, rows, 0.09, inclusive=True), sel,
                     dsa.paged_attn(q[:3], kv, rows, 0.09, sel=sel, inclusive=True)] +
                    [getattr(kv, x).view(torch.uint8)[first:first + n].clone() for x in ("k", "v")])
        dsa.check_device_errors()
        del kv
    for a, b in zip(*kept):
        assert torch.equal(a, b)


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
def test_a_captured_decode_step_follows_its_inputs(dsa, fmt):
    # append, selection and attention captured once and replayed with new rows
    # and positions give what eager calls give on a copy of the cache
    g = _gen(32)
    starts, page, n_kv, n_h, D, steps = [200, 37, 63], 64, 2, 8, 64, 4
    room = [s + steps + 1 for s in starts]
    table, t, n_pages = _table(room, [0] * 3, page, g)
    caches = [_pool(dsa, n_pages, page, n_kv, D, fmt) for _ in range(2)]
    k, v = _bf16(g, sum(starts), n_kv, D).cuda(), _bf16(g, sum(starts), n_kv, D).cuda()
    cos, sin = (x.cuda() for x in _angles(max(room), D))
    for kv in caches:
        dsa.paged_append(kv, dsa.PagedBatch.from_lens(starts, [0] * 3, t), k, v, cos, sin)
    pos = torch.tensor(starts, dtype=torch.int32, device="cuda")
    cu = torch.arange(4, dtype=torch.int32, device="cuda")
    batch = dsa.PagedBatch(cu, pos, t, total_q=3, max_Lq=1, max_Lk=max(room))
    x = [_bf16(g, 3, h, D).cuda() for h in (n_kv, n_kv, n_h)]

    def step(kv, out):
        qr = dsa.paged_append(kv, batch, x[0], x[1], cos, sin, q=x[2])
        sel = dsa.page_topk(qr, kv, batch, 2, inclusive=True)
        out[0].copy_(dsa.paged_attn(qr, kv, batch, 0.125, sel=sel, inclusive=True))
        out[1].copy_(dsa.paged_attn(qr, kv, batch, 0.125, inclusive=True))

    outs = [[torch.empty((3, n_h, D), dtype=torch.bfloat16, device="cuda") for _ in range(2)] for _ in range(2)]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            step(caches[0], outs[0])
        for i in range(steps):
            for y in x:
                y.copy_(_bf16(g, *y.shape, std=1.0 + i))
            graph.replay()
            step(caches[1], outs[1])
            s.synchronize()
            for a, b in zip(*outs):
                assert torch.equal(a, b)
            for name in ("k", "v", "k_scale", "sum", "sum_scale"):
                if getattr(caches[0], name) is not None:
                    assert torch.equal(*(getattr(c, name).view(torch.uint8) for c in caches)), name
            pos += 1
    dsa.check_device_errors()

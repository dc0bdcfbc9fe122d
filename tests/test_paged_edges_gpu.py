"""The paged-cache operators at the ends of their ranges: scores and scales
beyond what f32 or 8 bits hold, weights far below a row's largest, lists longer
than a row's pages, groups and contexts past the usual ones."""
import math

import pytest
import torch

import paged_ref as ref
from test_paged_gpu import _angles, _bf16, _filled, _gen, _pool, _table, dsa  # noqa: F401  (dsa: the fixture)

pytestmark = pytest.mark.gpu

MAX = 3.4028234663852886e38


def _guarded(shape, dtype, mark):
    """A contiguous tensor and the guard words behind it (64, set to mark)."""
    n = math.prod(shape)
    buf = torch.full((n + 64,), mark, dtype=dtype, device="cuda")
    return buf[:n].view(shape), buf[n:]


def _select(q_group, codes, scales, n, n_sel):
    """The selection's definition for n_first = n_last = 1, scores kept finite."""
    if n <= n_sel:
        return list(range(n)) + [-1] * (n_sel - n)
    qs = q_group.double().sum(0).float()
    c = (qs * (qs.abs().max().reciprocal() * 127.0)).round().to(torch.int64)
    x = (codes.to(torch.int64) * c).sum(1).float() * scales.float()
    x = torch.where(torch.isnan(x), torch.full_like(x, -MAX), x.clamp(-MAX, MAX)).tolist()
    return sorted(p for _, p in sorted((-math.inf if p in (0, n - 1) else -x[p], p) for p in range(n))[:n_sel])


def _check_selection(dsa, kv, batch, table, q_lens, starts, q, n_sel):
    """Every list by its definition, and nothing written behind the last."""
    page, n_kv, G = kv.k.shape[2], kv.k.shape[1], q.shape[1] // kv.k.shape[1]
    out, guard = _guarded((sum(q_lens), n_kv, n_sel), torch.int32, -77)
    dsa.page_topk(q.cuda(), kv, batch, n_sel, inclusive=True, out=out)
    dsa.check_device_errors()
    assert (guard == -77).all()
    out, codes, scales, r = out.cpu(), kv.sum.cpu(), kv.sum_scale.cpu(), 0
    for b, n in enumerate(q_lens):
        for i in range(n):
            vis = -(-(starts[b] + i + 1) // page)
            for h in range(n_kv):
                pages = table[b][:vis]
                want = _select(q[r, h * G:(h + 1) * G], codes[pages, h], scales[pages, h], vis, n_sel)
                assert out[r, h].tolist() == want, (b, i, h)
            r += 1


def _huge_keys(page):
    """Keys near 1e35, of alternating sign by page; every third page ordinary:
    page sums are finite, scores are not."""
    def hook(k, v):
        j = torch.arange(k.shape[0]) // page
        size = torch.where(j % 3 == 2, 1.0, 1e35) * torch.where(j % 2 == 0, 1.0, -1.0)
        k.copy_(((k.float() * 0.1 + 1.0) * size[:, None, None]).to(k.dtype))
    return hook


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("tokens", [400, 8000])
def test_selection_of_a_chunk_keeps_infinite_scores_apart_from_forced_pages(dsa, tokens, fmt):  # noqa: F811
    q_lens, starts = [9, 4], [tokens, tokens // 2]
    kv, mirror, batch, table, g = _filled(dsa, q_lens, starts, 2, 128, 16, fmt, 41, hook=_huge_keys(16))
    q = _bf16(g, 13, 8, 128) + 0.5
    _check_selection(dsa, kv, batch, table, q_lens, starts, q, 16)


@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("share", [0.1, 0.98, 1.0])
def test_selection_of_a_chunk_with_scales_that_no_call_wrote(dsa, share, value):  # noqa: F811
    # some, all but a few, or all of the summaries have a scale that is not finite
    q_lens, starts = [9, 4], [8000, 500]
    kv, mirror, batch, table, g = _filled(dsa, q_lens, starts, 2, 64, 16, "bf16", 42)
    kv.sum_scale[torch.rand(kv.sum_scale.shape, generator=g).cuda() < share] = value
    kv.sum[::5] = 0  # (a dot product of 0 times infinity)
    _check_selection(dsa, kv, batch, table, q_lens, starts, _bf16(g, 13, 4, 64), 16)


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("tokens", [400, 8000, 40000])
def test_selection_of_few_rows_with_infinite_scores(dsa, tokens, fmt):  # noqa: F811
    q_lens, starts = [1, 3], [tokens, tokens // 2]
    kv, mirror, batch, table, g = _filled(dsa, q_lens, starts, 2, 128, 16, fmt, 43, hook=_huge_keys(16))
    q = _bf16(g, 4, 8, 128) + 0.5
    _check_selection(dsa, kv, batch, table, q_lens, starts, q, 16)


@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("share", [0.1, 0.98, 1.0])
@pytest.mark.parametrize("tokens", [500, 40000])
def test_selection_of_few_rows_with_scales_that_no_call_wrote(dsa, tokens, share, value):  # noqa: F811
    q_lens, starts = [1, 1, 1], [tokens, 500, 130]
    kv, mirror, batch, table, g = _filled(dsa, q_lens, starts, 2, 64, 16, "bf16", 44)
    kv.sum_scale[torch.rand(kv.sum_scale.shape, generator=g).cuda() < share] = value
    kv.sum[::5] = 0
    _check_selection(dsa, kv, batch, table, q_lens, starts, _bf16(g, 3, 4, 64), 16)


@pytest.mark.parametrize("q_lens", [[1, 1], [6, 5]])
def test_selection_where_the_positions_run_ahead_of_the_cache(dsa, q_lens):  # noqa: F811
    # a first position beyond the appended tokens breaks the contract: the rows
    # are unspecified, but lists name visible pages and end where they should
    g, page, n_sel = _gen(45), 16, 8
    table, t, n_pages = _table([400, 400], [0, 0], page, g)
    kv = _pool(dsa, n_pages, page, 2, 64, "bf16")
    k = _bf16(g, 300, 2, 64).cuda()
    dsa.paged_append(kv, dsa.PagedBatch.from_lens([150, 150], [0, 0], t), k, k)
    total = sum(q_lens)
    batch = dsa.PagedBatch.from_lens(q_lens, [380, 300], t)
    out, guard = _guarded((total, 2, n_sel), torch.int32, -77)
    dsa.page_topk(_bf16(g, total, 4, 64).cuda(), kv, batch, n_sel, inclusive=True, out=out)
    dsa.check_device_errors()
    assert (guard == -77).all() and (out >= 0).all() and (out < 25).all()
    assert (out[..., 1:] > out[..., :-1]).all()


def _summaries(dsa, lens, page, n_kv, D, g):
    """A pool that has summaries alone (codes and scales drawn), with its table."""
    table, t, n_pages = _table(lens, [0] * len(lens), page, g, spare=1)
    kv = dsa.PagedKV.empty(n_pages, page, n_kv, D, fmt="e4m3")
    kv.sum.copy_(torch.randint(-127, 128, kv.sum.shape, generator=g, dtype=torch.int8))
    kv.sum_scale.copy_(torch.rand(kv.sum_scale.shape, generator=g) + 0.5)
    return kv, table, t


@pytest.mark.parametrize("spread", [0, 1, 900])
def test_selection_of_few_rows_with_crowded_scores(dsa, spread):  # noqa: F811
    # one page scores far above the others, which crowd into one of the equal
    # steps of value, with many or few different values among them
    g = _gen(46)
    kv, table, t = _summaries(dsa, [20000, 9000], 16, 2, 64, g)
    kv.sum.fill_(3)
    kv.sum_scale.copy_(1.0 + torch.randint(0, spread + 1, kv.sum_scale.shape, generator=g) * 2.0 ** -20)
    for b, far in ((0, 700), (1, 33)):
        kv.sum_scale[table[b][far]] = 1e6
    q = _bf16(g, 2, 4, 64) + 2
    _check_selection(dsa, kv, dsa.PagedBatch.from_lens([1, 1], [19999, 8999], t), table, [1, 1], [19999, 8999], q, 33)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("q_lens,ends", [([1], [49152 * 16]), ([6, 4], [6369 * 16, 49000 * 16 - 3]), ([6], [6368 * 16])])
def test_selection_among_the_most_pages(dsa, D, q_lens, ends):  # noqa: F811
    # up to the most pages of a sequence; chunks on both sides of what the
    # shared memory of the kernel for many rows holds
    g = _gen(47)
    kv, table, t = _summaries(dsa, ends, 16, 1, D, g)
    starts = [e - n for e, n in zip(ends, q_lens)]
    q = _bf16(g, sum(q_lens), 3, D)
    _check_selection(dsa, kv, dsa.PagedBatch.from_lens(q_lens, starts, t), table, q_lens, starts, q, 100)


def _whole(g, *shape, most=8, times=1.0):
    """Whole numbers from -most to most, times a power of two: exact in bf16, in
    E4M3 with a power-of-two scale, and in f32 sums of their products."""
    return (torch.randint(-most, most + 1, shape, generator=g).double() * times).to(torch.bfloat16)


def _check_one_hot(dsa, kv, mirror, batch, table, q_lens, starts, q, scale, sel=None):
    """Scores so far apart that the softmax is exactly uniform over the keys
    that share the largest one: out is the mean of their values.

    Tolerance: the weights of equal scores are equal, each rounded to 8
    significant bits as their common value (2^-8), f32 sums, and one rounding of
    the output to bf16 (2^-8): 2^-7 of the mean of |v|, in all."""
    n_h, n_kv, page = q.shape[1], kv.k.shape[1], kv.k.shape[2]
    G = n_h // n_kv
    total = sum(q_lens)
    lse, guard = _guarded((total, n_h), torch.float32, -77.0)
    out = dsa.paged_attn(q.cuda(), kv, batch, scale, sel=None if sel is None else sel.cuda(), inclusive=True, lse=lse)
    dsa.check_device_errors()
    out, lse, r = out.cpu().double(), lse.cpu().double(), 0
    for b, n in enumerate(q_lens):
        for h in range(n_kv):
            K, V = mirror.rows(table[b], h)
            for i in range(n):
                t = starts[b] + i + 1
                seen = torch.arange(K.shape[0]) < t
                if sel is not None:
                    chosen = torch.zeros(K.shape[0] // page, dtype=torch.bool)
                    chosen[sel[r + i, h].long()] = True
                    seen &= chosen.repeat_interleave(page)
                idx = torch.nonzero(seen).flatten()
                for x in range(G):
                    e = K[idx] @ q[r + i, h * G + x].double()
                    top = e.max()
                    ties = idx[e == top]
                    want, size = V[ties].mean(0), V[ties].abs().mean(0)
                    err = (out[r + i, h * G + x] - want).abs()
                    assert (err <= 2.0 ** -7 * size + 1e-30).all(), (b, i, h, x, float(err.max()), float(size.max()))
                    want_lse = scale * float(top) + math.log(len(ties))
                    assert abs(float(lse[r + i, h * G + x]) - want_lse) <= 2.0 ** -20 * abs(want_lse)
        r += n


def _equal_far_keys(dsa, q_lens, starts, D, page, fmt, times, seed):
    """Keys of whole numbers that repeat every 97 tokens, so that a row's largest
    score has ties in many pages, and values whose size differs between pages."""
    def hook(k, v):
        k.copy_(_whole(_gen(seed), 97, *k.shape[1:], times=times)[torch.arange(k.shape[0]) % 97])
        v.mul_((2.0 ** (torch.arange(v.shape[0]) // page * 3 % 7 - 3))[:, None, None].to(v.dtype))
    kv, mirror, batch, table, g = _filled(dsa, q_lens, starts, 2, D, page, fmt, seed + 1, hook=hook)
    return kv, mirror, batch, table, _whole(g, sum(q_lens), 8, D, times=times)


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("D,page,q_lens,starts", [(64, 64, [140, 70], [300, 0]), (128, 32, [140], [3000])])
@pytest.mark.parametrize("times,scale", [(1.0, 64.0), (2.0 ** 10, 2.0 ** 9), (2.0 ** 10, 2.0 ** 40), (1.0, 1e30)])
def test_prompts_with_scores_past_the_f32_fraction(dsa, times, scale, D, page, q_lens, starts, fmt):  # noqa: F811
    # scores of 2^29 to 1e34: rounding one moves it by more than a weight's range
    kv, mirror, batch, table, q = _equal_far_keys(dsa, q_lens, starts, D, page, fmt, times, 51)
    _check_one_hot(dsa, kv, mirror, batch, table, q_lens, starts, q, scale)


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("lq", [1, 4, 140])
def test_keys_whose_scores_are_minus_infinity(dsa, lq, fmt):  # noqa: F811
    # the first 192 keys have scores below the f32 range, the others lie around
    # -3,000: the softmax is that of the others
    def hook(k, v):
        k[:192] = -(2.0 ** 100)
        k[192:] = (k[192:].float() * 0.1 - 23.0).to(k.dtype) * 2.0 ** -100
    kv, mirror, batch, table, g = _filled(dsa, [lq], [500], 2, 128, 64, fmt, 53, hook=hook)
    q = (torch.ones(lq, 8, 128) * 2.0 ** 100).to(torch.bfloat16)
    lse = torch.empty((lq, 8), dtype=torch.float32, device="cuda")
    out = dsa.paged_attn(q.cuda(), kv, batch, 1.0, inclusive=True, lse=lse).cpu().double()
    dsa.check_device_errors()
    for h in range(2):
        K, V = mirror.rows(table[0], h)
        for i in {0, lq // 2, lq - 1}:
            seen = (torch.arange(K.shape[0]) >= 192) & (torch.arange(K.shape[0]) <= 500 + i)
            for x in range(4):
                want, want_lse, tol, tol_lse = ref.attend_row(q[i, h * 4 + x].double(), K, V, seen, 1.0)
                assert ((out[i, h * 4 + x] - want).abs() <= tol).all()
                assert abs(float(lse[i, h * 4 + x]) - want_lse) <= tol_lse


def _attend(dsa, kv, mirror, batch, table, q_lens, starts, q, scale, sel=None, rows=None, tol=None):
    """paged_attn (inclusive) against a plain form, with guards behind out and
    lse.  tol(q, K, V, seen, scale, vs) -> (out, lse, their tolerances); vs: the
    V scale of each position."""
    tol = tol or _loose
    n_h, D, n_kv, page = q.shape[1], q.shape[2], kv.k.shape[1], kv.k.shape[2]
    total, G = sum(q_lens), q.shape[1] // kv.k.shape[1]
    lse, g1 = _guarded((total, n_h), torch.float32, -77.0)
    out, g2 = _guarded((total, n_h, D), torch.bfloat16, -77.0)
    dsa.paged_attn(q.cuda(), kv, batch, scale, sel=None if sel is None else sel.cuda(), inclusive=True, out=out, lse=lse)
    dsa.check_device_errors()
    assert (g1 == -77).all() and (g2 == -77).all()
    out, lse, r = out.cpu().double(), lse.cpu().double(), 0
    for b, n in enumerate(q_lens):
        for h in range(n_kv if n else 0):
            if rows is not None and not any(r + i in rows for i in range(n)):
                continue
            K, V = mirror.rows(table[b], h)
            vs = mirror.vs[torch.tensor(table[b], dtype=torch.long), h].repeat_interleave(page)
            for i in range(n):
                if rows is not None and r + i not in rows:
                    continue
                seen = torch.arange(K.shape[0]) <= starts[b] + i
                if sel is not None:
                    chosen = torch.zeros(K.shape[0] // page, dtype=torch.bool)
                    lst = sel[r + i, h].long()
                    chosen[lst[(lst >= 0) & (lst < chosen.numel())]] = True
                    seen &= chosen.repeat_interleave(page)
                for x in range(h * G, h * G + G):
                    want, want_lse, tol_o, tol_l = tol(q[r + i, x].double(), K, V, seen, scale, vs)
                    err = (out[r + i, x] - want).abs()
                    assert (err <= tol_o).all(), (b, i, x, float((err / tol_o).max()))
                    got = float(lse[r + i, x])
                    assert got == want_lse if math.isinf(want_lse) else abs(got - want_lse) <= tol_l, (b, i, x, got, want_lse)
        r += n


def _loose(q, K, V, seen, scale, vs):
    top = float(vs[seen].max()) if seen.any() else 0.0
    return ref.attend_row(q, K, V, seen, scale, top if float(vs.max()) != 1.0 or float(vs.min()) != 1.0 else 0.0)


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("page,n_sel,starts", [(16, 300, [40, 0, 5000, 700]), (64, 40, [0, 130, 63, 900])])
def test_lists_much_longer_than_the_rows(dsa, page, n_sel, starts, fmt):  # noqa: F811
    # most CTAs begin past the last page of the row they begin in
    q_lens = [1] * 4
    kv, mirror, batch, table, g = _filled(dsa, q_lens, starts, 2, 64, page, fmt, 61)
    sel = torch.full((4, 2, n_sel), -1, dtype=torch.int32)
    for b, s in enumerate(starts):
        vis = s // page + 1
        for h in range(2):
            pick = torch.randperm(vis, generator=g)[:n_sel].int()
            sel[b, h, :len(pick)] = pick
    for shift in (0, 3):  # (also with holes before the entries)
        _attend(dsa, kv, mirror, batch, table, q_lens, starts, _bf16(g, 4, 8, 64, std=1.5), 0.125, sel=sel.roll(shift, 2))


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("D,page,q_lens,starts", [(64, 64, [1, 1], [3000, 400]), (128, 32, [3], [3000]), (128, 16, [1], [300])])
@pytest.mark.parametrize("times,scale", [(1.0, 64.0), (2.0 ** 10, 2.0 ** 9), (2.0 ** 10, 2.0 ** 40), (1.0, 1e30)])
@pytest.mark.parametrize("listed", [False, True])
def test_few_rows_with_scores_past_the_f32_fraction(dsa, times, scale, listed, D, page, q_lens, starts, fmt):  # noqa: F811
    kv, mirror, batch, table, q = _equal_far_keys(dsa, q_lens, starts, D, page, fmt, times, 54)
    sel = None
    if listed:
        vis = min(s // page + 1 for s in starts)
        sel = torch.stack([torch.randperm(vis, generator=_gen(r))[:vis // 2 + 1] for r in range(2 * sum(q_lens))])
        sel = sel.view(sum(q_lens), 2, -1).int().contiguous()
    _check_one_hot(dsa, kv, mirror, batch, table, q_lens, starts, q, scale, sel=sel)


def _tight(q, K, V, seen, scale, vs):
    """The numerics that the header states, term by term: scores as f32 sums of D
    products and their scaling (delta), each weight within 2^-8 of itself, for
    an 8-bit cache (vs not all 1) also within 2^-14 of the largest weight x V
    scale of its 128 keys and 2^-32 of the row's, f32 sums over the keys, one
    rounding of the output to bf16 (2^-8)."""
    idx = torch.nonzero(seen).flatten()
    n, D = int(idx.numel()), q.numel()
    e = torch.full((K.shape[0],), -math.inf, dtype=torch.float64)
    e[idx] = scale * (K[idx] @ q)
    lse = float(torch.logsumexp(e, 0))
    p = torch.exp(e - lse)[:, None]
    v = torch.where(seen[:, None], V, torch.zeros_like(V))
    out = (p * v).sum(0)
    delta = scale * float((K[idx].abs() @ q.abs()).max()) * (D + 8) * 2.0 ** -24
    tol = 2.0 ** -8 * out.abs() + (2.0 ** -8 + 2 * delta + (n + 16) * 2.0 ** -24) * (p * v.abs()).sum(0)
    if not bool((vs == 1.0).all()):
        scales = torch.where(seen, vs, torch.zeros_like(vs))
        pad = -p.shape[0] % 128
        top = torch.nn.functional.pad(p[:, 0] * scales, (0, pad)).view(-1, 128).max(1).values.repeat_interleave(128)[:p.shape[0]]
        codes = torch.where(scales[:, None] > 0, v / vs[:, None], torch.zeros_like(v))
        # (rounding to the nearest step is never off by more than the weight itself)
        off = torch.minimum(p[:, 0] * scales, 2.0 ** -14 * top + 2.0 ** -32 * top.max())
        tol = tol + (off[:, None] * codes.abs()).sum(0)
    return out, lse, tol + 1e-37, delta + (n + 16) * 2.0 ** -24 + 2.0 ** -22 * (1 + abs(lse))


@pytest.mark.parametrize("page", [16, 32, 64])
@pytest.mark.parametrize("lq,gap", [(1, 20.8), (3, 20.8), (1, 12.0), (40, 20.8), (40, 12.0)])
def test_the_largest_score_in_a_page_of_tiny_values(dsa, lq, gap, page):  # noqa: F811
    # pages alternate between V scales of about 2^-25 with scores near 0 and of
    # about 1 with scores `gap` (natural log) lower; both weigh on the output
    D = 64

    def hook(k, v):
        odd = ((torch.arange(k.shape[0]) // page) % 2).bool()
        k.mul_(0.05)
        k[..., 0] = torch.where(odd, -gap / 2, 0.0)[:, None].to(k.dtype)
        v.mul_(torch.where(odd, 1.0, 2.0 ** -25)[:, None, None].to(v.dtype))
    kv, mirror, batch, table, g = _filled(dsa, [lq], [700], 2, D, page, "e4m3", 71, hook=hook)
    q = _bf16(g, lq, 8, D, std=0.05)
    q[..., 0] = 2.0
    _attend(dsa, kv, mirror, batch, table, [lq], [700], q, 1.0, tol=_tight)


def _copies(dsa, batch, table, q_lens, starts, times):
    """The batch of one sequence, `times` times over the same pages: so many
    that no sequence's keys are split between CTAs."""
    t = batch.block_table.repeat(times, 1).contiguous()
    return dsa.PagedBatch.from_lens(q_lens * times, starts * times, t), table * times, q_lens * times, starts * times


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("gap", [10.0, 16.0, 17.0, 19.0])
@pytest.mark.parametrize("lq,page,listed", [(1, 64, False), (3, 16, False), (12, 64, False), (1, 128, True)])
def test_many_small_weights_behind_a_large_one(dsa, lq, page, listed, gap, fmt):  # noqa: F811
    # one token of tiny value draws each row (an attention sink), the others lie
    # `gap` (natural log) lower: together they decide the output
    n = 60000

    def hook(k, v):
        k.mul_(0.25)
        k[..., 0] = -gap
        k[5, :, 0] = 0.0
        v.copy_((v.float().abs() + 0.25).to(v.dtype))
        v[5] *= 2.0 ** -9
    kv, mirror, batch, table, g = _filled(dsa, [lq], [n], 1, 64, page, fmt, 81, hook=hook)
    batch, table, q_lens, starts = _copies(dsa, batch, table, [lq], [n], 320)
    q = _bf16(g, 320 * lq, 4, 64, std=0.125)
    q[..., 0] = 1.0
    sel = torch.arange(-(-(n + lq) // page), dtype=torch.int32).expand(320 * lq, 1, -1).contiguous() if listed else None
    _attend(dsa, kv, mirror, batch, table, q_lens, starts, q, 1.0, sel=sel, rows={0, lq - 1, 320 * lq - 1}, tol=_tight)


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("lq,page", [(1, 16), (2, 128), (12, 64)])
@pytest.mark.parametrize("depth", [6.0, 14.0, 60.0])
@pytest.mark.parametrize("times", [1, 160])
def test_references_that_rise_and_fall(dsa, times, depth, lq, page, fmt):  # noqa: F811
    # runs of 128 keys whose scores go down and up again by `depth`, with values
    # that grow where the weights shrink
    def hook(k, v):
        run = (torch.arange(k.shape[0]) // 128 * 5 % 7).float() / 6  # 0 .. 1
        k.mul_(0.25)
        k[..., 0] = (-depth * run)[:, None].to(k.dtype)
        v.mul_((2.0 ** (depth * run * 1.25).round())[:, None, None].to(v.dtype))
    kv, mirror, batch, table, g = _filled(dsa, [lq], [4000], 2, 128, page, fmt, 82, hook=hook)
    batch, table, q_lens, starts = _copies(dsa, batch, table, [lq], [4000], times)
    q = _bf16(g, times * lq, 8, 128, std=0.125)
    q[..., 0] = 1.0
    _attend(dsa, kv, mirror, batch, table, q_lens, starts, q, 1.0, rows={0, lq - 1, times * lq - 1}, tol=_tight)


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("n_h,n_kv,lq,n_sel,start", [(40, 1, 1, 40, 5000), (128, 1, 3, 20, 2000), (66, 2, 5, 3, 700), (128, 2, 1, 300, 300)])
def test_selected_pages_of_groups_above_32_heads(dsa, n_h, n_kv, lq, n_sel, start, fmt):  # noqa: F811
    # a group's heads are cut into blocks of 32, with and without a merge
    kv, mirror, batch, table, g = _filled(dsa, [lq], [start], n_kv, 64, 16, fmt, 91)
    q = _bf16(g, lq, n_h, 64, std=1.5)
    sel = torch.full((lq, n_kv, n_sel), -1, dtype=torch.int32)
    for r in range(lq):
        for h in range(n_kv):
            pick = torch.randperm((start + r) // 16 + 1, generator=g)[:n_sel].int()
            sel[r, h, :len(pick)] = pick
    _attend(dsa, kv, mirror, batch, table, [lq], [start], q, 0.125, sel=sel)


@pytest.mark.parametrize("D,page", [(64, 16), (128, 64), (128, 128), (64, 32)])
@pytest.mark.parametrize("cut", [False, True])
@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
def test_summaries_bit_for_bit(dsa, fmt, cut, D, page):  # noqa: F811
    # codes and scales by the header's rule, from the cache's own contents: f32
    # sums by halving, and each operation rounded
    g = _gen(92)
    lens = [3 * page, 2 * page + 5, page - 1]
    table, t, n_pages = _table(lens, [0] * 3, page, g)
    kv = _pool(dsa, n_pages, page, 2, D, fmt)
    k = _bf16(g, sum(lens), 2, D)
    if cut:  # in three calls, the second of which rescales older codes
        ks, at = k.split(lens), [0, 0, 0]
        for i in range(3):
            n = [len(x) // 3 if i < 2 else len(x) - a for x, a in zip(ks, at)]
            part = torch.cat([x[a:a + m] * (1 + 3 * i) for x, a, m in zip(ks, at, n)])
            dsa.paged_append(kv, dsa.PagedBatch.from_lens(n, at, t), part.cuda(), part.cuda())
            at = [a + m for a, m in zip(at, n)]
    else:
        dsa.paged_append(kv, dsa.PagedBatch.from_lens(lens, [0] * 3, t), k.cuda(), k.cuda())
    for b, n in enumerate(lens):
        for j in range(n // page):
            pg = table[b][j]
            for h in range(2):
                x = kv.k[pg, h].cpu().float()
                while x.shape[0] > 1:
                    half = x.shape[0] // 2
                    x = x[:half] + x[half:]
                x = x[0] * (kv.k_scale[pg, h].cpu() if fmt == "e4m3" else 1.0)
                top = x.abs().max()
                codes = (x * (top.reciprocal() * 127.0)).round().to(torch.int8)
                assert torch.equal(kv.sum[pg, h].cpu(), codes)
                assert kv.sum_scale[pg, h].item() == ((top * torch.tensor(1 / 127, dtype=torch.float32)) / page).item()
    assert torch.isnan(kv.sum_scale[table[2][0]]).all()  # (an incomplete page has none)


@pytest.mark.parametrize("page", [16, 64, 128])
@pytest.mark.parametrize("lq", [1, 3, 40])
@pytest.mark.parametrize("gap", [0.0, 30.0, 55.0, 75.0])
@pytest.mark.parametrize("tiny_first", [False, True])
def test_scales_a_hundred_octaves_apart(dsa, tiny_first, gap, lq, page):  # noqa: F811
    # pages alternate between V scales of about 2^-100 and of about 2; those with
    # tiny values have scores `gap` (natural log) higher, and so the softmax's mass
    def hook(k, v):
        big = ((torch.arange(k.shape[0]) // page) % 2 == int(tiny_first))
        k.mul_(0.05)
        k[..., 0] = torch.where(big, -gap / 2, 0.0)[:, None].to(k.dtype)
        v.mul_(torch.where(big, 512.0, 2.0 ** -93)[:, None, None].to(v.dtype))
    kv, mirror, batch, table, g = _filled(dsa, [lq], [900], 2, 64, page, "e4m3", 73, hook=hook)
    q = _bf16(g, lq, 8, 64, std=0.05)
    q[..., 0] = 2.0
    _attend(dsa, kv, mirror, batch, table, [lq], [900], q, 1.0, tol=_tight)

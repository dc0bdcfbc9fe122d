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

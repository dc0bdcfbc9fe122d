"""Plain 64-bit forms of the paged-cache operators for their tests (CPU
tensors, one loop per sequence, page and head; include/dsa.h states the
definitions)."""
from __future__ import annotations

import math

import torch

MIN_SCALE = 2.0 ** -100


def to_e4m3(x):
    """Nearest E4M3 value (4 significant bits, steps of 2^-9 below 2^-6, ties
    to even, saturating at 448; NaN stays NaN) of a float64 tensor."""
    _, e = torch.frexp(x)
    step = torch.ldexp(torch.ones_like(x), (e - 4).clamp_min(-9))
    y = ((x / step).round() * step).clamp(-448, 448)
    return torch.where(torch.isinf(x), torch.sign(x) * 448.0, y)


def rotate(x, cos, sin, pos, interleaved):
    """x [n, heads, D] float64 rotated by the angles of pos [n]."""
    half = 0 if cos is None else cos.shape[1]
    if half == 0:
        return x.clone()
    c, s = cos.double()[pos][:, None], sin.double()[pos][:, None]
    y = x.clone()
    a, b = (x[..., 0:2 * half:2], x[..., 1:2 * half:2]) if interleaved else (x[..., :half], x[..., half:2 * half])
    u, w = a * c - b * s, b * c + a * s
    if interleaved:
        y[..., 0:2 * half:2], y[..., 1:2 * half:2] = u, w
    else:
        y[..., :half], y[..., half:2 * half] = u, w
    return y


def pow2_scale(amax: float) -> float:
    if amax == 0:
        return MIN_SCALE
    m, e = math.frexp(amax)  # amax = m 2^e, 0.5 <= m < 1; 448 = 0.875 * 2^9
    return max(MIN_SCALE, 2.0 ** (e - 9 + (m > 0.875)))


class Cache:
    """A float64 mirror of a PagedKV: values before the scale (codes), the
    scales, and the summaries."""

    def __init__(self, kv):
        self.f8 = kv.k_scale is not None
        up = (lambda t: t.cpu().float().double()) if self.f8 else (lambda t: t.cpu().double())
        self.k, self.v = up(kv.k), up(kv.v)
        n, h, self.page, self.D = self.k.shape
        one = torch.ones((n, h), dtype=torch.float64)
        self.ks = kv.k_scale.cpu().double() if self.f8 else one
        self.vs = kv.v_scale.cpu().double() if self.f8 else one.clone()
        self.sum = None if kv.sum is None else kv.sum.cpu().clone()
        self.sum_scale = None if kv.sum is None else kv.sum_scale.cpu().clone()

    def append(self, q_lens, starts, table, k, v, cos, sin, interleaved, touched=None):
        """k, v [total, n_kv, D] CPU bf16; table: lists of pool pages."""
        at = 0
        for b, n in enumerate(q_lens):
            pos = torch.arange(starts[b], starts[b] + n)
            new = {"k": rotate(k[at:at + n].double(), cos, sin, pos, interleaved), "v": v[at:at + n].double()}
            for j in range(starts[b] // self.page, -(-(starts[b] + n) // self.page) if n else 0):
                lo, hi = max(starts[b], j * self.page), min(starts[b] + n, (j + 1) * self.page)
                pg, a = table[b][j], lo - j * self.page
                for name, pool, scale in (("k", self.k, self.ks), ("v", self.v, self.vs)):
                    x = new[name][lo - starts[b]:hi - starts[b]].transpose(0, 1)  # [n_kv, m, D]
                    if not self.f8:
                        pool[pg, :, a:a + hi - lo] = x.float().to(torch.bfloat16).double()
                        continue
                    for h in range(pool.shape[1]):
                        fin = x[h][torch.isfinite(x[h].float())]
                        X = pow2_scale(float(fin.abs().max()) if fin.numel() else 0.0)
                        if a:
                            X = max(X, float(scale[pg, h]))
                            pool[pg, h, :a] = to_e4m3(pool[pg, h, :a] * (float(scale[pg, h]) / X))
                        scale[pg, h] = X
                        pool[pg, h, a:a + hi - lo] = to_e4m3(x[h] / X)
                if touched is not None:
                    touched.add(pg)
                if hi == (j + 1) * self.page and self.sum is not None:
                    total = self.k[pg].sum(1) * self.ks[pg][:, None]
                    for h in range(total.shape[0]):
                        top = float(total[h].abs().max())
                        ok = math.isfinite(top) and top >= 3.8e-37
                        inv = torch.tensor(top).float().reciprocal() * 127.0 if ok else 0.0
                        self.sum[pg, h] = (total[h].float() * inv).round().to(torch.int8) if ok else 0
                        self.sum_scale[pg, h] = top / 127.0 / self.page if ok else 0.0
            at += n

    def rows(self, pages, head):
        """Dequantised K and V of a sequence's pages, [len(pages) * page, D]."""
        pages = torch.as_tensor(pages, dtype=torch.long)
        K = (self.k[pages, head] * self.ks[pages, head][:, None, None]).reshape(-1, self.D)
        V = (self.v[pages, head] * self.vs[pages, head][:, None, None]).reshape(-1, self.D)
        return K, V


def select_row(q_group, codes, scales, n, n_sel, n_first, n_last):
    """q_group [G, D] float64; codes [n, D] and scales [n] of the visible
    pages.  Python integers, so the scores are exact."""
    if n <= n_sel:
        return list(range(n)) + [-1] * (n_sel - n)
    qs = q_group.sum(0).float()
    top = qs.abs().max()
    ok = bool(torch.isfinite(top)) and float(top) >= 3.8e-37
    c = (qs * (top.reciprocal() * 127.0)).round().to(torch.int64) if ok else torch.zeros(qs.shape, dtype=torch.int64)
    dots = (codes.to(torch.int64) * c).sum(1).float()
    score = [float(x) for x in dots * scales.float()]
    key = [(-math.inf if (p < n_first or p >= n - n_last) else -score[p], p) for p in range(n)]
    return sorted(p for _, p in sorted(key)[:n_sel])


def attend_row(q, K, V, seen, scale, vs_max=0.0):
    """q [D] float64 over K, V [L, D] where seen [L]; returns (out, lse, the
    tolerance of out, the tolerance of lse).

    The tolerances count the roundings of the numerics that the header states:
    an f32 sum of D exact products and its scaling (delta), weights with 8
    significant bits (2^-8), f32 sums over the n keys, and one rounding of the
    output to bf16 (2^-8 relative).  An 8-bit cache's weights have in addition
    an absolute step of 2^-23 of the largest weighted scale (vs_max * 448)."""
    idx = torch.nonzero(seen).flatten()
    n = int(idx.numel())
    if n == 0:
        return torch.zeros_like(q), -math.inf, torch.full_like(q, 0.0), 0.0
    k, v = K[idx], V[idx]
    e = scale * (k @ q)
    lse = float(torch.logsumexp(e, 0))
    p = torch.exp(e - lse)
    out = p @ v
    delta = float((scale * (k.abs() @ q.abs())).max()) * (q.numel() + 8) * 2.0 ** -24
    w = p @ v.abs()
    tol = 2.0 ** -8 * out.abs() + (2.0 ** -8 + 2 * delta + (n + 16) * 2.0 ** -24) * w + n * 2.0 ** -23 * 448 * vs_max * float(p.max())
    return out, lse, tol + 1e-30, delta + (n + 16) * 2.0 ** -24 + 2.0 ** -22 * (1 + abs(lse))

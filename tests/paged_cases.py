"""Paged-cache cases and the operators in 64 bits, for the tests of
paged_append, paged_attention, paged_key_weights and paged_evict.

A case's pools hold NaN in every row that no sequence owns, its block table
holds nonsense in every entry that no slot needs, and its token arrays end in
rows that belong to nobody.

Tolerances are bounds, element by element, of what the kernels may round:
  u_T = eps(T)/2 for a rounding to T, u = 2^-24 for one to fp32.
  scores   a dot product of D terms in fp32 (any order) is off by at most
           D u sum|q_d k_d|, then scaled and subtracted: g = scale (D + 4) u max_j sum|q k|
           plus 2^-21 for 2^x (the hardware's approximation, 2^-22, and the
           rounding of its argument's products)
  output   p_j rounded to T (u_T), weights p_j off by a factor within 1 +- 2 g', the sums of n
           terms by n u each, and the quotient rounded to T:
           |err| <= u_T |o| + (u_T + 2 (g + 2^-21) + 2 n u) sum_j p_j |v_j|   (times 1 + 2^-6 for the
           products of these terms)
"""
from __future__ import annotations

import math

import torch

DT = {"fp16": torch.float16, "bf16": torch.bfloat16}
U32 = 2.0 ** -24
SLACK = 1 + 2.0 ** -6


def u_of(dtype):
    return torch.finfo(DT[dtype]).eps / 2


def tiny_of(dtype):
    """Half a step of the subnormals of T."""
    return torch.finfo(DT[dtype]).smallest_normal * u_of(dtype)


class Case:
    """Sequences with past[b] cached tokens and new[b] new ones on random
    pages; everything on the CPU (`cuda()` copies it to the device)."""

    def __init__(self, dtype="bf16", H=8, Hkv=2, D=128, page=16, past=(5, 0, 40), new=(1, 1, 1), window=0, seed=0,
                 tail_rows=3, scale=0.0, qk=1.0, extra_pages=4, columns_extra=2, fill_new=True):
        g = torch.Generator().manual_seed(seed)
        self.dtype, self.H, self.Hkv, self.D, self.page, self.window = dtype, H, Hkv, D, page, window
        self.past, self.new, self.scale = list(past), list(new), scale
        self.B = len(self.past)
        t = DT[dtype]
        self.t = t
        total = [p + n for p, n in zip(past, new)]
        self.total = max(max(total), 1)
        self.max_new = max(max(new), 1)
        self.tokens = sum(new)
        rows = self.tokens + tail_rows
        need = [-(-x // page) for x in total]
        self.num_pages = sum(need) + extra_pages
        cols = max(need) + columns_extra
        perm = torch.randperm(self.num_pages, generator=g).to(torch.int32)
        self.table = torch.randint(-(1 << 30), 1 << 30, (self.B, cols), generator=g, dtype=torch.int32)
        self.table[self.table.abs() < self.num_pages] = -1
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = perm[at:at + n]
            at += n
        self.free = perm[at:]
        cu = [0]
        for n in new:
            cu.append(cu[-1] + n)
        self.cu = torch.tensor(cu, dtype=torch.int32)
        self.seqlens = torch.tensor(self.past, dtype=torch.int32)
        self.query = (torch.randn(rows, H * D, generator=g) * qk).to(t)
        self.key = torch.randn(rows, Hkv * D, generator=g).to(t)
        self.value = torch.randn(rows, Hkv * D, generator=g).to(t)
        self.k_pages = torch.full((self.num_pages, Hkv, page, D), float("nan"), dtype=t)
        self.v_pages = torch.full_like(self.k_pages, float("nan"))
        self.weights = torch.full((self.num_pages, Hkv, page), float("nan"))
        for b in range(self.B):
            n = total[b] if fill_new else self.past[b]
            j = torch.arange(n)
            pg = self.table[b, j // page].long()
            self.k_pages[pg, :, j % page] = (torch.randn(n, Hkv, D, generator=g) * qk).to(t)
            self.v_pages[pg, :, j % page] = torch.randn(n, Hkv, D, generator=g).to(t)
            self.weights[pg, :, j % page] = torch.rand(n, Hkv, generator=g)
        self.sm_scale = scale if scale > 0 else 1 / math.sqrt(D)

    NAMES = ("table", "cu", "seqlens", "query", "key", "value", "k_pages", "v_pages", "weights")

    def cuda(self, device="cuda"):
        return {n: getattr(self, n).to(device) for n in self.NAMES}

    def slots(self, b, n):
        j = torch.arange(n)
        return self.table[b, j // self.page].long(), j % self.page

    def gather(self, pool, b, n):
        """Rows of the first n slots of sequence b: [Hkv, n, ...]."""
        pg, off = self.slots(b, n)
        return pool[pg, :, off].transpose(0, 1)


def visible(case, b):
    """[new, past + new] truth values: token i sees slot j."""
    p, n = case.past[b], case.new[b]
    i = torch.arange(p, p + n)[:, None]
    j = torch.arange(p + n)[None]
    v = j <= i
    if case.window > 0:
        v &= j > i - case.window
    return v


def ref_attention(case, k_pages=None, v_pages=None, query=None):
    """(out, lse, tolerance of out, tolerance of lse) in float64, NaN in rows
    that belong to nobody."""
    k_pages = case.k_pages if k_pages is None else k_pages
    v_pages = case.v_pages if v_pages is None else v_pages
    query = case.query if query is None else query
    H, Hkv, D = case.H, case.Hkv, case.D
    G = H // Hkv
    rows = query.shape[0]
    out = torch.full((rows, H, D), float("nan"), dtype=torch.float64)
    lse = torch.full((rows, H), float("nan"), dtype=torch.float64)
    otol, ltol = torch.zeros_like(out), torch.zeros_like(lse)
    ut = u_of(case.dtype)
    for b in range(case.B):
        n = case.new[b]
        if n == 0:
            continue
        r = slice(int(case.cu[b]), int(case.cu[b]) + n)
        L = case.past[b] + n
        k, v = case.gather(k_pages, b, L).double(), case.gather(v_pages, b, L).double()
        q = query[r].double().view(n, Hkv, G, D)
        seen = visible(case, b)
        for h in range(Hkv):
            s = torch.einsum("igd,jd->gij", q[:, h], k[h]) * case.sm_scale
            mag = torch.einsum("igd,jd->gij", q[:, h].abs(), k[h].abs()) * case.sm_scale
            mag = torch.where(seen, mag, torch.zeros((), dtype=torch.float64)).amax(-1)      # [G, n]
            s = torch.where(seen, s, torch.full((), -math.inf, dtype=torch.float64))
            ls = torch.logsumexp(s, -1)
            p = torch.exp(s - ls[..., None])
            o = torch.einsum("gij,jd->igd", p, v[h])
            a = torch.einsum("gij,jd->igd", p, v[h].abs())
            g = (D + 4) * U32 * mag + 2.0 ** -21                                             # [G, n]
            nn = seen.sum(-1).double()
            hs = slice(h * G, (h + 1) * G)
            out[r, hs], lse[r, hs] = o, ls.T
            c = (ut + 2 * g + 2 * nn * U32).T[..., None]
            otol[r, hs] = SLACK * (ut * o.abs() + c * a) + tiny_of(case.dtype)
            ltol[r, hs] = SLACK * (g + nn * U32 + 2 * U32 * (ls.abs() + s.amax(-1).abs())).T
    return out, lse, otol, ltol


def ref_weights(case, lse, weights_in=None, k_pages=None, query=None):
    """(weights, tolerance, written) in float64 for the given lse."""
    k_pages = case.k_pages if k_pages is None else k_pages
    query = case.query if query is None else query
    weights_in = case.weights if weights_in is None else weights_in
    H, Hkv, D = case.H, case.Hkv, case.D
    G = H // Hkv
    w = weights_in.double().clone()
    tol = torch.zeros_like(w)
    written = torch.zeros(w.shape, dtype=torch.bool)
    for b in range(case.B):
        n, P = case.new[b], case.past[b]
        if n == 0:
            continue
        r = slice(int(case.cu[b]), int(case.cu[b]) + n)
        k = case.gather(k_pages, b, P + n).double()
        q = query[r].double().view(n, Hkv, G, D)
        seen = visible(case, b)
        lo = max(0, P + 1 - case.window) if case.window > 0 else 0
        pg, off = case.slots(b, P + n)
        j = torch.arange(P + n)
        for h in range(Hkv):
            s = torch.einsum("igd,jd->gij", q[:, h], k[h]) * case.sm_scale
            mag = torch.einsum("igd,jd->gij", q[:, h].abs(), k[h].abs()) * case.sm_scale
            z = lse[r].double().view(n, Hkv, G)[:, h].T[..., None]
            p = torch.where(seen, torch.exp(s - z), torch.zeros((), dtype=torch.float64))
            # the exponent's error: the dot product, the scaling and the
            # subtraction (of the magnitude of its two terms), then 2^x
            e = (D + 4) * U32 * mag + 4 * U32 * (mag + z.abs()) + 2.0 ** -21
            got = p.sum((0, 1))
            err = (p * e).sum((0, 1)) + G * n * U32 * got
            old = torch.where(j < P, weights_in[pg, h, off].double(), torch.zeros((), dtype=torch.float64))
            new = got + old
            sel = j >= lo
            w[pg[sel], h, off[sel]] = new[sel]
            tol[pg[sel], h, off[sel]] = (SLACK * (err + U32 * new.abs()) + 1e-38)[sel]
            written[pg[sel], h, off[sel]] = True
    return w, tol, written


def ref_kept(weights, recent, budget):
    """Old slots of the kept tokens of one (sequence, KV head), ascending."""
    n = len(weights)
    if n <= budget:
        return list(range(n))
    key = [(-math.inf if math.isnan(x) else x, 1 if math.isnan(x) else 0) for x in weights]
    cand = sorted(range(n - recent), key=lambda i: (-key[i][0], key[i][1], i))
    return sorted(cand[:budget - recent]) + list(range(n - recent, n))


def rotate_fp32(x, cos, sin, interleaved):
    """The rotation in fp32, products first (numpy-like: no contraction)."""
    x, c, s = x.float(), cos.float()[:, None], sin.float()[:, None]
    half = x.shape[-1] // 2
    a, b = (x[..., 0::2], x[..., 1::2]) if interleaved else (x[..., :half], x[..., half:])
    y1, y2 = (a * c) - (b * s), (b * c) + (a * s)
    return torch.stack((y1, y2), -1).flatten(-2) if interleaved else torch.cat((y1, y2), -1)


def ref_rows(x, weight, eps, cos, sin, interleaved, dtype):
    """(rows, tolerance) in float64: per-head norm, then rotation.  x [tokens,
    heads, D]; weight [D] or None; cos/sin [tokens, D/2] or None."""
    D = x.shape[-1]
    y = x.double()
    rel = 0.0
    if weight is not None:
        y = y / torch.sqrt((y * y).mean(-1, keepdim=True) + eps) * weight.double()
        # the sum of squares (D u, halved by the root), the division, the sum
        # with eps, 1/sqrt (2^-22: two units in the last place) and two products
        rel = (D / 2 + 4) * U32 + 2.0 ** -22
    mag = y.abs()
    if cos is not None:
        c, s = cos.double()[:, None], sin.double()[:, None]
        half = D // 2
        if interleaved:
            a, b = y[..., 0::2], y[..., 1::2]
            ma, mb = mag[..., 0::2], mag[..., 1::2]
        else:
            a, b, ma, mb = y[..., :half], y[..., half:], mag[..., :half], mag[..., half:]
        y1, y2 = a * c - b * s, b * c + a * s
        m1, m2 = ma * c.abs() + mb * s.abs(), mb * c.abs() + ma * s.abs()
        if interleaved:
            y, mag = torch.stack((y1, y2), -1).flatten(-2), torch.stack((m1, m2), -1).flatten(-2)
        else:
            y, mag = torch.cat((y1, y2), -1), torch.cat((m1, m2), -1)
        rel += 2 * U32  # a product and the sum
    return y, SLACK * (u_of(dtype) * y.abs() + rel * mag) + tiny_of(dtype)


def caches(rows, D, dtype, seed=0):
    inv = 10000.0 ** (-torch.arange(D // 2, dtype=torch.float64) * 2 / D)
    ang = torch.arange(rows, dtype=torch.float64)[:, None] * inv
    return torch.cos(ang).to(DT[dtype]), torch.sin(ang).to(DT[dtype])


def assert_close(got, ref, tol, what=""):
    got = got.double().cpu()
    bad = ~((got - ref).abs() <= tol)
    if bad.any():
        i = tuple(torch.nonzero(bad)[0].tolist())
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} out of tolerance; first at {i}: got "
                             f"{got[i].item()!r}, exact {ref[i].item()!r}, tolerance {tol[i].item():.3e}")


def same_bits(a, b):
    """Bitwise equality, NaN included."""
    a, b = a.cpu().contiguous(), b.cpu().contiguous()
    w = torch.int16 if a.element_size() == 2 else torch.int32
    return a.dtype == b.dtype and torch.equal(a.view(w), b.view(w))

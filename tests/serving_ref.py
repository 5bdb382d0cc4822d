"""Plain float64 definitions of the serving operators, one sequence, head and
page at a time on the CPU (test infrastructure; shares nothing with the
library), and bounds of what the kernels' roundings may add.

Bounds. u = eps / 2 of a type is the most one rounding is off, relative to the
value. A score s = scale sum_d q_d k_d of exact products summed in float32 is
off by at most (D + 2) 2^-24 S, S = |scale| sum_d |q_d| |k_d|; a probability
2^(s log2 e - reference) relative to its exact value by that (times e^that),
plus 2^-24 |s| for each of the products with log2 e and the difference, plus
2^-22 for the exponential; sums of n float32 terms by n 2^-24. `slack` is twice
their total, relative to A = sum_j p_j |v_j|.
"""

import math

import torch

E24 = 2.0 ** -24
NAN8 = 0x7F


def u(dtype):
    return torch.finfo(dtype).eps / 2


def rel_slack(S, D, n):
    """Relative error of a probability or of a sum of n of them (S: largest |scale| sum |q||k| of the row)."""
    return 2 * ((D + 8) * E24 * S + 2.0 ** -21 + (n + 32) * E24)


def rows(q, k, scale, lim):
    """Scores [n_q, n_k] of one head in float64, -inf past each row's last key lim[i], and S per row."""
    q, k = q.double(), k.double()
    s = scale * (q @ k.T)
    S = abs(scale) * (q.abs() @ k.abs().T)
    j = torch.arange(k.shape[0])
    gone = j[None, :] > lim[:, None]
    s = s.masked_fill(gone, -math.inf)
    S = S.masked_fill(gone, 0.0)
    return s, (S.amax(1) if k.shape[0] else torch.zeros(q.shape[0], dtype=torch.float64))


def softmax(s):
    """(P, LSE); dead rows give 0 and -inf."""
    if s.shape[1] == 0:
        return s.clone(), torch.full((s.shape[0],), -math.inf, dtype=torch.float64)
    lse = torch.logsumexp(s, 1)
    p = torch.where(torch.isneginf(lse)[:, None], torch.zeros_like(s), torch.exp(s - lse[:, None]))
    return p, lse


def limits(n_q, n_k, causal, align):
    i = torch.arange(n_q)
    if not causal:
        return torch.full((n_q,), n_k - 1)
    return i + (n_k - n_q if align == "bottom_right" else 0)


def odd_values(kept, v):
    """What the values that are not finite add to each row that keeps their key (0 elsewhere)."""
    x = torch.where(torch.isfinite(v), torch.zeros_like(v), v)
    j = (x != 0).any(1).nonzero()[:, 0]
    if not len(j):
        return torch.zeros(kept.shape[0], v.shape[1], dtype=torch.float64)
    return torch.where(kept[:, j, None], x[None, j], torch.zeros_like(x[None, j])).sum(1)


def prompt(q, k, v, cu_q, cu_k, causal=True, align="top_left", scale=None):
    """(O, LSE, bound of O, bound of LSE) of packed sequences; NaN at tokens of no sequence."""
    Tq, Hq, D = q.shape
    g = Hq // k.shape[1]
    scale = 1.0 / math.sqrt(D) if scale is None else scale
    o = torch.full((Tq, Hq, D), math.nan, dtype=torch.float64)
    lse = torch.full((Tq, Hq), math.nan, dtype=torch.float64)
    to, tl = torch.zeros_like(o), torch.zeros_like(lse)
    up = u(q.dtype) if q.dtype != torch.float32 else 0.0  # float32 probabilities are not rounded
    for b in range(len(cu_q) - 1):
        a, z, c, e = int(cu_q[b]), int(cu_q[b + 1]), int(cu_k[b]), int(cu_k[b + 1])
        lim = limits(z - a, e - c, causal, align)
        for h in range(Hq):
            s, S = rows(q[a:z, h], k[c:e, h // g], scale, lim)
            p, L = softmax(s)
            vv = v[c:e, h // g].double()
            kept = torch.where(p > 0, p, torch.zeros_like(p))
            o[a:z, h] = kept @ torch.nan_to_num(vv, 0.0, 0.0, 0.0) + odd_values(s > -math.inf, vv)
            A = kept @ torch.nan_to_num(vv.abs(), 0.0, 0.0, 0.0)
            sl = rel_slack(S, D, e - c)
            lse[a:z, h] = L
            to[a:z, h] = u(q.dtype) * torch.nan_to_num(o[a:z, h], 0.0, 0.0, 0.0).abs() + ((up + sl) * (1 + u(q.dtype)))[:, None] * A + 1e-30
            if q.dtype == torch.float16:
                # fp16 probabilities below 2^-14 and results near 0 round to steps of 2^-24; a row's reference is the
                # maximum of some of its scores, so its probabilities are taken with a sum of 1 at least
                to[a:z, h] += 2.0 ** -25 * (1 + (p > 0).double() @ torch.nan_to_num(vv.abs(), 0.0, 0.0, 0.0))
            tl[a:z, h] = sl + 2.0 ** -22 * torch.nan_to_num(L, 0.0, 0.0, 0.0).abs()
    return o, lse, to, tl


def weights(q, k, lse, cu_q, cu_k, max_k, causal=True, align="top_left", scale=None):
    """(W, bound) for the LSE given (float32)."""
    Tq, Hq, D = q.shape
    Hkv = k.shape[1]
    g = Hq // Hkv
    scale = 1.0 / math.sqrt(D) if scale is None else scale
    w = torch.zeros(len(cu_q) - 1, Hkv, max_k, dtype=torch.float64)
    t = torch.zeros_like(w)
    for b in range(len(cu_q) - 1):
        a, z, c, e = int(cu_q[b]), int(cu_q[b + 1]), int(cu_k[b]), int(cu_k[b + 1])
        lim = limits(z - a, e - c, causal, align)
        for h in range(Hq):
            s, S = rows(q[a:z, h], k[c:e, h // g], scale, lim)
            L = lse[a:z, h].double()
            p = torch.where(torch.isinf(L)[:, None], torch.zeros_like(s), torch.exp(s - L[:, None]))
            w[b, h // g, :e - c] += p.sum(0)
            # the float32 product of LSE with log2 e is off by 2^-24 |LSE| too
            t[b, h // g, :e - c] += ((rel_slack(S, D, z - a) + 4 * E24 * torch.nan_to_num(L, 0.0, 0.0, 0.0).abs())[:, None] * p).sum(0)
    return w, t + 1e-30


# ------------------------------------------------------------------ e4m3 cache


def values8(codes):
    """float64 values of e4m3 codes from their bits."""
    b = codes.view(torch.uint8).to(torch.int64)
    e, f = (b >> 3) & 15, b & 7
    x = torch.where(e > 0, (8 + f).double() * torch.exp2((e - 10).double()), f.double() * 2.0 ** -9)
    x = torch.where((b & 0x7F) == NAN8, torch.full_like(x, math.nan), x)
    return torch.where(b >= 128, -x, x)


_ALL = values8(torch.arange(256, dtype=torch.uint8))


def encode8(x):
    """Codes of float64 values of at most 448, to the nearest, ties to the even code; not finite: NaN."""
    pos = _ALL[:127]
    a = x.abs().nan_to_num(0.0, 0.0, 0.0)
    hi = torch.searchsorted(pos, a.contiguous()).clamp(max=126)
    lo = (hi - 1).clamp(min=0)
    dh, dl = pos[hi] - a, a - pos[lo]
    up = (dh < dl) | ((dh == dl) & (hi % 2 == 0))
    c = torch.where(up, hi, lo)
    c = torch.where(torch.isfinite(x), c, torch.full_like(c, NAN8))
    c = c + torch.where(torch.isfinite(x) & torch.signbit(x), 128, 0)
    return c.to(torch.uint8)


def scale_for(amax):
    """Smallest power of two s >= 2^-126 with amax <= 448 s (a float)."""
    s = 2.0 ** -126
    while amax > 448.0 * s:
        s *= 2.0
    return s


def append(cache, k, v, table, lens, cu):
    """The cache's tensors (codes as uint8) after the new tokens are written."""
    kc, vc = cache[0].view(torch.uint8).clone(), cache[1].view(torch.uint8).clone()
    ks, vs = cache[2].clone(), cache[3].clone()
    n_pages, H, P, D = kc.shape
    cap = table.shape[1] * P
    for b in range(len(lens)):
        n0 = min(max(int(lens[b]), 0), cap)
        n = min(int(cu[b + 1]) - int(cu[b]), cap - n0)
        at = n0
        while at < n0 + n:
            page, off = int(table[b, at // P]), at % P
            m = min(P - off, n0 + n - at)
            t0 = int(cu[b]) + at - n0
            if 0 <= page < n_pages:
                for h in range(H):
                    for c, s, x, last in ((kc, ks, k, False), (vc, vs, v, True)):
                        y = x[t0:t0 + m, h].double()
                        fin = y[torch.isfinite(y)].abs()
                        now = scale_for(float(fin.max()) if fin.numel() else 0.0)
                        pg = c[page, h].T if last else c[page, h]  # [P, D], a view
                        if off:
                            was = float(s[page, h])
                            now = max(now, was)
                            pg[:off] = encode8(values8(pg[:off].contiguous()) * (was / now))
                        s[page, h] = now
                        pg[off:off + m] = encode8(y / now)
            at += m
    return kc, vc, ks, vs


def gather(cache, table, b, n, h):
    """(k, v) [n, D] float64 and which of the n tokens exist (their page is in the pool)."""
    kc, vc, ks, vs = cache
    n_pages, H, P, D = kc.shape
    k, v = torch.zeros(n, D, dtype=torch.float64), torch.zeros(n, D, dtype=torch.float64)
    ok = torch.zeros(n, dtype=torch.bool)
    for p in range(-(-n // P)):
        page, m = int(table[b, p]), min(P, n - p * P)
        if 0 <= page < n_pages:
            k[p * P:p * P + m] = values8(kc[page, h].contiguous())[:m] * float(ks[page, h])
            v[p * P:p * P + m] = values8(vc[page, h].T.contiguous())[:m] * float(vs[page, h])
            ok[p * P:p * P + m] = True
    return k, v, ok


def attention(q, cache, table, lens, cu, causal=True, scale=None, w=None, max_kv=None):
    """(O, LSE, bound O, bound LSE, weights, bound of weights)."""
    T, Hq, D = q.shape
    Hkv, P = cache[0].shape[1], cache[0].shape[2]
    g = Hq // Hkv
    scale = 1.0 / math.sqrt(D) if scale is None else scale
    o = torch.full((T, Hq, D), math.nan, dtype=torch.float64)
    lse = torch.full((T, Hq), math.nan, dtype=torch.float64)
    to, tl = torch.zeros_like(o), torch.zeros_like(lse)
    wo = None if w is None else w.double().clone()
    tw = None if w is None else w.double().abs() * E24 + 1e-30
    for b in range(len(lens)):
        a, z = int(cu[b]), int(cu[b + 1])
        n, L = z - a, min(max(int(lens[b]), 0), table.shape[1] * P)
        if max_kv is not None:
            L = min(L, max_kv)
        lim = L - n + torch.arange(n) if causal else torch.full((n,), L - 1)
        for h in range(Hq):
            k, v, ok = gather(cache, table, b, L, h // g)
            s, S = rows(q[a:z, h], k, scale, lim)
            s = s.masked_fill(~ok[None, :], -math.inf)
            p, l = softmax(s)
            vz = torch.nan_to_num(v, 0.0, 0.0, 0.0)
            o[a:z, h] = p @ vz + odd_values(s > -math.inf, v)
            A = p @ vz.abs()
            sl = rel_slack(torch.nan_to_num(S, 0.0), D, L)
            lse[a:z, h] = l
            # probabilities as a bf16 rounding plus its bf16 residual: 2^-8 * 2^-8
            to[a:z, h] = u(q.dtype) * torch.nan_to_num(o[a:z, h], 0.0, 0.0, 0.0).abs() + ((2.0 ** -16 + sl) * (1 + u(q.dtype)))[:, None] * A + 1e-30
            if q.dtype == torch.float16:
                to[a:z, h] += 2.0 ** -25  # half of fp16's smallest step
            tl[a:z, h] = sl + 2.0 ** -22 * torch.nan_to_num(l, 0.0, 0.0, 0.0).abs()
            if w is not None:
                W = min(L, w.shape[2])
                wo[b, h // g, :W] += p.sum(0)[:W]
                # a probability is 2^(score - LSE): the stored LSE adds its own rounding
                rel = sl + 2.0 ** -22 * (1 + torch.nan_to_num(l, 0.0, 0.0, 0.0).abs())
                tw[b, h // g, :W] += (rel[:, None] * p).sum(0)[:W]
    if w is not None:
        tw = tw + 4 * E24 * wo.abs()
    return o, lse, to, tl, wo, tw


def evict(cache, table, lens, w, budget, recent, to):
    """(kept, new lengths, weights, k codes, v codes, scales) after the move."""
    kc, vc = cache[0].view(torch.uint8).clone(), cache[1].view(torch.uint8).clone()
    ks, vs = cache[2].clone(), cache[3].clone()
    n_pages, H, P, D = kc.shape
    B, W = w.shape[0], w.shape[2]
    kept = torch.full((B, H, budget), -1, dtype=torch.int32)
    new = torch.zeros(B, dtype=torch.int32)
    wo = torch.zeros_like(w)
    src = [t.clone() for t in (kc, vc, ks, vs)]
    for b in range(B):
        L = min(max(int(lens[b]), 0), table.shape[1] * P, W)
        n = min(L, budget)
        new[b] = n
        for h in range(H):
            late = L - min(recent, n)
            x = w[b, h, :late].tolist()
            key = [math.inf if math.isnan(y) else y for y in x]
            order = sorted(range(late), key=lambda j: (math.isnan(x[j]), key[j]), reverse=True)
            # reverse keeps equal elements in their order
            keep = sorted(order[:n - (L - late)]) + list(range(late, L))
            kept[b, h, :n] = torch.tensor(keep, dtype=torch.int32)
            wo[b, h, :n] = w[b, h, keep]
            for i in range(0, n, P):
                page_to = int(to[b, i // P])
                if not 0 <= page_to < n_pages:
                    continue
                part = keep[i:i + P]
                pages = [int(table[b, j // P]) for j in part]
                for c, s, c0, s0, last in ((kc, ks, src[0], src[2], False), (vc, vs, src[1], src[3], True)):
                    sc = [float(s0[p, h]) if 0 <= p < n_pages else 0.0 for p in pages]
                    top = max(max(sc), 2.0 ** -126)
                    pg = c[page_to, h].T if last else c[page_to, h]
                    pg[:] = 0
                    for r, (j, p, x8) in enumerate(zip(part, pages, sc)):
                        if 0 <= p < n_pages:
                            row = c0[p, h, :, j % P] if last else c0[p, h, j % P]
                            pg[r] = encode8(values8(row.contiguous()) * (x8 / top))
                    s[page_to, h] = top
    return kept, new, wo, kc, vc, ks, vs

"""Plain 64-bit implementations of the paged 8-bit cache operators (CPU)."""
import math

import torch

INF = math.inf


def e4m3_table():
    """The 256 values of e4m3: sign, 4 exponent bits (bias 7), 3 mantissa bits; 0x7F and 0xFF are NaN."""
    out = []
    for c in range(256):
        e, f = (c >> 3) & 15, c & 7
        v = math.ldexp(8 + f, e - 10) if e else math.ldexp(f, -9)
        v = math.nan if (c & 127) == 127 else v
        out.append(-v if c & 128 else v)
    return torch.tensor(out, dtype=torch.float64)


TABLE = e4m3_table()


def value(codes):
    return TABLE[codes.long()]


def round_e4m3(x):
    """float64 to the nearest e4m3 value, ties to the even mantissa, saturating."""
    a = x.abs().clamp(max=448.0)
    _, e = torch.frexp(a)
    step = torch.ldexp(torch.ones_like(a), (e - 1).clamp(min=-6) - 3)
    return torch.copysign(torch.round(a / step) * step, x)


def plan(lens, new, free, table, page, max_tokens):
    """-> slot_map, cu, lens_out, counts, table (new lists)."""
    table = [list(r) for r in table]
    slots, cu, taken = [], [0], 0
    for b, (n, a) in enumerate(zip(lens, new)):
        n, a = max(0, n), max(0, a)
        have = -(-n // page)
        for t in range(a):
            if len(slots) >= max_tokens:
                break
            pos = n + t
            at = pos // page
            got = -1
            if at < len(table[b]):
                if at >= have:
                    i = taken + at - have
                    if i < len(free):
                        got = free[i]
                        table[b][at] = got
                else:
                    got = table[b][at]
            slots.append(got * page + pos % page if got >= 0 else -1)
        taken += -(-(n + a) // page) - have
        cu.append(cu[-1] + a)
    slots += [-1] * (max_tokens - len(slots))
    return slots, cu, [max(0, n) + max(0, a) for n, a in zip(lens, new)], [cu[-1], taken], table


def append(x, slots, values, scales):
    """Rows x [T, H, d] (float64) into a cache given as values of codes [N, P, H, d] and scales [N, H] (float64, in place)."""
    N, P = values.shape[:2]
    slots = [s if 0 <= s < N * P else -1 for s in slots]
    t = 0
    while t < len(slots):
        if slots[t] < 0:
            t += 1
            continue
        page, end = slots[t] // P, t
        while end < len(slots) and slots[end] >= 0 and slots[end] // P == page:
            end += 1
        rows = x[t:end]
        first = min(slots[t:end]) % P
        amax = torch.where(rows.isfinite(), rows.abs(), 0.0).amax((0, 2))
        m, e = torch.frexp(amax)  # amax = m 2^e, m in [1/2, 1); 448 = 7/8 2^9
        e = torch.where(amax > 0, e.long() - 9 + (m > 0.875).long(), -60).clamp(min=-60)
        s = torch.ldexp(torch.ones_like(amax), e)
        if first > 0:
            s = torch.maximum(s, scales[page])
            values[page, :first] = round_e4m3(values[page, :first] * (scales[page] / s)[None, :, None])
        scales[page] = s
        for i in range(t, end):
            r = round_e4m3(x[i] / s[:, None])
            values[page, slots[i] % P] = torch.where(x[i].isfinite(), r, math.nan)
        t = end


def gather(values, scales, row, length):
    """Cached rows of one sequence: [length, H, d] float64."""
    N, P = values.shape[:2]
    pos = torch.arange(length)
    page = torch.tensor(row, dtype=torch.long)[pos // P].clamp(0, N - 1)
    return values[page, pos % P] * scales[page][:, :, None]


def attention(q, k, v, scale, n_new=None, causal=True, left=-1, right=-1):
    """q [n, Hq, d], k, v [L, Hkv, d] float64 -> (o, lse [n, Hq], weight) with weight = sum p |v| / sum p, the size
    that roundings of p are measured by, and dots = max_j sum |q k| scale per row."""
    n, hq, d = q.shape
    L, hkv = k.shape[:2]
    g = hq // hkv
    o = torch.zeros(n, hq, d, dtype=torch.float64)
    w = torch.zeros_like(o)
    lse = torch.full((n, hq), -INF, dtype=torch.float64)
    dots = torch.zeros(n, hq, dtype=torch.float64)
    if L == 0:
        return o, lse, w, dots
    pos = torch.arange(n)[:, None] + L - n
    at = torch.arange(L)[None]
    ok = torch.ones(n, L, dtype=torch.bool)
    if causal:
        ok &= at <= pos
    elif right >= 0:
        ok &= at <= pos + right
    if left >= 0:
        ok &= at >= pos - left
    for j in range(hq):
        kk, vv = k[:, j // g], v[:, j // g]
        s = torch.where(ok, q[:, j] @ kk.T * scale, -INF)
        some = ok.any(1)
        lse[:, j] = torch.where(some, torch.logsumexp(torch.where(some[:, None], s, 0.0), 1), -INF)
        p = torch.where(ok, torch.exp(s - torch.where(some, lse[:, j], 0.0)[:, None]), 0.0)
        for i in range(n):
            vis = ok[i]
            o[i, j] = p[i, vis] @ vv[vis]
            w[i, j] = p[i, vis] @ vv[vis].abs()
        dots[:, j] = torch.where(ok, q[:, j].abs() @ kk.abs().T * scale, 0.0).nan_to_num().amax(1)
    return o, lse, w, dots


def tolerances(o, w, dots, d, length):
    """Elementwise bounds of the kernels' error, by the roundings that they do.

    Scores: fp32 accumulation of d products (2^-23 a step, truncating) and two
    fp32 factors: d * 2^-23 * sum|qk| plus 2^-22 |x| <= (d + 2) 2^-23 dots; a
    query element below 2^-14 of its row's largest is off by 2^-25 of that
    largest, at most d * 2^-25 * dots together.  An absolute score error e
    changes p by the factor 1 + e.  P is rounded to f16, 2^-11 of itself;
    exponentials and logarithms are off by 2^-21, sums of up to `length` terms
    in fp32 by length * 2^-24.  O is rounded to bf16 once, 2^-8 of itself.
    """
    score = 1.25 * (d + 2) * 2.0 ** -23 * dots
    lse = score + 2.0 ** -20 + length * 2.0 ** -24
    rel_p = (2.0 ** -11 + 2.0 ** -20 + length * 2.0 ** -23 + 2 * score)[..., None]
    return 2.0 ** -8 * o.abs() + 1.01 * rel_p * w + 1e-30, lse

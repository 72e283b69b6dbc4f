"""Plain 64-bit references of the calls around the verify step, and seeded inputs for their tests.

Everything here is torch on the CPU, in float64 and whole numbers, one request (head, row) at a time.
"""
from __future__ import annotations

import math

import torch

FP8 = torch.float8_e4m3fn
E_MIN, E_MAX = -60, 60


# ------------------------------------------------------------------ the cache

def scale_exp(amax: float) -> int:
    """The smallest e in [-60, 60] with amax <= 448 * 2^e."""
    e = E_MIN
    while e < E_MAX and amax > 448.0 * 2.0 ** e:
        e += 1
    return e


def quantise(x: torch.Tensor, e: int) -> torch.Tensor:
    """float64 values as the codes' values at scale 2^e: nearest even on e4m3's grid, NaN past 448."""
    y = x.double() * 2.0 ** -e
    _, ex = torch.frexp(y)
    step = torch.ldexp(torch.ones_like(y), (ex - 1).clamp(min=-6) - 3)
    r = torch.round(y / step) * step  # torch.round ties to even
    return torch.where(y.abs() <= 448.0, r, torch.full_like(y, math.nan))


def accepted_rows(T, accepted=None, nodes=None):
    if accepted is None:
        return list(range(T))
    return [i if nodes is None or i == 0 else int(nodes[i - 1]) + 1 for i in range(int(accepted) + 1)]


def write_ref(codes, scales, x, table, length, rows):
    """One request's keys (or values) into float64 copies of the codes' values and scales, in place.
    codes [P, H, page, D], scales [P, H], x [T, H, D]."""
    page = codes.shape[2]
    at = 0
    while at < len(rows):
        j, first = divmod(length + at, page)
        take = rows[at:at + page - first]
        at += len(take)
        p = int(table[j])
        for h in range(codes.shape[1]):
            new = x[take, h].double()
            big = new.abs()
            big = big[big <= 448.0 * 2.0 ** E_MAX]
            e = scale_exp(float(big.max()) if big.numel() else 0.0)
            if first:
                e = max(e, int(math.log2(float(scales[p, h]))))
                k = e - int(math.log2(float(scales[p, h])))
                if k:
                    codes[p, h, :first] = quantise(codes[p, h, :first], k)
            scales[p, h] = 2.0 ** e
            codes[p, h, first:first + len(take)] = quantise(new, e)


def line(codes, scales, table, length):
    """The values of a request's tokens, [length, H, D] float64."""
    page = codes.shape[2]
    ids = table[:-(-length // page)].long()
    x = codes[ids].double() * scales[ids].double()[:, :, None, None]
    return x.permute(0, 2, 1, 3).flatten(0, 1)[:length]


# ------------------------------------------------------------------ trees

def path(parents, t):
    """Row t of a round and the rows before it on its path; parents None: a chain."""
    rows = [t]
    while rows[-1] > 0:
        i = rows[-1] - 1
        p = i - 1 if parents is None else int(parents[i])
        if not -1 <= p < i:
            break
        rows.append(p + 1)
    return rows


def random_parents(g, n):
    return torch.tensor([int(torch.randint(-1, i, (1,), generator=g)) if i else -1 for i in range(n)], dtype=torch.int32)


# ------------------------------------------------------------------ attention

def attention_ref(q, kc, vc, kn, vn, parents, n_rows, scale):
    """One request.  q [T, Hq, D]; kc, vc [L, Hkv, D] float64; kn, vn [T, Hkv, D] or None.
    Returns out, lse and, for the tolerances, per (row, head): the sum of p |v| [.., D], the number of
    tokens seen and the largest sum_d |q k| * scale among them."""
    T, hq, D = q.shape
    hkv = kc.shape[1]
    out = torch.zeros(T, hq, D, dtype=torch.float64)
    lse = torch.full((T, hq), -math.inf, dtype=torch.float64)
    absv = torch.zeros(T, hq, D, dtype=torch.float64)
    seen = torch.zeros(T, hq)
    size = torch.zeros(T, hq, dtype=torch.float64)
    for t in range(n_rows):
        new = [] if kn is None else sorted(path(parents, t))
        for h in range(hq):
            g = h // (hq // hkv)
            k, v = kc[:, g], vc[:, g]
            if kn is not None:
                k, v = torch.cat([k, kn[new, g].double()]), torch.cat([v, vn[new, g].double()])
            if not len(k):
                continue
            x = q[t, h].double()
            s = (k @ x) * scale
            lse[t, h] = torch.logsumexp(s, 0)
            p = torch.exp(s - lse[t, h])
            out[t, h] = p @ v
            absv[t, h] = p @ v.abs()
            seen[t, h] = len(k)
            size[t, h] = (k.abs() @ x.abs()).max() * scale
    return out, lse, absv, seen, size


def attention_tolerance(out, lse, absv, seen, size, vmax, D, dtype):
    """Bounds on |out - ref| and |lse - ref|, from the arithmetic the call documents:
      scores   D products summed in fp32: D 2^-23 of sum |q k|, and a few roundings of the exponent
      weights  rounded to a half for the product: 2^-11 relative, or 2^-32 of the largest weight
      sums     one fp32 rounding (2^-23) per token, and at the joins
      out      one rounding to its type"""
    lim = size.unsqueeze(-1)
    n = seen.unsqueeze(-1)
    ds = D * 2.0 ** -23 * lim + 2.0 ** -21 * (1 + lim)
    half = torch.finfo(dtype).eps / 2
    tol = (2.0 ** -11 + 4 * ds + (n + 64) * 2.0 ** -23) * absv + n * 2.0 ** -32 * vmax
    tol = tol + half * (out.abs() + tol) + (2.0 ** -25 if dtype == torch.float16 else 0.0)
    tl = 2 * ds[..., 0] + (seen + 64) * 2.0 ** -23 + 2.0 ** -22 * lse.abs().nan_to_num(posinf=0.0)
    return tol, tl


# ------------------------------------------------------------------ logits

def logits_ref(x, r, tokens, parents, history, pl, hl, rep, pres, freq, bias, allowed):
    """One row in float64.  x [V]; bias: list of (token, value) in order; allowed: bool [V] or None."""
    V = x.shape[0]
    y = x.double().clone()
    count, seen = {}, set()
    for i in range(hl):
        v = int(history[i])
        if 0 <= v < V:
            seen.add(v)
            if i >= pl:
                count[v] = count.get(v, 0) + 1
    for row in path(parents, r):
        if row > 0:
            v = int(tokens[row - 1])
            if 0 <= v < V:
                seen.add(v)
                count[v] = count.get(v, 0) + 1
    for v in seen:
        y[v] = y[v] / rep if y[v] > 0 else y[v] * rep
    for v, c in count.items():
        y[v] -= freq * c + pres
    for v, d in dict(bias).items():
        if 0 <= v < V:
            y[v] += d
    if allowed is not None:
        y[~allowed] = -math.inf
    return y

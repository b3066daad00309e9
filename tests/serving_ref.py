"""Plain 64-bit forms of the serving operators and the error bounds of the
kernels' arithmetic (helpers of the serving-operator tests)."""
import math

import torch


def unit(dtype):
    """Half a step relative to a value: the most one rounding to `dtype` is off."""
    return torch.finfo(dtype).eps / 2


def attend(q, k, v, seen, scale):
    """One head in 64 bits: q [n, hd], k and v [m, hd], seen [n, m] bool.  Returns
    (o, tolerance per element) for inputs of q's dtype."""
    dt = q.dtype
    q, k, v = q.double(), k.double(), v.double()
    n, m = q.shape[0], k.shape[0]
    if m == 0:
        return torch.zeros_like(q), torch.zeros_like(q)
    kz = torch.where(seen.any(0)[:, None], k, torch.zeros_like(k))
    z = (q @ kz.T) * scale
    mag = (q.abs() @ kz.abs().T) * abs(scale)
    z = torch.where(seen, z, torch.full_like(z, -math.inf))
    top = z.amax(1, keepdim=True)
    w = torch.where(seen, torch.exp(z - torch.where(top.isfinite(), top, torch.zeros_like(top))),
                    torch.zeros_like(z))
    w = w / w.sum(1, keepdim=True).clamp_min(1e-300)
    vis = torch.where(seen.any(0)[:, None], v, torch.zeros_like(v))
    o = w @ vis
    # Scores: hd products and sums in fp32 and a scaling, relative 2^-24 each against the sum of
    # magnitudes; subtracting the maximum rounds once more; e^x turns an absolute error of a score
    # into a relative one of its weight, and the sum of the weights carries as much again.
    f = 2.0 ** -24
    score = (mag.amax(1, keepdim=True) * (q.shape[1] + 4) * f
             + torch.where(seen, z.abs(), torch.zeros_like(z)).amax(1, keepdim=True) * 4 * f)
    rel = 2 * score + 2 * (m + 8) * f + 2.0 ** -19  # sums over m keys in fp32; e^x itself within 2^-20
    if dt == torch.bfloat16:
        rel = rel + unit(dt)  # weights are rounded to bf16 for the product with V
    else:
        rel = rel - 2.0 ** -19 + 2.0 ** -21
    tol = rel * (w @ vis.abs()) + unit(dt) * o.abs() + 1e-30
    return o, tol


def prompt(q, k, v, lq, lk, scale):
    """attn_prompt's definition: outputs and tolerances [n, H, hd] (zero outside)."""
    o = torch.zeros(q.shape, dtype=torch.float64, device=q.device)
    tol = torch.zeros_like(o)
    G = q.shape[1] // k.shape[1]
    a = b = 0
    for nq, nk in zip(lq, lk):
        seen = (torch.arange(nk, device=q.device)[None, :]
                <= (nk - nq + torch.arange(nq, device=q.device))[:, None])
        for h in range(q.shape[1]):
            o[a:a + nq, h], tol[a:a + nq, h] = attend(q[a:a + nq, h], k[b:b + nk, h // G],
                                                      v[b:b + nk, h // G], seen, scale)
        a, b = a + nq, b + nk
    return o, tol


def prefix(q, cache, rows, prefixes, tails, scale):
    """attn_prefix's definition: rows per group, prefix slot lists per group, tail
    slot lists per row."""
    n, H, hd = q.shape
    o = torch.zeros(q.shape, dtype=torch.float64, device=q.device)
    tol = torch.zeros_like(o)
    S = cache.shape[0]
    kv = cache.view(S, 2, -1, hd)
    G = H // kv.shape[2]
    r = 0
    for m, pre in zip(rows, prefixes):
        for i in range(r, r + m):
            idx = [s for s in list(pre) + list(tails[i]) if 0 <= s < S]
            idx = torch.tensor(idx, dtype=torch.long, device=q.device)
            seen = torch.ones(1, len(idx), dtype=torch.bool, device=q.device)
            for h in range(H):
                o[i, h], tol[i, h] = (x[0] for x in attend(q[i:i + 1, h], kv[idx, 0, h // G],
                                                           kv[idx, 1, h // G], seen, scale))
        r += m
    return o, tol


def verify(p, q, drafts, off, ua, ud):
    """lt_verify_drafts' definition (CPU tensors, Python floats are 64 bits)."""
    n, k = len(off) - 1, len(drafts)
    acc, tok = [], [-1] * (k + n)
    for s in range(n):
        o0, kk = off[s], off[s + 1] - off[s]
        a = 0
        while a < kk:
            x = drafts[o0 + a]
            if not 0 <= x < p.shape[1]:
                break
            qx = float(q[o0 + a, x]) if q is not None else 1.0
            if not float(ua[o0 + a]) * qx < float(p[o0 + s + a, x]):
                break
            tok[o0 + s + a] = x
            a += 1
        acc.append(a)
        row = p[o0 + s + a]
        w = row.clone()
        if a < kk:
            if q is not None:
                w = w - q[o0 + a]
            elif 0 <= drafts[o0 + a] < p.shape[1]:
                w[drafts[o0 + a]] = 0
        ok = lambda t: torch.where((t > 0) & t.isfinite(), t, torch.zeros_like(t)).double()  # noqa: E731
        w = ok(w)
        if float(w.sum()) == 0:
            w = ok(row)
        c = w.cumsum(0)
        if float(c[-1]) > 0:
            hit = torch.nonzero(c > float(ud[s]) * c[-1])
            tok[o0 + s + a] = int(hit[0]) if len(hit) else int(torch.nonzero(w > 0)[-1])
    return acc, tok

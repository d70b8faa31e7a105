"""Plain 64-bit forms of the softmax-attention operators (CPU), and how far a
kernel may be from them.

Tolerances count roundings, each at most half a step of its type (bf16 2^-8 of
the value, fp16 2^-11, fp32 2^-24, e4m3 2^-4):
- a score is a sum of 128 products in fp32 and a few more fp32 operations, so it
  is off by at most d = 160 * 2^-24 * (scale * sum |q||k| + cap + |x|), and a softmax weight by
  a factor within 1 +- 4 d (its exponential, and the sum it is divided by);
- the weight enters the product with v in bf16 (prefill) or fp16 (cache), where
  fp16 weights below 2^-14 of the largest are off by up to 2^-25 of it;
- the output is rounded to bf16 once.
"""
import torch

D = 128
F32 = 2.0 ** -24
BF16 = 2.0 ** -8
F16 = 2.0 ** -11


def visible(mask, n, prefix):
    i = torch.arange(n)
    if mask == "full":
        return torch.ones((n, n), dtype=torch.bool)
    seen = i[None, :] <= i[:, None]
    if mask == "prefix":
        seen = seen | (i[None, :] < prefix)
    return seen


def soft(q, k, scale, cap, slope, gap, seen):
    """Weights [R, L] and their relative error bound for fp32 scores; gap [R, L]."""
    q, k = q.double(), k.double()
    x = scale * (q @ k.T)
    d = scale * (q.abs() @ k.abs().T) + cap
    if cap > 0:
        x = cap * torch.tanh(x / cap)
    x = x - slope * gap.double().abs()
    d = 160 * F32 * (d + x.abs())
    x = torch.where(seen, x, -torch.inf)
    top = x.amax(1, keepdim=True)
    e = torch.exp(x - torch.where(torch.isfinite(top), top, 0.0))
    e = torch.where(seen, e, 0.0)
    total = e.sum(1, keepdim=True)
    p = e / torch.where(total > 0, total, 1.0)
    d = torch.where(seen, d, 0.0).amax(1, keepdim=True)
    return p, 4 * d


def prefill(q, k, v, scale, lengths, mask, cap=0.0, slopes=None, prefix=None):
    """(out, tolerance) [T, H, D] in 64 bits; the tensors are on the CPU."""
    T, H, _ = q.shape
    G = H // k.shape[1]
    out, tol = torch.zeros((T, H, D), dtype=torch.float64), torch.zeros((T, H, D), dtype=torch.float64)
    at = 0
    for s, n in enumerate(lengths):
        if n == 0:
            continue
        rows = slice(at, at + n)
        at += n
        seen = visible(mask, n, 0 if prefix is None else int(prefix[s]))
        gap = torch.arange(n)[:, None] - torch.arange(n)[None]
        for h in range(H):
            p, d = soft(q[rows, h], k[rows, h // G], scale, cap,
                        0.0 if slopes is None else float(slopes[h]), gap, seen)
            vv = v[rows, h // G].double()
            out[rows, h] = p @ vv
            tol[rows, h] = BF16 * out[rows, h].abs() * (1 + BF16) + (BF16 + d + 2.0 ** -15) * (p @ vv.abs())
    return out, tol


def rows_of(cache, table_row, h, n):
    """Dequantised keys and values, positions and the value scales of n slots of KV head h."""
    page = cache.k.shape[2]
    ids = [int(x) for x in table_row[: -(-n // page)]]
    if n == 0:
        z = torch.zeros((0, D), dtype=torch.float64)
        return z, z, torch.zeros(0, dtype=torch.int64), torch.zeros((0, 1), dtype=torch.float64), z
    k = torch.cat([cache.k[i, h].double() * cache.k_scale[i, h].double() for i in ids])[:n]
    v = torch.cat([cache.v[i, h].double() * cache.v_scale[i, h].double() for i in ids])[:n]
    pos = torch.cat([cache.pos[i, h] for i in ids])[:n].long()
    vs = torch.cat([cache.v_scale[i, h].double().expand(page) for i in ids])[:n, None]
    codes = torch.cat([cache.v[i, h].double() for i in ids])[:n]
    return k, v, pos, vs, codes


def cached(cache, q, table, lens, scale, counts, cap=0.0, slopes=None, positions=None):
    """(out, its tolerance, weight added, its tolerance); everything on the CPU."""
    T, H, _ = q.shape
    Hk, page = cache.k.shape[1], cache.k.shape[2]
    G = H // Hk
    out, tol = torch.zeros((T, H, D), dtype=torch.float64), torch.zeros((T, H, D), dtype=torch.float64)
    add, addtol = (torch.zeros(cache.weight.shape, dtype=torch.float64) for _ in range(2))
    at = 0
    for s, cnt in enumerate(counts):
        n = int(lens[s])
        for h in range(Hk):
            k, v, pos, vs, codes = rows_of(cache, table[s], h, n)
            if n == 0:
                continue
            if positions is not None:
                qp = positions[at:at + cnt].long()
            else:
                qp = pos[-1] - (cnt - 1 - torch.arange(cnt))
            gap = qp[:, None] - pos[None]
            total = torch.zeros(n, dtype=torch.float64)
            totaltol = torch.zeros(n, dtype=torch.float64)
            for g in range(G):
                head = h * G + g
                p, d = soft(q[at:at + cnt, head], k, scale, cap,
                            0.0 if slopes is None else float(slopes[head]), gap, gap >= 0)
                o = p @ v
                out[at:at + cnt, head] = o
                small = 2.0 ** -25 * (p * vs.T).amax(1, keepdim=True) * codes.abs().sum(0, keepdim=True)
                tol[at:at + cnt, head] = (BF16 * o.abs() * (1 + BF16) + (F16 + d + 2.0 ** -15) * (p @ v.abs())
                                          + 4 * small + 1e-30)
                total += p.sum(0)
                totaltol += ((d + 8 * F32) * p).sum(0)
            for j in range(-(-n // page)):
                m = min(page, n - j * page)
                add[int(table[s][j]), h, :m] += total[j * page:j * page + m]
                addtol[int(table[s][j]), h, :m] += totaltol[j * page:j * page + m] + cnt * G * F32 * total[j * page:j * page + m]
        at += cnt
    return out, tol, add, addtol


def exponent(amax):
    """Smallest e in [-64, 120] with amax <= 448 * 2^e."""
    e = -64
    while e < 120 and amax > 448 * 2.0 ** e:
        e += 1
    return e


def to_codes(x):
    """Nearest e4m3 value (ties to even) of 64-bit x; non-finite -> NaN."""
    mag = x.abs().clamp(max=448.0)
    _, e = torch.frexp(mag)                      # mag = m 2^e, 0.5 <= m < 1
    step = torch.exp2((e - 1).clamp(min=-6).double() - 3)
    r = torch.round(mag / step) * step           # torch.round: ties to even
    return torch.where(torch.isfinite(x), torch.copysign(r, x), torch.nan)


def append(cache, k, v, table, lens, counts, positions=None):
    """Appends in place to a cache whose codes are held as 64-bit values (CPU)."""
    page, at = cache["k"].shape[2], 0
    for s, cnt in enumerate(counts):
        n = int(lens[s])
        done = 0
        while done < cnt:
            slot = n + done
            pid, first = int(table[s][slot // page]), slot % page
            m = min(page - first, cnt - done)
            for h in range(k.shape[1]):
                for name, x in (("k", k), ("v", v)):
                    rows = x[at + done:at + done + m, h].double()
                    fine = rows[torch.isfinite(rows)]
                    sc = 2.0 ** exponent(float(fine.abs().max()) if fine.numel() else 0.0)
                    old = float(cache[name + "_scale"][pid, h])
                    if first and old > sc:
                        sc = old
                    if first:
                        cache[name][pid, h, :first] = to_codes(cache[name][pid, h, :first] * (old / sc))
                    cache[name][pid, h, first:first + m] = to_codes(rows / sc)
                    cache[name + "_scale"][pid, h] = sc
                cache["weight"][pid, h, first:first + m] = 0
                new = torch.arange(slot, slot + m) if positions is None else positions[at + done:at + done + m].long()
                cache["pos"][pid, h, first:first + m] = new
            done += m
        at += cnt


def kept_slots(weight, budget, recent):
    """Slots that stay of one (sequence, head), in order."""
    n = len(weight)
    if n <= budget:
        return list(range(n))
    old = n - recent
    ranked = sorted(range(old), key=lambda i: (-float(weight[i]), i))
    return sorted(ranked[: budget - recent]) + list(range(old, n))

"""Plain 64-bit forms of the short convolution, the state-space recurrence and the cache's page
tables (CPU), and how far a kernel may be from them.

Tolerances count roundings, each at most half a step of its type (bf16 2^-8 of the value, fp32
2^-24); an approximate exponential or reciprocal is off by 2^-22 of its value.
- step size d = softplus(v): v is rounded once (|v| 2^-24, by which d moves as much of itself at
  most), its two functions and the result by a few more: e_d = (8 + |v|) 2^-24 of d;
- decay e^{A d}: e_a = |A d| (e_d + 2^-22) + 2^-21 of itself;
- token by token, a state is multiplied and added to in fp32: each step adds 2^-23 (|a M| + |d x B|)
  to what the errors above make of it, and the output sums S products;
- in chunks of 128 tokens, sums of A d are off by 12 additions' roundings of their largest;
  the weights e^{l_i - l_j} d_j (C_i . B_j) and the copy of the state that the outputs see enter
  their products in bf16; x' enters its product in three bf16 addends (all 24 bits of fp32)
  where the final state is fp32, in two (2^-14, as upper 8 bits of what is left) where it
  is bf16, in one where there is none; a product adds 16 terms to an fp32 accumulator that may cut
  off instead of rounding (2^-23 of the largest each).
"""
import torch

F32 = 2.0 ** -24
BF16 = 2.0 ** -8
CHUNK = 128


def conv(x, w, bias, init, lengths, silu):
    """(out, tolerance, final state) of rows x [T, C]."""
    C, W = w.shape
    x, w = x.double(), w.double()
    b = bias.double() if bias is not None else torch.zeros(C, dtype=torch.float64)
    out, tol = torch.zeros_like(x), torch.zeros_like(x)
    fin = torch.zeros((len(lengths), W - 1, C), dtype=torch.float64)
    at = 0
    for n, length in enumerate(lengths):
        before = init[n].double() if init is not None else torch.zeros((W - 1, C), dtype=torch.float64)
        z = torch.cat([before, x[at:at + length]])
        y, mag = b.expand(length, C).clone(), b.abs().expand(length, C).clone()
        for j in range(W):
            y += z[j:j + length] * w[:, j]
            mag += (z[j:j + length] * w[:, j]).abs()
        o = y * torch.sigmoid(y) if silu else y
        e = (W + 1) * F32 * mag
        if silu:
            e = 1.1 * e + (y.abs() + 16) * F32 * o.abs() + 1e-30
        out[at:at + length], tol[at:at + length] = o, e + BF16 * (o.abs() + e)
        fin[n] = z[length:]
        at += length
    return out, tol, fin


def _steps(dt, A, dt_bias):
    v = dt.double() + (dt_bias.double() if dt_bias is not None else 0.0)
    d = torch.logaddexp(v, torch.zeros_like(v))
    return d, (8 + v.abs()) * F32


def ssm_step(x, dt, A, B, C, skip, dt_bias, init, lengths, state_dtype=torch.float32):
    """(out, tolerance, final state, tolerance) token by token."""
    T, H, P = x.shape
    G, S = B.shape[1:]
    d, ed = _steps(dt, A, dt_bias)
    x, A = x.double(), A.double()
    Bh, Ch = (t.double().repeat_interleave(H // G, 1) for t in (B, C))
    a = torch.exp(A * d)
    ea = (A * d).abs() * (ed + 2.0 ** -22) + 2.0 ** -21
    sk = skip.double()[:, None] if skip is not None else torch.zeros((H, 1), dtype=torch.float64)
    out, tol = torch.zeros_like(x), torch.zeros_like(x)
    N = len(lengths)
    fin, fin_tol = torch.zeros((N, H, P, S), dtype=torch.float64), torch.zeros((N, H, P, S), dtype=torch.float64)
    at = 0
    for n, length in enumerate(lengths):
        M = init[n].double().clone() if init is not None else torch.zeros((H, P, S), dtype=torch.float64)
        E = torch.zeros_like(M)
        for t in range(at, at + length):
            k, add = a[t][:, None, None], (d[t][:, None] * x[t])[..., None] * Bh[t][:, None]
            E = k * E + (k * M).abs() * (ea[t][:, None, None] + 2.0 ** -23) + add.abs() * (ed[t][:, None, None] + 2.0 ** -22)
            M = k * M + add
            y = torch.einsum("hps,hs->hp", M, Ch[t]) + sk * x[t]
            e = torch.einsum("hps,hs->hp", E + S * F32 * M.abs(), Ch[t].abs()) + 2 * F32 * (sk * x[t]).abs()
            out[t], tol[t] = y, e + BF16 * (y.abs() + e)
        at += length
        fin[n], fin_tol[n] = M, E + (BF16 * (M.abs() + E) if state_dtype == torch.bfloat16 else F32 * M.abs())
    return out, tol, fin, fin_tol


def ssm_chunks(x, dt, A, B, C, skip, dt_bias, init, lengths, state_dtype=torch.float32, final=True):
    """(out, tolerance, final state, tolerance) in chunks."""
    T, H, P = x.shape
    G, S = B.shape[1:]
    d, ed = _steps(dt, A, dt_bias)
    x, A = x.double(), A.double()
    Bh, Ch = (t.double().repeat_interleave(H // G, 1) for t in (B, C))
    sk = skip.double()[None, :, None] if skip is not None else torch.zeros((1, H, 1), dtype=torch.float64)
    ex = 0.0 if final and state_dtype == torch.float32 else 2.0 ** -14 if final else BF16  # x' in fewer addends
    out, tol = torch.zeros_like(x), torch.zeros_like(x)
    N = len(lengths)
    fin, fin_tol = torch.zeros((N, H, P, S), dtype=torch.float64), torch.zeros((N, H, P, S), dtype=torch.float64)
    at = 0
    for n, length in enumerate(lengths):
        M = init[n].double().clone() if init is not None else torch.zeros((H, P, S), dtype=torch.float64)
        E = torch.zeros_like(M)
        for c in range(at, at + length, CHUNK):
            r = slice(c, min(c + CHUNK, at + length))
            l = torch.cumsum(d[r] * A, 0).T                                  # [H, q]
            # exponents: 12 additions' roundings of the largest sum, and e_d of every step
            el = 1.45 * (12 * F32 * l.abs().amax(1) + ((d[r] * A).abs() * (ed[r] + 2 * F32)).sum(0)) + 2.0 ** -21  # [H]
            q = l.shape[1]
            X, Bc, Cc, dd = (t[r].transpose(0, 1) for t in (x, Bh, Ch, d[..., None]))  # [H, q, ...]
            edc = ed[r].amax(0)                                              # [H]
            w = torch.exp(torch.where(torch.ones(q, q, dtype=torch.bool).tril(), l[:, :, None] - l[:, None], -torch.inf))
            w = w * dd.transpose(1, 2)                                       # e^{l_i - l_j} d_j
            Pm = w * (Cc @ Bc.transpose(1, 2))
            Pa = w * (Cc.abs() @ Bc.abs().transpose(1, 2))
            ei = torch.exp(l)[..., None]
            off = Cc @ M.transpose(1, 2)                                     # [H, q, P]
            offa = Cc.abs() @ M.abs().transpose(1, 2)
            y = Pm @ X + ei * off + sk.transpose(0, 1) * X
            one = lambda t: t[:, None, None]  # noqa: E731
            e = (BF16 * Pm.abs() + (one(el + edc) + S * 2.0 ** -23) * Pa) @ X.abs() + q * 2.0 ** -23 * (Pa @ X.abs())
            e = e + ei * ((BF16 + one(el) + S * 2.0 ** -23) * offa + (1 + BF16) * (Cc.abs() @ E.transpose(1, 2)))
            e = e + 4 * F32 * (sk.transpose(0, 1) * X).abs() + 4 * F32 * y.abs()
            out[r], tol[r] = y.transpose(0, 1), (e + BF16 * (y.abs() + e)).transpose(0, 1)
            # the state: its decay, the weighted rows, 24 products' accumulations of up to all of it
            end = torch.exp(l[:, -1:] - l)[..., None] * dd                   # [H, q, 1]
            add = torch.einsum("hqp,hqs->hps", end * X, Bc)
            adda = torch.einsum("hqp,hqs->hps", (end * X).abs(), Bc.abs())
            k = torch.exp(l[:, -1])
            most = one(k) * M.abs() + adda
            E = one(k) * E + one(k) * M.abs() * (one(el) + 2.0 ** -22) + adda * (one(el + edc) + 2.0 ** -22 + ex) \
                + (3 * CHUNK // 16 + 18) * 2.0 ** -23 * most
            M = one(k) * M + add
        at += length
        fin[n], fin_tol[n] = M, E + (BF16 * (M.abs() + E) if state_dtype == torch.bfloat16 else F32 * M.abs())
    return out, tol, fin, fin_tol


def reserve(table, lens, new, free, count, page, rows, pages):
    """(table, lens, cu, slots, count) on lists; `table` is not changed."""
    table, width = [list(r) for r in table], len(table[0])
    up = lambda n: -(-n // page)  # noqa: E731
    out_lens, cu, slots, total, taken = [], [0], [], 0, 0
    for n, (length, add) in enumerate(zip(lens, new)):
        cu.append(cu[-1] + add)
        want = up(length + add) - up(length) if length + add <= width * page else 0
        fits = length + add <= width * page
        total += want
        ok = fits and (want == 0 or total <= count)
        if ok:
            for i in range(want):
                table[n][up(length) + i] = free[count - 1 - (total - want) - i]
            taken = total if want else taken
        out_lens.append(length + add if ok else length)
        slots += [table[n][p // page] * page + p % page if ok else -1 for p in range(length, length + add)]
    slots += [-1] * (rows - len(slots))
    return table, out_lens, cu, slots, count - taken


def release(table, lens, free, count, page, keep=None):
    free = list(free)
    up = lambda n: -(-n // page)  # noqa: E731
    for n, length in enumerate(lens):
        for j in range(up(keep[n]) if keep is not None else 0, up(length)):
            free[count] = table[n][j]
            count += 1
    return free, count

"""Cases of the softmax-attention operators that stand beside the KDA layers of a hybrid model.

A hybrid model puts an ordinary attention layer after every few linear (KDA) layers.  That layer
runs over the same packed rows ([T_total, H, 128] bf16, sequences cut by cu_seqlens) and keeps a
key/value cache.  Four operators make it up:

  prefill   attention over packed sequences (a document mask), with a causal, prefix or full mask
            inside each, scores capped by a tanh, a bias that falls with distance, shared KV heads
  append    new key/value rows into a paged cache held in e4m3 with one scale per (page, KV head)
  decode    attention of one or a few new tokens per sequence over that cache, which can add the
            attention weight that every cached token got to the cache's running sums
  evict     the tokens of least accumulated weight leave the cache: the others are packed into
            fresh pages, per KV head

Every case says which operator it is in "op".  ``own`` chooses between the plain form below and
the package's kernels.
"""
import random

import torch

own = False

D = 128
SCALE = D ** -0.5
E_MIN, E_MAX = -64, 120  # exponents of a block scale


# ---------------------------------------------------------------- cases

def listed():
    return [
        # a short prompt: one pass of a chat turn's first tokens, where launch latency counts
        dict(name="prefill 64", op="prefill", lo=64, hi=64, N=1, mix=0, H=16, Hk=4, mask="causal", cap=0.0, bias=True),
        # eight packed documents of equal length, capped scores
        dict(name="prefill 8x1024 capped", op="prefill", lo=1024, hi=1024, N=8, mix=0, H=32, Hk=8, mask="causal",
             cap=30.0, bias=False),
        # ragged documents whose first part is seen both ways (prefix mask), as in a prompt + answer batch
        dict(name="prefill ragged prefix", op="prefill", lo=1, hi=4096, N=8, mix=5, H=32, Hk=8, mask="prefix",
             cap=50.0, bias=False),
        # one long prompt with the distance bias
        dict(name="prefill 1x8192 bias", op="prefill", lo=8192, hi=8192, N=1, mix=0, H=64, Hk=8, mask="causal",
             cap=0.0, bias=True),
        # one serving step: a token of each of 256 sequences enters the cache
        dict(name="append 256x1", op="append", lo=1, hi=1, clo=0, chi=2048, N=256, mix=1, Hk=8, page=64),
        # the rows of a batch of ragged prompts enter it
        dict(name="append ragged prompts", op="append", lo=1, hi=4096, clo=0, chi=0, N=32, mix=2, Hk=8, page=64),
        # one user: a single sequence, where the split over its length counts
        dict(name="decode 1x4096", op="decode", lo=1, hi=1, clo=4096, chi=4096, N=1, mix=0, H=32, Hk=8, page=64,
             cap=0.0, bias=False, weights=False),
        # a full serving batch of ragged sequences, with the accumulated weights that eviction needs
        dict(name="decode 256 weights", op="decode", lo=1, hi=1, clo=1, chi=4096, N=256, mix=3, H=32, Hk=8, page=64,
             cap=0.0, bias=False, weights=True),
        # one long sequence, capped scores and the distance bias
        dict(name="decode 1x131072", op="decode", lo=1, hi=1, clo=131072, chi=131072, N=1, mix=0, H=32, Hk=8, page=64,
             cap=30.0, bias=True, weights=False),
        # several drafted tokens per sequence are checked at once
        dict(name="decode 32x4 tokens", op="decode", lo=4, hi=4, clo=16, chi=8192, N=32, mix=4, H=64, Hk=8, page=32,
             cap=0.0, bias=False, weights=False),
        # a single sequence over its budget
        dict(name="evict 1x4096", op="evict", clo=4096, chi=4096, N=1, mix=0, Hk=8, page=64, budget=1024, recent=128),
        # a batch of ragged sequences, some below the budget
        dict(name="evict 64 ragged", op="evict", clo=1, chi=16384, N=64, mix=6, Hk=8, page=64, budget=4096, recent=512),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(["prefill", "append", "decode", "evict"])
    Hk = rng.choice([1, 2, 4, 8])
    mix = rng.randrange(1, 1 << 20)
    page = rng.choice([16, 32, 64, 128])
    if op == "prefill":
        H = Hk * rng.choice([1, 2, 4, 8])
        hi = _log(rng, 16, 8192)
        N = _log(rng, 1, max(1, min(64, (1 << 31) // (H * hi * hi))))
        return dict(op=op, lo=max(0, hi // rng.choice([1, 2, 50])), hi=hi, N=N, mix=mix, H=H, Hk=Hk,
                    mask=rng.choice(["causal", "prefix", "full"]), cap=rng.choice([0.0, 20.0, 50.0]),
                    bias=rng.random() < 0.4)
    if op == "append":
        hi = _log(rng, 1, 8192)
        N = _log(rng, 1, max(1, min(256, (1 << 17) // hi)))
        return dict(op=op, lo=hi // rng.choice([1, 2, 50]), hi=hi, clo=0, chi=_log(rng, 1, 2048), N=N, mix=mix, Hk=Hk,
                    page=page)
    chi = _log(rng, 32, 131072)
    N = _log(rng, 1, max(1, min(256, (1 << 20) // chi)))
    if op == "decode":
        hi = rng.choice([1, 1, 1, 2, 5, 8])
        return dict(op=op, lo=rng.choice([1, hi]), hi=hi, clo=max(hi, chi // rng.choice([1, 2, 50])), chi=chi, N=N,
                    mix=mix, H=Hk * rng.choice([1, 2, 4, 8, 12, 16]), Hk=Hk, page=page,
                    cap=rng.choice([0.0, 0.0, 30.0]), bias=rng.random() < 0.4, weights=rng.random() < 0.5)
    budget = _log(rng, 16, max(17, chi // 2))
    return dict(op=op, clo=chi // rng.choice([1, 2, 50]), chi=chi, N=N, mix=mix, Hk=Hk, page=page, budget=budget,
                recent=rng.randrange(1, budget + 1))


def _lengths(lo, hi, N, mix):
    """N lengths in [lo, hi], the largest among them; they belong to the case, not to the seed."""
    r = random.Random(mix * 7919 + hi)
    v = [r.randint(lo, hi) for _ in range(N)]
    v[r.randrange(N)] = hi
    return v


def _new(case):
    return _lengths(case["lo"], case["hi"], case["N"], case["mix"])


def _cached(case):
    return _lengths(case["clo"], case["chi"], case["N"], case["mix"] + 1)


def _prefixes(case):
    r = random.Random(case["mix"] + 17)
    return [r.randint(0, n) for n in _new(case)]


def _pairs(case):
    """Visible (query, key) pairs of one head of a prefill."""
    total = 0
    for n, p in zip(_new(case), _prefixes(case)):
        if case["mask"] == "full":
            total += n * n
        elif case["mask"] == "causal":
            total += n * (n + 1) // 2
        else:
            total += n * (n + 1) // 2 + p * (p - 1) // 2
    return total


def work(case):
    N = case["N"]
    if case["op"] == "prefill":
        T = sum(_new(case))
        return {"bytes": 2 * D * T * (2 * case["H"] + 2 * case["Hk"]), "flops": 4 * D * case["H"] * _pairs(case)}
    row = case["Hk"] * D * 2  # bytes of one cached token's keys and values
    if case["op"] == "append":
        T = sum(_new(case))
        return {"bytes": T * (3 * row + 8 * case["Hk"]) + 4 * N, "flops": 4 * T * row}
    C = sum(_cached(case))
    if case["op"] == "decode":
        new = _new(case)
        pairs = sum(c * n for c, n in zip(_cached(case), new))
        extra = 8 * case["Hk"] * C if case["weights"] else 0
        extra += 4 * case["Hk"] * C if case["bias"] or case["hi"] > 1 else 0
        return {"bytes": C * row + extra + 4 * D * case["H"] * sum(new), "flops": 4 * D * case["H"] * pairs}
    kept = sum(min(c, case["budget"]) for c in _cached(case))
    return {"bytes": 4 * case["Hk"] * C + kept * (2 * row + 12 * case["Hk"]), "flops": kept * row}


# ---------------------------------------------------------------- inputs

def _cu(lengths):
    v = [0]
    v.extend(sum(lengths[: i + 1]) for i in range(len(lengths)))
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _slopes(H):
    """The usual geometric slopes, one per head: 2^(-8 (h + 1) / H)."""
    return torch.exp2(-8.0 * torch.arange(1, H + 1, device="cuda", dtype=torch.float32) / H)


def _pages(lengths, page):
    return [-(-n // page) for n in lengths]


def _table(counts, first, perm):
    """A block table [N, max pages]: sequence n owns counts[n] pages of `perm` from place first[n]; -1 past them."""
    width = max(1, max(counts))
    c = torch.tensor(counts, device="cuda")[:, None]
    f = torch.tensor(first, device="cuda")[:, None]
    j = torch.arange(width, device="cuda")[None]
    at = torch.where(j < c, f + j, 0)
    return torch.where(j < c, perm[at], -1).to(torch.int32).contiguous()


def _starts(counts):
    return [sum(counts[:i]) for i in range(len(counts))]


def _cache_rows(g, pages, Hk, page):
    """Codes and scales of a filled pool, as quantising keys and values of a few outlier channels leaves them."""
    k = torch.randn((pages, Hk, page, D), generator=g, device="cuda", dtype=torch.bfloat16)
    v = torch.randn((pages, Hk, page, D), generator=g, device="cuda", dtype=torch.bfloat16)
    ch = torch.exp(0.7 * torch.randn((1, Hk, 1, D), generator=g, device="cuda")).to(torch.bfloat16)
    k *= ch
    v *= torch.exp(0.5 * torch.randn((pages, Hk, 1, 1), generator=g, device="cuda")).to(torch.bfloat16)
    ek = _exponent(k.abs().amax((2, 3)).float())
    ev = _exponent(v.abs().amax((2, 3)).float())
    ks, vs = torch.exp2(ek), torch.exp2(ev)
    k = (k.float() / ks[:, :, None, None]).to(torch.float8_e4m3fn)
    v = (v.float() / vs[:, :, None, None]).to(torch.float8_e4m3fn)
    return k, v, ks, vs


def _exponent(amax):
    """Smallest e with amax <= 448 * 2^e, within [E_MIN, E_MAX] (448 is the largest e4m3 value)."""
    m, x = torch.frexp(amax)
    e = x - 9 + (m > 0.875).int()
    return torch.where(amax > 0, e, E_MIN).clamp(E_MIN, E_MAX).float()


def _positions(table, Hk, page, pages, lengths):
    """pos [pages, Hk, page]: the position of every cached token (nothing evicted yet), -1 elsewhere."""
    pos = torch.full((pages, page), -1, dtype=torch.int32, device="cuda")
    at = torch.arange(table.shape[1] * page, device="cuda", dtype=torch.int32).view(1, -1, page).expand(table.shape[0], -1, -1)
    own_page = table >= 0
    pos[table[own_page].long()] = at[own_page]
    return pos[:, None].repeat(1, Hk, 1).contiguous()


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    s = dict(case)
    op, N, Hk = case["op"], case["N"], case["Hk"]
    randn = lambda *shape: torch.randn(shape, generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
    if op == "prefill":
        n = _new(case)
        T = sum(n)
        s["q"] = 3.0 * randn(T, case["H"], D)
        s["k"] = randn(T, Hk, D)
        s["v"] = randn(T, Hk, D)
        s["cu"] = _cu(n)
        s["longest"] = max(n)
        s["slopes"] = _slopes(case["H"]) if case["bias"] else None
        s["prefix"] = torch.tensor(_prefixes(case), dtype=torch.int32, device="cuda") if case["mask"] == "prefix" else None
        return s
    page = case["page"]
    cached = _cached(case)
    if op == "append":
        n = _new(case)
        counts = _pages([a + b for a, b in zip(cached, n)], page)
    else:
        n = _new(case) if op == "decode" else None
        counts = _pages(cached, page)
    dst = _pages([min(c, case["budget"]) for c in cached], page) if op == "evict" else []
    pages = sum(counts) + sum(dst) + 3
    perm = torch.randperm(pages, generator=g, device="cuda")
    s["table"] = _table(counts, _starts(counts), perm)
    s["lens"] = torch.tensor(cached, dtype=torch.int32, device="cuda")
    s["kc"], s["vc"], s["ks"], s["vs"] = _cache_rows(g, pages, Hk, page)
    s["pos"] = _positions(s["table"], Hk, page, pages, cached)
    s["weight"] = torch.zeros((pages, Hk, page), device="cuda")
    s["longest"] = max(cached)
    if op == "append":
        T = sum(n)
        s["cu"] = _cu(n)
        size = torch.exp(0.6 * torch.randn((T, Hk, 1), generator=g, device="cuda"))
        s["k"] = (randn(T, Hk, D) * size).to(torch.bfloat16)
        s["v"] = (randn(T, Hk, D) * size).to(torch.bfloat16)
        s["new"] = max(n)
    elif op == "decode":
        s["q"] = 2.0 * randn(sum(n), case["H"], D)
        s["cu"] = _cu(n) if case["hi"] > 1 else None
        s["slopes"] = _slopes(case["H"]) if case["bias"] else None
        s["new"] = max(n)
    else:
        s["dst"] = _table(dst, [sum(counts) + f for f in _starts(dst)], perm)
        # a few tokens hold most of the weight; some never got any
        w = torch.exp(2.0 * torch.randn((pages, Hk, page), generator=g, device="cuda"))
        s["weight"] = torch.where(torch.rand((pages, Hk, page), generator=g, device="cuda") < 0.1, 0.0, w)
    return s


# ---------------------------------------------------------------- one pass

def run(s):
    return {"prefill": _prefill, "append": _append, "decode": _decode, "evict": _evict}[s["op"]](s)


def _cache(kda, s):
    return kda.KvCache(s["kc"], s["vc"], s["ks"], s["vs"], s["pos"], s["weight"])


def _pool(s):
    return {"k": s["kc"], "v": s["vc"], "k_scale": s["ks"], "v_scale": s["vs"], "pos": s["pos"], "weight": s["weight"]}


def _prefill(s):
    if own:
        import chunked_gated_delta_11_gb300 as kda
        return kda.kda_attn_fwd(s["q"], s["k"], s["v"], SCALE, mask=s["mask"], cap=s["cap"], slopes=s["slopes"],
                                prefix_lens=s["prefix"], cu_seqlens=s["cu"])
    N, H, Hk, L = s["N"], s["H"], s["Hk"], s["longest"]
    cu = s["cu"].long()
    n = cu[1:] - cu[:-1]
    i = torch.arange(L, device="cuda")
    there = i[None] < n[:, None]                                   # [N, L]
    at = torch.where(there, cu[:-1, None] + i[None], 0)
    q = s["q"][at].float().view(N, L, Hk, H // Hk, D).permute(0, 2, 3, 1, 4).reshape(N * Hk, (H // Hk) * L, D)
    k = s["k"][at].float().permute(0, 2, 3, 1).reshape(N * Hk, D, L)
    v = s["v"][at].float().permute(0, 2, 1, 3).reshape(N * Hk, L, D)
    x = torch.bmm(q, k).mul_(SCALE)
    if s["cap"]:
        x.div_(s["cap"]).tanh_().mul_(s["cap"])
    x = x.view(N, H, L, L)
    if s["slopes"] is not None:
        x.sub_(s["slopes"][None, :, None, None] * (i[:, None] - i[None]).abs())
    seen = there[:, None, :].expand(N, L, L)
    if s["mask"] != "full":
        back = i[None] <= i[:, None]
        if s["mask"] == "prefix":
            back = back[None] | (i[None, None] < s["prefix"][:, None, None])
        seen = seen & back
    x.masked_fill_(~seen[:, None], -torch.inf)
    x.sub_(x.amax(-1, keepdim=True)).exp_()
    x.div_(x.sum(-1, keepdim=True))
    o = torch.bmm(x.view(N * Hk, (H // Hk) * L, L), v)
    o = o.view(N, H, L, D).transpose(1, 2)[there]                  # [T, H, D]
    return o.to(torch.bfloat16)


def _append(s):
    if own:
        import chunked_gated_delta_11_gb300 as kda
        kda.kda_cache_append(_cache(kda, s), s["k"], s["v"], s["table"], s["lens"], cu_seqlens=s["cu"])
        return _pool(s)
    N, page, Hk = s["N"], s["page"], s["Hk"]
    cu, lens, table = s["cu"].long(), s["lens"].long(), s["table"].long()
    n = cu[1:] - cu[:-1]
    # the pages that get rows: the j-th of sequence b holds its slots from (lens // page + j) * page on
    J = (s["new"] + page - 1) // page + 1
    j = torch.arange(J, device="cuda")
    pj = lens[:, None] // page + j                                  # [N, J]
    live = (n[:, None] > 0) & (pj * page < (lens + n)[:, None])
    b, jj = torch.nonzero(live, as_tuple=True)
    pj = pj[b, jj]
    pid = table[b, pj]                                              # [M]
    slot = pj[:, None] * page + torch.arange(page, device="cuda")   # [M, page]
    fresh = (slot >= lens[b][:, None]) & (slot < (lens + n)[b][:, None])
    old = slot < lens[b][:, None]
    src = torch.where(fresh, cu[b][:, None] + slot - lens[b][:, None], 0)
    for_both = [(s["k"], s["kc"], s["ks"]), (s["v"], s["vc"], s["vs"])]
    _ = [_append_one(x, codes, scales, src, fresh, old, pid) for x, codes, scales in for_both]
    m, r = torch.nonzero(fresh, as_tuple=True)
    s["pos"][pid[m], :, r] = slot[m, r][:, None].int().expand(-1, Hk)
    s["weight"][pid[m], :, r] = 0.0
    return _pool(s)


def _append_one(x, codes, scales, src, fresh, old, pid):
    rows = x[src].float().transpose(1, 2)                           # [M, Hk, page, D]
    fine = torch.isfinite(rows) & fresh[:, None, :, None]
    need = torch.exp2(_exponent(torch.where(fine, rows.abs(), 0.0).amax((2, 3))))
    had = torch.where(old.any(1)[:, None], scales[pid], 0.0)
    scale = torch.maximum(need, had)[:, :, None, None]
    was = codes[pid]
    kept = was.float() * (had[:, :, None, None] / scale)
    new = torch.where(torch.isfinite(rows), rows / scale, torch.nan)
    out = torch.where(fresh[:, None, :, None], new, kept).to(torch.float8_e4m3fn)
    # rows that hold nothing yet stay as they are
    untouched = ~(fresh | old)[:, None, :, None]
    codes[pid] = torch.where(untouched, was.view(torch.uint8), out.view(torch.uint8)).view(torch.float8_e4m3fn)
    scales[pid] = scale[:, :, 0, 0]


def _decode(s):
    if own:
        import chunked_gated_delta_11_gb300 as kda
        o = kda.kda_cache_attn(_cache(kda, s), s["q"], s["table"], s["lens"], SCALE, cap=s["cap"], slopes=s["slopes"],
                               cu_seqlens=s["cu"], accumulate=s["weights"])
        return {"out": o, "weight": s["weight"]} if s["weights"] else {"out": o}
    N, H, Hk, page, R = s["N"], s["H"], s["Hk"], s["page"], s["new"]
    G = H // Hk
    lens, table = s["lens"].long(), s["table"].long()
    L = table.shape[1] * page
    pid = table.clamp(min=0)
    rows = lambda c, sc: (c[pid].float() * sc[pid][..., None, None]).transpose(1, 2).reshape(N * Hk, L, D)  # noqa: E731
    pos = s["pos"][pid].transpose(1, 2).reshape(N, Hk, L)
    held = torch.arange(L, device="cuda")[None] < lens[:, None]     # [N, L]
    cu = s["cu"].long() if s["cu"] is not None else torch.arange(N + 1, device="cuda")
    n = cu[1:] - cu[:-1]
    i = torch.arange(R, device="cuda")
    there = i[None] < n[:, None]                                    # [N, R]
    at = torch.where(there, cu[:-1, None] + i[None], 0)
    last = pos.gather(2, (lens - 1).clamp(min=0)[:, None, None].expand(N, Hk, 1))
    qpos = last - (n[:, None, None] - 1 - i[None, None])            # [N, Hk, R]
    q = s["q"][at].float().view(N, R, Hk, G, D).permute(0, 2, 3, 1, 4).reshape(N * Hk, G * R, D)
    x = torch.bmm(q, rows(s["kc"], s["ks"]).transpose(1, 2)).mul_(SCALE)
    if s["cap"]:
        x.div_(s["cap"]).tanh_().mul_(s["cap"])
    x = x.view(N, Hk, G, R, L)
    gap = qpos[..., None] - pos[:, :, None]                         # [N, Hk, R, L]
    if s["slopes"] is not None:
        x.sub_(s["slopes"].view(1, Hk, G, 1, 1) * gap[:, :, None].abs())
    seen = held[:, None, None] & there[:, None, :, None] & (gap >= 0)
    x.masked_fill_(~seen[:, :, None], -torch.inf)
    top = x.amax(-1, keepdim=True)
    x.sub_(torch.where(top > -torch.inf, top, 0.0)).exp_()
    total = x.sum(-1, keepdim=True)
    x.div_(torch.where(total > 0, total, 1.0))
    # a row's weights are zero where nothing is seen; codes in slots that hold nothing do not enter
    v = torch.where(held[:, None, :, None].expand(N, Hk, L, D).reshape(N * Hk, L, D), rows(s["vc"], s["vs"]), 0.0)
    o = torch.bmm(x.view(N * Hk, G * R, L), v).view(N, Hk, G, R, D).permute(0, 3, 1, 2, 4).reshape(N, R, H, D)
    o = o[there].to(torch.bfloat16)
    if not s["weights"]:
        return {"out": o}
    w = x.sum((2, 3)).view(N, Hk, -1, page).transpose(1, 2)         # [N, pages, Hk, page]
    mine = table >= 0
    s["weight"][table[mine]] += w[mine]
    return {"out": o, "weight": s["weight"]}


def _evict(s):
    if own:
        import chunked_gated_delta_11_gb300 as kda
        new = kda.kda_cache_evict(_cache(kda, s), s["table"], s["lens"], s["dst"], s["budget"], s["recent"])
        return {"lens": new, **_pool(s)}
    N, Hk, page, budget, recent = s["N"], s["Hk"], s["page"], s["budget"], s["recent"]
    lens, table, dst = s["lens"].long(), s["table"].long(), s["dst"].long()
    L = table.shape[1] * page
    new = lens.clamp(max=budget)
    flat = lambda x: x[table.clamp(min=0)].transpose(1, 2).reshape(N, Hk, L)  # noqa: E731
    i = torch.arange(L, device="cuda")
    w = flat(s["weight"])
    w = torch.where(i[None, None] < (lens - recent)[:, None, None], w, torch.inf)   # the newest always stay
    w = torch.where(i[None, None] < lens[:, None, None], w, -torch.inf)
    order = torch.sort(w, dim=-1, descending=True, stable=True).indices[..., :budget]
    order = torch.where(torch.arange(order.shape[-1], device="cuda") < new[:, None, None], order, L)
    order = torch.sort(order, dim=-1).values                        # kept slots in their old order, [N, Hk, <= budget]
    b, h, r = torch.nonzero(order < L, as_tuple=True)
    slot = order[b, h, r]
    sp, sr = table[b, slot // page], slot % page
    dp, dr = dst[b, r // page], r % page
    _ = [_evict_one(codes, scales, sp, sr, dp, dr, h) for codes, scales in ((s["kc"], s["ks"]), (s["vc"], s["vs"]))]
    s["pos"][dp, h, dr] = s["pos"][sp, h, sr]
    s["weight"][dp, h, dr] = s["weight"][sp, h, sr]
    return {"lens": new.int(), **_pool(s)}


def _evict_one(codes, scales, sp, sr, dp, dr, h):
    had = scales[sp, h]
    most = torch.zeros_like(scales)
    most.view(-1).scatter_reduce_(0, dp * scales.shape[1] + h, had, "amax")
    scale = most[dp, h]
    codes[dp, h, dr] = (codes[sp, h, sr].float() * (had / scale)[:, None]).to(torch.float8_e4m3fn)
    scales[dp, h] = scale


# ---------------------------------------------------------------- the definition in 64 bits

def exact(case, seed):
    return {"prefill": _exact_prefill, "append": _exact_append, "decode": _exact_decode,
            "evict": _exact_evict}[case["op"]](case, prepare(case, seed))


def _exact_prefill(case, s):
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lengths, prefixes, start = _new(case), _prefixes(case), 0
    group = case["H"] // case["Hk"]
    for n, p in zip(lengths, prefixes):
        row = torch.arange(n, device="cuda")[:, None]
        col = torch.arange(n, device="cuda")[None, :]
        hide = torch.zeros((n, n), dtype=torch.bool, device="cuda")
        if case["mask"] == "causal":
            hide = col > row
        elif case["mask"] == "prefix":
            hide = (col > row) & (col >= p)
        for h in range(case["H"]):
            if n == 0:
                continue
            q = s["q"][start:start + n, h].double()
            k = s["k"][start:start + n, h // group].double()
            v = s["v"][start:start + n, h // group].double()
            x = (q @ k.T) / D ** 0.5
            if case["cap"] > 0:
                x = case["cap"] * torch.tanh(x / case["cap"])
            if case["bias"]:
                x = x - 2.0 ** (-8.0 * (h + 1) / case["H"]) * (row - col).abs()
            x[hide] = float("-inf")
            out[start:start + n, h] = torch.softmax(x, dim=1) @ v
        start += n
    return out



def _exact_append(case, s):
    page = case["page"]
    out = {name: s[key].double() for name, key in (("k", "kc"), ("v", "vc"), ("k_scale", "ks"), ("v_scale", "vs"))}
    table, start = s["table"].tolist(), 0
    jobs = []
    for b, (c, n) in enumerate(zip(_cached(case), _new(case))):
        at = c
        while at < c + n:
            end = min((at // page + 1) * page, c + n)
            jobs.append((table[b][at // page], at % page, end - at, start + at - c))
            at = end
        start += n
    if len(jobs) > 8192:
        return None
    steps = torch.tensor([2.0 ** e for e in range(E_MIN, E_MAX + 1)], dtype=torch.float64, device="cuda")
    for name, key in (("k", "k"), ("v", "v")):
        codes, scales = out[name], out[name + "_scale"]
        for pid, first, count, row in jobs:
            x = s[key][row:row + count].double().transpose(0, 1)    # [Hk, count, D]
            need = steps[torch.searchsorted(448 * steps, x.abs().amax((1, 2)).contiguous())]
            new = torch.maximum(need, scales[pid]) if first else need
            if first:
                codes[pid, :, :first] *= (scales[pid] / new)[:, None, None]
            codes[pid, :, first:first + count] = x / new[:, None, None]
            scales[pid] = new
    return {**out, "pos": None, "weight": None}


def _exact_decode(case, s):
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    weight = s["weight"].double()
    lengths, new, group, page = _cached(case), _new(case), case["H"] // case["Hk"], case["page"]
    start = 0
    for b, (c, n) in enumerate(zip(lengths, new)):
        ids = s["table"][b, : -(-c // page)].long()
        if c and n:
            k = _value_rows(s, "k", ids, c)                          # [Hk, c, D]
            v = _value_rows(s, "v", ids, c)
            q = s["q"][start:start + n].double().view(n, case["Hk"], group, D).permute(1, 2, 0, 3)
            x = torch.einsum("hgnd,hcd->hgnc", q, k) / D ** 0.5
            if case["cap"] > 0:
                x = case["cap"] * torch.tanh(x / case["cap"])
            # nothing has been evicted here: slot and position are the same
            gap = (c - n + torch.arange(n, device="cuda"))[:, None] - torch.arange(c, device="cuda")[None]
            if case["bias"]:
                slope = 2.0 ** (-8.0 * torch.arange(1, case["H"] + 1, device="cuda", dtype=torch.float64) / case["H"])
                x = x - slope.view(case["Hk"], group, 1, 1) * gap.abs()
            x = x.masked_fill(gap < 0, float("-inf"))
            p = torch.nan_to_num(torch.softmax(x, dim=-1))
            out[start:start + n] = torch.einsum("hgnc,hcd->nhgd", p, v).reshape(n, case["H"], D)
            if case["weights"]:
                w = torch.zeros((case["Hk"], len(ids) * page), dtype=torch.float64, device="cuda")
                w[:, :c] = p.sum((1, 2))
                weight[ids] += w.view(case["Hk"], len(ids), page).transpose(0, 1)
        start += n
    return {"out": out, "weight": weight} if case["weights"] else {"out": out}


def _value_rows(s, key, ids, c):
    x = s[key + "c"][ids].double() * s[key + "s"][ids].double()[:, :, None, None]
    return x.transpose(0, 1).reshape(x.shape[1], -1, D)[:, :c]


def _exact_evict(case, s):
    page, budget, recent = case["page"], case["budget"], case["recent"]
    out = {name: s[key].double() for name, key in
           (("k", "kc"), ("v", "vc"), ("k_scale", "ks"), ("v_scale", "vs"), ("weight", "weight"))}
    for b, c in enumerate(_cached(case)):
        if not c:
            continue
        src = s["table"][b, : -(-c // page)].long()
        for h in range(case["Hk"]):
            w = s["weight"][src, h].reshape(-1)[:c]
            if c <= budget:
                keep = torch.arange(c, device="cuda")
            else:
                old = c - recent
                best = torch.argsort(-w[:old].double(), stable=True)[: budget - recent]
                keep = torch.cat([best, torch.arange(old, c, device="cuda")]).sort().values
            dst = s["dst"][b, : -(-len(keep) // page)].long()
            out["weight"][dst, h] = _fill(s["weight"][dst, h].double(), w[keep].double())
            for name, key in (("k", "k"), ("v", "v")):
                codes = s[key + "c"][src, h].double().reshape(-1, D)[keep]
                scale = s[key + "s"][src, h].double()[keep // page]
                group = torch.arange(len(keep), device="cuda") // page
                most = torch.stack([scale[i * page:(i + 1) * page].max() for i in range(len(dst))])
                out[name][dst, h] = _fill(s[key + "c"][dst, h].double(), codes * (scale / most[group])[:, None])
                out[name + "_scale"][dst, h] = most
    return {**out, "lens": None, "pos": None}


def _fill(old, rows):
    """`old` [pages, page, ...] with its first rows replaced."""
    flat = old.reshape(-1, *old.shape[2:]).clone()
    flat[: len(rows)] = rows
    return flat.view(old.shape)

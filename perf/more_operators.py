"""Cases of the operators that a hybrid model's recurrent layers and its serving loop need beside
the KDA passes and the paged attention cache.

A recurrent layer starts with a short causal convolution over its projected rows (KDA's q, k and v as
much as a state-space layer's x, B and C), and some layers of a hybrid model are selective state-space
layers: per head a matrix state with one decay per token.  The attention layers' cache lives in
pages that sequences take from a pool and give back.  Five operators:

  conv      a causal convolution of 2 to 4 taps per channel, SiLU after it, over packed rows, with the
            last rows of every sequence carried from call to call
  scan      the selective state-space recurrence over packed prompts, states in and out
  step      the same for one or a few new tokens per sequence, the state updated in place
  reserve   pages for every sequence's new tokens: the block table, the packed rows' cu_seqlens and
            the cache slot of every row, from the lengths on the device
  release   pages that sequences do not need any more go back to the pool

Every case says which operator it is in "op".  ``own`` chooses between the plain form below and
the package's kernels.
"""
import math
import random

import torch

own = False


# ---------------------------------------------------------------- cases

def listed():
    return [
        # the convolution of a KDA layer's q, k and v (3 x 32 heads of 128 channels) over a batch of ragged prompts
        dict(name="conv ragged qkv", op="conv", lo=1, hi=4096, N=8, mix=1, C=12288, W=4, pad=0, bias=False, states=True),
        # one serving step of a state-space layer (x, B and C, cut out of a wider projection), 256 sequences
        dict(name="conv 256x1", op="conv", lo=1, hi=1, N=256, mix=0, C=6144, W=4, pad=4160, bias=True, states=True),
        # a chat turn's short prompt: latency
        dict(name="scan 1x100", op="scan", lo=100, hi=100, N=1, mix=0, H=16, G=1, P=64, S=128, state="fp32", states=True),
        # one long prompt
        dict(name="scan 1x8192", op="scan", lo=8192, hi=8192, N=1, mix=0, H=64, G=8, P=64, S=128, state="fp32",
             states=False),
        # a batch of ragged prompts that go on from cached states, as in chunked prefill
        dict(name="scan ragged", op="scan", lo=1, hi=4096, N=16, mix=2, H=64, G=8, P=64, S=128, state="fp32", states=True),
        # wide heads with a small state, one group, states kept in bf16
        dict(name="scan 4x2048 wide", op="scan", lo=2048, hi=2048, N=4, mix=0, H=32, G=1, P=128, S=64, state="bf16",
             states=True),
        # one user's next token: latency
        dict(name="step 1x1", op="step", lo=1, hi=1, N=1, mix=0, H=64, G=8, P=64, S=128, state="fp32", states=True),
        # a full serving batch
        dict(name="step 256x1", op="step", lo=1, hi=1, N=256, mix=0, H=64, G=8, P=64, S=128, state="fp32", states=True),
        # a token of each of 256 sequences gets its place
        dict(name="reserve 256x1", op="reserve", lo=1, hi=1, clo=0, chi=4096, N=256, mix=3, page=64, room=1.0),
        # a batch of ragged prompts, more than the pool has pages for
        dict(name="reserve ragged prompts", op="reserve", lo=1, hi=8192, clo=0, chi=2048, N=64, mix=4, page=16, room=0.8),
        # drafted tokens that were not accepted: a few sequences lose a page
        dict(name="release 256 drafts", op="release", clo=16, chi=4096, N=256, mix=5, page=16, drop=8),
        # an eviction's old pages, all of them
        dict(name="release 64x16384", op="release", clo=1, chi=16384, N=64, mix=6, page=32, drop=0),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(["conv", "scan", "step", "reserve", "release"])
    mix = rng.randrange(1, 1 << 20)
    if op == "conv":
        C = 8 * _log(rng, 1, 1536)
        hi = _log(rng, 1, 8192)
        N = _log(rng, 1, max(1, min(256, (200 << 20) // (2 * hi * C))))
        return dict(op=op, lo=max(0, hi // rng.choice([1, 2, 50])), hi=hi, N=N, mix=mix, C=C, W=rng.choice([2, 3, 4]),
                    pad=8 * rng.choice([0, 0, 5, 64]), bias=rng.random() < 0.5, states=rng.random() < 0.7)
    if op in ("scan", "step"):
        G = rng.choice([1, 2, 4, 8])
        H = G * rng.choice([1, 2, 3, 4, 8])
        P, S = rng.choice([64, 64, 128]), rng.choice([128, 128, 64])
        case = dict(op=op, mix=mix, H=H, G=G, P=P, S=S, state=rng.choice(["fp32", "fp32", "bf16"]))
        if op == "step":
            hi = rng.choice([1, 1, 1, 2, 5, 8])
            return dict(case, lo=rng.choice([0, 1, hi]), hi=hi, N=_log(rng, 1, max(1, min(256, (1 << 27) // (H * P * S)))),
                        states=True)
        hi = _log(rng, 1, 8192)
        N = _log(rng, 1, max(1, min(32, (1 << 27) // (hi * H * P))))
        return dict(case, lo=max(0, hi // rng.choice([1, 2, 50])), hi=hi, N=N, states=rng.random() < 0.6)
    page = rng.choice([16, 32, 64, 128])
    chi = _log(rng, 16, 16384)
    N = _log(rng, 1, min(512, (1 << 20) // chi))
    case = dict(op=op, clo=chi // rng.choice([1, 2, 50]), chi=chi, N=N, mix=mix, page=page)
    if op == "release":
        return dict(case, drop=rng.choice([0, 0, 1, 7, 100]))
    hi = _log(rng, 1, max(1, min(8192, (1 << 18) // N)))
    return dict(case, lo=hi // rng.choice([1, 2, 50]), hi=hi, room=rng.choice([1.0, 1.0, 0.5]))


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


def work(case):
    N, op = case["N"], case["op"]
    if op == "conv":
        T = sum(_new(case))
        row = 2 * case["C"]
        state = 2 * N * (case["W"] - 1) * row if case["states"] else N * (case["W"] - 1) * row
        return {"bytes": 2 * T * row + state + row * case["W"], "flops": 2 * case["W"] * T * case["C"]}
    if op in ("scan", "step"):
        T, H = sum(_new(case)), case["H"]
        cell = case["P"] * case["S"]
        state = N * H * cell * (4 if case["state"] == "fp32" else 2) * (2 if case["states"] else 1)
        rows = 4 * T * (H * case["P"] + case["G"] * case["S"]) + 2 * T * H
        return {"bytes": rows + state, "flops": 4 * T * H * cell}
    page = case["page"]
    if op == "reserve":
        T = sum(_new(case))
        return {"bytes": 8 * T + 8 * (T // page) + 20 * N, "flops": 4 * T}
    pages = sum(-(-c // page) for c in _cached(case)) if case["drop"] == 0 else N
    return {"bytes": 8 * pages + 8 * N, "flops": 4 * N}


# ---------------------------------------------------------------- inputs

def _cu(lengths):
    v = [0]
    v.extend(sum(lengths[: i + 1]) for i in range(len(lengths)))
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _type(case):
    return torch.float32 if case["state"] == "fp32" else torch.bfloat16


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    s = dict(case)
    op, N = case["op"], case["N"]
    randn = lambda *shape: torch.randn(shape, generator=g, device="cuda")  # noqa: E731
    half = lambda *shape: randn(*shape).to(torch.bfloat16)  # noqa: E731
    rand = lambda *shape: torch.rand(shape, generator=g, device="cuda")  # noqa: E731
    if op == "conv":
        n, C, W = _new(case), case["C"], case["W"]
        s["cu"] = _cu(n)
        s["longest"] = max(n)
        s["x"] = half(sum(n), C + case["pad"])[:, :C]
        s["w"] = (randn(C, W) * W ** -0.5).to(torch.bfloat16)
        s["b"] = (0.2 * randn(C)).to(torch.bfloat16) if case["bias"] else None
        s["held"] = half(N, W - 1, C) if case["states"] else None
        return s
    if op in ("scan", "step"):
        n, H, G, P, S = _new(case), case["H"], case["G"], case["P"], case["S"]
        T = sum(n)
        s["cu"] = _cu(n)
        s["longest"] = max(n)
        # rows of x, B and C side by side, as the convolution before the scan leaves them
        rows = torch.nn.functional.silu(half(T, H * P + 2 * G * S))
        s["x"] = rows[:, : H * P].view(T, H, P)
        s["B"] = rows[:, H * P: H * P + G * S].view(T, G, S)
        s["C"] = rows[:, H * P + G * S:].view(T, G, S)
        # steps from about 1e-3 to 0.1 at rest, larger and smaller from token to token; decay rates 1 to 16
        step = torch.exp(math.log(1e-3) + rand(H) * math.log(100.0))
        s["dt_bias"] = step + torch.log(-torch.expm1(-step))
        s["dt"] = half(T, H)
        s["A"] = -(1.0 + 15.0 * rand(H))
        s["skip"] = 1.0 + 0.1 * randn(H)
        s["held"] = (0.3 * randn(N, H, P, S)).to(_type(case)) if case["states"] else None
        return s
    page, cached = case["page"], _cached(case)
    counts = [-(-c // page) for c in cached]
    if op == "reserve":
        new = _new(case)
        after = [-(-(a + b) // page) for a, b in zip(cached, new)]
        free = int(case["room"] * (sum(after) - sum(counts))) + (7 if case["room"] == 1.0 else 0)
        s["new"] = torch.tensor(new, dtype=torch.int32, device="cuda")
        s["rows"] = sum(new)
        width = max(1, max(after))
    else:
        free = 11
        width = max(1, max(counts))
        s["keep"] = torch.tensor([max(0, c - case["drop"]) for c in cached], dtype=torch.int32, device="cuda") \
            if case["drop"] else None
    pages = sum(counts) + free
    perm = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    j = torch.arange(width, device="cuda")[None]
    c = torch.tensor(counts, device="cuda")[:, None]
    at = torch.where(j < c, torch.cumsum(c, 0) - c + j, 0)
    s["table"] = torch.where(j < c, perm[at], -1).to(torch.int32).contiguous()
    s["lens"] = torch.tensor(cached, dtype=torch.int32, device="cuda")
    s["free"] = torch.full((pages,), -1, dtype=torch.int32, device="cuda")
    s["free"][:free] = perm[pages - free:]
    s["count"] = torch.tensor([free], dtype=torch.int32, device="cuda")
    s["pages"] = pages
    return s


# ---------------------------------------------------------------- one pass

def run(s):
    return {"conv": _conv, "scan": _scan, "step": _scan, "reserve": _reserve, "release": _release}[s["op"]](s)


def _padded(s):
    """Row number of every (sequence, place) of the padded batch [N, L], and whether it exists."""
    cu = s["cu"].long()
    i = torch.arange(max(1, s["longest"]), device="cuda")
    there = i[None] < (cu[1:] - cu[:-1])[:, None]
    return torch.where(there, cu[:-1, None] + i[None], 0), there


def _conv(s):
    if own:
        import chunked_gated_delta_11_gb300 as kda
        out, state = kda.kda_conv_fwd(s["x"], s["w"], s["b"], initial_state=s["held"], cu_seqlens=s["cu"],
                                      final_state=s["held"])
        return {"out": out, "state": state}
    x, w, N, C, W = s["x"].float(), s["w"].float(), s["N"], s["C"], s["W"]
    cu = s["cu"].long()
    T = x.shape[0]
    # every sequence's carried rows stand before its own: row i of sequence n is row i + n (W - 1) of `all`
    n = torch.searchsorted(cu, torch.arange(T, device="cuda"), right=True) - 1
    at = torch.arange(T, device="cuda") + (n + 1) * (W - 1)
    first = (cu[:-1] + torch.arange(N, device="cuda") * (W - 1))[:, None] + torch.arange(W - 1, device="cuda")
    rows = torch.zeros((T + N * (W - 1), C), device="cuda")
    rows[at] = x
    if s["held"] is not None:
        rows[first] = s["held"].float()
    y = sum(rows[at - (W - 1 - j)] * w[:, j] for j in range(W))
    if s["b"] is not None:
        y += s["b"].float()
    y *= torch.sigmoid(y)
    state = rows[first + (cu[1:] - cu[:-1])[:, None]].to(torch.bfloat16)
    if s["held"] is not None:
        state = s["held"].copy_(state)
    return {"out": y.to(torch.bfloat16), "state": state}


def _scan(s):
    if own:
        import chunked_gated_delta_11_gb300 as kda
        a = (s["x"], s["dt"], s["A"], s["B"], s["C"], s["skip"], s["dt_bias"])
        if s["op"] == "step":
            out, state = kda.kda_ssm_step(*a, initial_state=s["held"], cu_seqlens=s["cu"], final_state=s["held"])
        else:
            # the old states stay as they were, for a second try with other tokens
            new = torch.empty((s["N"], s["H"], s["P"], s["S"]), dtype=_type(s), device="cuda")
            out, state = kda.kda_ssm_fwd(*a, initial_state=s["held"], cu_seqlens=s["cu"], final_state=new)
        return {"out": out, "state": state}
    N, H, G, P, S = s["N"], s["H"], s["G"], s["P"], s["S"]
    Q = min(64, max(1, s["longest"]))
    at, there = _padded(s)
    L = -(-at.shape[1] // Q) * Q
    c = L // Q
    more = L - at.shape[1]
    at, there = torch.nn.functional.pad(at, (0, more)), torch.nn.functional.pad(there, (0, more))
    d = torch.nn.functional.softplus(s["dt"].double() + s["dt_bias"].double())[at]
    d = torch.where(there[..., None], d, 0.0)
    l = torch.cumsum((d * s["A"].double()).view(N, c, Q, H), 2)  # log of the decay since the chunk's start
    l = l.permute(0, 3, 1, 2).contiguous()                    # [N, H, c, Q]
    x = torch.where(there[..., None, None], s["x"][at].float(), 0.0) * d.float()[..., None]
    x = x.view(N, c, Q, H, P).permute(0, 3, 1, 2, 4)          # [N, H, c, Q, P]
    heads = lambda t: t[at].float().view(N, c, Q, G, 1, S).expand(-1, -1, -1, -1, H // G, -1).reshape(N, c, Q, H, S) \
        .permute(0, 3, 1, 2, 4)  # noqa: E731
    B, C = heads(s["B"]), heads(s["C"])
    i = torch.arange(Q, device="cuda")
    decay = torch.where(i[:, None] >= i[None], l[..., :, None] - l[..., None, :], -torch.inf).exp().float()
    y = torch.matmul(torch.matmul(C, B.transpose(-1, -2)) * decay, x)
    # what a chunk adds to the state by its end, and the states that chunks start from
    end = l[..., -1:]
    adds = torch.matmul((x * (end - l).exp().float()[..., None]).transpose(-1, -2), B)     # [N, H, c, P, S]
    state = torch.zeros((N, H, P, S), device="cuda") if s["held"] is None else s["held"].float()
    adds = torch.cat([state[:, :, None], adds], 2)
    e = torch.cumsum(torch.nn.functional.pad(end[..., 0], (1, 0)), 2)                      # [N, H, c + 1]
    k = torch.arange(c + 1, device="cuda")
    carry = torch.where(k[:, None] >= k[None], e[..., :, None] - e[..., None, :], -torch.inf).exp().float()
    starts = torch.matmul(carry, adds.reshape(N, H, c + 1, P * S)).view(N, H, c + 1, P, S)
    y += torch.matmul(C * l.exp().float()[..., None], starts[:, :, :-1].transpose(-1, -2))
    y = y.permute(0, 2, 3, 1, 4).reshape(N, L, H, P)[there]
    y = (y + s["skip"][:, None] * s["x"].float()).to(torch.bfloat16)
    state = starts[:, :, -1].to(_type(s))
    return {"out": y, "state": s["held"].copy_(state) if s["op"] == "step" else state}


def _reserve(s):
    if own:
        import chunked_gated_delta_11_gb300 as kda
        r = kda.kda_cache_reserve(s["table"], s["lens"], s["new"], s["free"], s["count"], s["page"], rows=s["rows"])
        return {"table": s["table"], "lens": r.lens, "cu": r.cu_seqlens, "slots": r.slots, "count": r.free_count}
    page, table, width, T = s["page"], s["table"], s["table"].shape[1], s["rows"]
    lens, new = s["lens"].long(), s["new"].long()
    had = (lens + page - 1) // page
    after = (lens + new + page - 1) // page
    fits = after <= width
    want = torch.where(fits, after - had, 0)
    upto = torch.cumsum(want, 0)
    granted = fits & ((want == 0) | (upto <= s["count"]))
    got = torch.where(granted, want, 0)
    # place j of the table gets a page if it lies between what the sequence had and what it has now
    j = torch.arange(width, device="cuda")[None]
    fresh = (j >= had[:, None]) & (j < (had + got)[:, None])
    at = s["count"] - 1 - (upto - want)[:, None] - (j - had[:, None])
    table.copy_(torch.where(fresh, s["free"][torch.where(fresh, at, 0)], table))
    cu = torch.nn.functional.pad(torch.cumsum(new, 0), (1, 0))
    t = torch.arange(T, device="cuda")
    n = (torch.searchsorted(cu, t, right=True) - 1).clamp(max=s["N"] - 1)
    p = lens[n] + t - cu[n]
    slots = torch.where(granted[n], table[n, (p // page).clamp(max=width - 1)].long() * page + p % page, -1)
    return {"table": table, "lens": torch.where(granted, lens + new, lens).int(), "cu": cu.int(), "slots": slots,
            "count": (s["count"] - got.sum()).int()}


def _release(s):
    if own:
        import chunked_gated_delta_11_gb300 as kda
        count = kda.kda_cache_release(s["table"], s["lens"], s["free"], s["count"], s["page"], keep=s["keep"])
        return {"free": s["free"], "count": count}
    page, width = s["page"], s["table"].shape[1]
    up = lambda x: (x.long() + page - 1) // page  # noqa: E731
    last = up(s["lens"])[:, None]
    first = up(s["keep"])[:, None] if s["keep"] is not None else 0
    j = torch.arange(width, device="cuda")[None]
    back = ((j >= first) & (j < last)).flatten()
    at = s["count"] + torch.cumsum(back, 0) - 1
    room = torch.nn.functional.pad(s["free"], (0, 1))
    room.scatter_(0, torch.where(back, at, s["pages"]), s["table"].flatten())
    s["free"].copy_(room[:-1])
    return {"free": s["free"], "count": (s["count"] + back.sum()).int()}


# ---------------------------------------------------------------- the definition in 64 bits

def exact(case, seed):
    if case["op"] == "conv":
        return _exact_conv(case, prepare(case, seed))
    if case["op"] in ("scan", "step"):
        return _exact_scan(case, prepare(case, seed))
    return None  # the block tables hold whole numbers only


def _exact_conv(case, s):
    C, W = case["C"], case["W"]
    w = s["w"].double()
    out = torch.empty((sum(_new(case)), C), dtype=torch.float64, device="cuda")
    state = torch.empty((case["N"], W - 1, C), dtype=torch.float64, device="cuda")
    start = 0
    for b, n in enumerate(_new(case)):
        before = s["held"][b].double() if case["states"] else torch.zeros((W - 1, C), dtype=torch.float64, device="cuda")
        z = torch.cat([before, s["x"][start:start + n].double()])
        y = torch.zeros((n, C), dtype=torch.float64, device="cuda")
        for j in range(W):
            y = torch.addcmul(y, z[j:j + n], w[:, j])
        if case["bias"]:
            y = y + s["b"].double()
        out[start:start + n] = y / (1.0 + torch.exp(-y))
        state[b] = z[n:]
        start += n
    return {"out": out, "state": state}


def _exact_scan(case, s):
    """Token by token, all sequences and heads at once."""
    lengths, N, H, G, P, S = _new(case), case["N"], case["H"], case["G"], case["P"], case["S"]
    n = torch.tensor(lengths, device="cuda")
    start = torch.cumsum(n, 0) - n
    h = torch.zeros((N, H, P, S), dtype=torch.float64, device="cuda") if s["held"] is None else s["held"].double()
    out = torch.zeros((sum(lengths), H, P), dtype=torch.float64, device="cuda")
    order = sorted(range(N), key=lambda b: -lengths[b])      # those that still have a token are the first ones
    order_t = torch.tensor(order, device="cuda")
    h, start = h[order_t].view(N, G, H // G, P, S), start[order_t]
    dt = torch.logaddexp(s["dt"].double() + s["dt_bias"].double(), torch.zeros((), dtype=torch.float64, device="cuda"))
    keep = torch.exp(s["A"].double() * dt)
    live = N
    for t in range(max(lengths)):
        while live and lengths[order[live - 1]] <= t:
            live -= 1
        row = start[:live] + t
        x = s["x"][row].double().view(live, G, H // G, P)
        hh = h[:live]
        hh *= keep[row].view(live, G, H // G, 1, 1)
        hh += (x * dt[row].view(live, G, H // G, 1))[..., None] * s["B"][row].double()[:, :, None, None, :]
        y = torch.matmul(hh, s["C"][row].double()[:, :, None, :, None])[..., 0]
        out[row] = (y + s["skip"].double().view(G, H // G, 1) * x).view(live, H, P)
    state = torch.empty((N, H, P, S), dtype=torch.float64, device="cuda")
    state[order_t] = h.reshape(N, H, P, S)
    return {"out": out, "state": state}

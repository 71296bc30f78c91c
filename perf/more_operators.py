"""What the paged language streams' operators are measured on: norm and rotation
of heads, attention of new tokens over a paged cache, the attention weight that
keys gather, and eviction by that weight.

Where `own` is false, run() computes each operator from its formula with
elementary torch operations in 32 bits (64 for the angles); where it is true it
makes the calls a user of the package makes.  Both work on what prepare()
returns.
"""
import math

import torch

own = False

BF16, F32, F64, I32 = torch.bfloat16, torch.float32, torch.float64, torch.int32
INF = float("inf")


# --------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------
def _rotate(B, T, new, Hq, Hkv, D, page, axes, rot, norm, adjacent, held):
    """page 0: keys and values go to dense outputs, else to pages."""
    return {"op": "rotate", "B": B, "T": T, "new": new, "Hq": Hq, "Hkv": Hkv, "D": D, "page": page, "axes": axes,
            "rot": rot, "norm": norm, "adjacent": adjacent, "held": held}


def _attend(B, T, new, Hq, Hkv, D, page, lo, hi, prefix, P, N, F):
    """lo, hi: the keys that streams hold before the step; N = 0: no shared store."""
    return {"op": "attend", "B": B, "T": T, "new": new, "Hq": Hq, "Hkv": Hkv, "D": D, "page": page, "lo": lo,
            "hi": hi, "prefix": prefix, "P": P, "N": N, "F": F}


def _weigh(B, T, new, Hq, Hkv, D, page, lo, hi, prefix, decay):
    return {"op": "weigh", "B": B, "T": T, "new": new, "Hq": Hq, "Hkv": Hkv, "D": D, "page": page, "lo": lo,
            "hi": hi, "prefix": prefix, "decay": decay}


def _evict(B, Hkv, D, page, lo, hi, sink, recent, budget):
    return {"op": "evict", "B": B, "Hkv": Hkv, "D": D, "page": page, "lo": lo, "hi": hi, "sink": sink,
            "recent": recent, "budget": budget}


def listed():
    return [
        # One decoded token for each of 16 streams: the smallest call, where latency counts.
        dict(_rotate(16, 1, "all", 8, 1, 256, 64, 1, 256, False, False, 2000), name="rotate_decode"),
        # Eight camera frames of 256 tokens with time, height and width, normed heads, dense keys and values.
        dict(_rotate(8, 256, "all", 8, 1, 256, 0, 3, 256, True, False, 0), name="rotate_frames"),
        # Prompts of up to 1999 tokens for 16 streams, 8 K/V heads, half of each head rotated.
        dict(_rotate(16, 1999, "ragged", 32, 8, 128, 16, 1, 64, True, True, 700), name="rotate_prompts"),
        # One token for each of 16 streams over the shared store, short tails.
        dict(_attend(16, 1, "all", 8, 1, 256, 64, 0, 30, False, 64, 8, 256), name="attend_decode"),
        # Long dialogues: one token for each of 32 streams, 8 K/V heads, small pages, no store.
        dict(_attend(32, 1, "all", 32, 8, 128, 16, 0, 16000, False, 0, 0, 0), name="attend_long"),
        # A new prompt of 512 tokens enters while 16 streams decode, over the long history.
        dict(_attend(17, 512, "one", 8, 1, 256, 64, 0, 2000, False, 256, 32, 256), name="attend_mixed"),
        # Chunks of up to 999 tokens with odd lengths, each prompt's start seen by all of it.
        dict(_attend(5, 999, "ragged", 32, 8, 128, 32, 100, 7000, True, 37, 3, 100), name="attend_prompts"),
        # The largest: chunks of 2048 tokens for 8 streams over the long history and tails to 6000 tokens.
        dict(_attend(8, 2048, "all", 8, 1, 256, 128, 0, 6000, False, 256, 32, 256), name="attend_most"),
        # The weight of one decoded token for each of 16 streams.
        dict(_weigh(16, 1, "all", 8, 1, 256, 64, 500, 2000, False, 0.5), name="weigh_decode"),
        # The weight of prompts' chunks, 8 K/V heads.
        dict(_weigh(5, 999, "ragged", 32, 8, 128, 32, 100, 7000, True, 1.0), name="weigh_prompts"),
        # 16 streams cut back to 1024 keys.
        dict(_evict(16, 1, 256, 64, 900, 1500, 4, 256, 1024), name="evict_streams"),
        # 64 long dialogues, 8 K/V heads, cut back to 4096 keys.
        dict(_evict(64, 8, 128, 16, 3000, 9000, 4, 1000, 4096), name="evict_most"),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rotate", "attend", "attend", "weigh", "evict"])
    Hkv, G, D = rng.choice([(1, 8, 256), (1, 8, 256), (8, 4, 128), (2, 8, 128), (1, 2, 64), (4, 1, 64)])
    page, new = rng.choice([16, 32, 64, 128]), rng.choice(["all", "ragged", "one"])
    if op == "rotate":
        B = _log(rng, 1, 64)
        T = _log(rng, 1, max(1, min(2048, 16 * 1999 * 48 * 128 // (B * (G + 2) * Hkv * D))))
        axes = rng.choice([1, 1, 2, 3])
        return _rotate(B, T, new, G * Hkv, Hkv, D, rng.choice([0, page]), axes, rng.choice([D, D, D // 2]),
                       rng.random() < 0.5, rng.random() < 0.3, rng.randint(0, 3000))
    if op == "evict":
        B = _log(rng, 1, 64)
        hi = _log(rng, 20, max(21, min(16000, 64 * 9000 * 8 * 128 // (B * Hkv * D) // 2)))
        budget = _log(rng, 4, hi)
        sink = rng.randint(0, min(8, budget // 4))
        return _evict(B, Hkv, D, page, rng.randint(0, hi), hi, sink, rng.randint(0, (budget - sink) // 2), budget)
    B = _log(rng, 1, 64)
    T = rng.choice([1, _log(rng, 1, max(1, min(2048, 16384 // B)))])
    hi = _log(rng, 8, max(9, min(12000, 32 * 16000 * 8 * 128 // (B * Hkv * D) // 2, 8 * 2048 * 8 * 6000 // (B * T * G * Hkv))))
    lo = rng.randint(0, hi)
    if op == "weigh":
        return _weigh(B, T, new, G * Hkv, Hkv, D, page, lo, hi, rng.random() < 0.3, rng.choice([0.0, 0.5, 1.0]))
    N = rng.choice([0, rng.randint(1, 32)])
    return _attend(B, T, new, G * Hkv, Hkv, D, page, lo, hi, rng.random() < 0.3, rng.randint(0, 300) if N else 0, N,
                   rng.choice([16, 50, 100, 256]) if N else 0)


def _spread(lo, hi, n):
    return [lo + (hi - lo) * i // max(1, n - 1) for i in range(n)]


def _lengths(case):
    """(keys held before the step, new tokens) of each stream, in an order that
    is not sorted."""
    B = case["B"]
    step = next(s for s in (7, 5, 3, 1) if math.gcd(s, B) == 1)
    held = _spread(0, case["held"], B) if case["op"] == "rotate" else _spread(case["lo"], case["hi"], B)
    held = [held[(step * b) % B] for b in range(B)]
    if case["op"] == "evict":
        return held, [0] * B
    T = case["T"]
    return held, [{"all": T, "ragged": T - T * ((3 * b + 1) % 8) // 8, "one": T if b == 0 else 1}[case["new"]]
                  for b in range(B)]


# --------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------
def _values(g, shape):
    """Keys and values as a model makes them: unit scale, one entry in a hundred far out."""
    x = torch.randn(shape, device="cuda", dtype=F32, generator=g)
    return torch.where(torch.rand(shape, device="cuda", generator=g) < 0.01, 4 * x, x).to(BF16)


def _ints(v):
    return torch.tensor(v, dtype=I32, device="cuda")


def _tables(g, case, lens):
    """Tables of the streams' pages, drawn from a pool in random order (unused entries -1); lens may hold two
    lists, the second for pages of a copy."""
    page, counts = case["page"], [[-(-n // case["page"]) for n in ln] for ln in lens]
    n_pages = sum(sum(c) for c in counts) + 3
    order = torch.randperm(n_pages, generator=g, device="cuda").to(I32)
    out, at = [], 0
    for c in counts:
        each = _ints(c)
        before = torch.cumsum(each, 0) - each + at
        j = torch.arange(max(1, max(c)), device="cuda")
        idx = (before[:, None] + j).clamp(max=n_pages - 1).long()
        out.append(torch.where(j < each[:, None], order[idx], torch.full_like(order[idx], -1)).contiguous())
        at += sum(c)
    return n_pages, out


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    st = {"case": case}
    held, new = _lengths(case)
    B, Hkv, D, page = case["B"], case["Hkv"], case["D"], case["page"]
    after = [h + n for h, n in zip(held, new)]
    start = [sum(new[:b]) for b in range(B + 1)]
    N = start[B]
    if case["op"] == "evict":
        st["n_pages"], (st["table"], st["to"]) = _tables(g, case, [held, [min(h, case["budget"]) for h in held]])
        st["len"], st["new_len"] = _ints(held), _ints(held)
    elif page:
        st["n_pages"], (st["table"],) = _tables(g, case, [after])
        st["len"], st["held"], st["new_len"] = _ints(after), _ints(held), _ints(after)
    if case["op"] != "evict":
        st["q_start"] = _ints(start)
    if page:
        pool = (st["n_pages"], page, Hkv, D)
        st["k_pages"], st["v_pages"] = _values(g, pool), _values(g, pool)
        w = torch.rand(pool[:3], device="cuda", generator=g) ** 4
        st["weight"] = torch.where(torch.rand(pool[:3], device="cuda", generator=g) < 0.05, torch.zeros_like(w), w)
    if case["op"] == "evict":
        st["kept"] = torch.zeros((B, Hkv, case["budget"]), dtype=I32, device="cuda")
    if case["op"] == "rotate":
        R = case["rot"]
        st["x"] = _values(g, (N, (case["Hq"] + 2 * Hkv) * D))
        st["freq"] = (10000.0 ** (-torch.arange(0, R, 2, device="cuda", dtype=F64) / R)).float()
        st["sections"] = {1: (R // 2,), 2: (R // 4, R // 2 - R // 4),
                          3: (R // 2 - 2 * (R // 6), R // 6, R // 6)}[case["axes"]]
        at = torch.cat([torch.arange(h, h + n, device="cuda") for h, n in zip(held, new)])
        grid = [at, at // 16 % 16, at % 16]        # a token's time, row and column
        st["pos"] = torch.stack([grid[0] if case["axes"] == 1 else grid[0] // 256, *grid[1:]][:case["axes"]]).to(I32)
        if case["norm"]:
            st["q_weight"], st["k_weight"] = (1 + 0.1 * torch.randn(D, device="cuda", generator=g) for _ in range(2))
        else:
            st["q_weight"] = st["k_weight"] = None
        return st
    if case["op"] == "evict":
        return st
    st["q"] = torch.randn((N, case["Hq"], D), device="cuda", generator=g).to(BF16)
    st["prefix"] = _ints([a // 3 for a in after]) if case["prefix"] else None
    if case["op"] == "weigh":
        st["lse"] = _attention(st)[1]
        st["to"] = st["weight"].clone()
        return st
    P, n_frames, F = case["P"], case["N"], case["F"]
    if n_frames:
        st["k_shared"], st["v_shared"] = _values(g, (P + n_frames * F, Hkv, D)), _values(g, (P + n_frames * F, Hkv, D))
        if own:   # the handle that a program keeps, holding the prefix and the window
            from partitioned_kv_cache_gb300 import rx
            c = rx.Cache(1, case["Hq"], Hkv, D, P, n_frames, F, 1)
            c.pin_prefix(st["k_shared"][None, :P].contiguous(), st["v_shared"][None, :P].contiguous())
            for i in range(P, P + n_frames * F, F):
                c.push_frame(st["k_shared"][None, i:i + F].contiguous(), st["v_shared"][None, i:i + F].contiguous())
            st["cache"] = c
    return st


# --------------------------------------------------------------------------
# one pass
# --------------------------------------------------------------------------
def _run_rotate(s):
    c = s["case"]
    Hq, Hkv, D, R, page = c["Hq"], c["Hkv"], c["D"], c["rot"], c["page"]
    if own:
        from partitioned_kv_cache_gb300 import rx
        heads = rx.Heads(Hq, Hkv, D, s["freq"], s["sections"], s["q_weight"], s["k_weight"], 1e-6, c["adjacent"])
        if not page:
            q, k, v = rx.rotate_heads(s["x"], heads, s["pos"])
            return {"q": q, "k": k, "v": v}
        pages = rx.Pages(s["k_pages"], s["v_pages"], s["table"], s["weight"])
        q = rx.rotate_heads_paged(s["x"], heads, s["pos"], pages, s["q_start"], s["held"], new_len=s["new_len"])
        return {"q": q, "k": s["k_pages"], "v": s["v_pages"], "weight": s["weight"], "new_len": s["new_len"]}
    N = s["x"].shape[0]
    x = s["x"].view(N, Hq + 2 * Hkv, D)
    y = x[:, :Hq + Hkv].float()
    if c["norm"]:
        w = torch.cat([s["q_weight"].expand(Hq, D), s["k_weight"].expand(Hkv, D)])
        y = y * torch.rsqrt(y.square().mean(-1, keepdim=True) + 1e-6) * w
    axis = torch.repeat_interleave(torch.arange(len(s["sections"]), device="cuda"),
                                   torch.tensor(s["sections"], device="cuda"), output_size=R // 2)
    turn = s["pos"][axis].T.double() * s["freq"].double()                     # [N][R/2]
    cos, sin = torch.cos(turn).float()[:, None], torch.sin(turn).float()[:, None]
    pairs = y[..., :R].unflatten(-1, (R // 2, 2) if c["adjacent"] else (2, R // 2))
    a, b = pairs.unbind(-1 if c["adjacent"] else -2)
    turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1 if c["adjacent"] else -2)
    y = torch.cat([turned.flatten(-2), y[..., R:]], -1).to(BF16)
    q, k, v = y[:, :Hq], y[:, Hq:], x[:, Hq + Hkv:]
    if not page:
        return {"q": q.contiguous(), "k": k.contiguous(), "v": v.contiguous()}
    n = torch.arange(N, device="cuda", dtype=I32)
    b = torch.searchsorted(s["q_start"][1:], n, right=True)
    place = s["held"][b] + n - s["q_start"][b]
    at = (s["table"][b, (place // page).long()] * page + place % page).long()
    s["k_pages"].view(-1, Hkv, D)[at] = k
    s["v_pages"].view(-1, Hkv, D)[at] = v
    s["weight"].view(-1, Hkv)[at] = 0
    torch.add(s["held"], s["q_start"][1:] - s["q_start"][:-1], out=s["new_len"])
    return {"q": q.contiguous(), "k": s["k_pages"], "v": s["v_pages"], "weight": s["weight"], "new_len": s["new_len"]}


def _slots(s):
    """[B][keys] place of every key in the pool, and which of them are held."""
    page, table = s["case"]["page"], s["table"]
    j = torch.arange(table.shape[1] * page, device="cuda")
    live = j < s["len"][:, None]
    at = table[:, j // page].long() * page + j % page
    return torch.where(live, at, torch.zeros_like(at)), live


def _scores(s):
    """Queries of the streams side by side, [Hkv][B][T][G][D], the scores against the pages with the mask, which
    rows are tokens, and their places among the packed ones."""
    c = s["case"]
    Hkv, D, T = c["Hkv"], c["D"], c["T"]
    G = c["Hq"] // Hkv
    at, live = _slots(s)
    B, L = at.shape
    n = s["q_start"][1:] - s["q_start"][:-1]
    t = torch.arange(T, device="cuda")
    token = t < n[:, None]                                                    # [B][T]
    packed = torch.where(token, s["q_start"][:-1, None] + t, torch.zeros_like(token, dtype=torch.int64)).long()
    x = s["q"].float().view(-1, Hkv, G, D)[packed].permute(2, 0, 1, 3, 4) / math.sqrt(D)
    seen = (s["len"] - n)[:, None] + t + 1
    if s["prefix"] is not None:
        seen = torch.maximum(seen, torch.minimum(s["prefix"], s["len"])[:, None])
    mask = (torch.arange(L, device="cuda") < seen[..., None]) & live[:, None]  # [B][T][L]
    k = s["k_pages"].view(-1, Hkv, D)[at].float()                             # [B][L][Hkv][D]
    z = x.reshape(Hkv, B, T * G, D) @ k.permute(2, 0, 3, 1)
    z = z.view(Hkv, B, T, G, L).masked_fill_(~mask[None, :, :, None], -INF)
    return x, z, at, live, token, packed


def _attention(s):
    c = s["case"]
    Hkv, D = c["Hkv"], c["D"]
    x, z, at, live, token, packed = _scores(s)
    _, B, T, G, L = z.shape
    top = z.amax(-1)
    if "k_shared" in s:
        zs = (x.reshape(Hkv, B * T * G, D) @ s["k_shared"].float().permute(1, 2, 0)).view(Hkv, B, T, G, -1)
        top = torch.maximum(top, zs.amax(-1))
    z = z.sub_(top[..., None]).exp_()
    total = z.sum(-1)
    v = s["v_pages"].view(-1, Hkv, D)[at].float()
    v = torch.where(live[:, :, None, None], v, torch.zeros_like(v))
    o = (z.view(Hkv, B, T * G, L) @ v.permute(2, 0, 1, 3)).view(Hkv, B, T, G, D)
    if "k_shared" in s:
        zs = zs.sub_(top[..., None]).exp_()
        total = total + zs.sum(-1)
        o = o + (zs.view(Hkv, B * T * G, -1) @ s["v_shared"].float().permute(1, 0, 2)).view(Hkv, B, T, G, D)
    o = (o / total[..., None]).permute(1, 2, 0, 3, 4)[token]                  # [N][Hkv][G][D], in packed order
    lse = (top + torch.log(total)).permute(1, 2, 0, 3)[token]
    return o.reshape(-1, c["Hq"], D).to(BF16), lse.reshape(-1, c["Hq"]).contiguous()


def _run_attend(s):
    if own:
        from partitioned_kv_cache_gb300 import rx
        pages = rx.Pages(s["k_pages"], s["v_pages"], s["table"])
        if "cache" in s:
            return s["cache"].attend_pages(0, s["q"], pages, s["q_start"], s["len"], prefix=s["prefix"], lse=True)
        return rx.attend_pages(s["q"], pages, s["q_start"], s["len"], prefix=s["prefix"], lse=True)
    return _attention(s)


def _run_weigh(s):
    decay = s["case"]["decay"]
    if own:
        from partitioned_kv_cache_gb300 import rx
        pages = rx.Pages(s["k_pages"], s["v_pages"], s["table"], s["weight"])
        return rx.weigh_pages(s["q"], s["lse"], pages, s["q_start"], s["len"], prefix=s["prefix"], decay=decay,
                              out=s["to"])
    _, z, at, live, token, packed = _scores(s)
    Hkv, B, T, G, L = z.shape
    lse = s["lse"].view(-1, Hkv, G)[packed].masked_fill(~token[..., None, None], INF).permute(2, 0, 1, 3)
    z = z.sub_(lse[..., None]).exp_()
    got = decay * s["weight"].view(-1, Hkv)[at] + z.sum((2, 3)).permute(1, 2, 0)   # [B][L][Hkv]
    s["to"].view(-1, Hkv)[at[live]] = got[live]
    return s["to"]


def _run_evict(s):
    c = s["case"]
    Hkv, D, page, sink, recent, budget = (c[k] for k in ("Hkv", "D", "page", "sink", "recent", "budget"))
    if own:
        from partitioned_kv_cache_gb300 import rx
        pages = rx.Pages(s["k_pages"], s["v_pages"], s["table"], s["weight"])
        rx.evict_pages(pages, s["len"], budget, sink=sink, recent=recent, to=s["to"], new_len=s["new_len"],
                       kept=s["kept"])
    else:
        at, live = _slots(s)
        B, L = at.shape
        j = torch.arange(L, device="cuda")
        w = s["weight"].view(-1, Hkv)[at].permute(0, 2, 1)                        # [B][Hkv][L]
        fixed = live & ((j < sink) | (j >= s["len"][:, None] - recent))
        w = w.masked_fill(fixed[:, None], INF).masked_fill(~live[:, None], -INF)
        some = min(L, budget)
        best = torch.sort(w, dim=-1, descending=True, stable=True).indices[..., :some]
        best = torch.where(best < s["len"][:, None, None], best, torch.full_like(best, L))   # beyond a short stream
        best = torch.sort(best, -1).values
        there = best < L                                                          # [B][Hkv][some]
        s["kept"].fill_(-1)[..., :some] = torch.where(there, best, torch.full_like(best, -1)).to(I32)
        b, h, i = torch.nonzero(there, as_tuple=True)
        src = at[b, best[b, h, i]]
        dst = s["to"][b, i // page].long() * page + i % page
        for pool in (s["k_pages"], s["v_pages"], s["weight"]):
            pool = pool.view(-1, Hkv, D) if pool.dim() == 4 else pool.view(-1, Hkv)
            pool[dst, h] = pool[src, h]
        torch.clamp(s["len"], max=budget, out=s["new_len"])
    return {"k": s["k_pages"], "v": s["v_pages"], "weight": s["weight"], "kept": s["kept"], "new_len": s["new_len"]}


def run(state):
    return {"rotate": _run_rotate, "attend": _run_attend, "weigh": _run_weigh, "evict": _run_evict}[state["case"]["op"]](state)


# --------------------------------------------------------------------------
# what a pass cannot do without
# --------------------------------------------------------------------------
def work(case):
    held, new = _lengths(case)
    Hkv, D, N = case["Hkv"], case["D"], sum(new)
    if case["op"] == "evict":
        kept = sum(min(h, case["budget"]) for h in held) * Hkv
        return {"bytes": 4 * Hkv * sum(held) + kept * (8 * D + 12), "flops": Hkv * sum(held)}
    Hq = case["Hq"]
    if case["op"] == "rotate":
        turned = N * (Hq + Hkv)
        return {"bytes": 4 * N * (Hq + 2 * Hkv) * D + 4 * N * case["axes"] + (4 * N * Hkv if case["page"] else 0),
                "flops": turned * (3 * case["rot"] + (4 * D if case["norm"] else 0))}
    keys = seen = 0
    for h, n in zip(held, new):
        first = (h + n) // 3 if case["prefix"] else 0
        seen += sum(max(h + t + 1, first) for t in range(n))
        keys += h + n
    if case["op"] == "weigh":
        return {"bytes": keys * Hkv * (2 * D + 8) + N * Hq * (2 * D + 4), "flops": 2 * D * Hq * seen}
    shared = case["P"] + case["N"] * case["F"]
    return {"bytes": (shared + keys) * Hkv * D * 4 + N * Hq * (4 * D + 4), "flops": 4 * D * Hq * (seen + shared * N)}


# --------------------------------------------------------------------------
# the definitions in 64 bits
# --------------------------------------------------------------------------
def _places(s, b, n):
    """The places in the pool of the first n keys of stream b."""
    page = s["case"]["page"]
    return [int(p) * page + i for p in s["table"][b].tolist() if p >= 0 for i in range(page)][:n]


def _exact_rotate(s, held, new):
    c = s["case"]
    Hq, Hkv, D, R = c["Hq"], c["Hkv"], c["D"], c["rot"]
    x = s["x"].double().reshape(-1, Hq + 2 * Hkv, D)
    out = x.clone()
    for kind, lo, hi in (("q", 0, Hq), ("k", Hq, Hq + Hkv)):
        part = x[:, lo:hi]
        if c["norm"]:
            part = part / torch.sqrt((part * part).sum(-1, keepdim=True) / D + 1e-6) * s[kind + "_weight"].double()
        done, i = part.clone(), 0
        for axis, count in enumerate(s["sections"]):
            for i in range(i, i + count):
                one, two = (2 * i, 2 * i + 1) if c["adjacent"] else (i, i + R // 2)
                turn = (s["pos"][axis].double() * s["freq"][i].double())[:, None]
                z = torch.complex(part[..., one], part[..., two]) * torch.complex(torch.cos(turn), torch.sin(turn))
                done[..., one], done[..., two] = z.real, z.imag
            i += 1 if count else 0
        out[:, lo:hi] = done
    q, k, v = out[:, :Hq], out[:, Hq:Hq + Hkv], out[:, Hq + Hkv:]
    if not c["page"]:
        return {"q": q, "k": k, "v": v}
    kp, vp = s["k_pages"].double(), s["v_pages"].double()
    weight, at = s["weight"].double(), 0
    for b, (h, n) in enumerate(zip(held, new)):
        to = torch.tensor(_places(s, b, h + n)[h:], device="cuda", dtype=torch.int64)
        kp.view(-1, Hkv, D)[to], vp.view(-1, Hkv, D)[to] = k[at:at + n], v[at:at + n]
        weight.view(-1, Hkv)[to] = 0
        at += n
    return {"q": q, "k": kp, "v": vp, "weight": weight, "new_len": _ints([h + n for h, n in zip(held, new)])}


def _exact_evict(s, held):
    c = s["case"]
    Hkv, D, page, budget = c["Hkv"], c["D"], c["page"], c["budget"]
    kp, vp, weight = s["k_pages"].double(), s["v_pages"].double(), s["weight"].double()
    kept = torch.full_like(s["kept"], -1)
    for b, n in enumerate(held):
        src = torch.tensor(_places(s, b, n), device="cuda", dtype=torch.int64)
        dst = torch.tensor([int(p) * page + i for p in s["to"][b].tolist() if p >= 0 for i in range(page)],
                           device="cuda", dtype=torch.int64)
        for h in range(Hkv):
            lo, hi = min(n, c["sink"]), max(min(n, c["sink"]), n - c["recent"])
            if n <= budget:
                keep = list(range(n))
            else:
                w = s["weight"].view(-1, Hkv)[src[lo:hi], h].double().cpu()
                order = sorted(zip((-w).tolist(), range(lo, hi)))[:budget - lo - (n - hi)]
                keep = list(range(lo)) + sorted(i for _, i in order) + list(range(hi, n))
            kept[b, h, :len(keep)] = torch.tensor(keep, dtype=I32)
            keep = src[torch.tensor(keep, device="cuda", dtype=torch.int64)]
            for new, old in ((kp.view(-1, Hkv, D), s["k_pages"].view(-1, Hkv, D)), (vp.view(-1, Hkv, D), s["v_pages"].view(-1, Hkv, D)),
                             (weight.view(-1, Hkv), s["weight"].view(-1, Hkv))):
                new[dst[:len(keep)], h] = old[keep, h].double()
    return {"k": kp, "v": vp, "weight": weight, "kept": kept, "new_len": _ints([min(n, budget) for n in held])}


def exact(case, seed):
    s = prepare(case, seed)
    held, new = _lengths(case)
    if case["op"] == "evict":
        return _exact_evict(s, held)
    if case["op"] == "rotate":
        return _exact_rotate(s, held, new)
    Hkv, D = case["Hkv"], case["D"]
    G, at = case["Hq"] // Hkv, 0
    out = torch.empty(s["q"].shape, dtype=F64, device="cuda")
    lse = torch.empty(s["q"].shape[:2], dtype=F64, device="cuda")
    weight = s["weight"].double()
    for b, (h, n) in enumerate(zip(held, new)):
        src = torch.tensor(_places(s, b, h + n), device="cuda", dtype=torch.int64)
        seen = torch.arange(h + 1, h + n + 1, device="cuda")
        if case["prefix"]:
            seen = seen.clamp(min=(h + n) // 3)
        hidden = torch.arange(h + n, device="cuda") >= seen[:, None]
        for kv in range(Hkv):
            heads = slice(kv * G, kv * G + G)
            q = s["q"][at:at + n, heads].double()
            k, v = s["k_pages"].view(-1, Hkv, D)[src, kv].double(), s["v_pages"].view(-1, Hkv, D)[src, kv].double()
            z = torch.einsum("tgd,kd->tgk", q, k) / math.sqrt(D)
            z = z.masked_fill(hidden[:, None], -INF)
            if case["op"] == "weigh":
                p = torch.exp(z - s["lse"][at:at + n, heads, None].double())
                weight.view(-1, Hkv)[src, kv] = case["decay"] * weight.view(-1, Hkv)[src, kv] + p.sum((0, 1))
                continue
            if case["N"]:
                z = torch.cat([torch.einsum("tgd,kd->tgk", q, s["k_shared"][:, kv].double()) / math.sqrt(D), z], -1)
                v = torch.cat([s["v_shared"][:, kv].double(), v])
            lse[at:at + n, heads] = torch.logsumexp(z, -1)
            out[at:at + n, heads] = torch.einsum("tgk,kd->tgd", torch.softmax(z, -1), v)
        at += n
    return weight if case["op"] == "weigh" else (out, lse)

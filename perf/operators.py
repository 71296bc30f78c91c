"""What the language streams' operators are measured on: appending to 8-bit
tails, attention over the shared store and those tails, and the verification
of drafted tokens.

Where `own` is false, run() computes each operator from its formula with
elementary torch operations in 32 bits (64 for the cumulative sums of the
verification); where it is true it makes the calls a user of the package
makes.  Both work on what prepare() returns.
"""
import math

import torch

own = False

BF16, F32, E4M3 = torch.bfloat16, torch.float32, torch.float8_e4m3fn


# --------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------
def _append(B, T, Hkv, D, cap, ragged):
    return {"op": "append", "B": B, "T": T, "Hkv": Hkv, "D": D, "cap": cap, "ragged": ragged}


def _attend(B, T, Hq, Hkv, D, P, N, F, cap, lo, hi, ragged):
    return {"op": "attend", "B": B, "T": T, "Hq": Hq, "Hkv": Hkv, "D": D, "P": P, "N": N, "F": F,
            "cap": cap, "lo": lo, "hi": hi, "ragged": ragged}


def _verify(B, T, V, dtype, draft_probs):
    return {"op": "verify", "B": B, "T": T, "V": V, "dtype": dtype, "draft_probs": draft_probs}


def listed():
    return [
        # One decoded token for each of 16 streams: the smallest call, where latency counts.
        dict(_append(16, 1, 1, 256, 32, False), name="append_decode"),
        # Up to 8 drafted tokens for each of 61 streams, 8 K/V heads, tails with odd capacity.
        dict(_append(61, 8, 8, 128, 517, True), name="append_drafts"),
        # Prompts of up to 8191 tokens for 24 streams at once.
        dict(_append(24, 8191, 1, 256, 8192, True), name="append_prompts"),
        # The shared-cache batch: one token for each of 16 streams, tails of 0 to 30 tokens.
        dict(_attend(16, 1, 8, 1, 256, 64, 8, 256, 32, 0, 30, False), name="attend_decode"),
        # Drafts of up to 5 tokens over the long history, tails of up to 2000 tokens.
        dict(_attend(16, 5, 8, 1, 256, 256, 32, 256, 2048, 5, 2000, True), name="attend_drafts"),
        # Grouped heads of width 128, odd prefix, odd frames, odd tails.
        dict(_attend(7, 3, 32, 8, 128, 37, 3, 100, 1001, 3, 1001, True), name="attend_grouped"),
        # Long dialogues: one token for each of 32 streams, tails of 1 to 16000 tokens.
        dict(_attend(32, 1, 8, 1, 256, 64, 8, 256, 16384, 1, 16000, False), name="attend_long"),
        # The largest: drafts of 8 tokens for 64 streams over tails of 8000 to 16384 tokens.
        dict(_attend(64, 8, 8, 1, 256, 256, 8, 256, 16384, 8000, 16384, False), name="attend_most"),
        # A few streams with a small vocabulary.
        dict(_verify(4, 4, 32000, "float32", True), name="verify_few"),
        # An odd vocabulary in 16 bits, 7 drafted tokens.
        dict(_verify(16, 7, 50257, "bfloat16", True), name="verify_odd"),
        # Drafts without probabilities (looked up, not sampled).
        dict(_verify(32, 5, 151936, "float32", False), name="verify_lookup"),
        # A large vocabulary for 64 streams.
        dict(_verify(64, 4, 257152, "float32", True), name="verify_most"),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "attend", "attend", "verify"])
    if op == "append":
        Hkv, D = rng.choice([1, 2, 8]), rng.choice([64, 128, 256])
        B = _log(rng, 1, 64)
        T = _log(rng, 1, max(1, min(8191, 24 * 8191 * 256 // (B * Hkv * D))))
        return _append(B, T, Hkv, D, T + _log(rng, 1, 2048), rng.random() < 0.5)
    if op == "attend":
        Hkv, G, D = rng.choice([(1, 8, 256), (1, 8, 256), (8, 4, 128), (2, 8, 128), (1, 2, 64), (4, 1, 64)])
        B, T = _log(rng, 1, 64), rng.randint(1, 8)
        cap = T + _log(rng, 8, max(9, min(16384, 64 * 16384 * 256 // (B * Hkv * max(D, 128)) // 2)))
        hi = rng.randint(max(T, cap // 2), cap)
        return _attend(B, T, Hkv * G, Hkv, D, rng.randint(0, 300), rng.randint(1, 32), rng.choice([16, 50, 100, 256]),
                       cap, rng.randint(T, hi), hi, rng.random() < 0.5)
    return _verify(_log(rng, 1, 64), rng.randint(1, 8), _log(rng, 100, 257152), rng.choice(["float32", "bfloat16"]),
                   rng.random() < 0.75)


def _spread(lo, hi, n):
    return [lo + (hi - lo) * i // max(1, n - 1) for i in range(n)]


def _lengths(case):
    """Tail lengths and new-token counts of a case's streams, in an order that
    is not sorted (a stride through the evenly spread values)."""
    B, T = case["B"], case["T"]
    step = next(s for s in (7, 5, 3, 1) if math.gcd(s, B) == 1)
    new = [T - T * ((3 * b + 1) % 8) // 8 for b in range(B)] if case["ragged"] else [T] * B
    if case["op"] == "append":
        lens = _spread(0, case["cap"] - T, B)
    else:
        lens = _spread(case["lo"], case["hi"], B)
    return [lens[(step * b) % B] for b in range(B)], new


# --------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------
def _scale_of(byte):
    """2^(byte - 127) in 32 bits; 255 stands for NaN."""
    e = byte.to(torch.int32)
    s = torch.where(e == 0, torch.full_like(e, 0x00400000), e << 23).view(F32)
    return torch.where(e == 255, torch.full_like(s, float("nan")), s)


def _quantise(x):
    """x [..., D] -> e4m3 codes and the byte of the power-of-two scale: the
    smallest scale under which the largest magnitude is at most 448."""
    x = x.float()
    top = x.abs().amax(-1)
    m, e = torch.frexp(top)
    byte = (e - 9 + (m > 0.875).int() + 127).clamp(min=0)
    byte = torch.where(top == 0, torch.zeros_like(byte), byte)
    byte = torch.where(torch.isfinite(top), byte, torch.full_like(byte, 255))
    up = torch.where(byte == 255, torch.zeros_like(byte), 254 - byte)      # 2^(127 - byte)
    up = (up << 23).view(F32)
    y = torch.where((byte == 255).unsqueeze(-1), torch.zeros_like(x), x * up.unsqueeze(-1))
    return y.to(E4M3), byte.to(torch.uint8)


def _values(g, shape):
    """Keys and values as a model makes them: unit scale, one entry in a hundred far out."""
    x = torch.randn(shape, device="cuda", dtype=F32, generator=g)
    return torch.where(torch.rand(shape, device="cuda", generator=g) < 0.01, 4 * x, x).to(BF16)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    st = {"case": case}
    if case["op"] == "verify":
        B, T, V, t = case["B"], case["T"], case["V"], getattr(torch, case["dtype"])
        logits = 2.5 * torch.randn((B, T + 1, V), device="cuda", generator=g)
        near = logits[:, :T] + 0.7 * torch.randn((B, T, V), device="cuda", generator=g)
        st["p"] = torch.softmax(logits, -1).to(t)
        q = torch.softmax(near, -1)
        st["draft"] = torch.multinomial(q.view(B * T, V), 1, generator=g).view(B, T).to(torch.int32)
        st["q"] = q.to(t) if case["draft_probs"] else None
        st["u"] = torch.rand((B, T), device="cuda", generator=g)
        st["r"] = torch.rand((B,), device="cuda", generator=g)
        st["n_draft"] = torch.randint(0, T + 1, (B,), device="cuda", generator=g, dtype=torch.int32)
        st["tail_len"] = torch.randint(0, 4096, (B,), device="cuda", generator=g, dtype=torch.int32)
        return st
    lens, new = _lengths(case)
    B, T, Hkv, D, cap = case["B"], case["T"], case["Hkv"], case["D"], case["cap"]
    st["tail_len"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    st["n_new"] = torch.tensor(new, dtype=torch.int32, device="cuda") if case["ragged"] else None
    st["k_tail"], st["k_exp"] = _quantise(_values(g, (B, cap, Hkv, D)))
    st["v_tail"], st["v_exp"] = _quantise(_values(g, (B, cap, Hkv, D)))
    if case["op"] == "append":
        st["k_new"], st["v_new"] = _values(g, (B, T, Hkv, D)), _values(g, (B, T, Hkv, D))
        st["new_len"] = torch.empty_like(st["tail_len"])
        return st
    Hq, P, N, F = case["Hq"], case["P"], case["N"], case["F"]
    st["q"] = torch.randn((B, T, Hq, D), device="cuda", generator=g).to(BF16)
    st["out"] = torch.zeros_like(st["q"])
    st["k_shared"], st["v_shared"] = _values(g, (P + N * F, Hkv, D)), _values(g, (P + N * F, Hkv, D))
    if own:   # the handle that a program keeps, holding the prefix and the window
        from partitioned_kv_cache_gb300 import rx
        c = rx.Cache(1, Hq, Hkv, D, P, N, F, 1, cap, B * T)
        c.pin_prefix(st["k_shared"][None, :P].contiguous(), st["v_shared"][None, :P].contiguous())
        for i in range(P, P + N * F, F):
            c.push_frame(st["k_shared"][None, i:i + F].contiguous(), st["v_shared"][None, i:i + F].contiguous())
        st["cache"] = c
    return st


# --------------------------------------------------------------------------
# one pass
# --------------------------------------------------------------------------
def _run_append(s):
    names = ("k_tail", "v_tail", "k_exp", "v_exp")
    if own:
        from partitioned_kv_cache_gb300 import rx
        rx.tail_append_quant(s["k_tail"], s["v_tail"], s["k_exp"], s["v_exp"], s["tail_len"], s["k_new"], s["v_new"],
                             n_new=s["n_new"], new_len=s["new_len"])
    else:
        cap, T = s["k_tail"].shape[1], s["k_new"].shape[1]
        n = torch.full_like(s["tail_len"], T) if s["n_new"] is None else s["n_new"]
        t = torch.arange(T, device="cuda")
        at = s["tail_len"][:, None] + t
        b, t = torch.nonzero((t < n[:, None]) & (at < cap), as_tuple=True)
        at = at[b, t].long()
        for x in ("k", "v"):
            codes, byte = _quantise(s[x + "_new"][b, t])
            s[x + "_tail"].view(torch.uint8)[b, at] = codes.view(torch.uint8)
            s[x + "_exp"][b, at] = byte
        torch.minimum(s["tail_len"] + n, torch.full_like(n, cap), out=s["new_len"])
    return {k: s[k] for k in names + ("new_len",)}


def _run_attend(s):
    q, out = s["q"], s["out"]
    if own:
        return s["cache"].attend_streams_quant(0, q, s["k_tail"], s["v_tail"], s["k_exp"], s["v_exp"], s["tail_len"],
                                               n_new=s["n_new"], out=out)
    B, T, Hq, D = q.shape
    cap, Hkv = s["k_tail"].shape[1:3]
    G = Hq // Hkv
    n = torch.full_like(s["tail_len"], T) if s["n_new"] is None else s["n_new"]
    t = torch.arange(T, device="cuda")
    seen = (s["tail_len"] - n)[:, None] + t + 1                               # [B][T] tail keys
    mask = torch.arange(cap, device="cuda") < seen[..., None]                 # [B][T][cap]
    live = torch.arange(cap, device="cuda") < s["tail_len"][:, None]          # [B][cap]
    k = s["k_tail"].float() * _scale_of(s["k_exp"])[..., None]                # [B][cap][Hkv][D]
    v = s["v_tail"].float() * _scale_of(s["v_exp"])[..., None]
    v = torch.where(live[:, :, None, None], v, torch.zeros_like(v))
    x = q.float().view(B, T, Hkv, G, D).permute(2, 0, 1, 3, 4) / math.sqrt(D)  # [Hkv][B][T][G][D]
    ks, vs = s["k_shared"].float(), s["v_shared"].float()
    shared = x.reshape(Hkv, B * T * G, D) @ ks.permute(1, 2, 0)               # [Hkv][B*T*G][keys]
    tail = x.reshape(Hkv, B, T * G, D) @ k.permute(2, 0, 3, 1)                # [Hkv][B][T*G][cap]
    tail = tail.view(Hkv, B, T, G, cap).masked_fill(~mask[None, :, :, None], float("-inf"))
    top = torch.maximum(shared.amax(-1).view(Hkv, B, T, G), tail.amax(-1))[..., None]
    shared = torch.exp(shared.view(Hkv, B, T, G, -1) - top)
    tail = torch.exp(tail - top)
    total = shared.sum(-1) + tail.sum(-1)
    o = (shared.view(Hkv, B * T * G, -1) @ vs.permute(1, 0, 2)).view(Hkv, B, T, G, D)
    o = o + (tail.view(Hkv, B, T * G, cap) @ v.permute(2, 0, 1, 3)).view(Hkv, B, T, G, D)
    o = (o / total[..., None]).permute(1, 2, 0, 3, 4).reshape(B, T, Hq, D).to(BF16)
    rows = (t < n[:, None])[..., None, None]
    return out.copy_(torch.where(rows, o, out))


def _run_verify(s):
    p, q, draft, u, r, n = s["p"], s["q"], s["draft"], s["u"], s["r"], s["n_draft"]
    if own:
        from partitioned_kv_cache_gb300 import rx
        tokens, count, length = rx.verify_drafts(p, q, draft, u, r, n_draft=n, tail_len=s["tail_len"])
        return {"tokens": tokens, "n_accept": count, "new_len": length}
    B, T = draft.shape
    b, t = torch.arange(B, device="cuda"), torch.arange(T, device="cuda")
    x = draft.long()[..., None]
    at_p = p[:, :T].gather(2, x)[..., 0].double()
    at_q = torch.ones_like(at_p) if q is None else q.gather(2, x)[..., 0].double()
    fine = (u.double() * at_q < at_p) & (t < n[:, None])
    a = fine.int().cumprod(1).sum(1)                                          # accepted tokens
    row = p[b, a].double()
    refused = (a < n)[:, None]
    at = a.clamp(max=T - 1)
    if q is None:
        less = torch.zeros_like(row).scatter_(1, draft.long()[b, at][:, None], float("inf"))
    else:
        less = q[b, at].double()
    w = torch.where(refused, (row - less).clamp(min=0), row)
    w = torch.where((w > 0).any(1, keepdim=True), w, row)
    total = w.cumsum(1)
    nxt = (total <= r.double()[:, None] * total[:, -1:]).sum(1).to(torch.int32)
    i = torch.arange(T + 1, device="cuda")
    tokens = torch.cat([draft, draft[:, :1]], 1)
    tokens = torch.where(i < a[:, None], tokens, torch.where(i == a[:, None], nxt[:, None], torch.full_like(tokens, -1)))
    a = a.to(torch.int32)
    return {"tokens": tokens, "n_accept": a, "new_len": s["tail_len"] + 1 + a}


def run(state):
    return {"append": _run_append, "attend": _run_attend, "verify": _run_verify}[state["case"]["op"]](state)


# --------------------------------------------------------------------------
# what a pass cannot do without
# --------------------------------------------------------------------------
def work(case):
    if case["op"] == "verify":
        size = 4 if case["dtype"] == "float32" else 2
        rows = 2 if case["draft_probs"] else 1
        return {"bytes": case["B"] * (rows * case["V"] * size + case["T"] * 24), "flops": 2 * rows * case["B"] * case["V"]}
    lens, new = _lengths(case)
    Hkv, D = case["Hkv"], case["D"]
    if case["op"] == "append":
        n = sum(new) * Hkv
        return {"bytes": n * (2 * D * 2 + 2 * D + 2), "flops": 4 * n * D}
    Hq, shared = case["Hq"], case["P"] + case["N"] * case["F"]
    seen = sum((ln - n + 1 + t) for ln, n in zip(lens, new) for t in range(n) if ln - n + 1 + t > 0)
    held = sum(lens)
    return {"bytes": shared * Hkv * D * 4 + held * Hkv * (2 * D + 2) + sum(new) * Hq * D * 4,
            "flops": 4 * D * Hq * (seen + shared * sum(new))}


# --------------------------------------------------------------------------
# the definitions in 64 bits
# --------------------------------------------------------------------------
def _two(e):
    """2^e in 64 bits, made from its bits (pow may be off in the last one)."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _exact_e4m3(x):
    """The e4m3 value nearest to x (ties to the even code), |x| <= 448."""
    mag = x.abs()
    _, e = torch.frexp(mag)
    ulp = _two((e - 1).clamp(min=-6) - 3)
    return torch.round(mag / ulp) * ulp * torch.sign(x)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "append":
        lens, new = _lengths(case)
        got = {k: s[k].double() if k.endswith("tail") else s[k].clone() for k in ("k_tail", "v_tail", "k_exp", "v_exp")}
        for b, (ln, n) in enumerate(zip(lens, new)):
            n = min(n, case["cap"] - ln)
            for x in ("k", "v"):
                v = s[x + "_new"][b, :n].double()
                top = v.abs().amax(-1)
                e = torch.ceil(torch.log2(top / 448))
                e = torch.where(top > 0, e, torch.full_like(e, -127))
                e = torch.where(448 * _two(e - 1) >= top, e - 1, e)
                e = torch.where(448 * _two(e) < top, e + 1, e).clamp(min=-127)
                got[x + "_tail"][b, ln:ln + n] = _exact_e4m3(v * _two(-e)[..., None])
                got[x + "_exp"][b, ln:ln + n] = (e + 127).to(torch.uint8)
        got["new_len"] = torch.tensor([min(ln + n, case["cap"]) for ln, n in zip(lens, new)], dtype=torch.int32)
        return got
    if case["op"] == "attend":
        lens, new = _lengths(case)
        G, out = case["Hq"] // case["Hkv"], torch.zeros_like(s["q"], dtype=torch.float64)
        for b, (ln, n) in enumerate(zip(lens, new)):
            for h in range(case["Hkv"]):
                k = s["k_tail"][b, :ln, h].double() * _two(s["k_exp"][b, :ln, h].long() - 127)[:, None]
                v = s["v_tail"][b, :ln, h].double() * _two(s["v_exp"][b, :ln, h].long() - 127)[:, None]
                k, v = torch.cat([s["k_shared"][:, h].double(), k]), torch.cat([s["v_shared"][:, h].double(), v])
                z = torch.einsum("tgd,kd->tgk", s["q"][b, :n, h * G:(h + 1) * G].double(), k) / math.sqrt(case["D"])
                hidden = torch.arange(len(k), device="cuda") > (len(k) - n + torch.arange(n, device="cuda"))[:, None]
                z = torch.softmax(z.masked_fill(hidden[:, None], float("-inf")), -1)
                out[b, :n, h * G:(h + 1) * G] = torch.einsum("tgk,kd->tgd", z, v)
        return out
    B, T, V = case["B"], case["T"], case["V"]
    tokens, count = torch.full((B, T + 1), -1, dtype=torch.int32), torch.zeros(B, dtype=torch.int32)
    draft, u, r, n = s["draft"].tolist(), s["u"].tolist(), s["r"].tolist(), s["n_draft"].tolist()
    for b in range(B):
        a = 0
        while a < n[b]:
            x = draft[b][a]
            if not u[b][a] * (1.0 if s["q"] is None else float(s["q"][b, a, x])) < float(s["p"][b, a, x]):
                break
            tokens[b, a] = x
            a += 1
        row = s["p"][b, a].double()
        w = row
        if a < n[b]:
            if s["q"] is None:
                w = row.clone()
                w[draft[b][a]] = 0.0
            else:
                w = torch.relu(row - s["q"][b, a].double())
            w = w if float(w.sum()) > 0 else row
        c = torch.cumsum(w, 0)
        tokens[b, a] = int(torch.searchsorted(c, r[b] * c[-1:], right=True))
        count[b] = a
    return {"tokens": tokens, "n_accept": count, "new_len": (s["tail_len"].cpu() + 1 + count).to(torch.int32)}

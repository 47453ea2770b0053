"""Cases that time the operators of the 4-bit key/value cache and what they compute.

Four operators, used in this order by a program that answers token by token:

* ``weights``: the attention weight every key of a prompt has received
  (the sum of its probabilities over the queries and the q heads of its
  group), from the prompt's Q, K and logsumexp under a block mask;
* ``append``: keys and values into a cache that holds them in 4 bits;
* ``fwd``: attention of a few new tokens over that cache, which may also add
  their probabilities to the keys' accumulated weights;
* ``evict``: the keys of the largest accumulated weights, compacted.

The 4-bit cache.  For a key (or value) row of D elements and each group of 32
consecutive elements: s = bf16(amax / 7), code = round_half_even(x / s) + 8 (8
when s is 0), value = s * (code - 8).  Element d of a K row (g = d // 32, t = d
% 32 // 8, j = d % 8) is nibble j of the 32-bit word t * (D / 32) + g; element
d of a V row (g = d // 32, p = d % 32 // 4, j = d % 4) is nibble j of the 16-bit
word p * (D / 32) + g; nibble j sits in byte j // 2, low half first.  With D =
128 the byte index of a V row is XORed with 32 where the slot has bit 1 set.
"""
import math

import torch

own = False

GROUP = 32


def listed():
    return [
        # one new token for each of 16 running sequences: the append of a decode step
        {"name": "append_step", "op": "append", "B": 16, "Hkv": 8, "D": 128, "T": 1, "capacity": 8192, "ragged": False},
        # a batch of padded prompts of unequal lengths, an odd number of tokens, the small head size
        {"name": "append_ragged", "op": "append", "B": 4, "Hkv": 16, "D": 64, "T": 2049, "capacity": 4096, "ragged": True},
        # the keys and values of long prompts
        {"name": "append_prompt", "op": "append", "B": 4, "Hkv": 8, "D": 128, "T": 8192, "capacity": 8192, "ragged": False},
        # one token against one short sequence: all latency
        {"name": "fwd_small", "op": "fwd", "B": 1, "Hq": 2, "Hkv": 2, "D": 64, "T": 1, "len": 512, "ragged": False,
         "accumulate": False, "cap": 0.0, "sinks": 0},
        # the decode step of 16 sequences of unequal lengths, weights accumulated for a later eviction
        {"name": "fwd_gqa_weights", "op": "fwd", "B": 16, "Hq": 32, "Hkv": 8, "D": 128, "T": 1, "len": 8192, "ragged": True,
         "accumulate": True, "cap": 0.0, "sinks": 0},
        # one long document: few rows, a long axis to split
        {"name": "fwd_long", "op": "fwd", "B": 1, "Hq": 32, "Hkv": 8, "D": 128, "T": 1, "len": 65536, "ragged": False,
         "accumulate": False, "cap": 0.0, "sinks": 0},
        # a large batch of long sequences: all bandwidth
        {"name": "fwd_batch", "op": "fwd", "B": 64, "Hq": 32, "Hkv": 8, "D": 128, "T": 1, "len": 8191, "ragged": False,
         "accumulate": False, "cap": 0.0, "sinks": 0},
        # four drafted tokens a sequence, one key head for 16 query heads, soft cap and sinks
        {"name": "fwd_mqa_draft", "op": "fwd", "B": 8, "Hq": 16, "Hkv": 1, "D": 128, "T": 4, "len": 16384, "ragged": True,
         "accumulate": False, "cap": 30.0, "sinks": 4},
        # the weights of a long GQA prompt's keys under the causal mask
        {"name": "weights_gqa_causal", "op": "weights", "B": 1, "Hq": 32, "Hkv": 8, "S": 8192, "D": 128, "mask": "causal",
         "param": 0, "ragged": False},
        # two padded prompts under a local window, one q head a key head
        {"name": "weights_local", "op": "weights", "B": 2, "Hq": 16, "Hkv": 16, "S": 4096, "D": 64, "mask": "local",
         "param": 1024, "ragged": True},
        # running sequences brought back to their budget
        {"name": "evict_step", "op": "evict", "B": 16, "Hkv": 8, "D": 128, "len": 1088, "keep": 1024, "recent": 128,
         "ragged": True},
        # a long prompt's cache compressed to an eighth
        {"name": "evict_prompt", "op": "evict", "B": 1, "Hkv": 8, "D": 128, "len": 65536, "keep": 8192, "recent": 512,
         "ragged": False},
    ]


def _spread(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "fwd", "fwd", "weights", "evict"])
    D = rng.choice([64, 128])
    if op == "append":
        B, Hkv, T = _spread(rng, 1, 16), rng.choice([1, 2, 4, 8, 16]), _spread(rng, 1, 8192)
        while B * Hkv * T > 1 << 18:
            T = T // 2 + 1
        return {"op": op, "B": B, "Hkv": Hkv, "D": D, "T": T, "capacity": -(-(T + rng.randrange(1024)) // 16) * 16,
                "ragged": rng.random() < 0.5}
    if op == "fwd":
        Hkv, G, T = rng.choice([1, 2, 4, 8, 16]), rng.choice([1, 2, 3, 4, 8, 16]), rng.choice([1, 1, 1, 2, 3, 4, 5])
        B, n = _spread(rng, 1, 64), _spread(rng, 1, 65536)
        while B * Hkv * n > 1 << 22 or B * Hkv * G * T * n > 1 << 24:
            B, n = max(1, B // 2), max(1, n * 3 // 4)
        return {"op": op, "B": B, "Hq": Hkv * G, "Hkv": Hkv, "D": D, "T": T, "len": max(n, T), "ragged": rng.random() < 0.5,
                "accumulate": rng.random() < 0.5, "cap": rng.choice([0.0, 0.0, 30.0]), "sinks": rng.choice([0, 0, 1, 4])}
    if op == "weights":
        Hkv, G = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 4])
        B, S = rng.choice([1, 1, 2]), 128 * _spread(rng, 1, 64)
        while B * Hkv * G * S * S > 32 * 8192 * 8192:
            S = S // 256 * 128
        mask = rng.choice(["causal", "local", "chunked", "full"])
        return {"op": op, "B": B, "Hq": Hkv * G, "Hkv": Hkv, "S": S if mask != "full" else min(S, 4096), "D": D,
                "mask": mask, "param": _spread(rng, 64, 2048), "ragged": rng.random() < 0.5}
    B, Hkv, n = _spread(rng, 1, 16), rng.choice([1, 2, 4, 8, 16]), _spread(rng, 2, 65536)
    while B * Hkv * n > 1 << 19:
        n = n // 2 + 1
    keep = min(_spread(rng, 1, n), max(1, (1 << 17) // (B * Hkv)))
    return {"op": op, "B": B, "Hkv": Hkv, "D": D, "len": n, "keep": keep, "recent": rng.randrange(min(keep, 512) + 1),
            "ragged": rng.random() < 0.5}


# ------------------------------------------------------------------ inputs

def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(shape, g):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)


def _keys_values(B, H, n, D, g):
    """Rows with channels of unequal size, as projections give them."""
    k = _randn((B, H, n, D), g).mul_(torch.exp(0.5 * _randn((1, H, 1, D), g))).to(torch.bfloat16)
    v = _randn((B, H, n, D), g).to(torch.bfloat16)
    return k, v


def _lengths(B, n, ragged, g, least=1):
    """int32 [B]: n for each sequence, or lengths of [n / 8, n] with the longest among them."""
    if not ragged:
        return torch.full((B,), n, dtype=torch.int32, device="cuda")
    lens = torch.randint(max(least, n // 8), n + 1, (B,), generator=g, device="cuda", dtype=torch.int32)
    lens[0] = n
    return lens


def _round16(n):
    return -(-n // 16) * 16


def _make_cache(B, Hkv, D, capacity, n, g):
    """A cache whose first n slots hold quantised random rows."""
    k, v = _keys_values(B, Hkv, n, D, g)
    cache = {}
    for name, x in (("k", k), ("v", v)):
        codes, scales, _ = _quantise(x)
        whole = torch.full((B, Hkv, capacity, D // 2), 0x88, dtype=torch.uint8, device="cuda")
        whole[:, :, :n] = _pack(codes, name, torch.arange(n, device="cuda"))
        all_scales = torch.zeros((B, Hkv, capacity, D // GROUP), dtype=torch.bfloat16, device="cuda")
        all_scales[:, :, :n] = scales
        cache[name + "_codes"], cache[name + "_scales"] = whole, all_scales
        del codes, scales
    cache["weights"] = torch.rand((B, Hkv, capacity), generator=g, device="cuda", dtype=torch.float32).square_()
    cache["positions"] = torch.arange(capacity, device="cuda", dtype=torch.int32).expand(B, Hkv, capacity).contiguous()
    return cache


def _visible(case, q0, q1):
    """bool [q1 - q0, S]: which keys queries q0 .. q1 - 1 see."""
    S, p = case["S"], case["param"]
    q = torch.arange(q0, q1, device="cuda")[:, None]
    k = torch.arange(S, device="cuda")[None, :]
    if case["mask"] == "causal":
        return k <= q
    if case["mask"] == "local":
        return (k <= q) & (k >= q - p)
    if case["mask"] == "chunked":
        return (k <= q) & (k // p == q // p)
    return torch.ones((q1 - q0, S), dtype=torch.bool, device="cuda")


def prepare(case, seed):
    g = _generator(seed)
    op, D = case["op"], case["D"]
    if op == "append":
        B, Hkv, T, cap = case["B"], case["Hkv"], case["T"], case["capacity"]
        k, v = _keys_values(B, Hkv, T, D, g)
        cache = {"k_codes": torch.zeros((B, Hkv, cap, D // 2), dtype=torch.uint8, device="cuda"),
                 "k_scales": torch.zeros((B, Hkv, cap, D // GROUP), dtype=torch.bfloat16, device="cuda"),
                 "weights": torch.zeros((B, Hkv, cap), dtype=torch.float32, device="cuda"),
                 "positions": torch.zeros((B, Hkv, cap), dtype=torch.int32, device="cuda")}
        cache["v_codes"], cache["v_scales"] = cache["k_codes"].clone(), cache["k_scales"].clone()
        start = torch.randint(0, cap - T + 1, (B,), generator=g, device="cuda", dtype=torch.int32)
        return {"case": case, "cache": cache, "k": k, "v": v, "start": start,
                "n_new": _lengths(B, T, case["ragged"], g)}
    if op == "fwd":
        B, Hq, Hkv, T, n = case["B"], case["Hq"], case["Hkv"], case["T"], case["len"]
        cache = _make_cache(B, Hkv, D, _round16(n), n, g)
        q = _randn((B, Hq, T, D), g).to(torch.bfloat16)
        sinks = _randn((Hkv, case["sinks"]), g) if case["sinks"] else None
        return {"case": case, "cache": cache, "q": q, "lens": _lengths(B, n, case["ragged"], g, T), "sinks": sinks}
    if op == "weights":
        B, Hq, Hkv, S = case["B"], case["Hq"], case["Hkv"], case["S"]
        q = _randn((B, Hq, S, D), g).to(torch.bfloat16)
        k, _ = _keys_values(B, Hkv, S, D, g)
        lse = torch.empty((B, Hq, S), dtype=torch.float32, device="cuda")
        kt = k.float().transpose(2, 3)[:, :, None]
        for i in range(0, S, 1024):  # the prompt's logsumexp, a strip of queries at a time
            j = min(S, i + 1024)
            s = torch.matmul(q[:, :, i:j].float().view(B, Hkv, Hq // Hkv, j - i, D), kt).mul_(1 / math.sqrt(D))
            s.masked_fill_(~_visible(case, i, j), -math.inf)
            lse[:, :, i:j] = torch.logsumexp(s, -1).view(B, Hq, j - i)
            del s
        info = None
        if own:  # the compiled mask is kept by a user's program
            import block_sparse_attention_process_gb300 as bsa
            kw = {"local": {"local_left": case["param"], "local_right": 0}, "chunked": {"chunk": case["param"]}}
            info = bsa.mask_compile(case["mask"], S, S, orientation="dkv", **kw.get(case["mask"], {}))
        return {"case": case, "q": q, "k": k, "lse": lse, "info": info,
                "q_lens": _lengths(B, S, case["ragged"], g)}
    B, Hkv, n, keep = case["B"], case["Hkv"], case["len"], case["keep"]
    cache = _make_cache(B, Hkv, D, _round16(n), n, g)
    into = {name: torch.zeros((B, Hkv, _round16(keep)) + t.shape[3:], dtype=t.dtype, device="cuda")
            for name, t in cache.items()}
    return {"case": case, "cache": cache, "into": into, "lens": _lengths(B, n, case["ragged"], g)}


# ------------------------------------------------------------------ plain forms

def _quantise(x):
    """codes (0..15) and bf16 scales of each 32 elements of the last axis, and the values they stand for in fp32."""
    x = x.float().unflatten(-1, (-1, GROUP))
    s = (x.abs().amax(-1) / 7).to(torch.bfloat16)
    s32 = s.float()[..., None]
    codes = torch.where(s32 > 0, torch.round(x / s32), torch.zeros_like(x))
    values = (codes * s32).flatten(-2)
    return (codes + 8).to(torch.uint8).flatten(-2), s, values


def _swap(x, slots):
    """V rows of 64 bytes: halves exchanged where the slot has bit 1 set."""
    if x.shape[-1] != 64:
        return x
    return torch.where(((slots & 2) != 0)[..., None], x.roll(32, -1), x)


def _pack(codes, name, slots):
    G = codes.shape[-1] // GROUP
    x = codes.unflatten(-1, (G, 4, 8) if name == "k" else (G, 8, 4)).transpose(-3, -2).flatten(-3)
    x = x[..., 0::2] | (x[..., 1::2] << 4)
    return x if name == "k" else _swap(x, slots)


def _values(cache, name):
    """fp32 [B, H, capacity, D]: what a cache's codes stand for."""
    x = cache[name + "_codes"]
    G = x.shape[-1] * 2 // GROUP
    if name == "v":
        x = _swap(x, torch.arange(x.shape[2], device=x.device))
    x = torch.stack((x & 15, x >> 4), -1).flatten(-2)
    x = x.unflatten(-1, (4, G, 8) if name == "k" else (8, G, 4)).transpose(-3, -2)
    x = x.to(torch.float32).sub_(8).mul_(cache[name + "_scales"].float()[..., None, None])
    return x.flatten(-3)


def _plain_append(state):
    cache, k, v = state["cache"], state["k"], state["v"]
    B, H, T, D = k.shape
    t = torch.arange(T, device="cuda")
    slots = state["start"].long()[:, None] + t                      # [B, T]
    new = t < state["n_new"][:, None]
    b = torch.arange(B, device="cuda")[:, None]
    rows = {"weights": torch.zeros((B, T, 1), device="cuda"), "positions": slots.to(torch.int32)[..., None]}
    out = []
    for name, x in (("k", k), ("v", v)):
        codes, scales, values = _quantise(x)
        rows[name + "_codes"] = _pack(codes, name, slots[:, None]).transpose(1, 2)
        rows[name + "_scales"] = scales.transpose(1, 2)
        out.append((values * new[:, None, :, None]).to(torch.bfloat16))
    for name, x in rows.items():
        old = cache[name][b, :, slots]                              # [B, T, H, ...]
        cache[name][b, :, slots] = torch.where(new.view(B, T, *[1] * (old.dim() - 2)), x, old)
    return out


def _plain_fwd(state):
    case, cache, q = state["case"], state["cache"], state["q"]
    B, Hq, T, D = q.shape
    Hkv, cap = cache["weights"].shape[1:]
    G = Hq // Hkv
    s = torch.matmul(q.float().view(B, Hkv, G * T, D), _values(cache, "k").transpose(2, 3)) * (1 / math.sqrt(D))
    if case["cap"]:
        s = case["cap"] * torch.tanh(s / case["cap"])
    first = state["lens"][:, None] - T + torch.arange(T, device="cuda")   # the last key each new token sees
    seen = torch.arange(cap, device="cuda") <= first[..., None]           # [B, T, cap]
    s = s.view(B, Hkv, G, T, cap).masked_fill(~seen[:, None, None], -math.inf)
    m = s.amax(-1)
    if state["sinks"] is not None:
        z = state["sinks"][None, :, None, None, :]
        m = torch.maximum(m, z.amax(-1))
    e = torch.exp(s - m[..., None])
    total = e.sum(-1)
    if state["sinks"] is not None:
        total = total + torch.exp(z - m[..., None]).sum(-1)
    p = e / total[..., None]
    o = torch.matmul(p.view(B, Hkv, G * T, cap), _values(cache, "v")).view(B, Hq, T, D).to(torch.bfloat16)
    lse = (m + torch.log(total)).view(B, Hq, T)
    if case["accumulate"]:
        cache["weights"] += p.sum((2, 3))
        return {"o": o, "lse": lse, "weights": cache["weights"]}
    return {"o": o, "lse": lse}


def _plain_weights(state):
    case, q, k, lse = state["case"], state["q"], state["k"], state["lse"]
    B, Hq, S, D = q.shape
    Hkv = k.shape[1]
    s = torch.matmul(q.float().view(B, Hkv, -1, D), k.float().transpose(2, 3)).mul_(1 / math.sqrt(D))
    p = s.view(B, Hq, S, S).sub_(lse[..., None]).exp_()
    counted = _visible(case, 0, S) & (torch.arange(S, device="cuda") < state["q_lens"][:, None])[:, :, None]
    p.masked_fill_(~counted[:, None], 0.0)
    return p.view(B, Hkv, -1, S).sum(2)


def _plain_evict(state):
    case, cache, into, lens = state["case"], state["cache"], state["into"], state["lens"]
    keep, recent = case["keep"], case["recent"]
    slots = torch.arange(cache["weights"].shape[2], device="cuda")
    held = slots < lens[:, None, None]
    w = torch.where(cache["positions"] >= lens[:, None, None] - recent, math.inf, cache["weights"])
    w = torch.where(held, w, -math.inf)
    order = torch.sort(w, dim=-1, descending=True, stable=True).indices[..., :keep]
    n = lens.clamp(max=keep)
    kept = torch.arange(keep, device="cuda") < n[:, None, None]
    index = torch.sort(torch.where(kept, order, w.shape[-1]), dim=-1).values
    src = torch.where(kept, index, 0)
    index = torch.where(kept, index, -1).to(torch.int32)
    out = {"index": index, "lens": n}
    for name in ("k", "v"):
        codes = torch.gather(cache[name + "_codes"], 2, src[..., None].expand(-1, -1, -1, cache[name + "_codes"].shape[3]))
        if name == "v":
            codes = _swap(codes, src ^ torch.arange(keep, device="cuda"))
        scales = torch.gather(cache[name + "_scales"], 2, src[..., None].expand(-1, -1, -1, cache[name + "_scales"].shape[3]))
        into[name + "_codes"][:, :, :keep] = torch.where(kept[..., None], codes, into[name + "_codes"][:, :, :keep])
        into[name + "_scales"][:, :, :keep] = torch.where(kept[..., None], scales, into[name + "_scales"][:, :, :keep])
        out[name] = (_values(into, name)[:, :, :keep] * kept[..., None]).to(torch.bfloat16)
    for name in ("weights", "positions"):
        into[name][:, :, :keep] = torch.where(kept, torch.gather(cache[name], 2, src), into[name][:, :, :keep])
        out[name] = into[name]
    return out


# ------------------------------------------------------------------ one pass

def run(state):
    case = state["case"]
    if own:
        import block_sparse_attention_process_gb300 as bsa
        if case["op"] == "weights":
            return bsa.key_weights(state["q"], state["k"], state["lse"], state["info"], q_lens=state["q_lens"])
        cache = bsa.KV4Cache(**state["cache"])
        if case["op"] == "append":
            return bsa.kv4_append(cache, state["k"], state["v"], state["start"], n_new=state["n_new"], values=True)
        if case["op"] == "fwd":
            o, lse = bsa.kv4_fwd(state["q"], cache, state["lens"], logits_soft_cap=case["cap"] or None,
                                 sinks=state["sinks"], accumulate=case["accumulate"])
            return {"o": o, "lse": lse, "weights": cache.weights} if case["accumulate"] else {"o": o, "lse": lse}
        into = bsa.KV4Cache(**state["into"])
        lens, index, k, v = bsa.kv4_evict(cache, state["lens"], case["keep"], recent=case["recent"], out=into, values=True)
        return {"index": index, "lens": lens, "k": k, "v": v, "weights": into.weights, "positions": into.positions}
    return {"append": _plain_append, "fwd": _plain_fwd, "weights": _plain_weights, "evict": _plain_evict}[case["op"]](state)


# ------------------------------------------------------------------ work

def _blocks(case):
    """Blocks of 128 x 128 that hold a visible pair, of one head."""
    n = case["S"] // 128
    p = case["param"]
    if case["mask"] == "full":
        return n * n
    if case["mask"] == "causal":
        return n * (n + 1) // 2
    total = 0
    for i in range(n):
        q0, q1 = i * 128, i * 128 + 127
        lo = max(0, q0 - p) if case["mask"] == "local" else q0 // p * p
        total += q1 // 128 - lo // 128 + 1
    return total


def work(case):
    D, B, Hkv = case["D"], case["B"], case["Hkv"]
    row4 = D // 2 + 2 * (D // GROUP)   # one key or value row in the cache
    part = (1 + 0.5625 * (B - 1)) / B if case["ragged"] else 1.0   # mean of the lengths that _lengths draws
    if case["op"] == "append":
        n = B * Hkv * case["T"] * part
        return {"bytes": n * (2 * (2 * D + row4 + 2 * D) + 8), "flops": n * 2 * D * 4}
    if case["op"] == "fwd":
        n = B * Hkv * case["len"] * part
        rows = case["Hq"] // Hkv * case["T"]
        q = B * case["Hq"] * case["T"]
        return {"bytes": n * (2 * row4 + (8 if case["accumulate"] else 0)) + q * (4 * D + 4), "flops": n * rows * 4 * D}
    if case["op"] == "weights":
        q, k = B * case["Hq"] * case["S"], B * Hkv * case["S"]
        return {"bytes": q * (2 * D + 4) + k * (2 * D + 4), "flops": part * B * case["Hq"] * _blocks(case) * 2 * 128 * 128 * D}
    n = B * Hkv * case["len"] * part
    kept = B * Hkv * min(case["keep"], case["len"])
    return {"bytes": n * 8 + kept * (2 * 2 * row4 + 2 * 2 * D + 8 + 4), "flops": n * 4}


# ------------------------------------------------------------------ 64 bits

def _decode64(cache, name, b):
    """fp64 [H, capacity, D] of sequence b: every element by its own byte and shift."""
    codes, scales = cache[name + "_codes"][b], cache[name + "_scales"][b].double()
    D = codes.shape[-1] * 2
    d = torch.arange(D, device="cuda")
    if name == "k":
        byte, shift = 4 * (d % 32 // 8 * (D // 32) + d // 32) + d % 8 // 2, 4 * (d % 2)
    else:
        byte, shift = 2 * (d % 32 // 4 * (D // 32) + d // 32) + d % 4 // 2, 4 * (d % 2)
    byte = byte[None].repeat(codes.shape[1], 1)
    if name == "v" and D == 128:
        byte ^= 32 * (torch.arange(codes.shape[1], device="cuda")[:, None] >> 1 & 1)
    c = torch.gather(codes, 2, byte[None].expand(codes.shape[0], -1, -1)).int() >> shift & 15
    return (c - 8).double() * scales.repeat_interleave(32, -1)


def _rounded64(x, valid):
    """bf16 of the values that rows x (fp64, [.., D]) take in 4 bits; zero where not valid."""
    x = x.unflatten(-1, (-1, 32))
    top = x.abs().max(-1, keepdim=True).values
    s = (top / 7).to(torch.bfloat16).double()
    q = torch.where(s == 0, 0.0, torch.round(x / torch.where(s == 0, 1.0, s)))
    return (q * s).flatten(-2).masked_fill(~valid, 0.0).to(torch.bfloat16)


def exact(case, seed):
    state = prepare(case, seed)
    if case["op"] == "append":
        valid = (torch.arange(case["T"], device="cuda") < state["n_new"][:, None])[:, None, :, None]
        return [_rounded64(state["k"].double(), valid).double(), _rounded64(state["v"].double(), valid).double()]
    if case["op"] == "fwd":
        q, cache = state["q"].double(), state["cache"]
        B, Hq, T, D = q.shape
        Hkv = case["Hkv"]
        o = torch.zeros((B, Hq, T, D), dtype=torch.float64, device="cuda")
        lse = torch.zeros((B, Hq, T), dtype=torch.float64, device="cuda")
        w = cache["weights"].double()
        for b, n in enumerate(state["lens"].tolist()):
            k, v = _decode64(cache, "k", b)[:, :n], _decode64(cache, "v", b)[:, :n]
            for t in range(T):
                end = n - T + 1 + t
                s = torch.einsum("hgd,hnd->hgn", q[b, :, t].view(Hkv, -1, D), k[:, :end]) * D ** -0.5
                if case["cap"]:
                    s = case["cap"] * torch.tanh(s / case["cap"])
                z = s if state["sinks"] is None else torch.cat(
                    (s, state["sinks"].double()[:, None].expand(-1, s.shape[1], -1)), -1)
                l = torch.logsumexp(z, -1, keepdim=True)
                p = torch.exp(s - l)
                o[b, :, t] = torch.einsum("hgn,hnd->hgd", p, v[:, :end]).reshape(Hq, D)
                lse[b, :, t] = l.reshape(Hq)
                w[b, :, :end] += p.sum(1)
        return {"o": o, "lse": lse, "weights": w} if case["accumulate"] else {"o": o, "lse": lse}
    if case["op"] == "weights":
        q, k, lse = state["q"].double(), state["k"].double(), state["lse"].double()
        B, Hq, S, D = q.shape
        Hkv = case["Hkv"]
        out = torch.zeros((B, Hkv, S), dtype=torch.float64, device="cuda")
        for b, n in enumerate(state["q_lens"].tolist()):
            for i in range(0, n, 2048):
                j = min(n, i + 2048)
                seen = _visible(case, i, j)
                for h in range(Hq):
                    s = q[b, h, i:j] @ k[b, h // (Hq // Hkv)].T * D ** -0.5 - lse[b, h, i:j, None]
                    out[b, h // (Hq // Hkv)] += torch.where(seen, torch.exp(s), 0.0).sum(0)
        return out
    cache, into, keep = state["cache"], state["into"], case["keep"]
    B, H = cache["weights"].shape[:2]
    index = torch.full((B, H, keep), -1, dtype=torch.int32)
    values = {x: torch.zeros((B, H, keep, case["D"]), dtype=torch.float64, device="cuda") for x in "kv"}
    weights, positions = into["weights"].double(), into["positions"].clone()
    lens = state["lens"].tolist()
    for b, n in enumerate(lens):
        k, v = _decode64(cache, "k", b), _decode64(cache, "v", b)
        for h in range(H):
            w = cache["weights"][b, h, :n].tolist()
            p = cache["positions"][b, h, :n].tolist()
            first = sorted(range(n), key=lambda i: (p[i] < n - case["recent"], -w[i], i))[:keep]
            first.sort()
            at = torch.tensor(first, device="cuda")
            m = len(first)
            index[b, h, :m] = at.int().cpu()
            values["k"][b, h, :m], values["v"][b, h, :m] = k[h, at], v[h, at]
            weights[b, h, :m], positions[b, h, :m] = cache["weights"][b, h, at].double(), cache["positions"][b, h, at]
    bf16 = {x: values[x].to(torch.bfloat16).double() for x in "kv"}
    return {"index": index, "lens": torch.tensor([min(n, keep) for n in lens], dtype=torch.int32), "k": bf16["k"],
            "v": bf16["v"], "weights": weights, "positions": positions}

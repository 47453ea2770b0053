"""Cases that time the operators of the paged key/value cache and what they compute.

Four operators, used in this order by a program that answers many sequences token by token:

* ``resize``: sequences get longer or shorter; pages go from a free stack into their tables and back, and every
  new token gets its slot;
* ``append``: keys and values of new tokens into their slots, with the bounds of each page's keys;
* ``fwd``: attention of a few new tokens over the pages of their sequence;
* ``sparse``: the pages whose bounds promise the largest scores, chosen for each query, and attention over them.

The cache: k, v bf16 [pages, Hkv, page, D]; the table int32 [B, M] names the pages of each sequence in order; the
slot of token i of a sequence is table[b, i // page] * page + i % page.  The free stack: entries used .. pages - 1 of
``free`` are the pages that belong to no sequence; the next one taken is entry ``used``.

The bounds of a page and key head, bf16 [pages, Hkv, 2, D]: with m the largest magnitude of its keys and e =
max(floor(log2 m) - 7, -100), the largest and smallest key of every channel rounded up and down to multiples of
2^e; plus and minus infinity throughout where m is not below 2^100.

The score of a page for a query (a new token and key head, its q heads taken together): q as whole numbers qc =
round_half_even(q / 2^f), f = max(floor(log2 max|q|) - 6, -100) (0 where max|q| is not below 2^100), and the maximum over the q heads of
sum_d max(qc_d hi_d, qc_d lo_d); infinite where that is not finite.  Whole numbers below 2^22 times a power of two: exact
in 32 bits in any order.
"""
import math

import numpy as np
import torch

own = False


def listed():
    return [
        # a decode step of 256 running sequences: one token each, a sixteenth of them finished
        {"name": "resize_step", "op": "resize", "B": 256, "page": 16, "M": 512, "T": 1, "admit": False},
        # prompts of up to 8192 tokens taken into the places of a batch of 64
        {"name": "resize_admit", "op": "resize", "B": 64, "page": 16, "M": 512, "T": 8192, "admit": True},
        # one new token for each of 64 running sequences: the append of a decode step
        {"name": "append_step", "op": "append", "B": 64, "Hkv": 8, "D": 128, "T": 1, "page": 16, "bounds": True, "ragged": False},
        # long prompts of an odd number of tokens, the bounds of their pages with them
        {"name": "append_prompt", "op": "append", "B": 4, "Hkv": 8, "D": 128, "T": 8191, "page": 64, "bounds": True,
         "ragged": False},
        # one token against one short sequence: all latency
        {"name": "fwd_small", "op": "fwd", "B": 1, "Hq": 2, "Hkv": 2, "D": 64, "T": 1, "len": 512, "page": 16, "ragged": False,
         "mask": "causal", "param": 0, "cap": 0.0, "sinks": 0},
        # the decode step of 16 sequences of unequal lengths
        {"name": "fwd_gqa_ragged", "op": "fwd", "B": 16, "Hq": 32, "Hkv": 8, "D": 128, "T": 1, "len": 8192, "page": 16,
         "ragged": True, "mask": "causal", "param": 0, "cap": 0.0, "sinks": 0},
        # one long document: few rows, a long axis to split
        {"name": "fwd_long", "op": "fwd", "B": 1, "Hq": 32, "Hkv": 8, "D": 128, "T": 1, "len": 65536, "page": 64,
         "ragged": False, "mask": "causal", "param": 0, "cap": 0.0, "sinks": 0},
        # a large batch of long sequences: all bandwidth
        {"name": "fwd_batch", "op": "fwd", "B": 64, "Hq": 32, "Hkv": 8, "D": 128, "T": 1, "len": 8191, "page": 16,
         "ragged": False, "mask": "causal", "param": 0, "cap": 0.0, "sinks": 0},
        # four drafted tokens a sequence, one key head for 16 query heads, soft cap and sinks
        {"name": "fwd_mqa_draft", "op": "fwd", "B": 8, "Hq": 16, "Hkv": 1, "D": 128, "T": 4, "len": 16384, "page": 32,
         "ragged": True, "mask": "causal", "param": 0, "cap": 30.0, "sinks": 4},
        # two drafted tokens against short sequences, a few of their pages each, the small head size
        {"name": "sparse_draft", "op": "sparse", "B": 4, "Hq": 16, "Hkv": 4, "D": 64, "T": 2, "len": 2048, "page": 16, "keep": 16,
         "ragged": True},
        # one long document: an eighth of its pages
        {"name": "sparse_long", "op": "sparse", "B": 1, "Hq": 32, "Hkv": 8, "D": 128, "T": 1, "len": 131072, "page": 64,
         "keep": 256, "ragged": False},
        # a batch of long sequences, an eighth of the longest one's pages
        {"name": "sparse_batch", "op": "sparse", "B": 16, "Hq": 32, "Hkv": 8, "D": 128, "T": 1, "len": 32768, "page": 64,
         "keep": 64, "ragged": True},
    ]


def _spread(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["resize", "append", "fwd", "fwd", "sparse", "sparse"])
    page = rng.choice([16, 32, 64, 128])
    if op == "resize":
        B, T = _spread(rng, 1, 1024), _spread(rng, 1, 8192)
        while B * T > 64 * 8192:
            T = T // 2 + 1
        return {"op": op, "B": B, "page": page, "M": -(-(T + _spread(rng, 1, 8192)) // page), "T": T, "admit": rng.random() < 0.5}
    D = rng.choice([64, 128])
    if op == "append":
        B, Hkv, T = _spread(rng, 1, 64), rng.choice([1, 2, 4, 8, 16]), _spread(rng, 1, 8192)
        while B * Hkv * T > 1 << 18:
            T = T // 2 + 1
        return {"op": op, "B": B, "Hkv": Hkv, "D": D, "T": T, "page": page, "bounds": rng.random() < 0.7, "ragged": rng.random() < 0.5}
    Hkv, G, T = rng.choice([1, 2, 4, 8, 16]), rng.choice([1, 2, 3, 4, 5, 8, 16]), rng.choice([1, 1, 1, 2, 3, 4, 5])
    B, n = _spread(rng, 1, 64), _spread(rng, 1, 65536)
    while B * Hkv * n > 1 << 22 or B * Hkv * G * T * n > 1 << 24:
        B, n = max(1, B // 2), max(1, n * 3 // 4)
    case = {"op": op, "B": B, "Hq": Hkv * G, "Hkv": Hkv, "D": D, "T": T, "len": max(n, T), "page": page, "ragged": rng.random() < 0.5}
    if op == "fwd":
        mask = rng.choice(["causal", "causal", "local", "chunked"])
        return {**case, "mask": mask, "param": 0 if mask == "causal" else _spread(rng, 16, 4096), "cap": rng.choice([0.0, 0.0, 30.0]),
                "sinks": rng.choice([0, 0, 1, 4])}
    keep = _spread(rng, 2, 256)
    while B * Hkv * T * keep * page > 1 << 21:
        keep = max(2, keep // 2)
        B = max(1, B // 2)
    return {**case, "B": B, "keep": keep}


# ------------------------------------------------------------------ inputs

def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(shape, g):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)


def _rand_bf16(shape, g, channels=None):
    """Random rows, with channels of unequal size as projections give them where `channels` is given."""
    out = torch.empty(shape, dtype=torch.bfloat16, device="cuda")
    step = max(1, (1 << 26) // max(1, out[0].numel()))
    for i in range(0, shape[0], step):
        x = _randn((min(step, shape[0] - i),) + tuple(shape[1:]), g)
        out[i:i + step] = x if channels is None else x.mul_(channels)
    return out


def _lengths(B, n, ragged, g, least=1):
    """int32 [B]: n for each sequence, or lengths of [n / 8, n] with the longest among them."""
    if not ragged:
        return torch.full((B,), n, dtype=torch.int32, device="cuda")
    lens = torch.randint(max(least, n // 8), n + 1, (B,), generator=g, device="cuda", dtype=torch.int32)
    lens[0] = n
    return lens


def _ceil(a, b):
    return -(-a // b)


def _tables(B, M, pages, have, g):
    """A table whose rows hold `have` pages each in no order (others: -1), and the free stack beside it."""
    order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    j = torch.arange(M, device="cuda")
    at = (torch.cumsum(have, 0) - have)[:, None] + j
    held = j < have[:, None]
    table = torch.where(held, order[torch.where(held, at, 0)], -1).contiguous()
    used = have.sum().to(torch.int32).view(1)
    free = torch.where(torch.arange(pages, device="cuda") < used, -1, order)
    return table, free, used


def prepare(case, seed):
    g = _generator(seed)
    op, page, B, T = case["op"], case["page"], case["B"], case["T"]
    if op == "resize":
        M = case["M"]
        longest = M * page
        lens = torch.randint(0, max(1, longest - T + 1), (B,), generator=g, device="cuda", dtype=torch.int32)
        chance = torch.rand((B,), generator=g, device="cuda")
        if case["admit"]:  # three of four places are empty and take a prompt; of the others half have finished
            empty = chance < 0.75
            lens = torch.where(empty, 0, lens)
            prompt = torch.randint(max(1, T // 16), T + 1, (B,), generator=g, device="cuda", dtype=torch.int32)
            new = torch.where(empty, prompt, torch.where(chance < 0.875, 0, lens))
        else:
            new = torch.where(chance < 1 / 16, 0, lens + T)
        # (a pool that the batch nearly fills: it may be that the last ones have to wait)
        pages = max(1, int(B * M * 0.6)) if B > 8 else B * M
        have = _ceil(lens, page).long()
        while int(have.sum()) > pages:
            pages = pages * 5 // 4 + 1
        table, free, used = _tables(B, M, pages, have, g)
        return {"case": case, "table": table, "free": free, "used": used, "lens": lens, "new": new.to(torch.int32)}
    Hkv, D = case["Hkv"], case["D"]
    channels = torch.exp(0.5 * _randn((1, Hkv, 1, D), g))
    if op == "append":
        lens = torch.randint(0, 256, (B,), generator=g, device="cuda", dtype=torch.int32)
        n_new = _lengths(B, T, case["ragged"], g)
        M = _ceil(T + 256, page)
        pages = B * M + 7
        table, _, _ = _tables(B, M, pages, _ceil(lens + n_new, page).long(), g)
        kc, vc = _rand_bf16((pages, Hkv, page, D), g, channels), _rand_bf16((pages, Hkv, page, D), g)
        i = torch.arange(T, device="cuda")
        at = lens[:, None].long() + i
        new = i < n_new[:, None]
        slots = torch.where(new, torch.gather(table, 1, torch.where(new, at // page, 0)) * page + at % page, -1).to(torch.int32)
        cache = {"k": kc, "v": vc, "bounds": _bounds(kc, kc.new_full((pages,), page, dtype=torch.long)) if case["bounds"] else None}
        return {"case": case, "cache": cache, "k": _rand_bf16((B, Hkv, T, D), g, channels), "v": _rand_bf16((B, Hkv, T, D), g),
                "slots": slots.contiguous()}
    n, Hq = case["len"], case["Hq"]
    lens = _lengths(B, n, case["ragged"], g, T)
    M = _ceil(n, page)
    pages = B * M + 5
    table, _, _ = _tables(B, M, pages, _ceil(lens, page).long(), g)
    kc, vc = _rand_bf16((pages, Hkv, page, D), g, channels), _rand_bf16((pages, Hkv, page, D), g)
    state = {"case": case, "cache": {"k": kc, "v": vc, "bounds": None}, "table": table, "lens": lens,
             "q": _randn((B, Hq, T, D), g).to(torch.bfloat16)}
    if op == "fwd":
        return {**state, "sinks": _randn((Hkv, case["sinks"]), g) if case["sinks"] else None}
    fill = torch.full((pages,), page, dtype=torch.long, device="cuda")
    last = torch.gather(table, 1, (_ceil(lens, page).long() - 1)[:, None])[:, 0].long()
    fill[last] = (lens - 1).long() % page + 1
    state["cache"]["bounds"] = _bounds(kc, fill)
    return state


# ------------------------------------------------------------------ plain forms

def _power(x, bits):
    """2^max(floor(log2 x) - bits, -100) of non-negative numbers below 2^100."""
    e = torch.frexp(x).exponent - 1 - bits
    return torch.ldexp(torch.ones_like(x), torch.where(x > 0, e, -100).clamp(min=-100))


def _bounds(k, fill):
    """bf16 [n, Hkv, 2, D]: bounds of the first fill[i] keys of pages k [n, Hkv, page, D]."""
    out = torch.empty((k.shape[0], k.shape[1], 2, k.shape[3]), dtype=torch.bfloat16, device=k.device)
    step = max(1, (1 << 26) // max(1, k[0].numel()))
    for i in range(0, k.shape[0], step):
        x = k[i:i + step].float()
        out_of = (torch.arange(k.shape[2], device=k.device) >= fill[i:i + step, None])[:, None, :, None]
        top = x.abs().masked_fill(out_of, 0.0).amax((2, 3), keepdim=True)
        usual = top < 2.0 ** 100
        s = _power(torch.where(usual, top, 1.0), 7)
        hi = torch.ceil(x.masked_fill(out_of, -math.inf).amax(2, keepdim=True) / s) * s
        lo = torch.floor(x.masked_fill(out_of, math.inf).amin(2, keepdim=True) / s) * s
        out[i:i + step] = torch.cat((torch.where(usual, hi, math.inf), torch.where(usual, lo, -math.inf)), 2)
    return out


def _plain_resize(state):
    case, table, free, lens = state["case"], state["table"], state["free"], state["lens"].long()
    page, T, M, pages = case["page"], case["T"], case["M"], free.numel()
    j = torch.arange(M, device="cuda")
    new = state["new"].long()
    new = torch.where((new >= 0) & (new <= M * page) & (new - lens <= T), new, lens)
    have, want = _ceil(lens, page), _ceil(new, page)
    drop, need = (have - want).clamp(min=0), (want - have).clamp(min=0)
    base = state["used"].long() - drop.sum()
    # pages given back, then pages taken; the entry one past the stack takes what is not moved
    stack = torch.cat((free, free.new_zeros(1)))
    gone = (j >= want[:, None]) & (j < have[:, None])
    stack[torch.where(gone, base + (torch.cumsum(drop, 0) - drop)[:, None] + j - want[:, None], pages)] = table
    before = torch.cumsum(need, 0) - need
    served = (need == 0) | (before + need <= pages - base)
    new = torch.where(served, new, lens)
    need = torch.where(served, need, 0)
    taken = (j >= have[:, None]) & (j < (have + need)[:, None])
    table.copy_(torch.where(taken, stack[torch.where(taken, base + before[:, None] + j - have[:, None], 0)], table))
    free.copy_(stack[:pages])
    i = torch.arange(T, device="cuda")
    at = lens[:, None] + i
    added = at < new[:, None]
    slots = torch.where(added, torch.gather(table, 1, torch.where(added, at // page, 0)).long() * page + at % page, -1)
    return {"lens": new.to(torch.int32), "used": (base + need.sum()).to(torch.int32), "slots": slots.to(torch.int32),
            "table": table, "free": free}


def _plain_append(state):
    cache, slots = state["cache"], state["slots"].long()
    pages, _, page, _ = cache["k"].shape
    new = slots >= 0
    at = slots[new]
    for name in ("k", "v"):
        cache[name][at // page, :, at % page] = state[name].transpose(1, 2)[new]
    if cache["bounds"] is None:
        return {"k": cache["k"], "v": cache["v"]}
    fill = torch.zeros(pages, dtype=torch.long, device="cuda").scatter_reduce_(0, at // page, at % page + 1, "amax")
    touched = torch.nonzero(fill)[:, 0]
    cache["bounds"][touched] = _bounds(cache["k"][touched], fill[touched])
    return dict(cache)


def _limits(state):
    """[B, T]: the position of each new token (the last key it sees)."""
    T = state["q"].shape[2]
    return state["lens"][:, None].long() - T + torch.arange(T, device="cuda")


def _first(case, pos):
    """The first key that a token at `pos` sees."""
    if case.get("mask") == "local":
        return (pos - case["param"]).clamp(min=0)
    if case.get("mask") == "chunked":
        return pos // case["param"] * case["param"]
    return torch.zeros_like(pos)


def _softmax_values(case, s, v, z):
    """(o, lse) of scores s [.., R, n] (-inf: not seen) over values v [.., n, D], with sinks z [.., R, m] or None."""
    if case.get("cap"):
        s = torch.where(torch.isfinite(s), case["cap"] * torch.tanh(s / case["cap"]), s)
    m = s.amax(-1, keepdim=True)
    if z is not None:
        m = torch.maximum(m, z.amax(-1, keepdim=True))
    e = torch.exp(s - m)
    total = e.sum(-1, keepdim=True)
    if z is not None:
        total = total + torch.exp(z - m).sum(-1, keepdim=True)
    return torch.matmul(e, v) / total, (m + torch.log(total))[..., 0]


def _plain_fwd(state):
    case, cache, table, q = state["case"], state["cache"], state["table"], state["q"]
    B, Hq, T, D = q.shape
    Hkv, page = cache["k"].shape[1:3]
    G, n = Hq // Hkv, table.shape[1] * page
    pos = _limits(state)
    key = torch.arange(n, device="cuda")
    o, lse = torch.empty_like(q), torch.empty((B, Hq, T), dtype=torch.float32, device="cuda")
    step = max(1, (1 << 27) // (Hkv * n * D))
    for b in range(0, B, step):
        t = table[b:b + step].clamp(min=0).long()
        c = t.shape[0]
        k, v = (cache[x][t].transpose(1, 2).reshape(c, Hkv, n, D).float() for x in "kv")
        s = torch.matmul(q[b:b + c].float().view(c, Hkv, G * T, D), k.transpose(2, 3)) * (1 / math.sqrt(D))
        p = pos[b:b + c, :, None]
        seen = (key <= p) & (key >= _first(case, p))
        s = s.view(c, Hkv, G, T, n).masked_fill(~seen[:, None, None], -math.inf).view(c, Hkv, G * T, n)
        v = v.masked_fill((key >= state["lens"][b:b + c, None])[:, None, :, None], 0.0)
        z = None if state["sinks"] is None else state["sinks"][None, :, None].expand(c, -1, G * T, -1)
        x, l = _softmax_values(case, s, v, z)
        o[b:b + c] = x.view(c, Hq, T, D).to(torch.bfloat16)
        lse[b:b + c] = l.view(c, Hq, T)
    return {"o": o, "lse": lse}


def _plain_select(state):
    """int32 [B, Hkv, T, keep]: the pages of each query in order, -1 behind the last one."""
    case, table, q = state["case"], state["table"], state["q"].float()
    B, Hq, T, D = q.shape
    bounds = state["cache"]["bounds"]
    Hkv, M, keep = bounds.shape[1], table.shape[1], case["keep"]
    q = q.view(B, Hkv, Hq // Hkv, T, D)
    top = q.abs().amax((2, 4), keepdim=True)
    usual = top < 2.0 ** 100
    qc = torch.where(usual, torch.round(q / _power(torch.where(usual, top, 1.0), 6)), 0.0)
    b = bounds[table.clamp(min=0).long()].float().permute(0, 2, 3, 4, 1)               # [B, Hkv, 2, D, M]
    s = torch.matmul(torch.cat((qc.clamp(min=0), qc.clamp(max=0)), -1).flatten(2, 3), b.flatten(2, 3))
    s = s.view(B, Hkv, -1, T, M).amax(2)                                                # [B, Hkv, T, M]
    n = _ceil(_limits(state) + 1, case["page"])[:, None, :, None]                       # pages that a query sees
    j = torch.arange(M, device="cuda")
    s = torch.where(torch.isfinite(s), s.double(), 1e300)
    s = torch.where((j < 1) | (j >= n - 1), 1e301, s)                                   # the first and the last one always
    s = torch.where(j < n, s, -math.inf)
    order = torch.sort(s, dim=-1, descending=True, stable=True).indices[..., :keep]
    if M < keep:
        order = torch.nn.functional.pad(order, (0, keep - M))
    kept = torch.arange(keep, device="cuda") < n
    index = torch.sort(torch.where(kept, order, M), dim=-1).values
    return torch.where(kept, index, -1).to(torch.int32)


def _plain_sparse(state):
    case, cache, table, q = state["case"], state["cache"], state["table"], state["q"]
    B, Hq, T, D = q.shape
    Hkv, page = cache["k"].shape[1:3]
    index = _plain_select(state)
    keep, G = index.shape[3], Hq // Hkv
    o, lse = torch.empty_like(q), torch.empty((B, Hq, T), dtype=torch.float32, device="cuda")
    pos = _limits(state)
    step = max(1, (1 << 27) // (Hkv * T * keep * page * D))
    heads = torch.arange(Hkv, device="cuda")[:, None, None]
    for b in range(0, B, step):
        x = index[b:b + step].long()
        c = x.shape[0]
        at = torch.gather(table[b:b + c, None, None].expand(c, Hkv, T, -1).long(), 3, x.clamp(min=0)).clamp(min=0)
        key = (x[..., None] * page + torch.arange(page, device="cuda")).flatten(3)                       # [c, Hkv, T, n]
        seen = ((x >= 0)[..., None].expand(*x.shape, page).flatten(3)) & (key <= pos[b:b + c, None, :, None])
        k, v = (cache[y][at, heads].flatten(3, 4).float() for y in "kv")                                 # [c, Hkv, T, n, D]
        r = q[b:b + c].float().view(c, Hkv, G, T, D).transpose(2, 3)
        s = (torch.matmul(r, k.transpose(3, 4)) * (1 / math.sqrt(D))).masked_fill(~seen[:, :, :, None], -math.inf)
        y, l = _softmax_values(case, s, v.masked_fill(~seen[..., None], 0.0), None)
        o[b:b + c] = y.transpose(2, 3).reshape(c, Hq, T, D).to(torch.bfloat16)
        lse[b:b + c] = l.transpose(2, 3).reshape(c, Hq, T)
    return {"index": index, "o": o, "lse": lse}


# ------------------------------------------------------------------ one pass

def run(state):
    case = state["case"]
    if not own:
        return {"resize": _plain_resize, "append": _plain_append, "fwd": _plain_fwd, "sparse": _plain_sparse}[case["op"]](state)
    import block_sparse_attention_process_gb300 as bsa
    if case["op"] == "resize":
        lens, used, slots = bsa.paged_resize(state["table"], state["free"], state["used"], state["lens"], state["new"], case["page"],
                                             case["T"])
        return {"lens": lens, "used": used, "slots": slots, "table": state["table"], "free": state["free"]}
    cache = bsa.PagedCache(**state["cache"])
    if case["op"] == "append":
        bsa.paged_append(cache, state["k"], state["v"], state["slots"])
        return {x: y for x, y in state["cache"].items() if y is not None}
    if case["op"] == "fwd":
        window = {"local": {"local_left": case["param"]}, "chunked": {"chunk": case["param"]}}.get(case["mask"], {})
        o, lse = bsa.paged_fwd(state["q"], cache, state["table"], state["lens"], logits_soft_cap=case["cap"] or None,
                               sinks=state["sinks"], **window)
        return {"o": o, "lse": lse}
    index = bsa.paged_select(state["q"], cache, state["table"], state["lens"], case["keep"], first=1, recent=1)
    o, lse = bsa.paged_fwd(state["q"], cache, state["table"], state["lens"], select=index)
    return {"index": index, "o": o, "lse": lse}


# ------------------------------------------------------------------ work

def work(case):
    B, T, page = case["B"], case["T"], case["page"]
    if case["op"] == "resize":
        # a slot for each token of the map, and the table and stack entries that change
        moved = B * (0.75 * 0.53 * T / page if case["admit"] else (T / page + case["M"] / 32))
        return {"bytes": B * 12 + 4 * B * T + 12 * moved, "flops": B * T * 4}
    D, Hkv = case["D"], case["Hkv"]
    part = (1 + 0.5625 * (B - 1)) / B if case["ragged"] else 1.0   # mean of the lengths that _lengths draws
    if case["op"] == "append":
        n = B * Hkv * T * part
        touched = B * Hkv * (T * part / page + 1)
        begun = B * Hkv * page / 2
        return {"bytes": n * 8 * D + 4 * B * T + (touched * 4 * D + begun * 2 * D if case["bounds"] else 0), "flops": n * D * 4}
    q = B * case["Hq"] * T
    if case["op"] == "fwd":
        n = case["len"] * part
        if case["mask"] != "causal":
            n = min(n, case["param"] + T if case["mask"] == "local" else case["param"] / 2 + T)
        return {"bytes": B * Hkv * n * 4 * D + q * (4 * D + 4), "flops": B * case["Hq"] * T * n * 4 * D}
    pages = case["len"] * part / page
    kept = min(case["keep"], pages)
    return {"bytes": B * Hkv * (pages * 4 * D + T * kept * (page * 4 * D + 4)) + q * (4 * D + 4),
            "flops": q * (pages * 4 * D + kept * page * 4 * D)}


# ------------------------------------------------------------------ 64 bits

def _exact_resize(state):
    case, page, T = state["case"], state["case"]["page"], state["case"]["T"]
    table, free = state["table"].cpu().numpy().copy(), state["free"].cpu().numpy().copy()
    lens, new, used = state["lens"].tolist(), state["new"].tolist(), int(state["used"][0])
    out, slots = list(lens), np.full((len(lens), T), -1, dtype=np.int32)
    fits = [0 <= w <= case["M"] * page and w - n <= T for n, w in zip(lens, new)]
    given = [p for b, n in enumerate(lens) if fits[b] for p in table[b, _ceil(new[b], page):_ceil(n, page)].tolist()]
    used -= len(given)
    free[used:used + len(given)] = given
    waits = False
    for b, n in enumerate(lens):
        if not fits[b]:
            continue
        more = _ceil(new[b], page) - _ceil(n, page)
        if more > 0:
            waits = waits or used + more > len(free)
            if waits:
                continue
            table[b, _ceil(n, page):_ceil(n, page) + more] = free[used:used + more]
            used += more
        out[b] = new[b]
        at = np.arange(n, max(n, new[b]))
        slots[b, :len(at)] = table[b, at // page] * page + at % page
    return {"lens": torch.tensor(out, dtype=torch.int32), "used": torch.tensor([used], dtype=torch.int32),
            "slots": torch.from_numpy(slots), "table": torch.from_numpy(table), "free": torch.from_numpy(free)}


def _unit64(top, bits):
    return 2.0 ** np.maximum(np.floor(np.log2(np.where(top > 0, top, 2.0 ** -120))) - bits, -100)


def _exact_append(state):
    cache = {x: y if y is None else y.double() for x, y in state["cache"].items()}
    page = cache["k"].shape[2]
    slots = state["slots"].cpu().numpy()
    last = {}
    for b in range(slots.shape[0]):
        n = int((slots[b] >= 0).sum())
        at = torch.from_numpy(slots[b, :n]).long().cuda()
        for x in "kv":
            cache[x][at // page, :, at % page] = state[x][b, :, :n].double().transpose(0, 1)
        for s in slots[b, :n].tolist():
            last[s // page] = s % page
    if cache["bounds"] is None:
        return {"k": cache["k"], "v": cache["v"]}
    for p, end in last.items():
        x = cache["k"][p, :, :end + 1].cpu().numpy()
        unit = _unit64(np.abs(x).max((1, 2)), 7)[:, None]
        cache["bounds"][p] = torch.from_numpy(np.stack((np.ceil(x.max(1) / unit) * unit, np.floor(x.min(1) / unit) * unit), 1)).cuda()
    return cache


def _exact_attend(case, q, k, v, z):
    """One query: q [Hkv, G, D], k and v [Hkv, n, D] of what it sees, z [Hkv, m] or None."""
    s = torch.einsum("hgd,hnd->hgn", q, k) * q.shape[-1] ** -0.5
    if case.get("cap"):
        s = case["cap"] * torch.tanh(s / case["cap"])
    a = s if z is None else torch.cat((s, z[:, None].expand(-1, s.shape[1], -1)), -1)
    l = torch.logsumexp(a, -1, keepdim=True)
    return torch.einsum("hgn,hnd->hgd", torch.exp(s - l), v).flatten(0, 1), l.flatten()


def exact(case, seed):
    state = prepare(case, seed)
    if case["op"] == "resize":
        return _exact_resize(state)
    if case["op"] == "append":
        return _exact_append(state)
    cache, table, page = state["cache"], state["table"].long(), case["page"]
    B, Hq, T, D = state["q"].shape
    Hkv = case["Hkv"]
    q = state["q"].double().view(B, Hkv, -1, T, D)
    o = torch.zeros((B, Hq, T, D), dtype=torch.float64, device="cuda")
    lse = torch.zeros((B, Hq, T), dtype=torch.float64, device="cuda")
    index = np.full((B, Hkv, T, case.get("keep", 0)), -1, dtype=np.int32)
    for b, n in enumerate(state["lens"].tolist()):
        mine = table[b, :_ceil(n, page)]
        if case["op"] == "fwd":
            k, v = (cache[x][mine].transpose(0, 1).flatten(1, 2) for x in "kv")
        else:
            limit = cache["bounds"][mine].double()                                      # [pages, Hkv, 2, D]
            for t in range(T):
                x = q[b, :, :, t]
                unit = torch.from_numpy(_unit64(x.abs().amax((1, 2)).cpu().numpy(), 6)).cuda()
                x = torch.round(x / unit[:, None, None])
                s = torch.maximum(x[:, None] * limit[:, :, 0].transpose(0, 1)[:, :, None],
                                  x[:, None] * limit[:, :, 1].transpose(0, 1)[:, :, None]) if mine.numel() * Hq * D < 1 << 27 else torch.stack(
                    [torch.maximum(x * y[:, 0, None], x * y[:, 1, None]) for y in limit], 1)
                s = s.sum(-1).amax(-1).cpu().numpy()                                    # [Hkv, pages]
                m = _ceil(n - T + t + 1, page)
                for h in range(Hkv):
                    rest = np.lexsort((np.arange(1, m - 1), -s[h, 1:m - 1])) + 1
                    chosen = sorted(({0, m - 1} | set(rest[:max(0, case["keep"] - len({0, m - 1}))].tolist())) if m else ())
                    index[b, h, t, :len(chosen)] = chosen
        for t in range(T):
            end = n - T + t + 1
            if case["op"] == "fwd":
                first = int(_first(case, torch.tensor(end - 1)))
                z = None if state["sinks"] is None else state["sinks"].double()
                x, l = _exact_attend(case, q[b, :, :, t], k[:, first:end].double(), v[:, first:end].double(), z)
                o[b, :, t], lse[b, :, t] = x, l
                continue
            for h in range(Hkv):
                own_pages = torch.from_numpy(index[b, h, t][index[b, h, t] >= 0]).long().cuda()
                at = own_pages[:, None] * page + torch.arange(page, device="cuda")
                k, v = (cache[y][mine[own_pages], h][at < end].double()[None] for y in "kv")
                x, l = _exact_attend(case, q[b, h, :, t][None], k, v, None)
                g = Hq // Hkv
                o[b, h * g:(h + 1) * g, t], lse[b, h * g:(h + 1) * g, t] = x, l
    out = {"o": o, "lse": lse}
    return {"index": torch.from_numpy(index), **out} if case["op"] == "sparse" else out

"""The 4-bit key/value cache on the GPU against the fp64 oracle: append (bit
for bit), attention, accumulated weights, eviction (exactly), a prompt's key
weights, and a run of them together.

Tolerances (none is a measured one).  A score is an fp32 sum of D exact
products: off by at most D 2^-24 sum|q k|, twice that where the tensor core
truncates, so |ds| <= 2^-16 A with A = scale * sum|q k| of the worst seen key;
the soft cap's tanh adds 2^-19 cap.  exp2 and the conversion to log2 units add
2^-20 relative, 2^-20 max(1, |lse|) to a logsumexp.
  LSE:      ds + 2^-20 max(1, |lse|)
  weights:  relative 2 ds + 2^-19
  O:        bf16 rounding 2^-8 |o|, plus (2^-10 + 2 ds) sum_j p_j max_d|v_jd|:
            a probability times its scale is held in fp16, half a step is 2^-11
            of it or, below 2^-14 of the row's largest, 2^-25 of that, which
            summed over up to 2^13 keys is at most 2^-11 of the sum
"""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

from helpers import ROOT, need_gpu
from oracle import kv4, masks

pytestmark = pytest.mark.gpu


def bsa_():
    need_gpu()
    import block_sparse_attention_process_gb300 as bsa
    return bsa


def host(t):
    return None if t is None else (t.float() if t.dtype == torch.bfloat16 else t).cpu().numpy()


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def rows(shape, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(shape, generator=g) * scale * torch.exp(0.5 * torch.randn(shape[-1], generator=g))
    return x.to(torch.bfloat16)


def filled(bsa, B, H, cap, D, seed, junk=True, k=None, v=None):
    """A cache with every slot written (by the oracle's packing) and the values it holds."""
    k = rows((B, H, cap, D), seed) if k is None else k
    v = rows((B, H, cap, D), seed + 1) if v is None else v
    out, val = [], []
    for name, x in (("k", k), ("v", v)):
        codes, s = kv4.quantise(x.double().numpy())
        out += [torch.from_numpy(kv4.pack(codes, name, np.arange(cap))).cuda(),
                torch.from_numpy(s).to(torch.bfloat16).cuda()]
        val.append(kv4.values(codes, s))
    g = torch.Generator().manual_seed(seed + 2)
    w = torch.rand((B, H, cap), generator=g).cuda()
    pos = torch.arange(cap, dtype=torch.int32).expand(B, H, cap).contiguous().cuda()
    return bsa.KV4Cache(*out, w, pos), val[0], val[1]


def poison(cache, lens):
    """Slots at and past the lengths get arbitrary codes and NaN scales."""
    for b, n in enumerate(lens):
        for c, s in ((cache.k_codes, cache.k_scales), (cache.v_codes, cache.v_scales)):
            c[b, :, n:] = 0x5A
            s[b, :, n:] = float("nan")


def within(name, got, want, tol):
    got, want = np.asarray(got, np.float64), np.asarray(want, np.float64)
    assert got.shape == want.shape, name
    assert np.array_equal(np.isfinite(got), np.isfinite(want)), f"{name}: non-finite pattern"
    f = np.isfinite(want)
    assert np.array_equal(got[~f & ~np.isnan(want)], want[~f & ~np.isnan(want)]) and np.array_equal(np.isnan(got), np.isnan(want)), name
    over = np.abs(got[f] - want[f]) - np.broadcast_to(tol, got.shape)[f]
    assert over.size == 0 or over.max() <= 0, f"{name}: {np.abs(got - want)[f].max():.3e}, over the tolerance by {over.max():.3e}"


def check_fwd(o, lse, dw, want, cap=0.0):
    wo, wl, ww, apv, aqk = want
    ds = 2.0 ** -16 * aqk + 2.0 ** -19 * (cap or 0.0)
    with np.errstate(invalid="ignore"):
        fin = np.where(np.isfinite(wl), np.abs(wl), 0)
    within("lse", host(lse), wl, ds + 2.0 ** -20 * np.maximum(1, fin))
    within("o", host(o), wo, 2.0 ** -8 * np.abs(wo) + (2.0 ** -10 + 2 * ds[..., None]) * apv)
    if dw is not None:
        # (fp32 addition to a weight of at most 1 rounds by 2^-24 of the sum)
        within("weights", dw, ww, ww * (2 * ds.max() + 2.0 ** -19) + 2.0 ** -23 * (1 + ww))


# ------------------------------------------------------------------ append

@pytest.mark.parametrize("B,H,T,D,cap", [(1, 1, 1, 64, 16), (1, 1, 1, 128, 16), (3, 2, 7, 128, 32), (2, 5, 130, 64, 256),
                                         (2, 3, 33, 128, 48)])
def test_append_is_bit_exact(B, H, T, D, cap):
    bsa = bsa_()
    k, v = rows((B, H, T, D), 1), rows((B, H, T, D), 2)
    k[0, 0, 0, :32] = 0                                       # a group of zeros
    v[-1, -1, -1, -32:] = 0
    k[0, -1, 0, 32:40] = torch.tensor([1, -1, 0.5, 0.25, 3, -7, 7, 3.5]) * 2.0 ** -120
    k[-1, 0, -1, 0] = 3e38
    cache = bsa.KV4Cache.empty(B, H, cap, D)
    for t in (cache.k_codes, cache.v_codes):
        t.fill_(0x77)
    cache.weights.fill_(5)
    start = [(cap - T) * (b + 1) // (B + 1) for b in range(B)]
    n_new = [max(0, T - 3 * b) for b in range(B)]
    w0 = torch.rand((B, H, T)).cuda()
    kv, vv = bsa.kv4_append(cache, k.cuda(), v.cuda(), i32(start), n_new=i32(n_new), positions=i32([100 + b for b in range(B)]),
                            weights=w0, values=True)
    assert bsa.get_device_error() == 0
    for name, x, codes, scales, vals in (("k", k, cache.k_codes, cache.k_scales, kv), ("v", v, cache.v_codes, cache.v_scales, vv)):
        c, s = kv4.quantise(x.double().numpy())
        got_c, got_s, val = host(codes), host(scales), host(vals)
        for b in range(B):
            n, at = n_new[b], start[b]
            assert np.array_equal(got_c[b, :, at:at + n], kv4.pack(c[b, :, :n], name, np.arange(at, at + n))), (name, b)
            assert np.array_equal(got_s[b, :, at:at + n], s[b, :, :n]), (name, b)
            assert np.array_equal(val[b, :, :n], kv4.bf16(kv4.values(c, s))[b, :, :n]) and (val[b, :, n:] == 0).all()
            assert (got_c[b, :, :at] == 0x77).all() and (got_c[b, :, at + n:] == 0x77).all()
            assert (got_s[b, :, :at] == 0).all() and (got_s[b, :, at + n:] == 0).all()
    w, pos = host(cache.weights), host(cache.positions)
    for b in range(B):
        n, at = n_new[b], start[b]
        assert np.array_equal(w[b, :, at:at + n], host(w0)[b, :, :n]) and (w[b, :, at + n:] == 5).all() and (w[b, :, :at] == 5).all()
        assert (pos[b, :, at:at + n] == 100 + b + np.arange(n)).all()


def test_append_of_infinities_and_nan():
    bsa = bsa_()
    k, v = rows((1, 1, 4, 64), 3), rows((1, 1, 4, 64), 4)
    k[0, 0, 0, 5], k[0, 0, 1, 40], v[0, 0, 2, 0], v[0, 0, 3, 63] = float("inf"), float("nan"), float("-inf"), float("nan")
    cache = bsa.KV4Cache.empty(1, 1, 16, 64)
    kv, vv = bsa.kv4_append(cache, k.cuda(), v.cuda(), i32([0]), values=True)
    for x, s, val in ((k, cache.k_scales, kv), (v, cache.v_scales, vv)):
        c, want = kv4.quantise(x.double().numpy())
        assert np.array_equal(host(s)[:, :, :4], want, equal_nan=True)
        assert np.array_equal(host(val), kv4.bf16(kv4.values(c, want)), equal_nan=True)


def test_append_takes_strided_rows_and_every_bf16_magnitude():
    bsa = bsa_()
    B, H, T, D = 2, 3, 5, 64
    wide = rows((B, T, 2 * H, D), 5).cuda()
    k, v = wide[:, :, :H].transpose(1, 2), wide[:, :, H:].transpose(1, 2)
    a, b = bsa.KV4Cache.empty(B, H, 16, D), bsa.KV4Cache.empty(B, H, 16, D)
    bsa.kv4_append(a, k, v, i32([3, 0]))
    bsa.kv4_append(b, k.contiguous(), v.contiguous(), i32([3, 0]))
    for n in ("k_codes", "k_scales", "v_codes", "v_scales", "weights", "positions"):
        assert torch.equal(getattr(a, n), getattr(b, n)), n
    assert (a.positions[0, :, 3:8].cpu() == torch.arange(3, 8)).all()
    # all finite bf16 values, ties among them: 65,280 values, 32 a group, sorted by magnitude and shuffled
    bits = torch.arange(1 << 16, dtype=torch.int32).to(torch.int16).view(torch.bfloat16)
    x = bits[torch.isfinite(bits.float())].double().numpy()
    for order in (np.argsort(np.abs(x), kind="stable"), np.random.default_rng(0).permutation(x.size)):
        y = torch.from_numpy(x[order]).to(torch.bfloat16).reshape(1, 1, -1, 64)
        n = y.shape[2]
        c = bsa.KV4Cache.empty(1, 1, (n + 15) // 16 * 16, 64)
        bsa.kv4_append(c, y.cuda(), y.cuda(), i32([0]))
        codes, s = kv4.quantise(y.double().numpy())
        assert np.array_equal(host(c.k_codes)[:, :, :n], kv4.pack(codes, "k", np.arange(n)))
        assert np.array_equal(host(c.v_codes)[:, :, :n], kv4.pack(codes, "v", np.arange(n)))
        assert np.array_equal(host(c.k_scales)[:, :, :n], s)


def test_append_outside_the_cache_is_dropped_and_reported():
    bsa = bsa_()
    k = rows((2, 1, 4, 64), 6).cuda()
    cache = bsa.KV4Cache.empty(2, 1, 16, 64)
    bsa.kv4_append(cache, k, k, i32([14, -2]))
    with pytest.raises(bsa.BsaError):
        bsa.get_device_error()
    assert bsa.get_device_error() == 0
    s = host(cache.k_scales)
    assert (s[0, 0, :14] == 0).all() and (s[0, 0, 14:] != 0).all()
    assert (s[1, 0, :2] != 0).all() and (s[1, 0, 2:] == 0).all()


# ------------------------------------------------------------------ attention

FWD = [
    # B, Hq, Hkv, T, D, capacity, lens, q_lens, cap, sinks
    (1, 1, 1, 1, 64, 16, [1], None, 0, None),
    (1, 2, 2, 1, 128, 16, [16], None, 0, None),
    (4, 4, 2, 1, 128, 160, [0, 1, 129, 160], None, 0, None),
    (4, 4, 2, 1, 64, 160, [0, 15, 17, 159], None, 0, None),
    (3, 8, 1, 1, 128, 272, [127, 128, 257], None, 0, None),
    (2, 6, 2, 3, 128, 144, [3, 140], None, 0, None),
    (3, 6, 2, 3, 64, 144, [2, 0, 137], None, 0, None),              # more new tokens than keys
    (3, 4, 4, 4, 128, 144, [50, 1, 144], [4, 1, 0], 0, None),       # padded queries
    (2, 16, 1, 4, 128, 400, [399, 255], None, 30.0, (1, 4)),
    (2, 9, 3, 1, 64, 208, [200, 3], None, 1.5, (2,)),
    (2, 4, 4, 2, 128, 64, [0, 1], None, 0, (4, 3)),                 # rows with the sinks alone
    (1, 40, 1, 1, 128, 144, [130], None, 0, None),                  # a large group
    (2, 10, 2, 7, 64, 208, [205, 100], None, 0, None),              # 35 rows a key head
    (1, 8, 2, 1, 128, 2064, [2049], None, 0, None),
    (1, 32, 8, 1, 128, 1040, [1033], None, 0, None),
    (8, 2, 1, 1, 64, 1104, [1101, 3, 700, 64, 0, 999, 128, 1], None, 0, None),
]


@pytest.mark.parametrize("case", FWD, ids=lambda c: f"b{c[0]}h{c[1]}-{c[2]}t{c[3]}d{c[4]}n{max(c[6])}")
def test_fwd_matches_oracle(case):
    bsa = bsa_()
    B, Hq, Hkv, T, D, cap, lens, q_lens, softcap, sink_shape = case
    cache, kv, vv = filled(bsa, B, Hkv, cap, D, 10)
    poison(cache, lens)
    q = rows((B, Hq, T, D), 13, 1.5)
    sinks = None if sink_shape is None else np.random.default_rng(5).standard_normal(
        (Hkv, sink_shape[1]) if len(sink_shape) == 2 else sink_shape).astype(np.float32)
    sd = None if sinks is None else torch.from_numpy(sinks).cuda()
    want = kv4.forward(q.double().numpy(), kv, vv, lens, q_lens, cap=softcap, sinks=sinks)
    for accumulate in (False, True):
        before = cache.weights.clone()
        o, lse = bsa.kv4_fwd(q.cuda(), cache, i32(lens), q_lens=None if q_lens is None else i32(q_lens),
                             logits_soft_cap=softcap or None, sinks=sd, accumulate=accumulate)
        assert bsa.get_device_error() == 0
        dw = cache.weights.double().cpu().numpy() - before.double().cpu().numpy()
        if not accumulate:
            assert (dw == 0).all()
        else:
            for b, n in enumerate(lens):
                assert (dw[b, :, n:] == 0).all()
        check_fwd(o, lse, dw if accumulate else None, want, softcap)


def test_fwd_repeats_bit_for_bit_and_takes_strides():
    bsa = bsa_()
    B, Hq, Hkv, T, D = 3, 8, 2, 2, 128
    cache, _, _ = filled(bsa, B, Hkv, 528, D, 20)
    lens = i32([528, 77, 300])
    base = rows((B, T, Hq, D), 21).cuda()
    q = base.transpose(1, 2)
    w0 = cache.weights.clone()
    o, lse = bsa.kv4_fwd(q, cache, lens, accumulate=True)
    w1 = cache.weights.clone()
    out = torch.full((B, T, Hq, D), float("nan"), dtype=torch.bfloat16, device="cuda").transpose(1, 2)
    for _ in range(3):
        cache.weights.copy_(w0)
        o2, lse2 = bsa.kv4_fwd(q.contiguous(), cache, lens, o=out, accumulate=True)
        assert o2 is out and torch.equal(o2, o) and torch.equal(lse2, lse) and torch.equal(cache.weights, w1)


def test_fwd_with_far_apart_magnitudes():
    """Values of very different size with weights the other way round, large scores, an explicit scale."""
    bsa = bsa_()
    B, H, n, D = 1, 2, 64, 64
    k, v = rows((B, H, n, D), 30), rows((B, H, n, D), 31)
    q = rows((B, H, 1, D), 32)
    k[0, 0, 7] = (q[0, 0, 0].float() * 8).to(torch.bfloat16)      # one key far ahead of the others ...
    v[0, 0, 7] = (v[0, 0, 7].float() * 2.0 ** -30).to(torch.bfloat16)   # ... of tiny values
    v[0, 0, 9] = (v[0, 0, 9].float() * 2.0 ** 20).to(torch.bfloat16)
    v[0, 1, 3] = (v[0, 1, 3].float() * 2.0 ** 100).to(torch.bfloat16)   # huge, of weight ~2^-100
    k[0, 1, 3] = (q[0, 1, 0].float() * -16).to(torch.bfloat16)
    cache, kv, vv = filled(bsa, B, H, n, D, 33, k=k, v=v)
    o, lse = bsa.kv4_fwd(q.cuda(), cache, i32([n]), softmax_scale=0.25)
    check_fwd(o, lse, None, kv4.forward(q.double().numpy(), kv, vv, [n], scale=0.25))
    for factor in (2.0 ** -100, 2.0 ** 60):                         # queries of any size
        q2 = (q.float() * factor).to(torch.bfloat16)
        o, lse = bsa.kv4_fwd(q2.cuda(), cache, i32([n]), softmax_scale=0.25 / factor)
        check_fwd(o, lse, None, kv4.forward(q2.double().numpy(), kv, vv, [n], scale=0.25 / factor))


def test_fwd_nan_stays_with_its_head():
    bsa = bsa_()
    B, H, n, D = 2, 2, 80, 128
    k, v = rows((B, H, n, D), 40), rows((B, H, n, D), 41)
    v[0, 1, 11, 3] = float("nan")        # visible to (0, 1) alone
    k[1, 0, 60, 0] = float("inf")        # behind sequence 1's length
    cache, kv, vv = filled(bsa, B, H, n, D, 42, k=k, v=v)
    q = rows((B, 4, 1, D), 43)
    o, lse = bsa.kv4_fwd(q.cuda(), cache, i32([n, 60]))
    with np.errstate(invalid="ignore"):
        want = kv4.forward(q.double().numpy(), np.nan_to_num(kv), np.nan_to_num(vv), [n, 60])
    o, lse = host(o), host(lse)
    assert np.isnan(o[0, 2:, :, :32]).all() and np.isfinite(o[0, 2:, :, 32:]).all()   # NaN in its group alone
    assert np.isfinite(o[0, :2]).all() and np.isfinite(o[1]).all() and np.isfinite(lse).all()
    within("o", o[1], want[0][1], 2.0 ** -8 * np.abs(want[0][1]) + 2.0 ** -9 * want[3][1])


def test_fwd_lengths_outside_the_cache_are_clamped_and_reported():
    bsa = bsa_()
    cache, kv, vv = filled(bsa, 2, 1, 32, 64, 50)
    q = rows((2, 1, 1, 64), 51)
    o, lse = bsa.kv4_fwd(q.cuda(), cache, i32([1000, -5]))
    with pytest.raises(bsa.BsaError):
        bsa.get_device_error()
    check_fwd(o, lse, None, kv4.forward(q.double().numpy(), kv, vv, [32, 0]))


def test_append_and_fwd_in_a_replayed_graph_and_on_another_stream():
    bsa = bsa_()
    B, Hq, Hkv, D, cap = 2, 4, 2, 128, 320
    cache, _, _ = filled(bsa, B, Hkv, cap, D, 60)
    lens = i32([0, 0])
    q, k, v = (torch.zeros((B, h, 1, D), dtype=torch.bfloat16, device="cuda") for h in (Hq, Hkv, Hkv))

    def step():
        bsa.kv4_append(cache, k, v, lens)
        return bsa.kv4_fwd(q, cache, lens + 1, accumulate=True)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, lse = step()
    side = torch.cuda.Stream()
    for i, ls in enumerate(([5, 300], [0, 1], [319, 128])):
        lens.copy_(i32(ls))
        for t, s in ((q, 61), (k, 62), (v, 63)):
            t.copy_(rows(t.shape, s + 10 * i))
        w0 = cache.weights.clone()
        graph.replay()
        got = o.clone(), lse.clone(), cache.weights.clone()
        cache.weights.copy_(w0)
        side.wait_stream(torch.cuda.current_stream())
        bsa.kv4_append(cache, k, v, lens, stream=side)
        lens1 = lens + 1
        side.wait_stream(torch.cuda.current_stream())
        o2, lse2 = bsa.kv4_fwd(q, cache, lens1, accumulate=True, stream=side)
        torch.cuda.current_stream().wait_stream(side)
        assert torch.equal(o2, got[0]) and torch.equal(lse2, got[1]) and torch.equal(cache.weights, got[2])
    assert bsa.get_device_error() == 0


# ------------------------------------------------------------------ eviction

EVICT = [
    # B, H, D, capacity, lens, keep, recent
    (1, 1, 64, 16, [1], 1, 0),
    (1, 2, 128, 16, [16], 1, 1),
    (2, 3, 128, 208, [200, 130], 128, 16),
    (3, 2, 64, 48, [48, 20, 0], 20, 7),
    (2, 1, 128, 1104, [1100, 1025], 1024, 0),
    (2, 2, 128, 3088, [3085, 2000], 700, 128),
    (1, 1, 64, 20016, [20011], 5000, 40),
]


@pytest.mark.parametrize("in_place", [False, True], ids=["into", "in-place"])
@pytest.mark.parametrize("weights", ["random", "ties", "odd"])
@pytest.mark.parametrize("case", EVICT, ids=lambda c: f"n{max(c[4])}k{c[5]}")
def test_evict_is_exact(case, weights, in_place):
    bsa = bsa_()
    B, H, D, cap, lens, keep, recent = case
    rng = np.random.default_rng(7)
    codes = [torch.from_numpy(rng.integers(0, 256, (B, H, cap, D // 2)).astype(np.uint8)).cuda() for _ in "kv"]
    scales = [torch.from_numpy(rng.standard_normal((B, H, cap, D // 32)).astype(np.float32)).to(torch.bfloat16).cuda() for _ in "kv"]
    w = rng.random((B, H, cap)).astype(np.float32) ** 4
    if weights == "ties":
        w = rng.integers(0, 3, (B, H, cap)).astype(np.float32)
    if weights == "odd":
        w = np.where(rng.random(w.shape) < 0.1, np.float32(-0.0), w)
        w = np.where(rng.random(w.shape) < 0.1, np.float32(np.nan), w)
        w = np.where(rng.random(w.shape) < 0.1, np.float32(np.inf), w)
        w = np.where(rng.random(w.shape) < 0.1, -w, w)
    pos = np.stack([[rng.permutation(cap) for _ in range(H)] for _ in range(B)]).astype(np.int32)
    cache = bsa.KV4Cache(codes[0], scales[0], codes[1], scales[1], torch.from_numpy(w).cuda(), torch.from_numpy(pos).cuda())
    seen = [cap + 3] * B
    want, new = kv4.evict(w, pos, lens, keep, recent, seen, in_place)
    src = {n: host(getattr(cache, n)).copy() for n in ("k_codes", "k_scales", "v_codes", "v_scales", "weights", "positions")}
    src["k_val"] = kv4.values(kv4.unpack(src["k_codes"], "k"), src["k_scales"])
    src["v_val"] = kv4.values(kv4.unpack(src["v_codes"], "v"), src["v_scales"])
    out = None
    if not in_place:
        out = bsa.KV4Cache.empty(B, H, (keep + 31) // 16 * 16, D)
        out.weights.fill_(9)
    new_lens, index, kv, vv = bsa.kv4_evict(cache, i32(lens), keep, recent=recent, seen=i32(seen), out=out, values=True)
    assert bsa.get_device_error() == 0
    assert np.array_equal(host(new_lens), new) and np.array_equal(host(index), want)
    dst = cache if in_place else out
    got = {n: host(getattr(dst, n)) for n in ("k_codes", "k_scales", "v_codes", "v_scales", "weights", "positions")}
    got["k_val"] = kv4.values(kv4.unpack(got["k_codes"], "k"), got["k_scales"])
    got["v_val"] = kv4.values(kv4.unpack(got["v_codes"], "v"), got["v_scales"])
    for b in range(B):
        n = int(new[b])
        for h in range(H):
            i = want[b, h, :n]
            for name in ("k_val", "v_val", "weights", "positions", "k_scales", "v_scales"):
                assert np.array_equal(got[name][b, h, :n], src[name][b, h, i], equal_nan=True), name
            for vals, name in ((kv, "k_val"), (vv, "v_val")):
                assert np.array_equal(host(vals)[b, h, :n], kv4.bf16(src[name][b, h, i])) and (host(vals)[b, h, n:] == 0).all()
        if not in_place:
            assert (got["weights"][b, :, n:] == 9).all() and (got["k_codes"][b, :, n:] == 0).all()


def test_evict_without_positions_and_without_values():
    bsa = bsa_()
    c, _, _ = filled(bsa, 2, 2, 64, 64, 80)
    plain = bsa.KV4Cache(c.k_codes, c.k_scales, c.v_codes, c.v_scales, c.weights)
    out = bsa.KV4Cache.empty(2, 2, 32, 64)
    new_lens, index = bsa.kv4_evict(plain, i32([64, 30]), 32, recent=5, out=out)
    want, new = kv4.evict(host(c.weights), None, [64, 30], 32, 5)
    assert np.array_equal(host(index), want) and np.array_equal(host(new_lens), new)
    assert np.array_equal(host(out.positions)[0], want[0])
    bsa.kv4_evict(plain, i32([200, -1]), 32, out=out)
    with pytest.raises(bsa.BsaError):
        bsa.get_device_error()


# ------------------------------------------------------------------ key weights

KEYS = [
    # B, Hq, Hkv, S_q, S_kv, D, mask, kwargs, q_lens, cap
    (1, 1, 1, 128, 128, 64, "causal", {}, None, 0),
    (1, 2, 2, 512, 512, 64, "causal", {}, None, 0),
    (2, 4, 2, 640, 640, 128, "causal", {}, [640, 333], 0),
    (1, 6, 2, 384, 384, 128, "full", {}, [1], 0),
    (2, 2, 1, 768, 768, 64, "local", {"local_left": 200, "local_right": 0}, [0, 768], 0),
    (1, 3, 3, 512, 512, 128, "local", {"local_left": 40, "local_right": 70}, None, 20.0),
    (1, 8, 1, 1024, 1024, 128, "chunked", {"chunk": 300}, [1000], 0),
    (1, 4, 2, 256, 512, 128, "dense", {}, None, 0),
    (2, 2, 2, 512, 256, 64, "dense", {}, [511, 130], 2.0),
    (1, 4, 2, 384, 384, 64, "perhead", {}, None, 0),
    (1, 20, 1, 256, 256, 64, "causal", {}, None, 0),
]


@pytest.mark.parametrize("case", KEYS, ids=lambda c: f"{c[6]}-b{c[0]}h{c[1]}-{c[2]}s{c[3]}-{c[4]}d{c[5]}")
def test_key_weights_match_oracle(case):
    bsa = bsa_()
    B, Hq, Hkv, Sq, Skv, D, kind, kw, q_lens, cap = case
    q, k = rows((B, Hq, Sq, D), 90), rows((B, Hkv, Skv, D), 91)
    rng = np.random.default_rng(92)
    heads = Hq if kind == "perhead" else 1
    if kind in ("dense", "perhead"):
        dense = (rng.random((heads, Sq, Skv)) < 0.3).astype(np.uint8)
        dense[:, 5] = 0                                                 # a row that sees nothing
        dense[:, :128, 128:256] = 0                                     # an empty and a full block
        dense[:, 128:256, :128] = 1
        dkv = bsa.mask_compile("dense", Sq, Skv, dense=torch.from_numpy(dense).cuda(), orientation="dkv")
        allowed = dense != 0
    else:
        dkv = bsa.mask_compile(kind, Sq, Skv, orientation="dkv", **kw)
        allowed = masks.materialise(kind, Sq, Skv, left=kw.get("local_left"), right=kw.get("local_right"), chunk=kw.get("chunk"))[None]
    qd, kd = q.double().numpy(), k.double().numpy()
    lse = np.full((B, Hq, Sq), -np.inf, np.float32)
    want, amax, top = np.zeros((B, Hkv, Skv)), 0.0, 1.0
    for b in range(B):
        n = Sq if q_lens is None else q_lens[b]
        for h in range(Hq):
            g = h // (Hq // Hkv)
            s = qd[b, h] @ kd[b, g].T * D ** -0.5
            amax = max(amax, (np.abs(qd[b, h]) @ np.abs(kd[b, g]).T).max() * D ** -0.5)
            if cap:
                s = cap * np.tanh(s / cap)
            s = np.where(allowed[h if heads > 1 else 0], s, -np.inf)
            some = np.isfinite(s).any(-1)
            m = np.where(some, s.max(-1), 0)
            with np.errstate(divide="ignore"):
                lse[b, h] = np.where(some, m + np.log(np.exp(s - m[:, None]).sum(-1)), -np.inf)
            p = np.exp(s - np.where(some, lse[b, h].astype(np.float64), 0)[:, None])
            want[b, g] += p[:n].sum(0)
            top = max(top, np.abs(lse[b, h][some]).max())
    args = (q.cuda(), k.cuda(), torch.from_numpy(lse).cuda(), dkv)
    kwargs = dict(q_lens=None if q_lens is None else i32(q_lens), logits_soft_cap=cap or None)
    got = bsa.key_weights(*args, **kwargs)
    assert bsa.get_device_error() == 0
    ds = 2.0 ** -16 * amax + 2.0 ** -19 * cap + 2.0 ** -23 * top
    # (the sum of up to Sq G positive terms: 2^-24 a step, far fewer steps in a row than 2^5)
    within("key weights", host(got), want, want * (2 * ds + 2.0 ** -18) + 1e-30)
    assert torch.equal(bsa.key_weights(*args, **kwargs), got)


def test_key_weights_of_fwd_sum_to_the_number_of_queries():
    bsa = bsa_()
    B, Hq, Hkv, S, D = 1, 8, 2, 2048, 128
    q, k = rows((B, Hq, S, D), 95).cuda(), rows((B, Hkv, S, D), 96).cuda()
    info, dkv = bsa.mask_compile("causal", S, S), bsa.mask_compile("causal", S, S, orientation="dkv")
    _, lse = bsa.fwd(q, k, k, info)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    w = bsa.key_weights(q, k, lse, dkv, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    total = w.double().sum(-1).cpu().numpy()
    # every query's probabilities sum to 1 up to the errors of its logsumexp (1e-5) and of the scores
    assert np.abs(total / (Hq // Hkv * S) - 1).max() < 2e-4


@pytest.mark.parametrize("D,cap", [(64, 0), (128, 0), (128, 10.0)])
def test_key_weights_keep_nan_and_infinities_where_they_are(D, cap):
    """Padded queries of NaN change nothing; a NaN query reaches the keys it sees, an infinite key itself alone."""
    bsa = bsa_()
    S, n = 384, 300
    q, k = rows((1, 4, S, D), 97).cuda(), rows((1, 2, S, D), 98).cuda()
    info, dkv = bsa.mask_compile("causal", S, S), bsa.mask_compile("causal", S, S, orientation="dkv")
    _, lse = bsa.fwd(q, k, k, info, logits_soft_cap=cap or None)
    weights = lambda q, k, lse: bsa.key_weights(q, k, lse, dkv, q_lens=i32([n]), logits_soft_cap=cap or None)
    clean = weights(q, k, lse)
    assert torch.isfinite(clean).all() and (clean[:, :, n:] == 0).all()
    q, lse = q.clone(), lse.clone()
    q[:, :, n:] = float("nan")
    lse[:, :, n:] = float("nan")
    lse[:, :, -1] = float("inf")
    assert torch.equal(weights(q, k, lse), clean)
    q[0, 1, 131] = float("nan")             # (of the first key head's group)
    lse[0, 1, 131] = float("nan")
    got = weights(q, k, lse)
    assert torch.isnan(got[0, 0, :132]).all() and torch.equal(got[0, 0, 132:], clean[0, 0, 132:]) and torch.equal(got[0, 1], clean[0, 1])
    k = k.clone()
    k[0, 1, 70, 3] = float("inf")
    got = weights(q, k, lse)
    keep = torch.arange(S, device="cuda") != 70
    assert not torch.equal(got[0, 1], clean[0, 1]) and torch.equal(got[0, 1, keep], clean[0, 1, keep])
    assert bsa.get_device_error() == 0


@pytest.mark.parametrize("scale", [0.0, 1e-30, -0.0, -0.07, 3.0])
def test_key_weights_of_any_scale(scale):
    bsa = bsa_()
    S, D = 256, 64
    q, k = rows((1, 2, S, D), 99), rows((1, 1, S, D), 100)
    s = np.where(np.tril(np.ones((S, S), bool)), scale * np.einsum("hid,jd->hij", q.double().numpy()[0], k.double().numpy()[0, 0]), -np.inf)
    lse = np.log(np.exp(s - s.max(-1, keepdims=True)).sum(-1)) + s.max(-1)
    l32 = lse.astype(np.float32)
    want = np.exp(s - l32[..., None].astype(np.float64)).sum((0, 1))
    dkv = bsa.mask_compile("causal", S, S, orientation="dkv")
    got = bsa.key_weights(q.cuda(), k.cuda(), torch.from_numpy(l32[None]).cuda(), dkv, softmax_scale=scale)
    assert bsa.get_device_error() == 0
    amax = abs(scale) * np.einsum("hid,jd->hij", np.abs(q.double().numpy()[0]), np.abs(k.double().numpy()[0, 0])).max()
    ds = 2.0 ** -16 * amax + 2.0 ** -23 * max(1.0, np.abs(lse).max())
    within("key weights", host(got)[0, 0], want, want * (2 * ds + 2.0 ** -18) + 1e-30)


# ------------------------------------------------------------------ together

def test_prompt_append_decode_evict_together():
    """A padded batch of prompts, its keys' weights, the cache, and 40 tokens with an eviction whenever the budget
    is exceeded.  The oracle follows with its own attention on the values the cache holds; what the library
    evicts must be what the oracle evicts given the library's accumulated weights."""
    bsa = bsa_()
    B, Hq, Hkv, D, S = 2, 4, 2, 64, 256
    prompt, keep, recent, cap = [256, 150], 176, 32, 272
    q, k, v = rows((B, Hq, S, D), 100), rows((B, Hkv, S, D), 101), rows((B, Hkv, S, D), 102)
    info, dkv = bsa.mask_compile("causal", S, S), bsa.mask_compile("causal", S, S, orientation="dkv")
    _, lse = bsa.fwd(q.cuda(), k.cuda(), v.cuda(), info)
    w = bsa.key_weights(q.cuda(), k.cuda(), lse, dkv, q_lens=i32(prompt))
    cache = bsa.KV4Cache.empty(B, Hkv, cap, D)
    bsa.kv4_append(cache, k.cuda(), v.cuda(), i32([0, 0]), n_new=i32(prompt), weights=w)

    def held():
        return [kv4.values(kv4.unpack(host(c), n), host(s)) for n, c, s in
                (("k", cache.k_codes, cache.k_scales), ("v", cache.v_codes, cache.v_scales))]

    lens, seen = i32(prompt), i32(prompt)
    for step in range(40):
        n_before = host(lens).copy()
        if (n_before > keep).any() and step % 4 == 0:
            w0, p0 = host(cache.weights).copy(), host(cache.positions).copy()
            want, new = kv4.evict(w0, p0, n_before, keep, recent, host(seen), in_place=True)
            lens, index = bsa.kv4_evict(cache, lens, keep, recent=recent, seen=seen)
            assert np.array_equal(host(index), want) and np.array_equal(host(lens), new)
            pos = host(cache.positions)
            for b in range(B):          # the last `recent` positions are still there
                for h in range(Hkv):
                    have = set(pos[b, h, :new[b]].tolist())
                    assert have >= set(range(int(host(seen)[b]) - recent, int(host(seen)[b]))) and len(have) == new[b]
        q1, k1, v1 = (rows((B, h, 1, D), 110 + 3 * step + i) for i, h in enumerate((Hq, Hkv, Hkv)))
        bsa.kv4_append(cache, k1.cuda(), v1.cuda(), lens, positions=seen)
        lens, seen = lens + 1, seen + 1
        w0 = cache.weights.double().cpu().numpy()
        o, l = bsa.kv4_fwd(q1.cuda(), cache, lens, accumulate=True)
        kk, vv = held()
        dw = cache.weights.double().cpu().numpy() - w0
        wo, wl, ww, apv, aqk = kv4.forward(q1.double().numpy(), kk, vv, host(lens))
        ds = 2.0 ** -16 * aqk
        within("lse", host(l), wl, ds + 2.0 ** -20 * np.maximum(1, np.abs(wl)))
        within("o", host(o), wo, 2.0 ** -8 * np.abs(wo) + (2.0 ** -10 + 2 * ds[..., None]) * apv)
        within("weights", dw, ww, ww * (2 * ds.max() + 2.0 ** -19) + 2.0 ** -23 * (np.abs(w0) + 1))
    assert bsa.get_device_error() == 0
    assert (host(lens) <= keep + 4).all()


# ------------------------------------------------------------------ work split over many sequences, long axes, streams, graphs

@pytest.mark.parametrize("B,Hq,Hkv,T,D,cap", [(70, 4, 2, 2, 64, 1040), (5, 3, 1, 5, 128, 4112), (24, 8, 8, 1, 128, 1024)])
def test_fwd_of_many_unequal_sequences(B, Hq, Hkv, T, D, cap):
    """Runs that hold parts of several pairs, sequences without keys or new tokens between them, pairs of more than
    eight rows, a capacity on either side of the one that a CTA takes alone."""
    bsa = bsa_()
    rng = np.random.default_rng(90)
    lens = rng.integers(0, cap + 1, B)
    lens[:5] = [cap, 0, 1, 129, 128]
    q_lens = rng.integers(0, T + 1, B)
    q_lens[0] = T
    cache, kv, vv = filled(bsa, B, Hkv, cap, D, 91)
    poison(cache, lens)
    cache.weights.zero_()
    q = rows((B, Hq, T, D), 92)
    sinks = rng.standard_normal((Hkv, 2)).astype(np.float32)
    want = kv4.forward(q.double().numpy(), kv, vv, lens, q_lens, sinks=sinks)
    o, lse = bsa.kv4_fwd(q.cuda(), cache, i32(lens), q_lens=i32(q_lens), sinks=torch.from_numpy(sinks).cuda(), accumulate=True)
    assert bsa.get_device_error() == 0
    check_fwd(o, lse, cache.weights.double().cpu().numpy(), want)


@pytest.mark.parametrize("exponent,spread,zeros", [(0, 40, 0), (0, 0, 700), (-120, 0, 0), (-120, 0, 2000), (80, 30, 33), (118, 0, 1)])
def test_fwd_joins_parts_of_far_apart_magnitudes(exponent, spread, zeros):
    """Values of any size, keys of very different ones, the first keys' (whole parts of them) all 0."""
    bsa = bsa_()
    n, D = 2050, 64
    k, v = rows((1, 1, n, D), 95), rows((1, 1, n, D), 96)
    e = exponent + np.random.default_rng(3).integers(-spread, spread + 1, (1, 1, n, 1))
    v = torch.ldexp(v.double(), torch.from_numpy(e)).to(torch.bfloat16)
    v[:, :, :zeros] = 0
    if spread:
        v[:, :, 300:700] *= 2.0 ** -20                  # whole parts of small values
    pad = torch.zeros((1, 1, 2064 - n, D), dtype=torch.bfloat16)
    cache, kv, vv = filled(bsa, 1, 1, 2064, D, 97, k=torch.cat((k, pad), 2), v=torch.cat((v, pad), 2))
    q = rows((1, 3, 1, D), 98)
    o, lse = bsa.kv4_fwd(q.cuda(), cache, i32([n]))
    check_fwd(o, lse, None, kv4.forward(q.double().numpy(), kv, vv, [n]))


@pytest.mark.parametrize("n", [100, 1100])
def test_fwd_key_without_values_takes_nearly_all_the_weight(n):
    bsa = bsa_()
    D, cap = 128, (n + 15) // 16 * 16
    k, v, q = rows((1, 1, cap, D), 103), rows((1, 1, cap, D), 104), rows((1, 2, 1, D), 105)
    k[0, 0, 0] = (q[0, 0, 0].float() * 2.0).to(torch.bfloat16)      # far ahead for the first row
    v[0, 0, 0] = 0
    cache, kv, vv = filled(bsa, 1, 1, cap, D, 106, k=k, v=v)
    want = kv4.forward(q.double().numpy(), kv, vv, [n])
    assert np.abs(want[0][0, 0]).max() < 2.0 ** -12 < np.abs(want[0][0, 1]).max()
    check_fwd(*bsa.kv4_fwd(q.cuda(), cache, i32([n])), None, want)


def test_fwd_sinks_of_minus_infinity():
    bsa = bsa_()
    cache, kv, vv = filled(bsa, 2, 2, 32, 64, 100)
    q = rows((2, 4, 1, 64), 101)
    lens = i32([0, 20])
    o, lse = bsa.kv4_fwd(q.cuda(), cache, lens, sinks=torch.full((3,), -float("inf"), device="cuda"))
    o2, lse2 = bsa.kv4_fwd(q.cuda(), cache, lens)
    assert (host(lse)[0] == -np.inf).all() and (host(o)[0] == 0).all()
    check_fwd(o, lse, None, kv4.forward(q.double().numpy(), kv, vv, [0, 20]))
    check_fwd(o2, lse2, None, kv4.forward(q.double().numpy(), kv, vv, [0, 20]))


def test_long_cache_past_32_bit_offsets():
    """2 heads of 20,000,000 slots (codes of 2.6 GB): three tokens of known scores at far slots among zeros, whose
    scores are 0; their weights from append, attention and eviction."""
    bsa = bsa_()
    if torch.cuda.mem_get_info()[0] < 12 << 30:
        pytest.skip("needs 12 GB")
    cap, D, H = 20_000_000, 128, 2
    cache = bsa.KV4Cache.empty(1, H, cap, D)
    at = [3, 12_345_678, cap - 1]
    k, v = rows((1, H, 3, D), 110), rows((1, H, 3, D), 111)
    q = rows((1, H, 1, D), 112)
    vals = []
    for i, slot in enumerate(at):
        vals.append([host(x)[0, :, 0].astype(np.float64) for x in
                     bsa.kv4_append(cache, k[:, :, i:i + 1].cuda(), v[:, :, i:i + 1].cuda(), i32([slot]), values=True)])
    # (values are rounded once more to bf16; the cache's own come from its codes, whose order depends on the slot mod 4)
    def held(name, codes, scales):
        return np.stack([kv4.values(kv4.unpack(np.repeat(host(codes[0, :, i:i + 1]), 4, 1), name)[:, i % 4], host(scales[0, :, i]))
                         for i in at], 1)
    idx = torch.tensor(at, device="cuda")
    kv, vv = held("k", cache.k_codes, cache.k_scales), held("v", cache.v_codes, cache.v_scales)
    for i in range(3):
        assert np.array_equal(vals[i][0], kv4.bf16(kv[:, i])) and np.array_equal(vals[i][1], kv4.bf16(vv[:, i]))
    qd = q.double().numpy()[0, :, 0]
    s = np.einsum("hd,hkd->hk", qd, kv)
    scale = 18.0 / np.abs(s).max()
    s, aqk = s * scale, scale * np.einsum("hd,hkd->hk", np.abs(qd), np.abs(kv)).max(1)
    zeros = cap - 3
    tot = zeros + np.exp(s).sum(1)
    p = np.exp(s) / tot[:, None]
    o, lse = bsa.kv4_fwd(q.cuda(), cache, i32([cap]), softmax_scale=float(scale), accumulate=True)
    assert bsa.get_device_error() == 0
    # l is a fp32 sum over 456 runs of up to 88,000 equal terms, four warps of 8 lanes each: a lane adds at most 2^12
    # times four, off by at most 2^-24 of the sum each time, 2^-12 in all
    ds = 2.0 ** -16 * aqk + 2.0 ** -12
    assert (np.abs(host(lse)[0, :, 0] - np.log(tot)) <= ds + 2.0 ** -20 * np.log(tot)).all()
    wo, apv = np.einsum("hk,hkd->hd", p, vv), (p * np.abs(vv).max(2)).sum(1)
    assert (np.abs(host(o)[0, :, 0] - wo) <= 2.0 ** -8 * np.abs(wo) + ((2.0 ** -10 + 2 * ds) * apv)[:, None]).all()
    w = cache.weights[0][:, idx].double().cpu().numpy()
    assert (np.abs(w - p) <= p * (2 * ds + 2.0 ** -19)[:, None]).all()
    low = cache.weights[0, :, 100].double().cpu().numpy()
    assert (np.abs(low * tot - 1) <= 2 * ds + 2.0 ** -19).all()
    keep = 4
    cache.weights[:] = 0
    cache.weights[0, 1, at[1]] = 2
    cache.weights[0, 1, at[2]] = 1
    out = bsa.KV4Cache.empty(1, H, 16, D)
    new_lens, index, kk, _ = bsa.kv4_evict(cache, i32([cap]), keep, out=out, values=True)
    assert bsa.get_device_error() == 0
    assert host(new_lens).tolist() == [keep] and host(index)[0].tolist() == [[0, 1, 2, 3], [0, 1, at[1], at[2]]]
    assert np.array_equal(host(kk)[0, 1, 2:], kv4.bf16(kv[1, 1:])) and np.array_equal(host(kk)[0, 0, 3], kv4.bf16(kv[0, 0]))


def test_more_heads_than_a_grid_has_rows():
    bsa = bsa_()
    B, H, cap, D, keep = 33_000, 2, 16, 64, 5
    cache = bsa.KV4Cache.empty(B, H, cap, D)
    g = torch.Generator(device="cuda").manual_seed(1)
    k = torch.randn((B, H, cap, D), generator=g, device="cuda").to(torch.bfloat16)
    w = torch.rand((B, H, cap), generator=g, device="cuda")
    start, lens = torch.zeros(B, dtype=torch.int32, device="cuda"), torch.full((B,), cap, dtype=torch.int32, device="cuda")
    kv, _ = bsa.kv4_append(cache, k, k, start, weights=w, values=True)
    new_lens, index, kk, vv = bsa.kv4_evict(cache, lens, keep, values=True)
    order = torch.sort(w, dim=-1, descending=True, stable=True).indices[..., :keep]
    assert torch.equal(torch.sort(index, dim=-1).values.long(), torch.sort(order, dim=-1).values)
    assert torch.equal(kk, torch.gather(kv, 2, index.long()[..., None].expand(-1, -1, -1, D))) and torch.equal(kk, vv)
    q = torch.randn((B, H, 1, D), generator=g, device="cuda").to(torch.bfloat16)
    o, lse = bsa.kv4_fwd(q, cache, new_lens)
    assert bsa.get_device_error() == 0
    pick = torch.tensor([0, 1, 16_383, 32_767, 32_999], device="cuda")
    sub = kv4.forward(q[pick].double().cpu().numpy(), *(kv4.values(kv4.unpack(host(c[pick]), n), host(s[pick])) for n, c, s in (
        ("k", cache.k_codes, cache.k_scales), ("v", cache.v_codes, cache.v_scales))), [keep] * 5)
    check_fwd(o[pick], lse[pick], None, sub)


def test_eviction_and_key_weights_in_a_replayed_graph():
    bsa = bsa_()
    B, H, cap, D, keep, S = 2, 2, 208, 64, 100, 256
    info = bsa.mask_compile("causal", S, S)
    dkv = bsa.mask_compile("causal", S, S, orientation="dkv")
    base, _, _ = filled(bsa, B, H, cap, D, 120)
    names = ("k_codes", "k_scales", "v_codes", "v_scales", "weights", "positions")
    clone = lambda c: bsa.KV4Cache(*(getattr(c, n).clone() for n in names))
    a, b = clone(base), bsa.KV4Cache.empty(B, H, 112, D)
    lens = i32([cap, 150])
    q, k, v = (torch.zeros((1, h, S, D), dtype=torch.bfloat16, device="cuda") for h in (4, 2, 2))

    lse = torch.zeros((1, 4, S), device="cuda")      # (the forward itself is not captured: it uploads its schedule)

    def step(a, b):
        w = bsa.key_weights(q, k, lse, dkv)
        into = bsa.kv4_evict(a, lens, keep, recent=8, out=b)
        return (w, *into, *bsa.kv4_evict(a, lens, keep, recent=8, values=True))

    step(clone(a), b)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(a, b)
    for i, ls in enumerate(([208, 101], [100, 0], [7, 208])):
        lens.copy_(i32(ls))
        for t, s in ((q, 121), (k, 122), (v, 123)):
            t.copy_(rows(t.shape, s + 10 * i))
        lse.copy_(bsa.fwd(q, k, v, info)[1])
        for n in names:
            getattr(a, n).copy_(getattr(base, n))
        a.weights.copy_(torch.rand(a.weights.shape, generator=torch.Generator().manual_seed(i)))
        a2, b2 = clone(a), clone(b)
        want = step(a2, b2)
        graph.replay()
        for x, y in zip(got, want):
            assert torch.equal(x, y)
        for n in names:
            assert torch.equal(getattr(a, n).view(torch.uint8), getattr(a2, n).view(torch.uint8)), n
            assert torch.equal(getattr(b, n).view(torch.uint8), getattr(b2, n).view(torch.uint8)), n
    assert bsa.get_device_error() == 0


def test_two_streams_at_once():
    bsa = bsa_()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    calls = []
    for i in range(2):
        cache, _, _ = filled(bsa, 3, 2, 2064, 128, 130 + 2 * i)
        q, lens = rows((3, 8, 1, 128), 140 + i).cuda(), i32([2064, 5, 1500 + i])
        out = bsa.KV4Cache.empty(3, 2, 1008, 128)
        calls.append(lambda cache=cache, q=q, lens=lens, out=out: (
            *bsa.kv4_fwd(q, cache, lens, accumulate=False), *bsa.kv4_evict(cache, lens, 1000, recent=9, out=out, values=True)))
    want = [c() for c in calls]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(20):
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                got[i].append(calls[i]())
    torch.cuda.synchronize()
    for i in range(2):
        for g in got[i]:
            assert all(torch.equal(x, y) for x, y in zip(g, want[i]))
    assert bsa.get_device_error() == 0


def test_range_checked_build_runs_the_cache_and_the_key_weights_clean():
    need_gpu()
    from block_sparse_attention_process_gb300 import build as b
    if os.environ.get("BSA_LIBRARY_VARIANT") == "debug":
        pytest.skip("this process runs the range-checked build")
    if not os.path.exists(b.LIB_DEBUG):
        b.build(debug=True)
    r = subprocess.run([sys.executable, "-m", "pytest", "-x", "-q", "-m", "gpu", "-p", "no:cacheprovider", __file__, "-k",
                        "bit_exact or matches_oracle or match_oracle or unequal or together or (is_exact and random)"],
                       env=dict(os.environ, BSA_LIBRARY_VARIANT="debug"), capture_output=True, text=True, timeout=900, cwd=ROOT)
    assert r.returncode == 0 and "passed" in r.stdout, r.stdout[-3000:] + r.stderr[-3000:]


# ------------------------------------------------------------------ groups of a value row, each for itself

def check_groups(o, lse, q, kv, vv, lens, bad=(), **kw):
    """Every 32 channels against the oracle, with a tolerance of their own values' size: beside the rounding of the
    result, 2^-11 of the sum of p |v| for a product held in fp16 and as much again for the products below 2^-14 of
    the group's largest (2^-25 of that each, over 2^13 keys or fewer), and what the scores' errors make of p.
    `bad`: groups that are NaN."""
    D = q.shape[-1]
    got = host(o)
    for g in range(D // 32):
        part = slice(32 * g, 32 * g + 32)
        if g in bad:
            assert np.isnan(got[..., part]).all()
            continue
        only = np.zeros_like(vv)
        only[..., part] = vv[..., part]
        wo, wl, _, apv, aqk = kv4.forward(q.double().numpy(), kv, only, lens, **kw)
        ds = 2.0 ** -16 * aqk
        within(f"o, group {g}", got[..., part], wo[..., part], 2.0 ** -8 * np.abs(wo[..., part]) + (2.0 ** -10 + 2 * ds[..., None]) * apv)
    within("lse", host(lse), wl, ds + 2.0 ** -20 * np.maximum(1, np.abs(wl)))


@pytest.mark.parametrize("size", [2.0 ** -5, 2.0 ** 5])
@pytest.mark.parametrize("n,cap", [(1, 16), (33, 48), (65, 1024), (97, 112), (1, 2064), (33, 2064), (2049, 2064)])
@pytest.mark.parametrize("D", [64, 128])
def test_fwd_nan_group_of_the_only_key_of_a_warp(D, n, cap, size):
    """The last key, alone among the keys that a warp starts with, has one group of NaN: the others keep their values."""
    bsa = bsa_()
    k, v, q = rows((1, 1, cap, D), 150), rows((1, 1, cap, D), 151, size), rows((1, 2, 1, D), 152)
    v[0, 0, n - 1, 40] = float("nan")
    cache, kv, vv = filled(bsa, 1, 1, cap, D, 153, k=k, v=v)
    vv[0, 0, n - 1, 32:64] = 0
    o, lse = bsa.kv4_fwd(q.cuda(), cache, i32([n]))
    assert bsa.get_device_error() == 0
    check_groups(o, lse, q, kv, vv, [n], bad=(1,))


def group_sized(v, e):
    """v (bf16 [.., D]) times 2^e, e whole numbers [.., D/32] (broadcast)."""
    e = np.broadcast_to(np.repeat(np.asarray(e), 32, -1), v.shape)
    return torch.ldexp(v.double(), torch.from_numpy(e.copy())).to(torch.bfloat16)


@pytest.mark.parametrize("n,cap", [(64, 64), (1010, 1024), (2050, 2064)])
@pytest.mark.parametrize("D,sizes", [(64, (0, -14)), (64, (-20, 3)), (64, (0, -30)), (128, (0, -18, -25, 10)), (128, (-60, 15, 0, -90)),
                                     (128, (-100, -112, 0, 30))])
def test_fwd_groups_of_unequal_size(D, sizes, n, cap):
    bsa = bsa_()
    k, v, q = rows((1, 2, cap, D), 160), rows((1, 2, cap, D), 161), rows((1, 6, 1, D), 162)
    cache, kv, vv = filled(bsa, 1, 2, cap, D, 163, k=k, v=group_sized(v, sizes))
    o, lse = bsa.kv4_fwd(q.cuda(), cache, i32([n]))
    assert bsa.get_device_error() == 0
    check_groups(o, lse, q, kv, vv, [n])


@pytest.mark.parametrize("n,cap", [(70, 80), (1024, 1024), (2050, 2064)])
@pytest.mark.parametrize("spread", [4, 12, 40])
@pytest.mark.parametrize("D", [64, 128])
def test_fwd_groups_of_sizes_that_change_from_key_to_key(D, spread, n, cap):
    bsa = bsa_()
    rng = np.random.default_rng(170)
    k, v, q = rows((2, 1, cap, D), 171), rows((2, 1, cap, D), 172), rows((2, 3, 2, D), 173)
    v = group_sized(v, rng.integers(-spread, spread + 1, (2, 1, cap, D // 32)))
    cache, kv, vv = filled(bsa, 2, 1, cap, D, 174, k=k, v=v)
    lens = [n, n // 2 + 1]
    poison(cache, lens)
    o, lse = bsa.kv4_fwd(q.cuda(), cache, i32(lens))
    assert bsa.get_device_error() == 0
    check_groups(o, lse, q, kv, vv, lens)


@pytest.mark.parametrize("n,cap", [(100, 112), (2050, 2064)])
@pytest.mark.parametrize("size", [None, -12, -40, -80])   # None: all zeros
@pytest.mark.parametrize("ahead", [0.25, 2.0])            # (of all the weight but 2^-7 or so, and but 2^-54 or so)
@pytest.mark.parametrize("at", [0, 31, 40, 96])
def test_fwd_key_of_nearly_all_the_weight_has_a_small_group(at, ahead, size, n, cap):
    """Key `at` takes nearly all the weight of the first row; its second group is far smaller than the others',
    or 0: what that group gets then comes from keys of little weight."""
    bsa = bsa_()
    D = 128
    k, v, q = rows((1, 1, cap, D), 180), rows((1, 1, cap, D), 181), rows((1, 2, 1, D), 182)
    k[0, 0, at] = (q[0, 0, 0].float() * ahead).to(torch.bfloat16)
    v[0, 0, at, 32:64] = 0 if size is None else torch.ldexp(v[0, 0, at, 32:64].double(), torch.tensor(size)).to(torch.bfloat16)
    cache, kv, vv = filled(bsa, 1, 1, cap, D, 183, k=k, v=v)
    o, lse = bsa.kv4_fwd(q.cuda(), cache, i32([n]))
    assert bsa.get_device_error() == 0
    check_groups(o, lse, q, kv, vv, [n])


@pytest.mark.parametrize("n,cap", [(500, 512), (2050, 2064)])
@pytest.mark.parametrize("zeros", [1, 33, 129, 400, 3000])
def test_fwd_group_that_begins_with_zeros(zeros, n, cap):
    """The first keys' last group is 0 (a head of 96 channels padded to 128, where all are), with a key of nearly
    all the weight among them."""
    bsa = bsa_()
    D = 128
    k, v, q = rows((1, 1, cap, D), 190), rows((1, 1, cap, D), 191), rows((1, 2, 1, D), 192)
    k[0, 0, 0] = (q[0, 0, 0].float() * 0.75).to(torch.bfloat16)
    v[0, 0, :zeros, 96:] = 0
    cache, kv, vv = filled(bsa, 1, 1, cap, D, 193, k=k, v=v)
    o, lse = bsa.kv4_fwd(q.cuda(), cache, i32([n]))
    assert bsa.get_device_error() == 0
    check_groups(o, lse, q, kv, vv, [n])


@pytest.mark.parametrize("cap", [256, 2064])
def test_fwd_does_not_depend_on_what_lies_behind_the_lengths(cap):
    bsa = bsa_()
    B, Hq, Hkv, T, D = 3, 4, 2, 2, 128
    cache, _, _ = filled(bsa, B, Hkv, cap, D, 200)
    q, lens = rows((B, Hq, T, D), 201).cuda(), [cap - 3, 33, cap // 2 + 1]
    want = bsa.kv4_fwd(q, cache, i32(lens))
    for scale in (0.0, float("nan"), 2.0 ** -60, 2.0 ** 60):
        poison(cache, lens)
        for b, n in enumerate(lens):
            cache.k_scales[b, :, n:] = scale
            cache.v_scales[b, :, n:] = scale
        got = bsa.kv4_fwd(q, cache, i32(lens))
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert bsa.get_device_error() == 0


# ------------------------------------------------------------------ NaN under a soft cap

@pytest.mark.parametrize("softcap", [None, 20.0])
@pytest.mark.parametrize("n,cap", [(1, 16), (90, 96), (2060, 2064)])
def test_fwd_nan_scores(n, cap, softcap):
    """A query of NaN is NaN itself alone; a key that reads as NaN makes its group's rows NaN that see it."""
    bsa = bsa_()
    D = 64
    k, v, q = rows((2, 2, cap, D), 210), rows((2, 2, cap, D), 211), rows((2, 4, 2, D), 212)
    q[0, 1, 0, 7] = float("nan")             # one row of (0, key head 0)
    k[1, 1, n - 1, 40] = float("nan")        # seen by the last token of (1, key head 1)
    cache, kv, vv = filled(bsa, 2, 2, cap, D, 213, k=k, v=v)
    before = cache.weights.clone()
    o, lse = bsa.kv4_fwd(q.cuda(), cache, i32([n, n]), logits_soft_cap=softcap, accumulate=True)
    assert bsa.get_device_error() == 0
    want = kv4.forward(np.nan_to_num(q.double().numpy()), np.nan_to_num(kv), vv, [n, n], cap=softcap or 0)
    nan = np.zeros((2, 4, 2), bool)
    nan[0, 1, 0] = n > 1                     # (of one key the last token alone sees it)
    nan[1, 2:, 1] = True
    o, lse, dw = host(o), host(lse), host(cache.weights - before)
    assert np.array_equal(np.isnan(lse), nan) and np.array_equal(np.isnan(o), np.broadcast_to(nan[..., None], o.shape))
    ds = (2.0 ** -16 * want[4] + 2.0 ** -19 * (softcap or 0))[~nan]
    within("lse", lse[~nan], want[1][~nan], ds + 2.0 ** -20 * np.maximum(1, np.nan_to_num(np.abs(want[1][~nan]), posinf=0)))
    within("o", o[~nan], want[0][~nan], 2.0 ** -8 * np.abs(want[0][~nan]) + (2.0 ** -10 + 2 * ds[:, None]) * want[3][~nan])
    seen = np.arange(cap) < n
    assert np.isnan(dw[1, 1, seen]).all() and np.isfinite(dw[0, 1]).all() and np.isfinite(dw[1, 0]).all()
    assert np.isnan(dw[0, 0, seen & (np.arange(cap) < n - 1)]).all() and (dw[:, :, ~seen] == 0).all()


@pytest.mark.parametrize("softcap", [None, 10.0])
@pytest.mark.parametrize("D", [64, 128])
def test_key_weights_of_nan_scores(D, softcap):
    """A NaN query whose logsumexp is finite makes the keys it sees NaN, a NaN key itself."""
    bsa = bsa_()
    S = 256
    q, k = rows((1, 2, S, D), 215).cuda(), rows((1, 2, S, D), 216).cuda()
    info, dkv = bsa.mask_compile("causal", S, S), bsa.mask_compile("causal", S, S, orientation="dkv")
    _, lse = bsa.fwd(q, k, k, info, logits_soft_cap=softcap)
    clean = bsa.key_weights(q, k, lse, dkv, logits_soft_cap=softcap)
    q, k = q.clone(), k.clone()
    q[0, 0, 131, 3] = float("nan")
    k[0, 1, 70, D - 1] = float("nan")
    got = bsa.key_weights(q, k, lse, dkv, logits_soft_cap=softcap)
    assert bsa.get_device_error() == 0
    nan = torch.zeros_like(clean, dtype=torch.bool)
    nan[0, 0, :132] = True
    nan[0, 1, 70] = True
    assert torch.equal(torch.isnan(got), nan) and torch.equal(got[~nan], clean[~nan])


def test_fwd_and_key_weights_of_scores_far_above_the_cap():
    bsa = bsa_()
    B, Hq, Hkv, S, D, softcap = 1, 2, 1, 128, 64, 3.0
    q, k, v = rows((B, Hq, S, D), 217, 60.0), rows((B, Hkv, S, D), 218), rows((B, Hkv, S, D), 219)
    cache, kv, vv = filled(bsa, B, Hkv, S, D, 0, k=k, v=v)
    want = kv4.forward(q[:, :, :1].double().numpy(), kv, vv, [S], cap=softcap)
    assert want[4].max() > 64 * softcap                            # (the exponential overflows from 45 of them)
    o, lse = bsa.kv4_fwd(q[:, :, :1].cuda(), cache, i32([S]), logits_soft_cap=softcap)
    # (a score's error reaches the capped one at most unchanged; the tanh's own and the rest as above)
    check_fwd(o, lse, None, want, softcap)
    dkv = bsa.mask_compile("full", S, S, orientation="dkv")
    qd, kd = q.double().numpy()[0], k.double().numpy()[0, 0]
    s = softcap * np.tanh(qd @ kd.T * D ** -0.5 / softcap)
    lse = np.log(np.exp(s).sum(-1)).astype(np.float32)
    want = np.exp(s - lse[..., None].astype(np.float64)).sum((0, 1))
    got = bsa.key_weights(q.cuda(), k.cuda(), torch.from_numpy(lse[None]).cuda(), dkv, logits_soft_cap=softcap)
    ds = 2.0 ** -16 * (np.abs(qd) @ np.abs(kd).T).max() * D ** -0.5 + 2.0 ** -19 * softcap + 2.0 ** -23 * np.abs(lse).max()
    within("key weights", host(got)[0, 0], want, want * (2 * ds + 2.0 ** -18) + 1e-30)
    assert bsa.get_device_error() == 0


@pytest.mark.parametrize("softcap,scale", [(None, None), (None, -0.05), (None, 0.0), (15.0, None)])
def test_key_weights_of_infinite_and_huge_logsumexps(softcap, scale):
    """Queries that count with a logsumexp of infinity, or of 300: their probabilities are 0."""
    bsa = bsa_()
    S, D = 256, 64
    q, k = rows((1, 2, S, D), 220), rows((1, 1, S, D), 221)
    sc = D ** -0.5 if scale is None else scale
    s = sc * np.einsum("hid,jd->hij", q.double().numpy()[0], k.double().numpy()[0, 0])
    if softcap:
        s = softcap * np.tanh(s / softcap)
    s = np.where(np.tril(np.ones((S, S), bool)), s, -np.inf)
    lse = np.log(np.exp(s - s.max(-1, keepdims=True)).sum(-1)) + s.max(-1)
    lse[0, [0, 100, 255]] = np.inf
    lse[1, [17, 130]] = 300
    l32 = lse.astype(np.float32)
    want = np.exp(s - l32[..., None].astype(np.float64)).sum((0, 1))
    dkv = bsa.mask_compile("causal", S, S, orientation="dkv")
    got = bsa.key_weights(q.cuda(), k.cuda(), torch.from_numpy(l32[None]).cuda(), dkv, softmax_scale=scale, logits_soft_cap=softcap)
    assert bsa.get_device_error() == 0
    amax = abs(sc) * np.einsum("hid,jd->hij", np.abs(q.double().numpy()[0]), np.abs(k.double().numpy()[0, 0])).max()
    top = np.abs(lse[np.isfinite(lse) & (lse != 300)]).max()
    ds = 2.0 ** -16 * amax + 2.0 ** -23 * max(1.0, top) + 2.0 ** -19 * (softcap or 0)
    within("key weights", host(got)[0, 0], want, want * (2 * ds + 2.0 ** -18) + 1e-30)


@pytest.mark.parametrize("B,cap,T,lens", [(1, 2064, 1, {0: -1}), (2, 2064, 1, {0: -1, 1: -7}), (33, 1040, 1, {32: -1}),
                                          (70, 1040, 1, {69: -3}), (40, 1040, 1, {35: 1041}), (2, 32, 9, {0: -2, 1: -1})])
def test_fwd_split_over_ctas_reports_lengths_outside_the_cache(B, cap, T, lens):
    """Wherever in the batch, and also where no sequence holds a key (T of 9 with weights is split at any capacity)."""
    bsa = bsa_()
    D = 64
    cache, kv, vv = filled(bsa, B, 1, cap, D, 230)
    q = rows((B, 1, T, D), 231)
    ls = [lens.get(b, 1 + 7 * b) for b in range(B)]
    o, lse = bsa.kv4_fwd(q.cuda(), cache, i32(ls), accumulate=T > 8)
    with pytest.raises(bsa.BsaError):
        bsa.get_device_error()
    assert bsa.get_device_error() == 0
    check_fwd(o, lse, None, kv4.forward(q.double().numpy(), kv, vv, [min(max(n, 0), cap) for n in ls]))


# ------------------------------------------------------------------ the documented loop

def test_the_documented_loop_keeps_the_newest_tokens():
    """The README's program, line by line; its token lines run again and again, past several evictions."""
    bsa = bsa_()
    with open(os.path.join(ROOT, "README.md")) as f:
        block = [b for b in f.read().split("```python\n")[1:] if "kv4_append" in b][0].split("```")[0]
    lines = block.splitlines()
    first = next(i for i, x in enumerate(lines) if x.startswith("bsa.kv4_append(cache, k1"))
    B, Hq, Hkv, D, S, budget = 2, 4, 2, 64, 256, 272
    q, k, v = (rows((B, h, S, D), 240 + i).cuda() for i, h in enumerate((Hq, Hkv, Hkv)))
    dkv = bsa.mask_compile("causal", S, S, orientation="dkv")
    _, lse = bsa.fwd(q, k, v, bsa.mask_compile("causal", S, S))
    q1, k1, v1 = (rows((B, h, 1, D), 243 + i).cuda() for i, h in enumerate((Hq, Hkv, Hkv)))
    ns = dict(bsa=bsa, q=q, k=k, v=v, lse=lse, dkv=dkv, B=B, Hkv=Hkv, D=D, capacity=320, pos=i32([0, 0]), q1=q1, k1=k1, v1=v1,
              budget=budget, lens=i32([S, S]), seen=i32([S, S]))
    exec("\n".join(lines[:first]), ns)
    for step in range(40):
        exec("\n".join(lines[first:]), ns)
        assert host(ns["seen"]).tolist() == [S + step + 1] * B and host(ns["lens"]).tolist() == [min(S + step + 1, budget)] * B
        pos = host(ns["cache"].positions)
        for b in range(B):
            for h in range(Hkv):
                have = pos[b, h, :min(S + step + 1, budget)].tolist()
                assert len(set(have)) == len(have) and set(have) >= set(range(S + step + 1 - 256, S + step + 1))
    assert bsa.get_device_error() == 0

"""The key/value cache in pages on the GPU against the fp64 oracle: tables and
slots, append and bounds, selected pages (all exact), attention over pages and
over selected ones, and a run of them together.

Tolerances (none is a measured one).  A score is an fp32 sum of D exact
products: off by at most D 2^-24 sum|q k|, twice that where the tensor core
truncates, so |ds| <= 2^-16 A with A = scale * sum|q k| of the worst seen key;
the soft cap's tanh adds 2^-19 cap.  exp2 and the conversion to log2 units add
2^-20 relative, 2^-20 max(1, |lse|) to a logsumexp.
  LSE:  ds + 2^-20 max(1, |lse|)
  O:    bf16 rounding 2^-8 |o|, plus (2^-8 + 2 ds + 2^-19) sum_j p_j |v_jd|: a
        probability is rounded to bf16 before it meets the value
"""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

from helpers import ROOT, need_gpu
from oracle import paged

pytestmark = pytest.mark.gpu


def bsa_():
    need_gpu()
    import block_sparse_attention_process_gb300 as bsa
    return bsa


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def rows(shape, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(shape, generator=g) * scale * torch.exp(0.5 * torch.randn(shape[-1], generator=g))
    return x.to(torch.bfloat16)


def f64(t):
    return t.double().cpu().numpy()


def within(name, got, want, tol):
    got, want = np.asarray(got, np.float64), np.asarray(want, np.float64)
    assert got.shape == want.shape, name
    assert np.array_equal(np.isnan(got), np.isnan(want)), f"{name}: NaN pattern"
    inf = np.isinf(want)
    assert np.array_equal(got[inf], want[inf]) and not np.isinf(got[~inf]).any(), f"{name}: infinities"
    f = np.isfinite(want)
    err = np.abs(got[f] - want[f])
    over = err - np.broadcast_to(tol, want.shape)[f]
    assert not err.size or over.max() <= 0, f"{name}: off by {err.max():.3e}, {over.max():.3e} too much"


def layout(k, kind):
    """A [P, H, page, D] tensor's memory: plain, tokens before heads, or beside another in one buffer."""
    if kind == "phtd":
        return k.cuda()
    if kind == "pthd":
        return k.transpose(1, 2).contiguous().cuda().transpose(1, 2)
    both = torch.full((k.shape[0], 2) + tuple(k.shape[1:]), float("nan"), dtype=torch.bfloat16, device="cuda")
    both[:, 1] = k.cuda()
    return both[:, 1]


# ------------------------------------------------------------------ tables

def check_resize(bsa, table, free, used, lens, new, page, T, word=0):
    td, fd = torch.from_numpy(table.copy()).cuda(), torch.from_numpy(free.copy()).cuda()
    ud, ld, nd = i32([used]), i32(list(lens)), i32(list(new))
    want_t, want_f = table.copy(), free.copy()
    want_lens, want_used, want_slots = paged.resize(want_t, want_f, used, list(lens), list(new), page, T)
    for _ in range(2):  # a repeated call gives the same
        lens_out, used_out, slots = bsa.paged_resize(td, fd, ud, ld, nd, page, T)
        assert lens_out.tolist() == want_lens and used_out.tolist() == [want_used]
        assert np.array_equal(slots.cpu().numpy(), want_slots)
        assert np.array_equal(td.cpu().numpy(), want_t) and np.array_equal(fd.cpu().numpy(), want_f)
    assert ld.tolist() == list(lens) and ud.tolist() == [used]
    errors(bsa, word)
    return want_t, want_f, want_used, want_lens


def errors(bsa, word):
    if word:
        with pytest.raises(bsa.BsaError):
            bsa.get_device_error()
    assert bsa.get_device_error() == 0


@pytest.mark.parametrize("B,M,page,T,pages,seed", [
    (1, 1, 16, 1, 1, 0), (1, 40, 16, 640, 40, 1), (3, 7, 32, 224, 12, 2), (17, 9, 64, 300, 60, 3), (64, 33, 16, 65, 700, 4),
    (255, 5, 128, 257, 400, 5), (257, 4, 16, 3, 300, 6), (1000, 3, 256, 40, 1700, 7), (4096, 2, 16, 8, 4000, 8), (2, 1100, 16, 700, 1500, 9),
])
def test_sequences_grow_and_end(B, M, page, T, pages, seed):
    bsa = bsa_()
    rng = np.random.default_rng(seed)
    table, free, used = np.full((B, M), -1, dtype=np.int32), rng.permutation(pages).astype(np.int32), 0
    lens = [0] * B
    for _ in range(6):
        new = []
        for n in lens:
            kind = rng.integers(4)
            w = 0 if kind == 0 else int(rng.integers(0, n + 1)) if kind == 1 else n + int(rng.integers(0, T + 1))
            new.append(min(w, M * page))
        table, free, used, lens = check_resize(bsa, table, free, used, lens, new, page, T)
        # no page twice: in the tables and on the stack
        held = [p for b, n in enumerate(lens) for p in table[b, :-(-n // page)].tolist()] + free[used:].tolist()
        assert sorted(held) == list(range(pages))


def test_resize_reports_what_it_refuses():
    bsa = bsa_()
    table = np.array([[0, 1, 2], [3, 4, 5], [6, 9, 7]], dtype=np.int32)
    free = np.array([-1] * 8, dtype=np.int32)
    check_resize(bsa, table, free, 8, [48, 48, 40], [49, 0, 40], 16, 16, word=2)        # longer than its row
    check_resize(bsa, table, free, 8, [48, 48, 40], [-1, 16, 40], 16, 16, word=2)
    check_resize(bsa, table, free, 8, [-5, 48, 40], [48, 16, 40], 16, 16, word=2)
    check_resize(bsa, table, free, 8, [0, 0, 40], [17, 16, 40], 16, 16, word=2)         # more new tokens than the map has
    check_resize(bsa, table, free, 2, [48, 48, 40], [0, 0, 40], 16, 16, word=2)         # gives back more than was taken
    check_resize(bsa, table, free, 9, [48, 48, 40], [0, 0, 40], 16, 16, word=2)
    check_resize(bsa, table, free, -1, [48, 48, 40], [0, 0, 40], 16, 16, word=2)
    check_resize(bsa, table, free, 8, [48, 48, 20], [48, 48, 25], 16, 16, word=2)       # page 9 of 8: no slot
    check_resize(bsa, table, free, 8, [2**31 - 1] * 3, [2**31 - 1] * 3, 16, 16, word=2)


def test_sums_of_pages_do_not_wrap():
    """Pages given back whose number passes 32 bits: more than any stack holds, so nothing changes."""
    bsa = bsa_()
    B, page, M = 4096, 16, 600_000
    table = torch.empty((B, M), dtype=torch.int32, device="cuda")
    free, used = torch.arange(8, dtype=torch.int32, device="cuda"), i32([8])
    lens = torch.full((B,), M * page, dtype=torch.int32, device="cuda")
    for shorter in (0, M * page - page * 2**20 // 2):   # sums of 2,457,600,000 and of exactly 2^31
        got, used_out, slots = bsa.paged_resize(table, free, used, lens, torch.full_like(lens, shorter), page, 1)
        assert torch.equal(got, lens) and used_out.tolist() == [8] and bool((slots == -1).all())
        assert free.tolist() == list(range(8))
        errors(bsa, 2)


# ------------------------------------------------------------------ append

@pytest.mark.parametrize("D,page,H,T,kind", [
    (128, 16, 2, 1, "phtd"), (64, 16, 1, 1, "pthd"), (128, 16, 3, 40, "pthd"), (64, 32, 2, 33, "both"), (128, 64, 1, 200, "phtd"),
    (64, 128, 2, 300, "pthd"), (128, 256, 2, 515, "both"), (64, 256, 1, 77, "phtd"), (128, 32, 5, 64, "phtd"),
])
@pytest.mark.parametrize("bounds", [True, False])
def test_append(D, page, H, T, kind, bounds):
    bsa = bsa_()
    rng = np.random.default_rng(D + page + T)
    starts = [0, 1, page - 1, page, 3 * page // 2, 0]
    counts = [T, max(1, T // 2), 1, T, T, 0]
    B = len(starts)
    M = -(-(T + 2 * page) // page)
    P = B * M + 1
    table = rng.permutation(P)[:B * M].reshape(B, M)
    k0, v0 = rows((P, H, page, D), 1), rows((P, H, page, D), 2)
    b0 = rows((P, H, 2, D), 3) if bounds else None
    cache = bsa.PagedCache(layout(k0, kind), layout(v0, kind), None if b0 is None else b0.cuda())
    k, v = rows((B, T, H, D), 4).transpose(1, 2), rows((B, H, T, D), 5)  # (k strided)
    slots = np.full((B, T), -1, dtype=np.int32)
    want_k, want_v, want_b = f64(k0), f64(v0), None if b0 is None else f64(b0)
    for b in range(B):
        for t in range(counts[b]):
            at = starts[b] + t
            p, i = table[b, at // page], at % page
            slots[b, t] = p * page + i
            want_k[p, :, i], want_v[p, :, i] = f64(k)[b, :, t], f64(v)[b, :, t]
        if bounds and counts[b]:
            end = starts[b] + counts[b]
            for j in range(starts[b] // page, -(-end // page)):
                for h in range(H):
                    want_b[table[b, j], h] = paged.bounds(want_k[table[b, j], h, :min(page, end - j * page)])
    bsa.paged_append(cache, k.cuda(), v.cuda(), torch.from_numpy(slots).cuda())
    assert np.array_equal(f64(cache.k), want_k) and np.array_equal(f64(cache.v), want_v)
    if bounds:
        assert np.array_equal(f64(cache.bounds), want_b)
    assert bsa.get_device_error() == 0


@pytest.mark.parametrize("D", [64, 128])
def test_bounds_of_unusual_keys(D):
    bsa = bsa_()
    special = [torch.zeros(16, D), torch.full((16, D), -0.0), torch.full((16, D), 2.0 ** -126), torch.randn(16, D) * 2.0 ** -120,
               torch.randn(16, D) * 2.0 ** 97, torch.full((16, D), 2.0 ** 100)]
    for x in (float("nan"), float("inf"), -float("inf"), 3.3e38):
        y = torch.randn(16, D)
        y[7, D // 3] = x
        special.append(y)
    y = torch.full((16, D), 2.0 ** -133)
    y[:, 1::2] *= -1
    y[3, 5] = 2.0 ** 99  # channels whose quotient by the unit is no longer a number of fp32
    special.append(y)
    y = torch.randn(16, D)
    y[:, 1:] = -y[:, 1:].abs()
    y[:, 0] = 1.9921875
    special.append(y)
    k = torch.stack(special)[:, None].to(torch.bfloat16)
    P = len(special)
    cache = bsa.PagedCache.empty(P, 1, 16, D)
    slots = torch.arange(P * 16, dtype=torch.int32, device="cuda").view(P, 16)
    bsa.paged_append(cache, k.cuda(), k.cuda(), slots)
    got, want = f64(cache.bounds), np.stack([paged.bounds(x)[None] for x in f64(k)[:, 0]])
    assert np.array_equal(got, want)
    f = np.isfinite(f64(k)).all((1, 2, 3)) & (np.abs(f64(k)) < 2.0 ** 100).all((1, 2, 3))
    assert (got[f][:, 0, 0] >= f64(k)[f][:, 0].max(1)).all() and (got[f][:, 0, 1] <= f64(k)[f][:, 0].min(1)).all()


def test_append_in_any_order_without_bounds():
    bsa = bsa_()
    rng = np.random.default_rng(0)
    cache = bsa.PagedCache.empty(9, 2, 16, 64, bounds=False)
    slots = rng.permutation(9 * 16)[:100].reshape(2, 50).astype(np.int32)
    slots[0, 3], slots[1, 7] = -1, -7
    k = rows((2, 2, 50, 64), 1)
    bsa.paged_append(cache, k.cuda(), (-k).cuda(), torch.from_numpy(slots).cuda())
    want = np.zeros((9, 2, 16, 64))
    for b in range(2):
        for t in range(50):
            if slots[b, t] >= 0:
                want[slots[b, t] // 16, :, slots[b, t] % 16] = f64(k)[b, :, t]
    assert np.array_equal(f64(cache.k), want) and np.array_equal(f64(cache.v), -want)
    assert bsa.get_device_error() == 0


@pytest.mark.parametrize("bounds", [True, False])
def test_slots_outside_the_cache_are_reported(bounds):
    bsa = bsa_()
    cache = bsa.PagedCache.empty(3, 1, 16, 64, bounds=bounds)
    k = rows((3, 1, 1, 64), 1).cuda()
    bsa.paged_append(cache, k, k, i32([[48], [2**31 - 1], [17]]))
    errors(bsa, 2)
    want = np.zeros((3, 1, 16, 64))
    want[1, 0, 1] = f64(k)[2, 0, 0]
    assert np.array_equal(f64(cache.k), want)


def test_tokens_out_of_order_are_not_stored_with_bounds():
    bsa = bsa_()
    cache = bsa.PagedCache.empty(4, 1, 16, 64)
    k = rows((2, 1, 20, 64), 1).cuda()
    good = torch.arange(8, 28, dtype=torch.int32, device="cuda")
    slots = torch.stack((good, good + 24))
    slots[0, 2] = 60     # another place
    slots[1, 8:] -= 1    # the second page begins a place early
    bsa.paged_append(cache, k, k, slots)
    errors(bsa, 2)
    want = np.zeros((64, 64))
    for t in range(20):
        if t != 2:
            want[8 + t] = f64(k)[0, 0, t]
        if t < 8:
            want[32 + t] = f64(k)[1, 0, t]
    assert np.array_equal(f64(cache.k).reshape(64, 64), want)


# ------------------------------------------------------------------ selection

def paged_batch(bsa, B, H, D, page, lens, seed, kind="phtd", M=None, junk=True, scale=1.0):
    """A cache that holds sequences of `lens` tokens in scattered pages, junk elsewhere; their keys and values."""
    rng = np.random.default_rng(seed)
    most = max(1, max(lens))
    M = M or -(-most // page)
    P = B * M + 3
    table = rng.permutation(P)[:B * M].reshape(B, M).astype(np.int32)
    k, v = rows((B, H, M * page, D), seed, scale), rows((B, H, M * page, D), seed + 1)
    kc = torch.full((P, H, page, D), float("nan") if junk else 0.0, dtype=torch.bfloat16)
    vc = kc.clone()
    bc = torch.full((P, H, 2, D), float("nan"), dtype=torch.bfloat16)
    for b, n in enumerate(lens):
        for j in range(-(-n // page)):
            m = min(page, n - j * page)
            kc[table[b, j], :, :m], vc[table[b, j], :, :m] = k[b, :, j * page:j * page + m], v[b, :, j * page:j * page + m]
            for h in range(H):
                bc[table[b, j], h] = torch.from_numpy(paged.bounds(f64(k[b, h, j * page:j * page + m]))).to(torch.bfloat16)
        table[b, -(-n // page):] = -1
    return bsa.PagedCache(layout(kc, kind), layout(vc, kind), bc.cuda()), torch.from_numpy(table).cuda(), k, v


def want_select(cache, table, q, lens, keep, first, recent, q_lens=None):
    B, Hq, T, D = q.shape
    H, page = cache.Hkv, cache.page
    out = np.full((B, H, T, keep), -1, dtype=np.int32)
    bounds, tab, qh = f64(cache.bounds), table.cpu().numpy(), f64(q)
    for b in range(B):
        nq = T if q_lens is None else q_lens[b]
        for t in range(nq):
            n = -(-max(0, lens[b] - nq + t + 1) // page)
            for h in range(H):
                g = Hq // H
                out[b, h, t] = paged.select(qh[b, h * g:(h + 1) * g, t], bounds[tab[b, :n], h], keep, first, recent)
    return out


@pytest.mark.parametrize("B,H,G,D,page,T,lens,keep,first,recent", [
    (1, 1, 1, 64, 16, 1, [1], 1, 0, 0), (2, 2, 4, 128, 16, 1, [200, 37], 4, 1, 1), (1, 1, 16, 64, 16, 2, [700], 7, 2, 3),
    (3, 2, 3, 128, 32, 3, [1000, 2, 0], 5, 0, 0), (1, 2, 5, 64, 64, 1, [4097], 64, 1, 1), (2, 1, 17, 128, 16, 1, [2500, 2049], 20, 1, 1),
    (1, 1, 40, 64, 128, 2, [1300], 3, 0, 1), (2, 8, 4, 128, 16, 1, [4100, 3000], 32, 1, 1), (1, 1, 2, 64, 16, 1, [70000], 300, 1, 1),
    (2, 2, 2, 64, 256, 5, [3, 4000], 2, 1, 1), (1, 2, 8, 128, 16, 4, [2048], 128, 1, 2), (1, 1, 1, 64, 16, 1, [16 * 600], 1, 0, 0),
])
def test_select(B, H, G, D, page, T, lens, keep, first, recent):
    bsa = bsa_()
    cache, table, _, _ = paged_batch(bsa, B, H, D, page, lens, 11)
    q = rows((B, T, H * G, D), 21).transpose(1, 2).cuda()
    got = bsa.paged_select(q, cache, table, i32(lens), keep, first=first, recent=recent)
    assert np.array_equal(got.cpu().numpy(), want_select(cache, table, q, lens, keep, first, recent))
    assert bsa.get_device_error() == 0


def test_select_with_padding_and_short_sequences():
    bsa = bsa_()
    lens, q_lens, T = [500, 300, 2, 0, 90], [3, 0, 3, 2, 1], 3
    cache, table, _, _ = paged_batch(bsa, 5, 2, 64, 16, lens, 5)
    q = rows((5, 8, T, 64), 6).cuda()
    got = bsa.paged_select(q, cache, table, i32(lens), 6, q_lens=i32(q_lens))
    assert np.array_equal(got.cpu().numpy(), want_select(cache, table, q, lens, 6, 1, 1, q_lens))


def test_select_ties_zeros_and_infinities():
    bsa = bsa_()
    n = 300 * 16
    cache, table, _, _ = paged_batch(bsa, 1, 1, 64, 16, [n], 9)
    tab = table[0].long()
    q = rows((1, 2, 1, 64), 3).cuda()
    one = cache.bounds[tab[5]].clone()
    cache.bounds[tab] = one                        # all scores equal
    for keep in (1, 2, 77):
        got = bsa.paged_select(q, cache, table, i32([n]), keep, first=0, recent=0)
        assert got.flatten().tolist() == list(range(keep))
    cache.bounds[tab[200:]] = one * 2
    got = bsa.paged_select(q, cache, table, i32([n]), 50, first=0, recent=0)
    assert np.array_equal(got.cpu().numpy(), want_select(cache, table, q, [n], 50, 0, 0))
    cache.bounds[tab[123], :, 0], cache.bounds[tab[123], :, 1] = float("inf"), -float("inf")   # a page with a NaN key
    got = bsa.paged_select(q, cache, table, i32([n]), 3, first=1, recent=1)
    assert got.flatten().tolist() == [0, 123, 299]
    for q2 in (torch.zeros_like(q), torch.full_like(q, float("nan")), q * float("inf"), torch.full_like(q, 2.0 ** 100)):
        got = bsa.paged_select(q2, cache, table, i32([n]), 4, first=0, recent=1)
        assert got.flatten().tolist() == [0, 1, 123, 299]
    for s in (2.0 ** -126, 2.0 ** -110, 2.0 ** 90):
        q2 = (rows((1, 2, 1, 64), 4).float() * s).to(torch.bfloat16).cuda()
        got = bsa.paged_select(q2, cache, table, i32([n]), 60, first=0, recent=0)
        assert np.array_equal(got.cpu().numpy(), want_select(cache, table, q2, [n], 60, 0, 0))


def test_select_sums_stay_exact():
    """The largest whole numbers the sums can hold, whose last bit decides."""
    bsa = bsa_()
    D, n = 128, 40
    cache, table, _, _ = paged_batch(bsa, 1, 1, D, 16, [n * 16], 9)
    b = np.zeros((n, 2, D))
    rng = np.random.default_rng(1)
    b[:, 0], b[:, 1] = 256, -256
    for j in range(n):
        b[j, 0, :] -= rng.permutation(np.arange(D) < 2 + j % 3)    # sums that differ by few units in 2^22
    b *= 2.0 ** -7
    cache.bounds[table[0].long()] = torch.from_numpy(b[:, None]).to(torch.bfloat16).cuda()
    q = torch.full((1, 1, 1, D), 1.9921875, dtype=torch.bfloat16)
    q[..., ::3] = 1.0
    q[..., 1::7] = 0.515625
    for keep in (1, 5, 13, 20, 39):
        got = bsa.paged_select(q.cuda(), cache, table, i32([n * 16]), keep, first=0, recent=0)
        assert np.array_equal(got.cpu().numpy(), want_select(cache, table, q, [n * 16], keep, 0, 0))


@pytest.mark.parametrize("n,queries,keep", [(49152, 1, 500), (20000, 1, 2049), (9000, 24, 33), (300, 600, 17)])
def test_select_of_many_pages(n, queries, keep):
    """Up to the most pages a sequence can have; many queries to a launch."""
    bsa = bsa_()
    D, P = 64, n + 1
    g = torch.Generator(device="cuda").manual_seed(n)
    k = torch.zeros((P, 1, 16, D), dtype=torch.bfloat16, device="cuda")
    code = torch.randint(-256, 257, (P, 1, 2, D), generator=g, device="cuda")
    bounds = (torch.sort(code, dim=2, descending=True).values * 2.0 ** torch.randint(-9, -6, (P, 1, 1, 1), generator=g, device="cuda")).to(torch.bfloat16)
    cache = bsa.PagedCache(k, k, bounds)
    table = torch.randperm(P, generator=g, device="cuda")[:n].to(torch.int32).expand(queries, n).contiguous()
    q = torch.randn((queries, 2, 1, D), generator=g, device="cuda").to(torch.bfloat16)
    got = bsa.paged_select(q, cache, table, i32([n * 16] * queries), keep, first=2, recent=1)
    qc = torch.ldexp(q.float(), 7 - torch.frexp(q.float().abs().amax((1, 2, 3), keepdim=True)).exponent).double()
    qc = torch.round(qc)[:, :, 0].flatten(0, 1)
    b = bounds[table[0].long(), 0].double()
    s = (qc.clamp(min=0) @ b[:, 0].T + qc.clamp(max=0) @ b[:, 1].T).view(queries, 2, n).amax(1)
    s[:, :2], s[:, -1] = float("inf"), float("inf")
    want = torch.sort(torch.sort(s, dim=-1, descending=True, stable=True).indices[:, :keep], dim=-1).values
    assert torch.equal(got.view(queries, keep).long(), want)
    with pytest.raises(bsa.BsaError):
        bsa.paged_select(q[:1], cache, torch.zeros((1, 49153), dtype=torch.int32, device="cuda"), i32([16]), 4)


def test_select_reports_bad_tables_and_lengths():
    bsa = bsa_()
    cache, table, _, _ = paged_batch(bsa, 1, 1, 64, 16, [160], 9)
    q = rows((1, 1, 1, 64), 3).cuda()
    bsa.paged_select(q, cache, table, i32([161]), 3)
    errors(bsa, 2)
    bsa.paged_select(q, cache, table, i32([-1]), 3)
    errors(bsa, 2)
    want = bsa.paged_select(q, cache, table, i32([160]), 9, first=0, recent=0).flatten().tolist()
    out = next(j for j in range(10) if j not in want)
    for bad in (-1, cache.pages, 2**31 - 1):
        table[0, out] = bad           # the page of the least score is still the one left out
        assert bsa.paged_select(q, cache, table, i32([160]), 9, first=0, recent=0).flatten().tolist() == want
        errors(bsa, 2)


# ------------------------------------------------------------------ attention

def check_fwd(bsa, cache, table, k, v, q, lens, *, q_lens=None, scale=None, cap=0.0, sinks=None, left=None, chunk=None, select=None,
              without=None, **kw):
    B, Hq, T, D = q.shape
    H, page = cache.Hkv, cache.page
    o, lse = bsa.paged_fwd(q, cache, table, i32(lens), q_lens=None if q_lens is None else i32(q_lens), softmax_scale=scale,
                           logits_soft_cap=cap or None, sinks=sinks, local_left=left, chunk=chunk,
                           select=None if select is None else torch.from_numpy(select).cuda(), **kw)
    s = D ** -0.5 if scale is None else scale
    want, wl, mass, ds = np.zeros((B, Hq, T, D)), np.zeros((B, Hq, T)), np.zeros((B, Hq, T, D)), np.zeros((B, Hq, T))
    qh, kh, vh = f64(q), f64(k), f64(v)
    for b in range(B):
        nq = T if q_lens is None else q_lens[b]
        for hq in range(Hq):
            h = hq // (Hq // H)
            z = None if sinks is None else f64(sinks[h] if sinks.dim() == 2 else sinks)
            for t in range(T):
                pos = lens[b] - nq + t
                seen = np.arange(paged.first_key(pos, left, chunk), pos + 1) if t < nq and pos >= 0 else np.zeros(0, int)
                seen = seen[seen // page != without] if without is not None else seen
                if select is not None:
                    pages = select[b, h, t][:-(-len(seen) // page)].tolist()
                    seen = np.array([i for j in pages if 0 <= j * page <= pos for i in range(j * page, min(pos + 1, j * page + page))], int)
                x, l, m, a = paged.attend(qh[b, hq, t], kh[b, h, seen], vh[b, h, seen], s, cap, z)
                want[b, hq, t], wl[b, hq, t], mass[b, hq, t], ds[b, hq, t] = x, l, m, 2.0 ** -16 * a + 2.0 ** -19 * cap
    within("lse", f64(lse), wl, ds + 2.0 ** -20 * np.maximum(1, np.abs(np.where(np.isfinite(wl), wl, 0))))
    within("o", f64(o), want, 2.0 ** -8 * np.abs(want) + (2.0 ** -8 + 2 * ds[..., None] + 2.0 ** -19) * mass)
    return o, lse


@pytest.mark.parametrize("B,H,G,D,page,T,lens,kind", [
    (1, 1, 1, 64, 16, 1, [1], "phtd"), (2, 2, 4, 128, 16, 1, [300, 17], "phtd"), (3, 2, 3, 64, 32, 1, [65, 64, 63], "pthd"),
    (1, 2, 8, 128, 64, 1, [3000], "both"), (2, 1, 16, 64, 16, 1, [1025, 1], "phtd"), (1, 1, 17, 128, 16, 1, [700], "pthd"),
    (2, 1, 5, 64, 128, 3, [520, 130], "phtd"), (1, 1, 16, 128, 32, 4, [2000], "phtd"), (2, 2, 10, 64, 16, 7, [90, 700], "both"),
    (1, 1, 100, 64, 256, 1, [600], "phtd"), (1, 1, 3, 128, 256, 40, [1111], "pthd"), (16, 2, 4, 64, 16, 1, list(range(1, 1600, 100)), "phtd"),
    (1, 1, 2, 128, 16, 1, [20000], "phtd"), (90, 2, 2, 64, 16, 1, [1 + 29 * i % 600 for i in range(90)], "pthd"),
    (80, 2, 20, 64, 16, 1, [1 + 7 * i % 90 for i in range(80)], "phtd"), (9, 1, 9, 64, 32, 5, [300 * i for i in range(9)], "phtd"), (40, 1, 1, 64, 16, 1, [5 + 37 * i % 900 for i in range(40)], "phtd"),
])
def test_fwd(B, H, G, D, page, T, lens, kind):
    bsa = bsa_()
    cache, table, k, v = paged_batch(bsa, B, H, D, page, lens, 31, kind)
    q = rows((B, T, H * G, D), 41).transpose(1, 2).cuda()
    check_fwd(bsa, cache, table, k, v, q, lens)
    assert bsa.get_device_error() == 0


@pytest.mark.parametrize("M", [None, 64])   # a pair whole to a CTA, and cut into runs
def test_fwd_of_empty_and_padded_sequences(M):
    bsa = bsa_()
    lens, q_lens, T = [0, 5, 2, 100, 33, 0], [3, 3, 3, 0, 1, 0], 3
    cache, table, k, v = paged_batch(bsa, 6, 2, 64, 16, lens, 5, M=M)
    q = rows((6, 8, T, 64), 6).cuda()
    q[3] = float("nan")                         # padding rows may hold anything
    q[4, :, 1:] = float("inf")
    o, lse = check_fwd(bsa, cache, table, k, v, q, lens, q_lens=q_lens)
    assert not o[3].any() and torch.isneginf(lse[3]).all() and not o[2, :, 0].any()
    z = torch.randn((2, 3), generator=torch.Generator().manual_seed(0)).cuda()
    o, lse = check_fwd(bsa, cache, table, k, v, q, lens, q_lens=q_lens, sinks=z)
    assert torch.isfinite(lse).all()
    assert bsa.get_device_error() == 0


@pytest.mark.parametrize("kw", [{"left": 0}, {"left": 15}, {"left": 16}, {"left": 100}, {"left": 5000}, {"left": -1}, {"chunk": 1},
                                {"chunk": 7}, {"chunk": 64}, {"chunk": 100}, {"chunk": 1 << 40}])
@pytest.mark.parametrize("T", [1, 5])
def test_fwd_local_and_chunked(kw, T):
    bsa = bsa_()
    lens = [900, 64, 3, 129]
    cache, table, k, v = paged_batch(bsa, 4, 2, 64, 32, lens, 7)
    q = rows((4, 6, T, 64), 8).cuda()
    check_fwd(bsa, cache, table, k, v, q, lens, **kw)


@pytest.mark.parametrize("D", [64, 128])
def test_fwd_cap_sinks_scale_and_given_outputs(D):
    bsa = bsa_()
    lens = [700, 40]
    cache, table, k, v = paged_batch(bsa, 2, 2, D, 16, lens, 9, scale=3.0)
    q = rows((2, 4, 2, D), 10, 3.0).cuda()
    check_fwd(bsa, cache, table, k, v, q, lens, cap=30.0, sinks=torch.tensor([0.5, -3.0]).cuda())
    check_fwd(bsa, cache, table, k, v, q, lens, scale=-0.25)
    check_fwd(bsa, cache, table, k, v, q, lens, scale=0.0)
    o = torch.full((2, 2, 4, D), float("nan"), dtype=torch.bfloat16, device="cuda").transpose(1, 2)
    lse = torch.empty((2, 4, 2), device="cuda")
    got, _ = check_fwd(bsa, cache, table, k, v, q, lens, o=o, lse=lse)
    assert got is o


def test_one_visible_key_returns_its_value():
    bsa = bsa_()
    cache, table, k, v = paged_batch(bsa, 3, 1, 128, 16, [1, 1, 1], 3)
    q = rows((3, 4, 1, 128), 4).cuda()
    o, _ = bsa.paged_fwd(q, cache, table, i32([1, 1, 1]))
    assert torch.equal(o, v[:, :, :1].expand(3, 4, 1, 128).cuda())


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("where", ["k", "v"])
@pytest.mark.parametrize("H,G,T", [(2, 4, 5), (1, 16, 4)])
def test_what_a_row_does_not_see_does_not_reach_it(bad, where, H, G, T):
    """Values that are not numbers in keys that only later (or, with a window, only earlier) tokens see."""
    bsa = bsa_()
    n = 600
    for left, key in ((None, n - 2), (None, n - T + 1), (50, n - T - 50), (50, n - T - 48)):
        cache, table, k, v = paged_batch(bsa, 1, H, 64, 16, [n], 13)
        (k if where == "k" else v)[0, :, key, 3] = bad
        c = cache.k if where == "k" else cache.v
        c[table[0, key // 16].long(), :, key % 16, 3] = bad
        q = rows((1, H * G, T, 64), 14).cuda()
        o, lse = bsa.paged_fwd(q, cache, table, i32([n]), local_left=left)
        sees = [key <= n - T + t and (left is None or key >= n - T + t - left) for t in range(T)]
        assert any(sees) and not all(sees)
        clean_k, clean_v = k.clone(), v.clone()
        (clean_k if where == "k" else clean_v)[0, :, key, 3] = 1.0
        c[table[0, key // 16].long(), :, key % 16, 3] = 1.0
        want_o, want_lse = check_fwd(bsa, cache, table, clean_k, clean_v, q, [n], left=left)
        for t in range(T):
            if not sees[t]:
                assert torch.equal(o[:, :, t], want_o[:, :, t]) and torch.equal(lse[:, :, t], want_lse[:, :, t])
            elif where == "v":
                x = o[0, :, t, 3].float()
                assert bool((torch.isnan(x) if bad != bad else x == bad).all())
                assert torch.isfinite(o[0, :, t, :3].float()).all() and torch.equal(lse[:, :, t], want_lse[:, :, t])
            elif bad != bad:
                assert torch.isnan(lse[0, :, t]).all() and torch.isnan(o[0, :, t].float()).all()


@pytest.mark.parametrize("B,H,G,D,page,T,lens,keep", [
    (1, 1, 4, 64, 16, 1, [1000], 5), (2, 2, 4, 128, 16, 3, [300, 40], 4), (2, 1, 16, 64, 64, 2, [1500, 64], 3), (1, 2, 5, 128, 32, 1, [4000], 64),
    (3, 1, 17, 64, 128, 1, [1000, 3, 0], 2), (2, 2, 3, 64, 16, 4, [2, 700], 7), (1, 1, 2, 64, 16, 1, [500], 64), (4, 2, 4, 128, 64, 1, [2000, 1999, 70, 64], 9),
])
def test_fwd_over_selected_pages(B, H, G, D, page, T, lens, keep):
    bsa = bsa_()
    cache, table, k, v = paged_batch(bsa, B, H, D, page, lens, 51)
    q = rows((B, H * G, T, D), 52).cuda()
    select = want_select(cache, table, q, lens, keep, 0, 0)
    got = bsa.paged_select(q, cache, table, i32(lens), keep, first=0, recent=0)
    assert np.array_equal(got.cpu().numpy(), select)
    check_fwd(bsa, cache, table, k, v, q, lens, select=select)
    check_fwd(bsa, cache, table, k, v, q, lens, select=select, cap=20.0, sinks=torch.ones(H, 1).cuda())
    assert bsa.get_device_error() == 0


def test_lists_in_any_order_and_with_padding():
    bsa = bsa_()
    lens, q_lens = [500, 200, 50], [2, 0, 1]
    cache, table, k, v = paged_batch(bsa, 3, 2, 64, 16, lens, 5)
    q = rows((3, 4, 2, 64), 6).cuda()
    select = want_select(cache, table, q, lens, 6, 1, 1, q_lens)
    check_fwd(bsa, cache, table, k, v, q, lens, select=select[..., ::-1].copy() if (select >= 0).all() else select, q_lens=q_lens)
    select[0] = select[0][..., ::-1]
    check_fwd(bsa, cache, table, k, v, q, lens, select=select, q_lens=q_lens)
    assert bsa.get_device_error() == 0


def test_bad_pages_and_lengths_are_reported_and_left_out():
    bsa = bsa_()
    n = 400
    cache, table, k, v = paged_batch(bsa, 1, 1, 64, 16, [n], 5)
    q = rows((1, 4, 1, 64), 6).cuda()
    select = np.array([[[[0, 24, 7, 3]]]], dtype=np.int32)
    check_fwd(bsa, cache, table, k, v, q, [n], select=select)
    for entry in (-1, 25, 2**31 - 1, -2**31):
        check_fwd(bsa, cache, table, k, v, q, [n], select=np.array([[[[0, 24, entry, 7, 3]]]], dtype=np.int32))
        errors(bsa, 2)
    for entry in (-1, cache.pages, 2**31 - 1):
        broken = table.clone()
        broken[0, 9] = entry
        check_fwd(bsa, cache, broken, k, v, q, [n], without=9)
        errors(bsa, 2)
    cache, table, k, v = paged_batch(bsa, 1, 1, 64, 16, [n], 5)
    for n_bad, n_good in ((n + 1, n), (2**31 - 1, n), (-3, 0)):
        a = bsa.paged_fwd(q, cache, table, i32([n_bad]))
        errors(bsa, 2)
        b = bsa.paged_fwd(q, cache, table, i32([n_good]))
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_offsets_past_32_bits():
    bsa = bsa_()
    page, H, D = 256, 8, 128
    P = (1 << 31) // (page * H * D) + 40      # more than 2^31 elements
    kv = torch.zeros((P, H, page, D), dtype=torch.bfloat16, device="cuda")
    cache = bsa.PagedCache(kv, kv, torch.zeros((P, H, 2, D), dtype=torch.bfloat16, device="cuda"))
    n = 700
    table = i32([[P - 1, 3, P - 2]])
    k = rows((1, H, n, D), 1).cuda()
    t = torch.arange(n, device="cuda")
    slots = (table[0, t // page] * page + t % page).to(torch.int32)[None]
    bsa.paged_append(cache, k, k, slots)
    assert torch.equal(kv[P - 1, :, :5], k[0, :, :5]) and torch.equal(kv[P - 2, :, n - 513], k[0, :, n - 1])
    want = np.stack([[paged.bounds(f64(k[0, h, j * page:min(n, (j + 1) * page)])) for h in range(H)] for j in range(3)])
    assert np.array_equal(f64(cache.bounds[table[0].long()]), want)
    q = rows((1, 16, 1, D), 2).cuda()
    check_fwd(bsa, cache, table, k, k, q, [n])
    got = bsa.paged_select(q, cache, table, i32([n]), 2)
    assert np.array_equal(got.cpu().numpy(), want_select(cache, table, q, [n], 2, 1, 1))
    bare = bsa.PagedCache(kv, kv)
    bsa.paged_append(bare, -k, -k, slots)
    assert torch.equal(kv[P - 1, :, :5], -k[0, :, :5])
    assert bsa.get_device_error() == 0


# ------------------------------------------------------------------ together

def test_sequences_answer_in_one_captured_step():
    """Sequences that start, grow a token a step, end and make room, through one captured graph, against contiguous
    keys on the host."""
    bsa = bsa_()
    B, H, G, D, page, M, P, T = 5, 2, 4, 64, 16, 12, 34, 1
    cache = bsa.PagedCache.empty(P, H, page, D)
    table, free, used = bsa.paged_table(P, B, M)
    lens = i32([0] * B)
    g = torch.Generator().manual_seed(0)
    hold = [(torch.zeros(H, 0, D, dtype=torch.bfloat16), torch.zeros(H, 0, D, dtype=torch.bfloat16)) for _ in range(B)]

    def prompt(b_lens):
        nonlocal lens, used
        new = [n if m == 0 else m for n, m in zip(b_lens, lens.tolist())]
        before = lens.tolist()
        lens, used, slots = bsa.paged_resize(table, free, used, lens, i32(new), page, 64)
        k, v = torch.randn((2, B, H, 64, D), generator=g).to(torch.bfloat16)
        bsa.paged_append(cache, k.cuda(), v.cuda(), slots)
        for b, n in enumerate(lens.tolist()):
            m = n - before[b]
            if m > 0:
                hold[b] = tuple(torch.cat((x, y[b, :, :m]), 1) for x, y in zip(hold[b], (k, v)))
        assert lens.tolist() == new

    prompt([33, 64, 1, 16, 40])
    s_lens, s_new, s_used = lens.clone(), lens.clone(), used.clone()
    k1, v1 = (torch.zeros((B, H, T, D), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    q1 = torch.zeros((B, H * G, T, D), dtype=torch.bfloat16, device="cuda")

    def step():
        n, u, slots = bsa.paged_resize(table, free, s_used, s_lens, s_new, page, T)
        bsa.paged_append(cache, k1, v1, slots)
        index = bsa.paged_select(q1, cache, table, n, 3)
        full = bsa.paged_fwd(q1, cache, table, n)
        sparse = bsa.paged_fwd(q1, cache, table, n, select=index)
        return n, u, index, full, sparse

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for i in range(30):
        k, v = torch.randn((2, B, H, T, D), generator=g).to(torch.bfloat16)
        q = torch.randn((B, H * G, T, D), generator=g).to(torch.bfloat16)
        k1.copy_(k), v1.copy_(v), q1.copy_(q)
        now = s_lens.tolist()
        new = [0 if (i + b) % 11 == 10 else n + 1 for b, n in enumerate(now)]
        s_new.copy_(i32(new))
        graph.replay()
        n, u, index, full, sparse = out
        got = n.tolist()
        for b in range(B):
            if new[b] == 0:
                hold[b] = (hold[b][0][:, :0], hold[b][1][:, :0])
            elif got[b] == new[b]:
                hold[b] = tuple(torch.cat((x, y[b]), 1) for x, y in zip(hold[b], (k, v)))
            assert got[b] in (new[b], now[b]) and hold[b][0].shape[1] == got[b]
        kk = torch.stack([torch.nn.functional.pad(x, (0, 0, 0, M * page - x.shape[1])) for x, _ in hold])
        vv = torch.stack([torch.nn.functional.pad(x, (0, 0, 0, M * page - x.shape[1])) for _, x in hold])
        want = want_select(cache, table, q1, got, 3, 1, 1)
        assert np.array_equal(index.cpu().numpy(), want)
        for x, kw in ((full, {}), (sparse, {"select": want})):
            a = check_fwd(bsa, cache, table, kk, vv, q1, got, **kw)
            assert torch.equal(a[0], x[0]) and torch.equal(a[1], x[1])
        s_lens.copy_(n), s_used.copy_(u)
    assert bsa.get_device_error() == 0


def test_two_streams_at_once_and_replayed():
    bsa = bsa_()
    lens = [3000, 1500, 7]
    cache, table, k, v = paged_batch(bsa, 3, 2, 128, 16, lens, 3)
    q = [rows((3, 8, 1, 128), s).cuda() for s in (1, 2)]
    n = i32(lens)
    want = [(bsa.paged_select(x, cache, table, n, 20), bsa.paged_fwd(x, cache, table, n)) for x in q]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(20):
        got = [(bsa.paged_select(x, cache, table, n, 20, stream=s), bsa.paged_fwd(x, cache, table, n, stream=s)) for x, s in zip(q, streams)]
    torch.cuda.synchronize()
    for (i, (o, l)), (j, (p, m)) in zip(got, want):
        assert torch.equal(i, j) and torch.equal(o, p) and torch.equal(l, m)


def test_wrong_tensors_are_refused():
    bsa = bsa_()
    cache, table, _, _ = paged_batch(bsa, 2, 2, 64, 16, [40, 20], 3)
    q, n = rows((2, 4, 1, 64), 1).cuda(), i32([40, 20])
    bare = bsa.PagedCache(cache.k, cache.v)
    k = rows((2, 2, 1, 64), 1).cuda()
    bad = [
        lambda: bsa.paged_fwd(q.float(), cache, table, n), lambda: bsa.paged_fwd(q.cpu(), cache, table, n),
        lambda: bsa.paged_fwd(q, cache, table.long(), n), lambda: bsa.paged_fwd(q, cache, table[:1], n),
        lambda: bsa.paged_fwd(q, cache, table, n.cpu()), lambda: bsa.paged_fwd(q, cache, table, n[:1]),
        lambda: bsa.paged_fwd(q, cache, table, None), lambda: bsa.paged_fwd(q, cache, table.t(), n),
        lambda: bsa.paged_fwd(q, cache, table, n, local_left=3, chunk=4), lambda: bsa.paged_fwd(q, cache, table, n, chunk=0),
        lambda: bsa.paged_fwd(q, cache, table, n, select=torch.zeros((2, 2, 1, 0), dtype=torch.int32, device="cuda")),
        lambda: bsa.paged_fwd(q, cache, table, n, select=torch.zeros((2, 4, 1, 3), dtype=torch.int32, device="cuda")),
        lambda: bsa.paged_fwd(q, cache, table, n, o=torch.empty_like(q[:1])),
        lambda: bsa.paged_fwd(q, cache, table, n, o=torch.empty((2, 1, 1, 64), dtype=torch.bfloat16, device="cuda").expand(2, 4, 1, 64)),
        lambda: bsa.paged_fwd(q, cache, table, n, sinks=torch.zeros(3, 1, device="cuda")),
        lambda: bsa.paged_select(q, bare, table, n, 3), lambda: bsa.paged_select(q, cache, table, n, 1),
        lambda: bsa.paged_select(q, cache, table, n, 0, first=0, recent=0), lambda: bsa.paged_select(q[:, :3], cache, table, n, 3),
        lambda: bsa.paged_append(cache, k, k, n), lambda: bsa.paged_append(cache, k, k[:1], i32([[0], [16]])),
        lambda: bsa.paged_append(cache, k[..., :32], k[..., :32], i32([[0], [16]])),
        lambda: bsa.paged_resize(table, n, n[:1], None, n, 16, 1), lambda: bsa.paged_resize(table, n, n[:1], n, n, 24, 1), lambda: bsa.paged_resize(table, n, n[:1], n, n, 16, 0),
        lambda: bsa.paged_resize(table, n, n, n, n, 16, 1), lambda: bsa.PagedCache(cache.k, cache.v[:1]),
        lambda: bsa.PagedCache(cache.k, cache.v, cache.bounds[:1]), lambda: bsa.PagedCache(cache.k[:, :, :8], cache.v[:, :, :8]) and bsa.paged_append(
            bsa.PagedCache(cache.k[:, :, :8], cache.v[:, :, :8]), k, k, i32([[0], [16]])),
        lambda: bsa.PagedCache(cache.k[:1].expand(4, 2, 16, 64), cache.v[:4]),
    ]
    for call in bad:
        with pytest.raises((ValueError, bsa.BsaError)):
            call()
    assert bsa.get_device_error() == 0


def test_output_over_the_queries():
    bsa = bsa_()
    lens = [3000, 40]
    cache, table, k, v = paged_batch(bsa, 2, 2, 64, 16, lens, 3)
    q = rows((2, 8, 3, 64), 1).cuda()
    want, lse = check_fwd(bsa, cache, table, k, v, q, lens)
    mine = q.clone()
    got, lse2 = bsa.paged_fwd(mine, cache, table, i32(lens), o=mine)
    assert got is mine and torch.equal(got, want) and torch.equal(lse, lse2)


def test_sequences_that_share_pages():
    bsa = bsa_()
    n = 1000
    cache, table, k, v = paged_batch(bsa, 1, 2, 64, 16, [n], 3)
    B, lens = 70, [n - 13 * b for b in range(70)]
    shared = table.expand(B, -1).contiguous()
    q = rows((B, 4, 1, 64), 1).cuda()
    index = bsa.paged_select(q, cache, shared, i32(lens), 9)
    assert np.array_equal(index.cpu().numpy(), want_select(cache, shared, q, lens, 9, 1, 1))
    kk, vv = k.expand(B, -1, -1, -1), v.expand(B, -1, -1, -1)
    check_fwd(bsa, cache, shared, kk, vv, q, lens)
    check_fwd(bsa, cache, shared, kk, vv, q, lens, select=index.cpu().numpy())


def test_the_same_results_again():
    """Sums run in a fixed order: results repeat bit for bit."""
    bsa = bsa_()
    lens = [5000, 17, 900, 2222]
    cache, table, _, _ = paged_batch(bsa, 4, 2, 128, 32, lens, 3)
    q = rows((4, 8, 2, 128), 1).cuda()
    want = bsa.paged_fwd(q, cache, table, i32(lens))
    for _ in range(10):
        got = bsa.paged_fwd(q, cache, table, i32(lens))
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_range_checked_build():
    """The same kernels in the build that checks pages, slots and records on the device: right, and nothing found."""
    if os.environ.get("BSA_LIBRARY_VARIANT") == "debug":
        pytest.skip("already in it")
    need_gpu()
    from block_sparse_attention_process_gb300 import build as b
    if not os.path.exists(b.LIB_DEBUG):
        b.build(debug=True)
    r = subprocess.run([sys.executable, "-m", "pytest", "-x", "-q", "-m", "gpu", os.path.abspath(__file__), "-k",
                        "test_fwd or test_append or test_select_with or test_sequences or selected"],
                       env=dict(os.environ, BSA_LIBRARY_VARIANT="debug"), capture_output=True, text=True, timeout=900, cwd=ROOT)
    assert r.returncode == 0, r.stdout[-3000:] + r.stderr[-2000:]

"""The cache in pages on the GPU where its rules meet: pages before a window, counts of new tokens that no call can
have, padding between tokens, caps of any size, probabilities that nearly cancel, the joins and walks of large
batches, replayed graphs with a workspace.

Tolerances (none is a measured one).  Scores as in test_gpu_paged: |ds| <= 2^-16 A, A = scale * sum|q k| of the worst
seen key.
"""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

from helpers import ROOT, need_gpu
from oracle import paged
from test_gpu_paged import bsa_, check_fwd, errors, f64, i32, layout, paged_batch, rows, want_select, within

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------ masks and lengths

@pytest.mark.parametrize("page", [16, 32, 64])
@pytest.mark.parametrize("kw", [{"left": 0}, {"left": 47}, {"left": 1000}, {"chunk": 16}, {"chunk": 100}, {"chunk": 1000}])
@pytest.mark.parametrize("G,T", [(2, 3), (16, 3), (3, 1)])
def test_pages_before_the_window_are_not_looked_up(page, kw, G, T):
    """A program that gives back pages behind the window may leave anything in their entries."""
    bsa = bsa_()
    lens = [2000, 85, 3, 1640]
    cache, table, k, v = paged_batch(bsa, 4, 2, 64, page, lens, 7)
    for b, n in enumerate(lens):
        table[b, :paged.first_key(max(n - T, 0), kw.get("left"), kw.get("chunk")) // page] = -1
    q = rows((4, 2 * G, T, 64), 8).cuda()
    check_fwd(bsa, cache, table, k, v, q, lens, **kw)
    assert bsa.get_device_error() == 0


@pytest.mark.parametrize("M", [None, 256])   # a pair whole to a CTA, and cut into runs
def test_counts_of_new_tokens_outside_the_call_are_reported(M):
    bsa = bsa_()
    lens, T = [300, 70], 3
    cache, table, k, v = paged_batch(bsa, 2, 2, 64, 16, lens, 7, M=M)
    q = rows((2, 4, T, 64), 8).cuda()
    for bad, good in ((T + 1, T), (2**31 - 1, T), (-1, 0), (-2**31, 0)):
        for b in range(2):
            given, taken = [2, 2], [2, 2]
            given[b], taken[b] = bad, good
            got = bsa.paged_fwd(q, cache, table, i32(lens), q_lens=i32(given))
            errors(bsa, 2)
            want = check_fwd(bsa, cache, table, k, v, q, lens, q_lens=taken)
            assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
            index = bsa.paged_select(q, cache, table, i32(lens), 4, q_lens=i32(given))
            errors(bsa, 2)
            assert np.array_equal(index.cpu().numpy(), want_select(cache, table, q, lens, 4, 1, 1, taken))
            got = bsa.paged_fwd(q, cache, table, i32(lens), q_lens=i32(given), select=index)
            errors(bsa, 2)
            want = bsa.paged_fwd(q, cache, table, i32(lens), q_lens=i32(taken), select=index)
            assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    for fine in ([0, T], [T, 1]):
        check_fwd(bsa, cache, table, k, v, q, lens, q_lens=fine)
    assert bsa.get_device_error() == 0


# ------------------------------------------------------------------ append

@pytest.mark.parametrize("D,page", [(64, 16), (128, 16), (128, 32), (64, 64), (128, 256)])
def test_padding_between_tokens_leaves_no_bound_too_small(D, page):
    """With bounds, padding belongs behind a sequence's last token.  Elsewhere it is reported, and the bounds hold for
    whatever the page's places contain, those left out among them."""
    bsa = bsa_()
    H, T, M = 2, 3 * page, 4
    cache = bsa.PagedCache.empty(4 * M, H, page, D)
    cache.k.fill_(100.0)    # (what an earlier sequence left)
    starts, holes = [3, 3, 0, page - 1], [[page // 2], [0], [page - 1, page], list(range(page + 1, 2 * page + 1))]
    slots = np.stack([b * M * page + s + np.arange(T) for b, s in enumerate(starts)]).astype(np.int32)
    for b, h in enumerate(holes):
        slots[b, h] = -1 - b
        cache.k[b * M, :, :starts[b]] = 0.0
    k = rows((4, H, T, D), 1).cuda()
    want = f64(cache.k)
    for b in range(4):
        first = {}    # of each page: its first new token
        for t in range(T):
            first.setdefault((starts[b] + t) // page, t)
        stored = [t for t in range(T) if slots[b, t] >= 0 and slots[b, first[(starts[b] + t) // page]] >= 0]
        if slots[b, 0] < 0:   # (no place to count from: the places of no page's first token are known)
            stored = []
        for t in stored:
            want[slots[b, t] // page, :, slots[b, t] % page] = f64(k)[b, :, t]
    bsa.paged_append(cache, k, k, torch.from_numpy(slots).cuda())
    errors(bsa, 2)
    assert np.array_equal(f64(cache.k), want)
    got = f64(cache.bounds)
    for b in range(4):
        for t in range(T):
            p, i = slots[b, t] // page, slots[b, t] % page
            if slots[b, t] >= 0 and np.array_equal(want[p, :, i], f64(k)[b, :, t]):
                held = want[p, :, :i + 1]
                assert (got[p, :, 0] >= held.max(1)).all() and (got[p, :, 1] <= held.min(1)).all()


def test_tokens_out_of_order_leave_no_bound_too_small():
    bsa = bsa_()
    cache = bsa.PagedCache.empty(4, 1, 16, 64)
    cache.k.fill_(100.0)
    cache.k[0, 0, :4] = 0.0
    k = rows((1, 1, 8, 64), 1).cuda()
    slots = torch.arange(4, 12, dtype=torch.int32, device="cuda")[None].clone()
    slots[0, 2] = 60
    bsa.paged_append(cache, k, k, slots)
    errors(bsa, 2)
    held = f64(cache.k)[0, 0, :12]
    assert held[6].tolist() == [100.0] * 64 and held[7].tolist() == f64(k)[0, 0, 3].tolist()
    assert (f64(cache.bounds)[0, 0, 0] >= held.max(0)).all() and (f64(cache.bounds)[0, 0, 1] <= held.min(0)).all()


# ------------------------------------------------------------------ scores and sums

def reference(cache, table, k, v, q, lens, *, q_lens=None, cap=0.0, scale=None):
    """O, LSE, sum p |v| and A of every row, fp64."""
    B, Hq, T, D = q.shape
    want, wl, mass, a = np.zeros((B, Hq, T, D)), np.zeros((B, Hq, T)), np.zeros((B, Hq, T, D)), np.zeros((B, Hq, T))
    qh, kh, vh = f64(q), f64(k), f64(v)
    for b in range(B):
        nq = T if q_lens is None else q_lens[b]
        for h in range(Hq):
            for t in range(T):
                n = max(lens[b] - nq + t + 1, 0) if t < nq else 0
                g = h // (Hq // cache.Hkv)
                want[b, h, t], wl[b, h, t], mass[b, h, t], a[b, h, t] = paged.attend(
                    qh[b, h, t], kh[b, g, :n], vh[b, g, :n], D ** -0.5 if scale is None else scale, cap)
    return want, wl, mass, a


@pytest.mark.parametrize("cap", [1.0, 5.0, 30.0, 1e3, 1e4, 1e6, 1e12, 1e30, 8e37])
@pytest.mark.parametrize("D,G,T", [(64, 4, 1), (128, 4, 1), (128, 16, 2)])
def test_a_cap_of_any_size(cap, D, G, T):
    """A capped score is no further off than its own size allows, however large the cap.

    tanh x as 1 - 2 / (1 + e^2x): e off by 2^-22 (exp2) + 2 |x| 2^-23 (its argument) relative, 1 + e by 2^-24, the reciprocal
    by 2^-23, the difference by 2^-24: 2^-20.8 absolute, of tanh x from 1/4 on 2^-18.8 relative.  Below 1/4 a polynomial, 2^-22
    relative.  |capped| <= A: ds = (2^-16 + 2^-18) A.  Four units in the last place of an exponential 2^-20, of a logarithm and its
    conversion 2^-20 max(1, |lse|)."""
    bsa = bsa_()
    lens = [700, 40]
    cache, table, k, v = paged_batch(bsa, 2, 2, D, 16, lens, 9, scale=2.0)
    q = rows((2, 2 * G, T, D), 10, 2.0).cuda()
    want, wl, mass, a = reference(cache, table, k, v, q, lens, cap=cap)
    ds = (2.0 ** -16 + 2.0 ** -18) * a
    for M in (None, 256):
        wide = table if M is None else torch.cat((table, table.new_full((2, M - table.shape[1]), -1)), 1).contiguous()
        o, lse = bsa.paged_fwd(q, cache, wide, i32(lens), logits_soft_cap=cap)
        within("lse", f64(lse), wl, ds + 2.0 ** -20 * np.maximum(1, np.abs(wl)))
        within("o", f64(o), want, 2.0 ** -8 * np.abs(want) + (2.0 ** -8 + 2 * ds[..., None] + 2.0 ** -19) * mass)
    assert bsa.get_device_error() == 0


def test_caps_and_infinities():
    """A NaN score stays one, an infinite one is the cap itself."""
    bsa = bsa_()
    n = 40
    cache, table, k, v = paged_batch(bsa, 1, 1, 64, 16, [n], 9)
    q = torch.ones((1, 4, 1, 64), dtype=torch.bfloat16, device="cuda")
    for bad, limit in ((float("inf"), 20.0), (-float("inf"), -20.0)):
        k[0, 0, 5] = bad
        cache.k[table[0, 0].long(), 0, 5] = bad
        s = 20.0 * np.tanh((f64(k)[0, 0, :n].sum(1) / 8) / 20.0)
        assert s[5] == limit
        want = np.log(np.exp(s).sum())
        _, lse = bsa.paged_fwd(q, cache, table, i32([n]), logits_soft_cap=20.0)
        a = np.delete(np.abs(f64(k)[0, 0, :n]).sum(1) / 8, 5).max()
        within("lse", f64(lse), np.full((1, 4, 1), want), (2.0 ** -16 + 2.0 ** -18) * max(a, 20.0) + 2.0 ** -20 * max(1, abs(want)))
    cache.k[table[0, 0].long(), 0, 5] = float("nan")
    o, lse = bsa.paged_fwd(q, cache, table, i32([n]), logits_soft_cap=20.0)
    assert torch.isnan(lse).all() and torch.isnan(o.float()).all()


def nearly_cancelling(D, G, seed):
    """q, k, v of two keys: with a_h the probability of key 1 relative to key 0's in head h, v0 is minus a_d rounded to bf16 in
    channel d and v1 is 1, so that O[h, h] is what rounding a_h to bf16 takes off."""
    g = torch.Generator().manual_seed(seed)
    q, k, v = torch.zeros((G, D)), torch.zeros((2, D)), torch.ones((2, D))
    q[:, 0] = -(0.2 + torch.rand(G, generator=g))
    q = q.to(torch.bfloat16)
    k[1, 0] = 1.0
    a = torch.exp(q[:, 0].double())
    v[0, :] = -0.5
    v[0, :min(G, D)] = -a[:D].to(torch.bfloat16).float()
    return q, k.to(torch.bfloat16), v.to(torch.bfloat16)


@pytest.mark.parametrize("D,G", [(64, 3), (64, 16), (128, 16), (64, 32), (128, 31), (64, 64), (128, 64)])
@pytest.mark.parametrize("cut,T", [(False, 1), (True, 1), (False, 2)])
def test_probabilities_are_not_rounded_to_a_value_s_eight_bits(D, G, cut, T):
    """A probability meets its value as two bf16 terms: the first at most 2^-8 + 2^-7 of it away, the second rounded, so
    3 2^-16 off, and the sums of few products 2^-23 each: with ds and an exponential's 2^-19 O is off by bf16's rounding and
    (2^-13 + 2 ds) sum p |v|."""
    bsa = bsa_()
    q, k, v = nearly_cancelling(D, G, G + D)
    page, keys = 16, T + 1
    cache = bsa.PagedCache.empty(3, 1, page, D)
    # key 1 is the last new token's own; with T = 2 the first one does not see it, and one of its values is a NaN
    kk, vv = torch.zeros((1, 1, keys, D), dtype=torch.bfloat16), torch.zeros((1, 1, keys, D), dtype=torch.bfloat16)
    kk[0, 0, 0], kk[0, 0, -1], vv[0, 0, 0], vv[0, 0, -1] = k[0], k[1], v[0], v[1]
    if T == 2:
        kk[0, 0, 1, 0] = 60.0             # between them one far below (q is negative)
    cache.k[1, 0, :keys], cache.v[1, 0, :keys] = kk[0, 0].cuda(), vv[0, 0].cuda()
    if T == 2:
        cache.v[1, 0, 2, D - 1] = float("nan")
    table = i32([[1] + [-1] * (255 if cut else 0)])
    qq = q.view(1, G, 1, D).expand(1, G, T, D).contiguous().cuda()
    o, _ = bsa.paged_fwd(qq, cache, table, i32([keys]), softmax_scale=1.0)
    want, _, mass, a = reference(cache, table, kk, vv, qq, [keys], scale=1.0)
    a = np.minimum(a, 2.0)                # (the key between has no weight: its own error counts for nothing)
    ds = 2.0 ** -16 * a
    c = slice(0, D - 1) if T == 2 else slice(0, D)
    within("o", f64(o)[..., c], want[..., c], (2.0 ** -8 * np.abs(want) + (2.0 ** -13 + 2 * ds[..., None]) * mass)[..., c])
    if T == 2:
        assert torch.isnan(o[:, :, 1, D - 1].float()).all() and torch.isfinite(o[:, :, 0].float()).all()


@pytest.mark.parametrize("bad", [float("inf"), -float("inf")])
@pytest.mark.parametrize("D,G", [(64, 4), (128, 4), (128, 20), (64, 40)])
def test_infinite_values_of_keys_that_all_rows_see(bad, D, G):
    bsa = bsa_()
    n = 300
    cache, table, k, v = paged_batch(bsa, 1, 1, D, 16, [n], 13)
    for key in (0, 17, 298, 299):
        p, i = int(table[0, key // 16]), key % 16
        old = cache.v[p, 0, i, 3].clone()
        cache.v[p, 0, i, 3] = bad
        o, lse = bsa.paged_fwd(rows((1, G, 1, D), 14).cuda(), cache, table, i32([n]))
        assert bool((o[..., 3] == bad).all())
        rest = torch.cat((o[..., :3], o[..., 4:]), -1)
        assert torch.isfinite(rest.float()).all() and torch.isfinite(lse).all()
        cache.v[p, 0, i, 3] = old


# ------------------------------------------------------------------ joins, walks, warps

def workspace(bsa, cache, q, M, keep=0):
    """Bytes that the call needs: none where no pair is cut."""
    import ctypes as C
    a, (B, Hq, T, D) = bsa._abi, q.shape
    I3 = C.c_int64 * 3
    st = I3(Hq * T * D, T * D, D)
    kv = a.PagedCache(cache.k.data_ptr(), cache.v.data_ptr(), I3(*cache.k.stride()[:3]), I3(*cache.v.stride()[:3]), None, cache.pages,
                      cache.Hkv, D, cache.page)
    x = a.PagedFwdArgs(kv, 16, 32, 48, st, st, 64, 80, None, 96 if keep else None, B, Hq, M, T, keep, a.MASK_CAUSAL, -1, 0, float("nan"),
                       0.0, None, 0, 0, None, 0)
    n = C.c_size_t(0)
    assert a.lib().bsa_paged_fwd_workspace(C.byref(x), C.byref(n)) == 0
    return n.value


def sms():
    return torch.cuda.get_device_properties(0).multi_processor_count


@pytest.mark.parametrize("B,H,G,D,T", [
    (45, 1, 2, 64, 1), (70, 1, 3, 128, 1), (45, 2, 20, 64, 1), (70, 1, 9, 128, 2), (40, 1, 70, 64, 1), (39, 1, 40, 128, 1), (33, 3, 5, 64, 5),
    (100, 1, 1, 128, 1), (20, 8, 4, 128, 1),
])
def test_many_sequences_cut_into_runs(B, H, G, D, T):
    """More pairs than a quarter of the SMs (a warp joins a row) and more than 32 sequences (a walk over several lanes' worth), some empty."""
    bsa = bsa_()
    page, M = 16, 256
    lens = [0 if b % 7 == 3 else 1 + 97 * b * b % 700 for b in range(B)]
    q_lens = None if T == 1 else [b % (T + 1) for b in range(B)]
    cache, table, k, v = paged_batch(bsa, B, H, D, page, lens, 17)
    table = torch.cat((table, table.new_full((B, M - table.shape[1]), -1)), 1).contiguous()
    q = rows((B, T, H * G, D), 18).transpose(1, 2).cuda()
    R = G * T
    pairs = B * H * -(-R // (16 if R <= 16 else 32 if R <= 32 else 64))
    assert workspace(bsa, cache, q, M) > 0 and 4 * pairs > sms()
    check_fwd(bsa, cache, table, k, v, q, lens, q_lens=q_lens)
    check_fwd(bsa, cache, table, k, v, q, lens, q_lens=q_lens, cap=25.0, sinks=torch.linspace(-1, 1, H).cuda().view(H, 1))
    assert bsa.get_device_error() == 0


@pytest.mark.parametrize("B,H,G,D,T", [(14, 2, 3, 64, 3), (50, 1, 4, 128, 1), (9, 1, 20, 64, 5), (13, 1, 40, 128, 3)])
def test_many_lists_cut_into_runs(B, H, G, D, T):
    bsa = bsa_()
    page, keep = 64, 70
    lens = [0 if b % 6 == 5 else 1 + 1931 * b % 5000 for b in range(B)]
    cache, table, k, v = paged_batch(bsa, B, H, D, page, lens, 19, M=90)
    q = rows((B, H * G, T, D), 20).cuda()
    assert workspace(bsa, cache, q, 90, keep) > 0 and 4 * B * T * H > sms() and B * T > 32
    select = want_select(cache, table, q, lens, keep, 1, 1)
    got = bsa.paged_select(q, cache, table, i32(lens), keep)
    assert np.array_equal(got.cpu().numpy(), select)
    check_fwd(bsa, cache, table, k, v, q, lens, select=select)
    assert bsa.get_device_error() == 0


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("G", [2, 20, 40])
@pytest.mark.parametrize("cap", [0.0, 25.0])
def test_more_whole_pairs_than_sms(D, G, cap):
    """Pairs that go whole to a CTA of four warps."""
    bsa = bsa_()
    B = sms() + 9
    lens = [1 + 37 * b % 130 for b in range(B)]
    cache, table, k, v = paged_batch(bsa, B, 1, D, 16, lens, 21)
    q = rows((B, G, 1, D), 22).cuda()
    assert workspace(bsa, cache, q, table.shape[1]) == 0
    check_fwd(bsa, cache, table, k, v, q, lens, cap=cap)
    assert bsa.get_device_error() == 0


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("where", ["k", "v"])
@pytest.mark.parametrize("D,H,G,T", [(128, 2, 4, 4), (128, 2, 4, 5), (128, 1, 16, 4), (64, 1, 3, 5)])
def test_what_a_row_does_not_see_does_not_reach_it_in_any_tile(bad, where, D, H, G, T):
    bsa = bsa_()
    n = 600
    for left, key in ((None, n - 2), (None, n - T + 1), (50, n - T - 50), (50, n - T - 48)):
        cache, table, k, v = paged_batch(bsa, 1, H, D, 16, [n], 13)
        c = cache.k if where == "k" else cache.v
        page = table[0, key // 16].long()
        c[page, :, key % 16, 3] = bad
        q = rows((1, H * G, T, D), 14).cuda()
        o, lse = bsa.paged_fwd(q, cache, table, i32([n]), local_left=left)
        sees = [key <= n - T + t and (left is None or key >= n - T + t - left) for t in range(T)]
        assert any(sees) and not all(sees)
        (k if where == "k" else v)[0, :, key, 3] = 1.0
        c[page, :, key % 16, 3] = 1.0
        want_o, want_lse = check_fwd(bsa, cache, table, k, v, q, [n], left=left)
        for t in range(T):
            if not sees[t]:
                assert torch.equal(o[:, :, t], want_o[:, :, t]) and torch.equal(lse[:, :, t], want_lse[:, :, t])
            elif where == "v":
                x = o[0, :, t, 3].float()
                assert bool((torch.isnan(x) if bad != bad else x == bad).all())
                assert torch.isfinite(torch.cat((o[0, :, t, :3], o[0, :, t, 4:]), -1).float()).all() and torch.equal(lse[:, :, t], want_lse[:, :, t])
            elif bad != bad:
                assert torch.isnan(lse[0, :, t]).all() and torch.isnan(o[0, :, t].float()).all()


@pytest.mark.parametrize("B,M", [(3, 300), (45, 256)])    # joined by a CTA a row, and by a warp
def test_replayed_with_a_workspace_and_a_join(B, M):
    """One captured step whose lengths change from replay to replay, two such graphs, other calls between them."""
    bsa = bsa_()
    H, G, D, page = 2, 2, 64, 16
    longest = 900
    cache, table, k, v = paged_batch(bsa, B, H, D, page, [longest] * B, 23, junk=False)
    table = torch.cat((table, table.new_full((B, M - table.shape[1]), -1)), 1).contiguous()
    q = [rows((B, H * G, 1, D), s).cuda() for s in (24, 25)]
    lens = [i32([1] * B) for _ in range(2)]
    assert workspace(bsa, cache, q[0], M) > 0
    graphs, outs = [], []
    for x, n in zip(q, lens):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(bsa.paged_fwd(x, cache, table, n))
        graphs.append(g)
    for step in range(4):
        now = [[(311 * b + 97 * step + 450 * i) % (longest + 1) for b in range(B)] for i in range(2)]
        for i in range(2):
            lens[i].copy_(i32(now[i]))
        for g in graphs:
            g.replay()
        other = bsa.paged_fwd(q[0], cache, table, i32([longest] * B))
        for i in range(2):
            want = check_fwd(bsa, cache, table, k, v, q[i], now[i])
            assert torch.equal(outs[i][0], want[0]) and torch.equal(outs[i][1], want[1])
        del other
    assert bsa.get_device_error() == 0


def test_paths_in_the_range_checked_build():
    """The same calls in the build that checks pages, slots and records on the device: right, and nothing found."""
    if os.environ.get("BSA_LIBRARY_VARIANT") == "debug":
        pytest.skip("already in it")
    need_gpu()
    from block_sparse_attention_process_gb300 import build as b
    if not os.path.exists(b.LIB_DEBUG):
        b.build(debug=True)
    r = subprocess.run([sys.executable, "-m", "pytest", "-x", "-q", "-m", "gpu", os.path.abspath(__file__), "-k",
                        "window or outside or padding_between or runs or whole or replayed"],
                       env=dict(os.environ, BSA_LIBRARY_VARIANT="debug"), capture_output=True, text=True, timeout=900, cwd=ROOT)
    assert r.returncode == 0, r.stdout[-3000:] + r.stderr[-2000:]


def test_without_the_allocator_s_own_call(monkeypatch):
    """Where torch does not offer it, the workspace is a tensor."""
    bsa = bsa_()
    lens = [5000, 17]
    cache, table, _, _ = paged_batch(bsa, 2, 2, 64, 16, lens, 3)
    q = rows((2, 4, 1, 64), 1).cuda()
    assert workspace(bsa, cache, q, table.shape[1]) > 0
    want = bsa.paged_fwd(q, cache, table, i32(lens))
    monkeypatch.setattr(bsa, "_raw_alloc", None)
    monkeypatch.setattr(bsa, "_raw_free", None)
    got = bsa.paged_fwd(q, cache, table, i32(lens))
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])

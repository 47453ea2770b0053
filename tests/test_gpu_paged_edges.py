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

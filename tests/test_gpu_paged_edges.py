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

"""Calls that the entry points of the cache in pages refuse, on the host, before
anything is launched (so they run without a GPU)."""
import ctypes as C
import math

import pytest
import torch

from helpers import ensure_built

I3 = C.c_int64 * 3


def _abi():
    ensure_built()
    from block_sparse_attention_process_gb300 import _abi as a
    return a


def cache(abi, **kw):
    c = abi.PagedCache(1 << 20, 1 << 21, I3(4096, 2048, 128), I3(4096, 2048, 128), 1 << 22, 8, 2, 128, 16)
    for k, v in kw.items():
        setattr(c, k, v)
    return c


def made(a, kw):
    for k, v in kw.items():
        setattr(a, k, v)
    return a


def resize_args(abi, **kw):
    return made(abi.PagedResizeArgs(16, 32, 48, 64, 80, 96, 112, 128, 2, 4, 16, 8, 16), kw)


def append_args(abi, cache_kw=None, **kw):
    return made(abi.PagedAppendArgs(cache(abi, **(cache_kw or {})), 16, 32, I3(256, 128, 128), I3(256, 128, 128), 48, 2, 1), kw)


def select_args(abi, cache_kw=None, **kw):
    return made(abi.PagedSelectArgs(cache(abi, **(cache_kw or {})), 16, I3(512, 128, 128), 32, 48, None, 64, 2, 4, 4, 1, 2, 1, 1), kw)


def fwd_args(abi, cache_kw=None, **kw):
    return made(abi.PagedFwdArgs(cache(abi, **(cache_kw or {})), 16, 32, 48, I3(512, 128, 128), I3(512, 128, 128), 64, 80, None,
                                 None, 2, 4, 64, 1, 0, abi.MASK_CAUSAL, -1, 0, math.nan, 0.0, None, 0, 0, 96, 1 << 40), kw)


def refused(abi, entry, a, status):
    L = abi.lib()
    assert getattr(L, entry)(C.byref(a), None) == getattr(abi, status), L.bsa_last_error()
    assert len(L.bsa_last_error()) > 0


BAD_CACHES = [({"D": 96}, "UNSUPPORTED"), ({"Hkv": 0}, "INVALID_ARG"), ({"page": 24}, "UNSUPPORTED"), ({"page": 8}, "UNSUPPORTED"),
              ({"page": 0}, "UNSUPPORTED"), ({"page": 512}, "UNSUPPORTED"), ({"pages": 0}, "INVALID_ARG"),
              ({"pages": 1 << 27}, "UNSUPPORTED"), ({"bounds": 8}, "INVALID_ARG")]
BAD_ROWS = [({"k": None}, "INVALID_ARG"), ({"v": 8}, "INVALID_ARG"), ({"k_stride": I3(4096, 2048, 4)}, "INVALID_ARG"),
            ({"v_stride": I3(-4096, 2048, 128)}, "INVALID_ARG"), ({"k_stride": I3(0, 2048, 128)}, "INVALID_ARG")]


@pytest.mark.parametrize("kw,status", BAD_CACHES)
@pytest.mark.parametrize("entry,make", [("bsa_paged_append", append_args), ("bsa_paged_select", select_args), ("bsa_paged_fwd", fwd_args)])
def test_bad_caches(entry, make, kw, status):
    abi = _abi()
    refused(abi, entry, make(abi, cache_kw=kw), status)


@pytest.mark.parametrize("kw,status", BAD_ROWS)
@pytest.mark.parametrize("entry,make", [("bsa_paged_append", append_args), ("bsa_paged_fwd", fwd_args)])
def test_bad_cache_rows(entry, make, kw, status):
    abi = _abi()
    refused(abi, entry, make(abi, cache_kw=kw), status)


@pytest.mark.parametrize("kw,status", [
    ({"table": None}, "INVALID_ARG"), ({"free_pages": 2}, "INVALID_ARG"), ({"used": None}, "INVALID_ARG"), ({"lens": None}, "INVALID_ARG"),
    ({"new_lens": 6}, "INVALID_ARG"), ({"lens_out": None}, "INVALID_ARG"), ({"slots": None}, "INVALID_ARG"),
    ({"lens_out": 64}, "INVALID_ARG"), ({"lens_out": 80}, "INVALID_ARG"), ({"used_out": 48}, "INVALID_ARG"),
    ({"slots": 16}, "INVALID_ARG"), ({"slots": 96}, "INVALID_ARG"), ({"free_pages": 16}, "INVALID_ARG"), ({"B": 0}, "INVALID_ARG"),
    ({"B": 4097}, "UNSUPPORTED"), ({"M": 0}, "INVALID_ARG"), ({"M": 1 << 27}, "UNSUPPORTED"), ({"T": 0}, "INVALID_ARG"),
    ({"T": 1 << 30}, "UNSUPPORTED"), ({"pages": 0}, "INVALID_ARG"), ({"pages": 1 << 27}, "UNSUPPORTED"), ({"page": 48}, "UNSUPPORTED"),
])
def test_resize_refuses(kw, status):
    abi = _abi()
    refused(abi, "bsa_paged_resize", resize_args(abi, **kw), status)


@pytest.mark.parametrize("kw,status", [
    ({"k": None}, "INVALID_ARG"), ({"v": 8}, "INVALID_ARG"), ({"slots": None}, "INVALID_ARG"), ({"slots": 50}, "INVALID_ARG"),
    ({"B": 0}, "INVALID_ARG"), ({"T": 0}, "INVALID_ARG"), ({"T": 1 << 30}, "UNSUPPORTED"), ({"src_k_stride": I3(256, 128, 4)}, "INVALID_ARG"),
    ({"src_v_stride": I3(1, 128, 128)}, "INVALID_ARG"),
])
def test_append_refuses(kw, status):
    abi = _abi()
    refused(abi, "bsa_paged_append", append_args(abi, **kw), status)


@pytest.mark.parametrize("kw,status", [
    ({"q": None}, "INVALID_ARG"), ({"q": 8}, "INVALID_ARG"), ({"table": None}, "INVALID_ARG"), ({"lens": 2}, "INVALID_ARG"),
    ({"q_lens": 2}, "INVALID_ARG"), ({"index": None}, "INVALID_ARG"), ({"Hq": 3}, "INVALID_ARG"), ({"B": 0}, "INVALID_ARG"),
    ({"T": 0}, "INVALID_ARG"), ({"T": 1 << 30}, "UNSUPPORTED"), ({"M": 0}, "INVALID_ARG"), ({"M": 1 << 27}, "UNSUPPORTED"),
    ({"keep": 0, "first": 0, "recent": 0}, "INVALID_ARG"), ({"keep": 1}, "INVALID_ARG"), ({"first": -1}, "INVALID_ARG"),
    ({"recent": -1}, "INVALID_ARG"), ({"recent": 1 << 62}, "INVALID_ARG"), ({"keep": 1 << 40}, "UNSUPPORTED"),
    ({"q_stride": I3(512, 12, 128)}, "INVALID_ARG"), ({"M": 49153}, "UNSUPPORTED"),
])
def test_select_refuses(kw, status):
    abi = _abi()
    refused(abi, "bsa_paged_select", select_args(abi, **kw), status)


def test_select_needs_bounds():
    abi = _abi()
    refused(abi, "bsa_paged_select", select_args(abi, cache_kw={"bounds": None}), "INVALID_ARG")


@pytest.mark.parametrize("kw,status", [
    ({"q": None}, "INVALID_ARG"), ({"o": 8}, "INVALID_ARG"), ({"lse": None}, "INVALID_ARG"), ({"lens": None}, "INVALID_ARG"),
    ({"table": None}, "INVALID_ARG"), ({"table": 2}, "INVALID_ARG"), ({"lens": 2}, "INVALID_ARG"), ({"q_lens": 2}, "INVALID_ARG"),
    ({"Hq": 3}, "INVALID_ARG"), ({"Hq": 0}, "INVALID_ARG"), ({"B": 0}, "INVALID_ARG"), ({"T": 0}, "INVALID_ARG"),
    ({"T": 1 << 30}, "UNSUPPORTED"), ({"M": 0}, "INVALID_ARG"), ({"M": 1 << 27}, "UNSUPPORTED"), ({"kind": 0}, "UNSUPPORTED"),
    ({"kind": 4}, "UNSUPPORTED"), ({"kind": 2, "local_left": -2}, "INVALID_ARG"), ({"kind": 3, "chunk": 0}, "INVALID_ARG"),
    ({"select": 112, "keep": 0}, "INVALID_ARG"), ({"select": 114, "keep": 2}, "INVALID_ARG"),
    ({"select": 112, "keep": 2, "kind": 2}, "UNSUPPORTED"), ({"select": 112, "keep": 1 << 28}, "UNSUPPORTED"),
    ({"q_stride": I3(512, 128, 4)}, "INVALID_ARG"), ({"o_stride": I3(512, 0, 128)}, "INVALID_ARG"),
    ({"logits_soft_cap": -1.0}, "INVALID_ARG"), ({"logits_soft_cap": math.inf}, "INVALID_ARG"), ({"softmax_scale": math.inf}, "INVALID_ARG"),
    ({"logits_soft_cap": 1e-30, "softmax_scale": 1e9}, "INVALID_ARG"), ({"logits_soft_cap": math.nan}, "INVALID_ARG"),
    ({"num_sinks": 65, "sinks": 96}, "UNSUPPORTED"), ({"num_sinks": 2}, "INVALID_ARG"), ({"num_sinks": 2, "sinks": 98}, "INVALID_ARG"),
    ({"M": 4096, "workspace": None}, "INVALID_ARG"), ({"M": 4096, "workspace": 8}, "INVALID_ARG"),
    ({"M": 4096, "workspace_bytes": 64}, "INVALID_ARG"),  # (sequences that long are cut into runs)
])
def test_fwd_refuses(kw, status):
    abi = _abi()
    refused(abi, "bsa_paged_fwd", fwd_args(abi, **kw), status)


@pytest.mark.parametrize("entry", ["bsa_paged_resize", "bsa_paged_append", "bsa_paged_select", "bsa_paged_fwd"])
def test_null_args(entry):
    abi = _abi()
    assert getattr(abi.lib(), entry)(None, None) == abi.INVALID_ARG


def test_binding_refuses_before_the_library():
    _abi()
    import block_sparse_attention_process_gb300 as bsa
    cpu = torch.zeros((4, 2, 16, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        bsa.PagedCache(cpu, cpu)
    t = torch.zeros((2, 4), dtype=torch.int32)
    with pytest.raises(ValueError):
        bsa.paged_resize(t, t[0], t[0, :1], t[:, 0], t[:, 1], 16, 1)

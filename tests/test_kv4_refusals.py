"""Calls that the entry points after the prompt refuse, on the host, before
anything is launched (so they run without a GPU)."""
import ctypes as C
import math

import pytest
import torch

from helpers import ensure_built


def _abi():
    ensure_built()
    from block_sparse_attention_process_gb300 import _abi as a
    return a


def cache(abi, base=1 << 20, **kw):
    c = abi.Kv4Cache(base, base + 16, base + 32, base + 48, base + 64, base + 80, 2, 2, 128, 64)
    for k, v in kw.items():
        setattr(c, k, v)
    return c


def append_args(abi, cache_kw=None, **kw):
    a = abi.Kv4AppendArgs(cache(abi, **(cache_kw or {})), 16, 32, (256, 128, 128), (256, 128, 128), 1, 48, None, None, None,
                          None, None)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


def fwd_args(abi, cache_kw=None, **kw):
    a = abi.Kv4FwdArgs(cache(abi, **(cache_kw or {})), 16, 32, 48, (512, 128, 128), (512, 128, 128), 4, 1, 64, None,
                       math.nan, 0.0, None, 0, 0, 0, 80, 1 << 40)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


def evict_args(abi, cache_kw=None, out_kw=None, **kw):
    a = abi.Kv4EvictArgs(cache(abi, **(cache_kw or {})), cache(abi, 1 << 21, **(out_kw or {})), 16, None, 32, 8, 32, 48,
                         None, None, 64, 1 << 40)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


def weights_args(abi, **kw):
    a = abi.KeyWeightsArgs(16, 32, 48, None, 64, 80, 1 << 40, 1, 4, 2, 128, 256, 256, math.nan, 0.0)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


BAD_CACHES = [
    ({"D": 96}, "UNSUPPORTED"), ({"B": 0}, "INVALID_ARG"), ({"Hkv": -1}, "INVALID_ARG"),
    ({"capacity": 0}, "INVALID_ARG"), ({"capacity": 72}, "INVALID_ARG"), ({"capacity": (1 << 30) + 16}, "UNSUPPORTED"),
    ({"B": 1 << 20, "Hkv": 1 << 20}, "UNSUPPORTED"), ({"k_codes": None}, "INVALID_ARG"), ({"v_scales": 8}, "INVALID_ARG"),
    ({"weights": 6}, "INVALID_ARG"), ({"positions": 6}, "INVALID_ARG"),
]


@pytest.mark.parametrize("kw,status", BAD_CACHES)
@pytest.mark.parametrize("entry,make", [("bsa_kv4_append", append_args), ("bsa_kv4_fwd", fwd_args),
                                        ("bsa_kv4_evict", evict_args)])
def test_bad_caches(entry, make, kw, status):
    abi = _abi()
    L = abi.lib()
    a = make(abi, cache_kw=kw)
    assert getattr(L, entry)(C.byref(a), None) == getattr(abi, status), L.bsa_last_error()
    assert len(L.bsa_last_error()) > 0


@pytest.mark.parametrize("kw,status", [
    ({"k": None}, "INVALID_ARG"), ({"v": 8}, "INVALID_ARG"), ({"start": None}, "INVALID_ARG"), ({"start": 2}, "INVALID_ARG"),
    ({"T": 0}, "INVALID_ARG"), ({"T": 1 << 30}, "UNSUPPORTED"), ({"k_stride": (C.c_int64 * 3)(256, 128, 4)}, "INVALID_ARG"),
    ({"v_stride": (C.c_int64 * 3)(1, 128, 128)}, "INVALID_ARG"), ({"k_values": 8}, "INVALID_ARG"),
    ({"weights0": 2}, "INVALID_ARG"), ({"n_new": 2}, "INVALID_ARG"), ({"first_position": 2}, "INVALID_ARG"),
])
def test_append_refuses(kw, status):
    abi = _abi()
    a = append_args(abi, **kw)
    assert abi.lib().bsa_kv4_append(C.byref(a), None) == getattr(abi, status), abi.lib().bsa_last_error()


@pytest.mark.parametrize("kw,status", [
    ({"q": None}, "INVALID_ARG"), ({"o": 8}, "INVALID_ARG"), ({"lse": None}, "INVALID_ARG"), ({"lens": None}, "INVALID_ARG"),
    ({"lens": 2}, "INVALID_ARG"), ({"q_lens": 2}, "INVALID_ARG"), ({"Hq": 3}, "INVALID_ARG"), ({"Hq": 0}, "INVALID_ARG"),
    ({"T": 0}, "INVALID_ARG"), ({"T": 1 << 30}, "UNSUPPORTED"), ({"q_stride": (C.c_int64 * 3)(512, 128, 4)}, "INVALID_ARG"),
    ({"o_stride": (C.c_int64 * 3)(512, 12, 128)}, "INVALID_ARG"), ({"logits_soft_cap": -1.0}, "INVALID_ARG"),
    ({"logits_soft_cap": math.inf}, "INVALID_ARG"), ({"num_sinks": 65, "sinks": 96}, "UNSUPPORTED"),
    ({"num_sinks": 2}, "INVALID_ARG"), ({"num_sinks": 2, "sinks": 98}, "INVALID_ARG"), ({"accumulate": 2}, "INVALID_ARG"),
])
def test_fwd_refuses(kw, status):
    abi = _abi()
    a = fwd_args(abi, **kw)
    assert abi.lib().bsa_kv4_fwd(C.byref(a), None) == getattr(abi, status), abi.lib().bsa_last_error()


def test_fwd_needs_weights_to_accumulate_and_its_workspace():
    abi = _abi()
    L = abi.lib()
    a = fwd_args(abi, cache_kw={"weights": None}, accumulate=1)
    assert L.bsa_kv4_fwd(C.byref(a), None) == abi.INVALID_ARG and b"weights" in L.bsa_last_error()
    need = C.c_size_t(0)
    a = fwd_args(abi, accumulate=1)
    assert L.bsa_kv4_fwd_workspace(C.byref(a), C.byref(need)) == abi.OK and need.value > 0
    a.workspace_bytes = need.value - 1
    assert L.bsa_kv4_fwd(C.byref(a), None) == abi.INVALID_ARG and b"workspace" in L.bsa_last_error()
    a = fwd_args(abi, accumulate=1, workspace=8)
    assert L.bsa_kv4_fwd(C.byref(a), None) == abi.INVALID_ARG
    assert L.bsa_kv4_fwd_workspace(C.byref(a), None) == abi.INVALID_ARG


@pytest.mark.parametrize("kw,status", [
    ({"keep": 0}, "INVALID_ARG"), ({"keep": 65}, "INVALID_ARG"), ({"recent": -1}, "INVALID_ARG"), ({"recent": 33}, "INVALID_ARG"),
    ({"lens": None}, "INVALID_ARG"), ({"new_lens": None}, "INVALID_ARG"), ({"new_lens": 16}, "INVALID_ARG"),
    ({"index": None}, "INVALID_ARG"), ({"index": 50}, "INVALID_ARG"), ({"seen": 2}, "INVALID_ARG"),
    ({"k_values": 8}, "INVALID_ARG"),
    ({"cache_kw": {"weights": None}}, "INVALID_ARG"),
    ({"out_kw": {"Hkv": 1}}, "INVALID_ARG"), ({"out_kw": {"D": 64}}, "INVALID_ARG"),
    ({"out_kw": {"k_codes": 1 << 20}}, "INVALID_ARG"),                   # one shared buffer
    ({"out_kw": {"weights": (1 << 20) + 64}}, "INVALID_ARG"),
])
def test_evict_refuses(kw, status):
    abi = _abi()
    a = evict_args(abi, **{"keep": 32, **kw})
    assert abi.lib().bsa_kv4_evict(C.byref(a), None) == getattr(abi, status), abi.lib().bsa_last_error()


def test_evict_in_place_needs_positions_and_the_whole_cache():
    abi = _abi()
    L = abi.lib()
    a = evict_args(abi, cache_kw={"positions": None}, recent=4)
    a.out = a.cache
    assert L.bsa_kv4_evict(C.byref(a), None) == abi.INVALID_ARG and b"positions" in L.bsa_last_error()
    a = evict_args(abi)
    a.out = a.cache
    a.out.capacity = 48
    assert L.bsa_kv4_evict(C.byref(a), None) == abi.INVALID_ARG
    a.out.capacity = 64
    a.workspace_bytes = 0
    assert L.bsa_kv4_evict(C.byref(a), None) == abi.INVALID_ARG and b"workspace" in L.bsa_last_error()


@pytest.mark.parametrize("kw,status", [
    ({"B": 0}, "INVALID_ARG"), ({"Hq": 3}, "INVALID_ARG"), ({"S_q": 200}, "INVALID_ARG"), ({"S_kv": 0}, "INVALID_ARG"),
    ({"D": 96}, "UNSUPPORTED"), ({"logits_soft_cap": math.nan}, "INVALID_ARG"), ({"q": None}, "INVALID_ARG"),
    ({"Hq": 2, "Hkv": 1, "S_q": (1 << 23) + 128}, "UNSUPPORTED"),
    ({"lse": 8}, "INVALID_ARG"), ({"q_lens": 2}, "INVALID_ARG"), ({"weights": None}, "INVALID_ARG"),
    ({"S_q": 1 << 30}, "UNSUPPORTED"),
])
def test_key_weights_refuses(kw, status):
    abi = _abi()
    a = weights_args(abi, **kw)
    L = abi.lib()
    assert L.bsa_key_weights(C.byref(a), C.c_void_p(1), None) == getattr(abi, status), L.bsa_last_error()


def test_key_weights_needs_a_maskinfo():
    abi = _abi()
    a = weights_args(abi)
    assert abi.lib().bsa_key_weights(C.byref(a), None, None) == abi.INVALID_ARG
    need = C.c_size_t(0)
    assert abi.lib().bsa_key_weights_workspace(C.byref(a), None, C.byref(need)) == abi.INVALID_ARG


def test_the_binding_refuses_tensors_on_the_cpu():
    ensure_built()
    import block_sparse_attention_process_gb300 as bsa
    with pytest.raises(ValueError, match="CUDA"):
        bsa.KV4Cache.empty(1, 1, 16, 64, device="cpu")
    q = torch.zeros((1, 2, 128, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        bsa.key_weights(q, q, torch.zeros((1, 2, 128)), None)


def test_evict_refuses_to_write_the_lengths_over_those_it_reads():
    abi = _abi()
    L = abi.lib()
    a = evict_args(abi, seen=32)             # (where new_lens is)
    assert L.bsa_kv4_evict(C.byref(a), None) == abi.INVALID_ARG and b"seen" in L.bsa_last_error()


@pytest.mark.parametrize("axis", [0, 1, 2])
def test_fwd_refuses_outputs_of_several_rows_in_one_place(axis):
    abi = _abi()
    L = abi.lib()
    strides = [512, 128, 128]
    strides[axis] = 0
    a = fwd_args(abi, o_stride=(C.c_int64 * 3)(*strides))
    if axis == 2:
        a.T = 2
        a.o_stride[1] = 256
    assert L.bsa_kv4_fwd(C.byref(a), None) == abi.INVALID_ARG and b"one place" in L.bsa_last_error()

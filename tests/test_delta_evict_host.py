"""Refusals of the delta rule's extend and step and of the eviction calls: everything that the
host can see is returned as a status before anything is enqueued (no GPU needed)."""
import ctypes

import pytest
import torch

import block_sparse_attention_40_b200 as qsa
from block_sparse_attention_40_b200 import binding as B

GOOD = 0x10000


def _p(v):
    return None if v is None else ctypes.c_void_p(v)


def _extend(q=GOOD, la=GOOD, cu=(0, 64), d_cu=GOOD, key_heads=2, heads=4, states=GOOD, slots=3,
            slot_ptr=GOOD, out=GOOD, ws=GOOD, ws_bytes=1 << 30):
    h = (ctypes.c_int32 * len(cu))(*cu)
    r = qsa.load().qsa_gated_deltanet_extend(
        _p(q), _p(GOOD), _p(GOOD), _p(la), _p(GOOD), _p(d_cu), h, len(cu) - 1, key_heads, heads,
        _p(states), slots, _p(slot_ptr), _p(out), _p(ws), ws_bytes, None)
    return B.STATUS[r]


@pytest.mark.parametrize("kw,want", [
    (dict(q=None), "QSA_ERR_INVALID_ARG"), (dict(q=GOOD + 2), "QSA_ERR_ALIGNMENT"),
    (dict(la=None), "QSA_ERR_INVALID_ARG"), (dict(la=GOOD + 2), "QSA_ERR_ALIGNMENT"),
    (dict(states=GOOD + 4), "QSA_ERR_ALIGNMENT"), (dict(out=None), "QSA_ERR_INVALID_ARG"),
    (dict(cu=(1, 64)), "QSA_ERR_INVALID_ARG"), (dict(cu=(0, 9, 8)), "QSA_ERR_INVALID_ARG"),
    (dict(d_cu=None), "QSA_ERR_INVALID_ARG"), (dict(key_heads=3), "QSA_ERR_INVALID_ARG"),
    (dict(key_heads=0), "QSA_ERR_INVALID_ARG"), (dict(heads=257, key_heads=257),
                                                 "QSA_ERR_INVALID_ARG"),
    (dict(slots=0), "QSA_ERR_INVALID_ARG"),
    (dict(cu=(0, 1, 2), slots=1, slot_ptr=None), "QSA_ERR_INVALID_ARG"),
    (dict(slot_ptr=GOOD + 2), "QSA_ERR_ALIGNMENT"), (dict(ws=None), "QSA_ERR_INVALID_ARG"),
    (dict(ws=GOOD + 8), "QSA_ERR_ALIGNMENT"), (dict(ws_bytes=16), "QSA_ERR_WORKSPACE"),
    (dict(cu=(0, 0, 0)), "QSA_OK"),      # nothing to do: nothing is enqueued
])
def test_extend_refusals(kw, want):
    assert _extend(**kw) == want


def test_extend_workspace_size_refuses():
    size = qsa.load().qsa_gated_deltanet_extend_workspace_size
    cu = (ctypes.c_int32 * 2)(0, 1000)
    assert size(cu, 1, 2, 4) >= 256
    for bad in ((cu, 0, 2, 4), (cu, 1, 3, 4), (cu, 1, 0, 4), (None, 1, 2, 4),
                ((ctypes.c_int32 * 2)(0, -1), 1, 2, 4)):
        assert size(*bad) == 0


def _step(q=GOOD, batch=2, n_new=1, counts=GOOD, key_heads=2, heads=4, states=GOOD, num_slots=3,
          slots=GOOD):
    r = qsa.load().qsa_gated_deltanet_step(_p(q), _p(GOOD), _p(GOOD), _p(GOOD), _p(GOOD), batch,
                                           n_new, _p(counts), key_heads, heads, _p(states),
                                           num_slots, _p(slots), _p(GOOD), None)
    return B.STATUS[r]


@pytest.mark.parametrize("kw,want", [
    (dict(q=None), "QSA_ERR_INVALID_ARG"), (dict(q=GOOD + 8), "QSA_ERR_ALIGNMENT"),
    (dict(batch=0), "QSA_ERR_INVALID_ARG"), (dict(batch=65536), "QSA_ERR_INVALID_ARG"),
    (dict(n_new=-1), "QSA_ERR_INVALID_ARG"), (dict(counts=GOOD + 1), "QSA_ERR_ALIGNMENT"),
    (dict(heads=5), "QSA_ERR_INVALID_ARG"), (dict(num_slots=0), "QSA_ERR_INVALID_ARG"),
    (dict(slots=None, num_slots=1), "QSA_ERR_INVALID_ARG"), (dict(n_new=0), "QSA_OK"),
])
def test_step_refusals(kw, want):
    assert _step(**kw) == want


# (64 tokens x 4 heads: 64 KB of v and out, 32 KB of q and k, 1 KB of gates, 768 KB of states)
@pytest.mark.parametrize("field,at", [
    ("q", 0x200000), ("k", 0x200000 + 65536 - 16), ("v", 0x200000 + 16), ("la", 0x200000 + 4),
    ("beta", 0x200000 - 1020), ("states", 0x200000 - 786432 + 16), ("q", 0x800000 + 786432 - 16),
    ("v", 0x800000 - 65536 + 16), ("la", 0x800000), ("out", 0x800000)])
@pytest.mark.parametrize("call", ["extend", "step"])
def test_delta_overlaps_are_refused(call, field, at):
    p = dict(q=0x2000000, k=0x2100000, v=0x2200000, la=0x2300000, beta=0x2400000, out=0x200000,
             states=0x800000)
    p[field] = at
    lib = qsa.load()
    lead = [_p(p[x]) for x in ("q", "k", "v", "la", "beta")]
    if call == "extend":
        h = (ctypes.c_int32 * 2)(0, 64)
        r = lib.qsa_gated_deltanet_extend(*lead, _p(GOOD), h, 1, 2, 4, _p(p["states"]), 3, _p(GOOD),
                                          _p(p["out"]), _p(0x4000000), 1 << 30, None)
    else:
        r = lib.qsa_gated_deltanet_step(*lead, 2, 32, None, 2, 4, _p(p["states"]), 3, _p(GOOD),
                                        _p(p["out"]), None)
    assert B.STATUS[r] == "QSA_ERR_INVALID_ARG"


def _cache(batch=2, cap=64, k=GOOD, length=GOOD):
    return B.CacheDesc(k, GOOD, GOOD, GOOD, length, batch, cap)


@pytest.mark.parametrize("kw,want", [
    (dict(q=None), "QSA_ERR_INVALID_ARG"), (dict(q=GOOD + 2), "QSA_ERR_ALIGNMENT"),
    (dict(mass=GOOD + 4), "QSA_ERR_ALIGNMENT"), (dict(topk=0), "QSA_ERR_INVALID_ARG"),
    (dict(topk=1025), "QSA_ERR_INVALID_ARG"), (dict(ws_bytes=16), "QSA_ERR_WORKSPACE"),
    (dict(cache=_cache(cap=66)), "QSA_ERR_INVALID_ARG"),
    (dict(cache=_cache(batch=0)), "QSA_ERR_INVALID_ARG"),
    (dict(cache=_cache(k=None)), "QSA_ERR_INVALID_ARG"),
])
def test_accumulate_refusals(kw, want):
    a = dict(q=GOOD, cache=_cache(), idx=GOOD, cnt=GOOD, topk=16, mass=GOOD, ws=GOOD,
             ws_bytes=1 << 20)
    a.update(kw)
    r = qsa.load().qsa_accumulate_weights(_p(a["q"]), ctypes.byref(a["cache"]), _p(a["idx"]),
                                          _p(a["cnt"]), a["topk"], _p(a["mass"]), _p(a["ws"]),
                                          a["ws_bytes"], None)
    assert B.STATUS[r] == want


@pytest.mark.parametrize("kw,want", [
    (dict(mass=None), "QSA_ERR_INVALID_ARG"), (dict(keep=0), "QSA_ERR_INVALID_ARG"),
    (dict(sinks=-1), "QSA_ERR_INVALID_ARG"), (dict(sinks=5, recent=4), "QSA_ERR_INVALID_ARG"),
    (dict(recent=9), "QSA_ERR_INVALID_ARG"), (dict(kept=GOOD + 4), "QSA_ERR_ALIGNMENT"),
    (dict(keep=1 << 20), "QSA_ERR_INVALID_ARG"), (dict(ws_bytes=256), "QSA_ERR_WORKSPACE"),
    (dict(cache=_cache(length=GOOD + 4)), "QSA_ERR_ALIGNMENT"),
])
def test_evict_refusals(kw, want):
    a = dict(cache=_cache(), mass=GOOD, keep=8, sinks=1, recent=2, kept=GOOD, ws=GOOD,
             ws_bytes=1 << 20)
    a.update(kw)
    r = qsa.load().qsa_evict(ctypes.byref(a["cache"]), _p(a["mass"]), a["keep"], a["sinks"],
                             a["recent"], _p(a["kept"]), _p(a["ws"]), a["ws_bytes"], None)
    assert B.STATUS[r] == want


def test_evict_workspace_and_paged_refusals():
    lib = qsa.load()
    c = _cache(batch=4, cap=1024)
    assert lib.qsa_evict_workspace_size(ctypes.byref(c), 100, 1, 2) >= 256 + 4 * 101 * 4
    assert lib.qsa_evict_workspace_size(ctypes.byref(c), 100, 60, 60) == 0
    bad = B.PagedCacheDesc(c, GOOD, 500, 8)
    r = lib.qsa_evict_paged(ctypes.byref(bad), _p(GOOD), 8, 0, 0, None, _p(GOOD), 1 << 20, None)
    assert B.STATUS[r] == "QSA_ERR_INVALID_ARG"
    r = lib.qsa_accumulate_weights_paged(_p(GOOD), ctypes.byref(bad), _p(GOOD), _p(GOOD), 16,
                                         _p(GOOD), _p(GOOD), 1 << 20, None)
    assert B.STATUS[r] == "QSA_ERR_INVALID_ARG"


def test_binding_refuses_cpu_tensors():
    x = torch.zeros((2, 1, 4, 128), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        qsa.gated_deltanet_step(x, x, x, x, x, x)
    with pytest.raises(ValueError, match="CUDA"):
        qsa.gated_deltanet_extend(x[:, 0], x[:, 0], x[:, 0], x, x, [0, 2], x)

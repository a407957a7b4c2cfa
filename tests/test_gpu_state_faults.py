"""Waits of the delta rule's scan and join and of eviction's move that run out, without faulting the
GPU: qsa_set_debug_fault leaves out one post and gives the call's waits a limit of 1 ms.  The call
reports QSA_ERR_TIMEOUT at the wait's site and unwinds; the next calls run clean."""
import time

import pytest
import torch

import block_sparse_attention_40_b200 as qsa
from block_sparse_attention_40_b200 import binding as B
from tests.gpu_helpers import needs_gpu
from tests.test_gpu_delta import DEV, _draw
from tests.test_gpu_evict import _cache, _mass

pytestmark = [pytest.mark.gpu, needs_gpu]


class _Fault:
    def __init__(self, kind):
        self.kind = kind

    def __enter__(self):
        assert B.load().qsa_set_debug_fault(self.kind) == 0

    def __exit__(self, *_):
        assert B.load().qsa_set_debug_fault(0) == 0


# one walk; several sequences and heads; a cut sequence, in its first walk, and in its join
@pytest.mark.parametrize("lens,heads,kind,sites", [
    ([100], 1, 1, range(330, 350)), ([200, 70], 4, 1, range(330, 350)),
    ([5000], 2, 1, range(330, 350)), ([5000], 2, 2, [350])])
def test_extend_wait_runs_out(lens, heads, kind, sites):
    w, states = _draw(lens, heads, heads, len(lens), seed=80)
    args = (w.q, w.k, w.v, w.log_alpha, w.beta)
    start, want = states.clone(), states.clone()
    ref = qsa.DeltaExtend(w.cu_seqlens, heads, DEV).run(*args, want)
    ctx = qsa.DeltaExtend(w.cu_seqlens, heads, DEV)
    torch.cuda.synchronize()
    t0 = time.perf_counter()
    with _Fault(kind):
        ctx.run(*args, states)
    torch.cuda.synchronize()
    assert time.perf_counter() - t0 < 1.0      # waits of 1 ms, not of 2 s
    status, site = ctx.device_error()
    assert status == "QSA_ERR_TIMEOUT" and site in sites
    # the same context right after, its tensor memory and shared memory free again
    states.copy_(start)
    out = ctx.run(*args, states)
    torch.cuda.synchronize()
    assert torch.equal(out, ref) and torch.equal(states, want)
    clean = qsa.DeltaExtend(w.cu_seqlens, heads, DEV)
    clean.run(*args, states)
    assert clean.device_error() == ("QSA_OK", 0)


def test_extend_faults_leave_other_calls_alone():
    # fault 2 in a call without a join, fault 3 in an extend: nothing happens
    w, states = _draw([100], 2, 2, 1, seed=81)
    ctx = qsa.DeltaExtend(w.cu_seqlens, 2, DEV)
    for kind in (2, 3):
        with _Fault(kind):
            ctx.run(w.q, w.k, w.v, w.log_alpha, w.beta, states)
        assert ctx.device_error() == ("QSA_OK", 0)


def test_evict_wait_runs_out():
    mass = _mass((2, 512), 83, "plain").to(DEV)
    mass[0, 3] = 0.0      # something goes near the front, so that blocks move over the first tile
    ev = qsa.Evictor(_cache([2000, 1500], 2048, 0, seed=82), 300, 0, 5, mass=mass)
    torch.cuda.synchronize()
    t0 = time.perf_counter()
    with _Fault(3):
        ev.evict()
    torch.cuda.synchronize()
    assert time.perf_counter() - t0 < 1.0
    assert ev.device_error() == ("QSA_ERR_TIMEOUT", 313)
    twins = [_cache([2000, 1500], 2048, 0, seed=82) for _ in range(2)]
    runs = [qsa.Evictor(c, 300, 0, 5, mass=_mass((2, 512), 83, "plain").to(DEV)) for c in twins]
    for r in runs:
        r.evict()
        assert r.device_error() == ("QSA_OK", 0)
    assert torch.equal(twins[0].k_blocks, twins[1].k_blocks)


def test_unknown_faults_are_refused():
    assert B.STATUS[B.load().qsa_set_debug_fault(4)] == "QSA_ERR_INVALID_ARG"

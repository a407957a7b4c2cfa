"""GPU parity of the gated delta rule from and to a pool of states (extend, step) against the
fp64 token-by-token oracle.

Tolerances, for unit-norm keys and queries and R the largest row norm of the states of the
sequence and head (start or end; a state's row is a sum of at most unit-norm writes):
* states (fp32): a token rounds a*s and the fused write once each and the dot S k in at most 19
  steps (16 in sequence, 3 joins), 21 half steps of 2^-24 relative to R; gates of mean 0.95 or
  less keep about 20 tokens of such errors: 420, taken as 512 * 2^-24 * R.
* out (bf16): half a step, 2^-8 of the value, and the state's own error.  In chunks the operands
  that feed only the output may be rounded to 11 bits once each: two half steps of 2^-11 more,
  2^-10 * R.
"""
import numpy as np
import pytest
import torch

import block_sparse_attention_40_b200 as qsa
from block_sparse_attention_40_b200 import workloads as W
from oracle.gated_deltanet import gated_delta_rule
from tests.gpu_helpers import needs_gpu

pytestmark = [pytest.mark.gpu, needs_gpu]
DEV = "cuda:0"
STATE_TOL = 512 * 2.0 ** -24


def _np(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def _draw(lens, heads, key_heads, slots, seed, gate=(0.9, 1.0), reset_every=0, state=0.3):
    w = W.gated_deltanet(lens, heads, seed=seed, gate=gate, reset_every=reset_every)
    w.q, w.k = w.q[:, :key_heads].contiguous(), w.k[:, :key_heads].contiguous()
    g = torch.Generator().manual_seed(seed + 91)
    states = state * torch.randn((slots, heads, 128, 128), generator=g)
    return w.to(DEV), states.to(DEV)


def _compare(got_out, got_state, w, a, b, start, chunked):
    """Tokens a..b-1 of w from `start` [H, 128, 128] against the oracle."""
    ref, ref_state = gated_delta_rule(*(_np(x[a:b]) for x in (w.q, w.k, w.v, w.log_alpha, w.beta)),
                                      _np(start))
    norm = max(np.linalg.norm(_np(start), axis=-1).max(), np.linalg.norm(ref_state, axis=-1).max(),
               1.0)
    err = np.abs(_np(got_state) - ref_state).max()
    assert err <= STATE_TOL * norm, (err, STATE_TOL * norm)
    if b > a:
        tol = 2.0 ** -8 * np.abs(ref) + (STATE_TOL + (2.0 ** -10 if chunked else 0.0)) * norm
        worst = (np.abs(_np(got_out) - ref) - tol).max()
        assert worst <= 0, worst


def _check_extend(lens, heads, key_heads, seed, slots=None, num_slots=None, **kw):
    num_slots = num_slots or len(lens)
    w, states = _draw(lens, heads, key_heads, num_slots, seed, **kw)
    before = states.clone()
    sl = None if slots is None else torch.tensor(slots, dtype=torch.int32, device=DEV)
    ctx = qsa.DeltaExtend(w.cu_seqlens, heads, DEV, key_heads)
    out = torch.full((sum(lens), heads, 128), 7.0, dtype=torch.bfloat16, device=DEV)
    ctx.run(w.q, w.k, w.v, w.log_alpha, w.beta, states, slots=sl, out=out)
    torch.cuda.synchronize()
    assert ctx.device_error() == ("QSA_OK", 0)
    cu = [int(x) for x in w.cu_seqlens]
    seen = set()
    for s in range(len(lens)):
        slot = s if slots is None else slots[s]
        a, b = cu[s], cu[s + 1]
        if not 0 <= slot < num_slots or (slot in seen):
            assert torch.all(out[a:b] == 7.0)
            continue
        seen.add(slot)
        _compare(out[a:b], states[slot], w, a, b, before[slot], True)
    for slot in set(range(num_slots)) - seen:
        assert torch.equal(states[slot], before[slot])


@pytest.mark.parametrize("lens", [[1], [64], [65], [1, 63, 64, 65, 0, 200, 1000, 0], [4097]])
def test_extend_lengths(lens):
    _check_extend(lens, 2, 2, seed=11)


@pytest.mark.parametrize("heads,key_heads", [(1, 1), (3, 1), (6, 3), (8, 2)])
def test_extend_grouped_heads(heads, key_heads):
    _check_extend([130, 77], heads, key_heads, seed=12)


def test_extend_strong_decay_and_resets():
    _check_extend([500, 129], 2, 1, seed=13, gate=(0.3, 0.8))
    _check_extend([500, 129], 2, 2, seed=14, reset_every=37)
    _check_extend([300], 2, 2, seed=15, reset_every=1)


def test_extend_slots_out_of_the_pool_and_named_twice():
    # -1 and 7 lie outside, 2 comes twice: the first row has it
    _check_extend([70, 10, 130, 64, 200], 2, 2, seed=16, slots=[2, -1, 0, 2, 7], num_slots=5)


def test_extend_many_short_sequences():
    _check_extend([5, 1, 0, 9, 3, 64, 2] * 6, 2, 1, seed=17)


def test_extend_zero_state_and_no_writes():
    w, states = _draw([300], 2, 2, 1, seed=18, state=0.0)
    w.beta.zero_()
    out = qsa.gated_deltanet_extend(w.q, w.k, w.v, w.log_alpha, w.beta, w.cu_seqlens, states)
    torch.cuda.synchronize()
    assert torch.count_nonzero(out).item() == 0 and torch.count_nonzero(states).item() == 0


@pytest.mark.parametrize("cuts", [[100, 37, 63], [64, 128, 8], [1, 1, 198]])
def test_pieces_and_steps_continue_one_sequence(cuts):
    heads, key_heads = 4, 2
    T = sum(cuts) + 5
    w, states = _draw([T], heads, key_heads, 3, seed=20)
    start = states[1].clone()
    slot = torch.tensor([1], dtype=torch.int32, device=DEV)
    outs, t = [], 0
    for c in cuts:
        x = [y[t:t + c] for y in (w.q, w.k, w.v, w.log_alpha, w.beta)]
        outs.append(qsa.gated_deltanet_extend(*x, [0, c], states, slots=slot))
        t += c
    for n in (1, 4):
        x = [y[t:t + n][None].contiguous() for y in (w.q, w.k, w.v, w.log_alpha, w.beta)]
        outs.append(qsa.gated_deltanet_step(*x, states, slots=slot)[0])
        t += n
    torch.cuda.synchronize()
    _compare(torch.cat(outs), states[1], w, 0, T, start, True)


def _check_step(B, n, heads, key_heads, seed, counts=None, slots=None, num_slots=None, **kw):
    num_slots = num_slots or B
    w, states = _draw([n] * B, heads, key_heads, num_slots, seed, **kw)
    before = states.clone()
    x = [y.view(B, n, *y.shape[1:]) for y in (w.q, w.k, w.v, w.log_alpha, w.beta)]
    dev = lambda z: None if z is None else torch.tensor(z, dtype=torch.int32, device=DEV)  # noqa: E731
    out = torch.full((B, n, heads, 128), 7.0, dtype=torch.bfloat16, device=DEV)
    qsa.gated_deltanet_step(*x, states, slots=dev(slots), counts=dev(counts), out=out)
    torch.cuda.synchronize()
    seen = set()
    for b in range(B):
        slot = b if slots is None else slots[b]
        c = n if counts is None else max(0, min(n, counts[b]))
        if not 0 <= slot < num_slots or slot in seen:
            c = 0
        else:
            seen.add(slot)
            _compare(out[b, :c], states[slot], w, b * n, b * n + c, before[slot], False)
        assert torch.all(out[b, c:] == 7.0)
    for slot in set(range(num_slots)) - seen:
        assert torch.equal(states[slot], before[slot])


@pytest.mark.parametrize("B,n,heads,key_heads", [(1, 1, 1, 1), (1, 1, 32, 16), (3, 1, 6, 2),
                                                 (64, 1, 4, 4), (5, 7, 3, 1), (2, 64, 2, 2)])
def test_step(B, n, heads, key_heads):
    _check_step(B, n, heads, key_heads, seed=30)


def test_step_counts_and_slots():
    _check_step(6, 4, 4, 2, seed=31, counts=[0, 1, 4, -3, 9, 2])
    _check_step(6, 3, 2, 2, seed=32, counts=[3, 2, 3, 0, 1, 3], slots=[4, -1, 4, 5, 99, 0],
                num_slots=6)


def test_step_resets():
    _check_step(4, 6, 2, 2, seed=33, reset_every=4)


def test_step_on_another_stream_in_a_graph():
    w, states = _draw([1] * 8, 4, 2, 8, seed=34)
    x = [y.view(8, 1, *y.shape[1:]) for y in (w.q, w.k, w.v, w.log_alpha, w.beta)]
    start = states.clone()
    want = states.clone()
    out = torch.empty((8, 1, 4, 128), dtype=torch.bfloat16, device=DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        qsa.gated_deltanet_step(*x, states, out=out)
    for _ in range(3):
        ref = qsa.gated_deltanet_step(*x, want)
    torch.cuda.synchronize()
    assert torch.equal(states, start)      # captured, not run
    for _ in range(3):
        g.replay()
    torch.cuda.synchronize()
    assert torch.equal(states, want) and torch.equal(out, ref)


def test_extend_contexts_in_two_graphs():
    # two contexts, two captured graphs, replayed in turn and over again
    heads = 4
    runs = []
    for seed, lens in ((35, [200, 64]), (36, [700])):
        w, states = _draw(lens, heads, heads, len(lens), seed=seed)
        ctx = qsa.DeltaExtend(w.cu_seqlens, heads, DEV)
        args = (w.q, w.k, w.v, w.log_alpha, w.beta)
        want = states.clone()
        ref = [ctx.run(*args, want) for _ in range(2)][-1]
        torch.cuda.synchronize()
        out = torch.empty_like(w.v)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            ctx.run(*args, states, out=out)
        runs.append((g, states, want, out, ref, (ctx, args)))   # the graph reads args
    for _ in range(2):
        for r in runs:
            r[0].replay()
    torch.cuda.synchronize()
    for _, states, want, out, ref, _ in runs:
        assert torch.equal(states, want) and torch.equal(out, ref)


def test_binding_refusals():
    w, states = _draw([10], 4, 2, 1, seed=37)
    ctx = qsa.DeltaExtend([0, 10], 4, DEV, 2)
    args = [w.q, w.k, w.v, w.log_alpha, w.beta]
    with pytest.raises(ValueError):
        ctx.run(*[x[:9] for x in args], states)
    with pytest.raises(ValueError):
        ctx.run(w.v, w.v, w.v, w.log_alpha, w.beta, states)
    with pytest.raises(TypeError):
        ctx.run(*args, states.half())
    with pytest.raises(ValueError):
        ctx.run(*args, states, slots=torch.zeros(2, dtype=torch.int32, device=DEV))
    with pytest.raises(qsa.QSAError):
        qsa.DeltaExtend([1, 10], 4, DEV, 2)
    with pytest.raises(ValueError):
        qsa.gated_deltanet_step(*[x[None] for x in args], states[:0])

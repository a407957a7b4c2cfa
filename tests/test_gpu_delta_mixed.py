"""GPU tests of extend calls that mix sequences in chunks with short ones (token by token) and empty
ones, which are listed on the device (tolerances of tests/test_gpu_delta.py)."""
import pytest
import torch

import block_sparse_attention_40_b200 as qsa
from block_sparse_attention_40_b200 import workloads as W
from tests.gpu_helpers import needs_gpu
from tests.test_gpu_delta import DEV, STATE_TOL, _check_extend, _draw

pytestmark = [pytest.mark.gpu, needs_gpu]


@pytest.mark.parametrize("lens,heads,key_heads", [
    ([0, 100, 0], 2, 1), ([0, 0, 70, 64, 0, 129, 0], 2, 2),
    ([1] * 80 + [300, 17, 16] + [0] * 5 + [65, 3] * 6, 2, 2),
    ([5000, 1, 0, 2100] + [2] * 160 + [700], 1, 1),              # cut into segments, of some one only
    ([0, 3000, 0, 40, 1400], 4, 2),
    ([3] * 1100 + [90], 1, 1)])                                  # more rows than one turn of the list
def test_extend_mixed(lens, heads, key_heads):
    _check_extend(lens, heads, key_heads, seed=90, gate=(0.95, 1.0))


def test_extend_mixed_slots():
    # a short row names the slot of a later long one and has it; a long one lies outside the pool
    lens = [9, 200, 70, 0, 300, 64] + [2] * 100
    slots = [2, 2, 900, 1, 0, 1] + [10 + i for i in range(100)]
    _check_extend(lens, 2, 1, seed=91, slots=slots, num_slots=120)


def test_extend_mixed_equals_its_parts():
    # 4,000 and 900 tokens beside 60 short pieces, against calls of their own
    lens, heads = [7] * 30 + [4000] + [1] * 30 + [0, 900], 4
    w, states = _draw(lens, heads, 2, len(lens), seed=92)
    args = (w.q, w.k, w.v, w.log_alpha, w.beta)
    got = states.clone()
    out = qsa.gated_deltanet_extend(*args, w.cu_seqlens, got)
    cu = [int(x) for x in w.cu_seqlens]
    norm = max(got.norm(dim=-1).max().item(), states.norm(dim=-1).max().item())
    for s in (0, 30, 31, 62):
        one = states[s:s + 1].clone()
        a = qsa.gated_deltanet_extend(*[x[cu[s]:cu[s + 1]] for x in args], [0, lens[s]], one)
        assert (one[0] - got[s]).abs().max().item() <= 2 * STATE_TOL * norm
        tol = 2.0 ** -7 * a.float().abs() + 4 * STATE_TOL * norm
        assert torch.all((a.float() - out[cu[s]:cu[s + 1]].float()).abs() <= tol)
    assert torch.equal(got[61], states[61])      # the empty one


def test_extend_mixed_in_a_graph():
    # the list is made anew in every replay, beside the short rows' launch
    for lens in ([3000] + [4] * 80, [500, 0, 0, 2000]):
        w, states = _draw(lens, 2, 2, len(lens), seed=93)
        args = (w.q, w.k, w.v, w.log_alpha, w.beta)
        ctx = qsa.DeltaExtend(w.cu_seqlens, 2, DEV)
        want = states.clone()
        ref = [ctx.run(*args, want).clone() for _ in range(3)][-1]
        torch.cuda.synchronize()
        out = torch.empty_like(w.v)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            ctx.run(*args, states, out=out)
        for _ in range(3):
            g.replay()
        torch.cuda.synchronize()
        assert torch.equal(states, want) and torch.equal(out, ref)
        assert ctx.device_error() == ("QSA_OK", 0)


def test_extend_mixed_in_passes():
    # records of more than the budget, short pieces and an index: heads in two passes
    lens, heads = [60000, 1, 70000, 60001] + [2] * 20, 16
    w, states = _draw(lens, heads, heads, len(lens), seed=94, gate=(0.95, 1.0))
    ctx = qsa.DeltaExtend(w.cu_seqlens, heads, DEV)
    got = states.clone()
    out = ctx.run(w.q, w.k, w.v, w.log_alpha, w.beta, got)
    torch.cuda.synchronize()
    assert ctx.device_error() == ("QSA_OK", 0) and ctx.ws.numel() <= (1 << 32) + 4096
    norm = got.norm(dim=-1).max().item()
    for h in (0, 8, 15):
        one = states[:, h:h + 1].contiguous()
        x = [y[:, h:h + 1].contiguous() for y in (w.q, w.k, w.v, w.log_alpha, w.beta)]
        alone = qsa.gated_deltanet_extend(*x, w.cu_seqlens, one)
        assert (one - got[:, h:h + 1]).abs().max().item() <= 2 * STATE_TOL * norm
        a = alone[:, 0].float()
        tol = 2.0 ** -7 * a.abs() + 4 * STATE_TOL * norm
        assert torch.all((a - out[:, h].float()).abs() <= tol)


@pytest.mark.parametrize("where", ["cpu", DEV])
def test_extend_context_keeps_its_own_lengths(where):
    # the caller's tensor of lengths is filled with other ones after the context was made
    w, states = _draw([130, 70], 2, 2, 2, seed=95)
    twin = states.clone()
    args = (w.q, w.k, w.v, w.log_alpha, w.beta)
    want = qsa.gated_deltanet_extend(*args, [0, 130, 200], twin)
    cu = torch.tensor([0, 130, 200], dtype=torch.int32, device=where)
    ctx = qsa.DeltaExtend(cu, 2, DEV)
    cu.copy_(torch.tensor([0, 3, 9], dtype=torch.int32))
    out = ctx.run(*args, states)
    torch.cuda.synchronize()
    assert ctx.device_error() == ("QSA_OK", 0)
    assert torch.equal(out, want) and torch.equal(states, twin)


def test_extend_on_two_streams_at_once():
    # two contexts and the prefill attention (which holds tensor memory too), each on a stream of its
    # own, over and over without a wait between them
    runs = []
    for seed, lens, heads in ((96, [3000, 200], 4), (97, [5] * 40 + [1500, 700], 8)):
        w, states = _draw(lens, heads, heads, len(lens), seed=seed)
        runs.append((qsa.DeltaExtend(w.cu_seqlens, heads, DEV),
                     (w.q, w.k, w.v, w.log_alpha, w.beta), states, states.clone()))
    p = W.prefill("tiny")
    d = p.to(DEV)
    pre = qsa.Prefill(p.cu_seqlens, DEV, p.topk)
    attention = lambda: pre.run(d.q, d.k, d.v, d.q_idx, d.k_idx, d.w)  # noqa: E731
    want = [[ctx.run(*args, twin).clone() for _ in range(6)] for ctx, args, _, twin in runs]
    ref = attention().clone()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    got, outs = [[], []], []
    for _ in range(6):
        for i, (ctx, args, states, _) in enumerate(runs):
            with torch.cuda.stream(streams[i]):
                got[i].append(ctx.run(*args, states))
        with torch.cuda.stream(streams[2]):
            outs.append(attention())
    torch.cuda.synchronize()
    for i, (ctx, _, states, twin) in enumerate(runs):
        assert ctx.device_error() == ("QSA_OK", 0) and torch.equal(states, twin)
        assert all(torch.equal(a, b) for a, b in zip(got[i], want[i]))
    assert pre.device_error() == ("QSA_OK", 0) and all(torch.equal(o, ref) for o in outs)


def test_extend_zeroes_the_rows_of_skipped_sequences_only():
    # cut into segments, in chunks, token by token: a new out is zero where a slot is outside or was
    # named before, also over memory that held something else; a given out keeps what it had
    for lens, slots in (([3000, 2500, 70], [-1, 0, 0]), ([2] * 150 + [90, 40, 300], [0] * 151 + [1, 500]),
                        ([9, 20, 3], [1, 1, -7])):
        w, states = _draw(lens, 2, 1, 3, seed=98)
        twin = states.clone()
        sl = torch.tensor(slots, dtype=torch.int32, device=DEV)
        args = (w.q, w.k, w.v, w.log_alpha, w.beta)
        ctx = qsa.DeltaExtend(w.cu_seqlens, 2, DEV, 1)
        given = torch.full_like(w.v, 7.0)
        ctx.run(*args, twin, slots=sl, out=given)
        junk = torch.full_like(w.v, float("nan"))
        del junk
        out = ctx.run(*args, states, slots=sl)
        torch.cuda.synchronize()
        assert ctx.device_error() == ("QSA_OK", 0) and torch.equal(states, twin)
        t = 0
        seen = set()
        for n, slot in zip(lens, slots):
            if 0 <= slot < 3 and slot not in seen:
                assert torch.equal(out[t:t + n], given[t:t + n])
            else:
                assert torch.count_nonzero(out[t:t + n]).item() == 0
                assert torch.all(given[t:t + n] == 7.0)
            seen.add(slot)
            t += n

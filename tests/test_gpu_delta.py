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


@pytest.mark.parametrize("lens", [[130, 3, 64], [20, 1], [9000]])
def test_out_in_place_of_v(lens):
    w, states = _draw(lens, 2, 1, len(lens), seed=38)
    twin = states.clone()
    want = qsa.gated_deltanet_extend(w.q, w.k, w.v, w.log_alpha, w.beta, w.cu_seqlens, states)
    v = w.v.clone()
    qsa.gated_deltanet_extend(w.q, w.k, v, w.log_alpha, w.beta, w.cu_seqlens, twin, out=v)
    torch.cuda.synchronize()
    assert torch.equal(v, want) and torch.equal(twin, states)
    x = [y[:12].view(2, 6, *y.shape[1:]) for y in (w.q, w.k, w.v, w.log_alpha, w.beta)]
    states, twin = states[:1].repeat(2, 1, 1, 1), twin[:1].repeat(2, 1, 1, 1)
    want = qsa.gated_deltanet_step(*x, states)
    x[2] = x[2].clone()
    qsa.gated_deltanet_step(*x, twin, out=x[2])
    torch.cuda.synchronize()
    assert torch.equal(x[2], want) and torch.equal(twin, states)


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


# ---- sequences cut into segments, scales, neighbours -------------------------------------------
@pytest.mark.parametrize("lens,heads", [([20000], 1), ([5000, 3100], 8), ([2500] * 3 + [40, 700], 4)])
def test_extend_long_sequences_are_cut(lens, heads):
    # long walks with few heads: segments from zero, transitions, joins over 4, 16 and 8 rows
    _check_extend(lens, heads, heads, seed=40, gate=(0.97, 1.0))


def test_extend_long_sequence_equals_its_pieces():
    # the outputs' tolerance twice: either side is off by as much
    T, heads = 9000, 2
    w, states = _draw([T], heads, 1, 1, seed=41)
    args = (w.q, w.k, w.v, w.log_alpha, w.beta)
    one, two = states.clone(), states.clone()
    a = qsa.gated_deltanet_extend(*args, [0, T], one)
    b = torch.cat([qsa.gated_deltanet_extend(*[x[i:i + 1500] for x in args], [0, 1500], two)
                   for i in range(0, T, 1500)])
    torch.cuda.synchronize()
    norm = max(one.norm(dim=-1).max().item(), states.norm(dim=-1).max().item())
    assert (one - two).abs().max().item() <= 2 * STATE_TOL * norm
    tol = 2.0 ** -7 * a.float().abs() + 2 * (STATE_TOL + 2.0 ** -10) * norm
    assert torch.all((a.float() - b.float()).abs() <= tol)


def test_extend_twice_is_the_same_bits():
    w, states = _draw([3000, 40, 700], 4, 2, 3, seed=42)
    ctx = qsa.DeltaExtend(w.cu_seqlens, 4, DEV, 2)
    runs = []
    for _ in range(2):
        st = states.clone()
        runs.append((ctx.run(w.q, w.k, w.v, w.log_alpha, w.beta, st).clone(), st))
    assert torch.equal(runs[0][0], runs[1][0]) and torch.equal(runs[0][1], runs[1][1])


@pytest.mark.parametrize("lens", [[1] * 40 + [100], [16, 3, 9] * 12 + [300, 64], [32, 31, 1], [7]])
def test_extend_short_pieces(lens):
    # token by token alone, or beside longer ones where there are many
    _check_extend(lens, 6, 2, seed=43)


def test_extend_no_tokens():
    states = torch.ones((3, 2, 128, 128), device=DEV)
    x = torch.empty((0, 2, 128), dtype=torch.bfloat16, device=DEV)
    g = torch.empty((0, 2), device=DEV)
    assert qsa.gated_deltanet_extend(x, x, x, g, g, [0, 0, 0], states).shape == (0, 2, 128)
    out = qsa.gated_deltanet_step(x[None], x[None], x[None], g[None], g[None], states)
    assert out.shape == (1, 0, 2, 128) and torch.all(states == 1)


def test_extend_gates_above_one():
    # alpha in (1, 1.02): what a token writes grows on its way to the chunk's end.  The recurrence
    # multiplies every error by the same alphas as the state, so tolerances stay relative to it.
    w, states = _draw([150], 2, 2, 1, seed=44)
    w.log_alpha.uniform_(0.0, 0.02, generator=torch.Generator(device=DEV).manual_seed(45))
    start = states.clone()
    out = qsa.gated_deltanet_extend(w.q, w.k, w.v, w.log_alpha, w.beta, w.cu_seqlens, states)
    torch.cuda.synchronize()
    _compare(out, states[0], w, 0, 150, start[0], True)


@pytest.mark.parametrize("scale", [1e-20, 1e-5, 1e6, 1e25])
def test_extend_and_step_of_any_size(scale):
    # the rule is linear in (v, S): powers of ten in, the same powers out.  The scale is a power of
    # two, so that the unscaled run is the exact reference up to the roundings that the tolerances
    # of _compare count for each of the two.
    s = 2.0 ** round(np.log2(scale))
    w, states = _draw([200], 2, 1, 1, seed=46)
    small, big = states.clone(), states * s
    args = (w.q, w.k)
    a = qsa.gated_deltanet_extend(*args, w.v, w.log_alpha, w.beta, w.cu_seqlens, small)
    b = qsa.gated_deltanet_extend(*args, (w.v.float() * s).to(torch.bfloat16), w.log_alpha, w.beta,
                                  w.cu_seqlens, big)
    torch.cuda.synchronize()
    norm = small.norm(dim=-1).max().item()
    assert (big / s - small).abs().max().item() <= 2 * STATE_TOL * norm
    tol = 2.0 ** -7 * a.float().abs() + 2 * (STATE_TOL + 2.0 ** -10) * norm
    assert torch.all((b.float() / s - a.float()).abs() <= tol)
    x = [y[None, :3].contiguous() for y in (w.q, w.k, w.v, w.log_alpha, w.beta)]
    p, q = states.clone(), states * s
    qsa.gated_deltanet_step(*x, p)
    x[2] = (x[2].float() * s).to(torch.bfloat16)
    qsa.gated_deltanet_step(*x, q)
    assert (q / s - p).abs().max().item() <= 2 * STATE_TOL * norm


def test_extend_neighbours_stay_apart():
    # NaN in one sequence reaches no other one, whatever shares its last chunk's rows
    lens = [70, 100, 33, 65]
    w, states = _draw(lens, 2, 2, 4, seed=47)
    clean, dirty = states.clone(), states.clone()
    a = qsa.gated_deltanet_extend(w.q, w.k, w.v, w.log_alpha, w.beta, w.cu_seqlens, clean)
    bad = [x.clone() for x in (w.q, w.k, w.v)]
    for x in bad:
        x[70:170] = float("nan")
    dirty[1] = float("inf")
    b = qsa.gated_deltanet_extend(*bad, w.log_alpha, w.beta, w.cu_seqlens, dirty)
    torch.cuda.synchronize()
    assert torch.equal(a[:70], b[:70]) and torch.equal(a[170:], b[170:])
    for s in (0, 2, 3):
        assert torch.equal(clean[s], dirty[s])


def test_extend_heads_in_passes():
    # more records than one pass holds (4 GB): heads run in passes, each like heads alone
    lens, heads = [60000, 70000, 60001], 16
    w, states = _draw(lens, heads, heads, 3, seed=48, gate=(0.95, 1.0))
    ctx = qsa.DeltaExtend(w.cu_seqlens, heads, DEV)
    assert ctx.ws.numel() < sum(lens) // 64 * heads * 91136
    got = states.clone()
    out = ctx.run(w.q, w.k, w.v, w.log_alpha, w.beta, got)
    torch.cuda.synchronize()
    assert ctx.device_error() == ("QSA_OK", 0)
    norm = got.norm(dim=-1).max().item()
    for h in (0, 8, 15):
        one = states[:, h:h + 1].contiguous()
        x = [y[:, h:h + 1].contiguous() for y in (w.q, w.k, w.v, w.log_alpha, w.beta)]
        alone = qsa.gated_deltanet_extend(*x, w.cu_seqlens, one)
        assert (one - got[:, h:h + 1]).abs().max().item() <= 2 * STATE_TOL * norm
        a = alone[:, 0].float()
        tol = 2.0 ** -7 * a.abs() + 2 * (STATE_TOL + 2.0 ** -10) * norm
        assert torch.all((a - out[:, h].float()).abs() <= tol)


def test_extend_cut_sequence_in_a_graph_on_another_stream():
    w, states = _draw([4000], 2, 2, 1, seed=49)
    args = (w.q, w.k, w.v, w.log_alpha, w.beta)
    ctx = qsa.DeltaExtend(w.cu_seqlens, 2, DEV)
    want, start = states.clone(), states.clone()
    ref = [ctx.run(*args, want) for _ in range(3)][-1]
    torch.cuda.synchronize()
    out = torch.empty_like(w.v)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        ctx.run(*args, states, out=out)
    assert torch.equal(states, start)
    for _ in range(3):
        g.replay()
    torch.cuda.synchronize()
    assert torch.equal(states, want) and torch.equal(out, ref)


def test_extend_reports_timeouts_as_ok_when_there_are_none():
    # many contexts one after the other on one stream, their launches overlapping
    ctxs = []
    for seed in range(6):
        w, states = _draw([130 + 64 * seed, 20], 2, 2, 2, seed=50 + seed)
        ctx = qsa.DeltaExtend(w.cu_seqlens, 2, DEV)
        start = states.clone()
        ctxs.append((ctx, w, states, start, ctx.run(w.q, w.k, w.v, w.log_alpha, w.beta, states)))
    torch.cuda.synchronize()
    for ctx, w, states, start, out in ctxs:
        assert ctx.device_error() == ("QSA_OK", 0)
        n = int(w.cu_seqlens[1])
        _compare(out[:n], states[0], w, 0, n, start[0], True)


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

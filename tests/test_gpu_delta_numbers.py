"""GPU tests of how exactly the delta rule's chunked form computes: cases whose result is known to the
bit, and cases whose magnitudes differ by many orders, against the fp64 oracle.

Tolerances.  Token by token in fp32 a step is off by at most 21 half steps (2^-24) of the largest
row norm R_t of the state it leaves (two roundings of the update, 19 of the dot S k), and what it is
off by goes on through the later gates (|I - beta k k^T| <= 1 for unit-norm keys).  So a state is off by
    E_T = 21 * 2^-24 * sum_t R_t prod_{t < s <= T} a_s
and an output, rounded once to bf16 (half a step: 2^-8 of the value), by 2^-8 |o_t| + E_t +
21 * 2^-24 R_t.  The chunked form is held to the same.
"""
import numpy as np
import pytest
import torch

import block_sparse_attention_40_b200 as qsa
from oracle.gated_deltanet import gated_delta_rule
from tests.gpu_helpers import needs_gpu
from tests.test_gpu_delta import DEV, STATE_TOL, _compare, _draw, _np

pytestmark = [pytest.mark.gpu, needs_gpu]
FINE = 1 + 2.0 ** -8 + 2.0 ** -13      # just above half way from 1 to the next bf16, 1 + 2^-7


def _blank(T, heads):
    """No decay, nothing written, all vectors zero."""
    x = torch.zeros((T, heads, 128), dtype=torch.bfloat16, device=DEV)
    g = torch.zeros((T, heads), device=DEV)
    return x, x.clone(), x.clone(), g, g.clone()


def test_out_is_rounded_once_from_the_state():
    # one-hot queries of a state that stays: every output is one of its entries
    T, heads = 100, 2
    q, k, v, la, beta = _blank(T, heads)
    g = torch.Generator().manual_seed(1)
    t = torch.arange(T)
    q[t, :, (7 * t) % 128] = 1.0
    k[:, :, 3] = 1.0
    i = torch.arange(128)
    sign = torch.where(torch.rand((heads, 128, 128), generator=g) < 0.5, -1.0, 1.0)
    states = (sign * FINE * 2.0 ** ((i[:, None] + i) % 5)).to(DEV)[None].contiguous()
    want = states[0][:, :, (7 * t) % 128].permute(2, 0, 1).to(torch.bfloat16)
    out = qsa.gated_deltanet_extend(q, k, v, la, beta, [0, T], states)
    assert torch.equal(out, want)


@pytest.mark.parametrize("fine", ["key product", "write"])
def test_out_is_rounded_once_from_the_writes(fine):
    # one token writes, all read it: the product q.k (1 + 2^-8 + 2^-13), or what is written
    T, heads = 100, 2
    q, k, v, la, beta = _blank(T, heads)
    states = torch.zeros((1, heads, 128, 128), device=DEV)
    sign = torch.where(torch.arange(128) % 3 == 0, -1.0, 1.0).to(DEV)
    v[0] = sign.to(torch.bfloat16)
    if fine == "write":
        k[0, :, 9] = 1.0
        q[:, :, 9] = 1.0
        beta[0] = FINE
    else:
        k[0, :, :3] = 1.0
        q[:, :, 0], q[:, :, 1], q[:, :, 2] = 1.0, 2.0 ** -8, 2.0 ** -13
        beta[0] = 1.0
    out = qsa.gated_deltanet_extend(q, k, v, la, beta, [0, T], states)
    assert torch.all(out == (sign * (1 + 2.0 ** -7)).to(torch.bfloat16))


def _carried(w, start):
    """fp64 outputs, final state, E_t and R_t (see above) of one sequence, per token and head."""
    x = [_np(y) for y in (w.q, w.k, w.v, w.log_alpha, w.beta)]
    S, outs, E, R = _np(start), [], [], []
    e = np.zeros(S.shape[0])
    for t in range(x[0].shape[0]):
        before = np.linalg.norm(S, axis=-1).max(axis=-1)
        o, S = gated_delta_rule(*(y[t:t + 1] for y in x), S)
        a = np.exp(np.maximum(x[3][t], -87.0))
        r = np.maximum(np.linalg.norm(S, axis=-1).max(axis=-1), a * before)
        e = a * e + 21 * 2.0 ** -24 * r
        outs.append(o[0])
        E.append(e)
        R.append(r)
    return np.stack(outs), S, np.stack(E), np.stack(R)


def _check_carried(w, states):
    start = states[0].clone()
    ref, ref_state, E, R = _carried(w, start)
    out = qsa.gated_deltanet_extend(w.q, w.k, w.v, w.log_alpha, w.beta, w.cu_seqlens, states)
    torch.cuda.synchronize()
    err = np.abs(_np(states[0]) - ref_state).max(axis=(1, 2))
    assert np.all(err <= E[-1]), (err, E[-1])
    tol = 2.0 ** -8 * np.abs(ref) + (E + 21 * 2.0 ** -24 * R)[..., None]
    assert np.all(np.abs(_np(out) - ref) <= tol), (np.abs(_np(out) - ref) - tol).max()


@pytest.mark.parametrize("big", [1e3, 1e6, 1e8])
def test_a_large_write_before_a_reset_leaves_nothing(big):
    # what token 5 wrote is gone at token 29, in the middle of its chunk
    w, states = _draw([150], 2, 1, 1, seed=60, state=0.0)
    w.v[5] *= big
    w.log_alpha[29] = float("-inf")
    _check_carried(w, states)


@pytest.mark.parametrize("size", [1e3, 1e6])
def test_a_large_start_that_decays(size):
    w, states = _draw([150], 2, 2, 1, seed=61, gate=(0.5, 1.0), state=0.3 * size)
    _check_carried(w, states)


def test_a_large_start_that_is_reset():
    w, states = _draw([100], 2, 2, 1, seed=62, state=3e7)
    w.log_alpha[40] = float("-inf")
    _check_carried(w, states)


# ---- rows that are skipped, gates that are no number ---------------------------------------------
def test_extend_out_of_skipped_rows_is_zero():
    lens = [70, 40, 65, 33]
    w, states = _draw(lens, 2, 2, 3, seed=63)
    slots = torch.tensor([1, -1, 1, 0], dtype=torch.int32, device=DEV)
    junk = torch.full_like(w.v, float("nan"))
    del junk      # its memory is the next tensor's of this size
    out = qsa.gated_deltanet_extend(w.q, w.k, w.v, w.log_alpha, w.beta, w.cu_seqlens, states,
                                    slots=slots)
    torch.cuda.synchronize()
    assert torch.count_nonzero(out[70:175]).item() == 0
    assert torch.all(torch.isfinite(out)) and torch.count_nonzero(out[:70]).item() > 0


@pytest.mark.parametrize("lens,at", [([100, 70], 40), ([20, 9], 11)])
def test_extend_a_gate_that_is_no_number_is_carried_on(lens, at):
    # in chunks and token by token: not taken for a reset; other heads and sequences do not see it
    w, states = _draw(lens, 3, 3, 2, seed=64)
    clean = states.clone()
    want = qsa.gated_deltanet_extend(w.q, w.k, w.v, w.log_alpha, w.beta, w.cu_seqlens, clean)
    w.log_alpha[at, 1] = float("nan")
    out = qsa.gated_deltanet_extend(w.q, w.k, w.v, w.log_alpha, w.beta, w.cu_seqlens, states)
    torch.cuda.synchronize()
    assert torch.all(torch.isnan(states[0, 1])) and torch.all(torch.isnan(out[at:lens[0], 1]))
    assert torch.equal(states[1], clean[1]) and torch.equal(out[lens[0]:], want[lens[0]:])
    for h in (0, 2):
        assert torch.equal(states[0, h], clean[0, h]) and torch.equal(out[:, h], want[:, h])


def test_step_a_gate_that_is_no_number_is_carried_on():
    w, states = _draw([3, 3], 2, 1, 2, seed=65)
    x = [y.view(2, 3, *y.shape[1:]) for y in (w.q, w.k, w.v, w.log_alpha, w.beta)]
    x[3][0, 1, 0] = float("nan")
    out = qsa.gated_deltanet_step(*x, states)
    torch.cuda.synchronize()
    assert torch.all(torch.isnan(states[0, 0])) and torch.all(torch.isnan(out[0, 1:, 0]))
    assert torch.all(torch.isfinite(out[0, 0])) and torch.all(torch.isfinite(states[0, 1]))
    assert torch.all(torch.isfinite(out[1])) and torch.all(torch.isfinite(states[1]))


# ---- keys and queries of any length --------------------------------------------------------------
@pytest.mark.parametrize("lens", [[200], [5000]])
@pytest.mark.parametrize("m", [-20, -3, 3, 20])
def test_keys_and_queries_of_any_length(lens, m):
    # k 2^m, beta 2^-2m and S 2^-m, q 2^m leave the outputs as they were: powers of two, so that the
    # unscaled run is the reference up to the roundings of the two runs
    w, states = _draw(lens, 2, 1, 1, seed=66, gate=(0.95, 1.0))
    s = 2.0 ** m
    one, two = states.clone(), states / s
    a = qsa.gated_deltanet_extend(w.q, w.k, w.v, w.log_alpha, w.beta, w.cu_seqlens, one)
    b = qsa.gated_deltanet_extend((w.q.float() * s).to(torch.bfloat16),
                                  (w.k.float() * s).to(torch.bfloat16), w.v, w.log_alpha,
                                  w.beta / s ** 2, w.cu_seqlens, two)
    torch.cuda.synchronize()
    norm = max(one.norm(dim=-1).max().item(), states.norm(dim=-1).max().item())
    assert (two * s - one).abs().max().item() <= 2 * STATE_TOL * norm
    tol = 2.0 ** -7 * a.float().abs() + 4 * STATE_TOL * norm
    assert torch.all((a.float() - b.float()).abs() <= tol)


def test_keys_of_different_lengths():
    # key rows of norm 2^-6 .. 2^3 (beta so that beta |k|^2 <= 1), queries of norm 2^-9 .. 2^9
    w, states = _draw([300, 70], 2, 2, 2, seed=67)
    g = torch.Generator().manual_seed(68)
    e = torch.randint(-6, 4, (370, 2), generator=g).to(DEV).float()
    f = torch.randint(-9, 10, (370, 2), generator=g).to(DEV).float()
    w.k = (w.k.float() * (2.0 ** e)[..., None]).to(torch.bfloat16)
    w.beta = w.beta * 2.0 ** (-2 * e).clamp_max(0.0)
    plain = w.q
    w.q = (w.q.float() * (2.0 ** f)[..., None]).to(torch.bfloat16)
    before = states.clone()
    out = qsa.gated_deltanet_extend(w.q, w.k, w.v, w.log_alpha, w.beta, w.cu_seqlens, states)
    torch.cuda.synchronize()
    out = (out.float() * (2.0 ** -f)[..., None]).to(torch.bfloat16)   # exact: as for unit queries
    w.q = plain
    # a write is at most beta |k| <= 2^6 times what it is with unit-norm keys, and so is R
    for s, (a, b) in enumerate(((0, 300), (300, 370))):
        _compare(out[a:b], states[s], w, a, b, before[s], True)


# ---- joins ---------------------------------------------------------------------------------------
@pytest.mark.parametrize("lens,heads", [([1000, 1000], 4), ([3000], 6), ([2000], 9)])
def test_extend_cut_with_few_pairs_of_sequence_and_head(lens, heads):
    # five to nine of them: joins of eight rows a block
    w, states = _draw(lens, heads, heads, len(lens), seed=69, gate=(0.97, 1.0))
    before = states.clone()
    ctx = qsa.DeltaExtend(w.cu_seqlens, heads, DEV)
    out = ctx.run(w.q, w.k, w.v, w.log_alpha, w.beta, states)
    torch.cuda.synchronize()
    assert ctx.device_error() == ("QSA_OK", 0)
    cu = [int(x) for x in w.cu_seqlens]
    for s in range(len(lens)):
        a, b = cu[s], cu[s + 1]
        _compare(out[a:b], states[s], w, a, b, before[s], True)


# ---- what is not finite --------------------------------------------------------------------------
@pytest.mark.parametrize("which", ["q", "k", "v", "log_alpha", "beta"])
def test_extend_not_finite_reaches_no_earlier_group_of_16(which):
    # token 105 of 200: tokens before 96 come out as without it, and so does the other head
    w, states = _draw([200], 2, 2, 1, seed=70)
    clean = states.clone()
    want = qsa.gated_deltanet_extend(w.q, w.k, w.v, w.log_alpha, w.beta, w.cu_seqlens, clean)
    getattr(w, which)[105, 1] = float("nan")
    out = qsa.gated_deltanet_extend(w.q, w.k, w.v, w.log_alpha, w.beta, w.cu_seqlens, states)
    torch.cuda.synchronize()
    assert torch.equal(out[:96], want[:96]) and torch.equal(out[:, 0], want[:, 0])
    assert torch.equal(states[0, 0], clean[0, 0]) and torch.all(torch.isnan(out[105, 1]))
    if which == "q":      # its own output only
        assert torch.equal(states, clean)
        rest = torch.arange(200, device=DEV) != 105
        assert torch.equal(out[rest], want[rest])
    else:
        assert torch.all(torch.isnan(out[106:, 1])) and torch.all(torch.isnan(states[0, 1]))

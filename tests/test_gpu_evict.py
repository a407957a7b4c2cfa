"""GPU tests of eviction by accumulated attention weight.

Weights: tolerance from fp32.  A logit is 128 exact bf16 products summed in fp32: at most
128 * 2^-24 of sum |q k| / sqrt(128), which N(0,1) inputs keep below 12, so 9.2e-5; exponentials,
logarithms and the sums add a few 2^-22.  A weight is off by as much, relatively: 1e-4 of it, and
half a step of the running weight that it is added to.  Choice and moves are exact."""
import numpy as np
import pytest
import torch

import block_sparse_attention_40_b200 as qsa
from block_sparse_attention_40_b200 import workloads as W
from oracle import evict as oracle_evict
from oracle.gated_deltanet import gated_delta_rule
from tests.gpu_helpers import needs_gpu

pytestmark = [pytest.mark.gpu, needs_gpu]
DEV = "cuda:0"
PAGES = [0, 512]


def _np(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def _cache(lens, capacity, page, seed):
    """A cache filled through append; a paged one on a shuffled table with spare pages."""
    B = len(lens)
    if page:
        capacity = (capacity + page - 1) // page * page
        per = capacity // page
        perm = torch.randperm(B * per + 3, generator=torch.Generator().manual_seed(seed))
        table = perm[:B * per].to(torch.int32).view(B, per).to(DEV)
        cache = qsa.PagedKVCache(B, capacity, page, B * per + 3, table, DEV)
    else:
        cache = qsa.KVCache(B, capacity, DEV)
    spec = W.small_decode_spec(batch=B, context=lens, capacity=capacity, topk=8, steps=1, seed=seed)
    k, v, ki = W.decode_context(spec)
    cache.append(k.to(DEV), v.to(DEV), ki.to(DEV), counts=list(lens))
    return cache


def _selection(lens, topk, seed):
    rng = np.random.default_rng(seed)
    idx = np.full((len(lens), topk), -1, np.int32)
    cnt = np.zeros(len(lens), np.int32)
    for b, n in enumerate(lens):
        own = (n - 1) // 4
        cnt[b] = min(own, topk) if b % 3 != 2 else rng.integers(0, min(own, topk) + 1)
        idx[b, :cnt[b]] = np.sort(rng.choice(own, cnt[b], replace=False))
    return idx, cnt


def _check_weights(ev, lens, q, idx, cnt, before, skip=()):
    got = _np(ev.mass)
    for b, n in enumerate(lens):
        want = before[b].copy()
        if b not in skip:
            keys = np.stack([_np(ev.cache.kv_rows(b, g, n)[0]) for g in range(2)])
            blocks = idx[b, :cnt[b]]
            w = oracle_evict.block_weights(_np(q[b]), keys, n, blocks)
            at = list(blocks) + [(n - 1) // 4]
            want[at] += w
        else:
            w, at = np.zeros(0), []
        tol = 2.0 ** -24 * np.abs(want)
        tol[at] += 1e-4 * w
        assert np.all(np.abs(got[b] - want) <= tol), b


@pytest.mark.parametrize("page", PAGES)
@pytest.mark.parametrize("lens,topk", [([1], 16), ([4], 1), ([5, 6, 7, 8], 3),
                                       ([2000, 1999, 61, 1], 512), ([4100], 1024),
                                       ([333] * 40, 64), ([90] * 160, 16)])
def test_weights(lens, topk, page):
    ev = qsa.Evictor(_cache(lens, 4104, page, seed=3), 8)
    ev.mass.copy_(torch.rand(ev.mass.shape, generator=torch.Generator().manual_seed(4)))
    before = _np(ev.mass)
    q = torch.randn((len(lens), 24, 128), generator=torch.Generator().manual_seed(5)) \
        .to(torch.bfloat16).to(DEV)
    idx, cnt = _selection(lens, topk, seed=6)
    got = ev.accumulate(q, torch.from_numpy(idx).to(DEV), torch.from_numpy(cnt).to(DEV))
    torch.cuda.synchronize()
    assert got is ev.mass and ev.device_error() == ("QSA_OK", 0)
    _check_weights(ev, lens, q, idx, cnt, before)


@pytest.mark.parametrize("batch", [12, 16, 24, 31, 40, 74, 80])
def test_weights_clusters_of_every_size(batch):
    # from eight CTAs a sequence down to two, and the narrow ones beyond
    lens = [600 - 7 * (b % 5) for b in range(batch)]
    ev = qsa.Evictor(_cache(lens, 600, 0, seed=66), 8)
    before = _np(ev.mass)
    q = torch.randn((batch, 24, 128), generator=torch.Generator().manual_seed(67)) \
        .to(torch.bfloat16).to(DEV)
    idx, cnt = _selection(lens, 100, seed=68)
    ev.accumulate(q, torch.from_numpy(idx).to(DEV), torch.from_numpy(cnt).to(DEV))
    torch.cuda.synchronize()
    assert ev.device_error() == ("QSA_OK", 0)
    _check_weights(ev, lens, q, idx, cnt, before)


def test_weights_twice_are_the_same_bits():
    lens = [1500, 700]
    ev = qsa.Evictor(_cache(lens, 2048, 0, seed=7), 8)
    q = torch.randn((2, 24, 128), generator=torch.Generator().manual_seed(8)).to(torch.bfloat16)
    idx, cnt = (torch.from_numpy(x).to(DEV) for x in _selection(lens, 200, seed=9))
    first = ev.accumulate(q.to(DEV), idx, cnt).clone()
    ev.mass.zero_()
    assert torch.equal(ev.accumulate(q.to(DEV), idx, cnt), first)


def test_weights_extreme_logits():
    # keys scaled so that one block takes nearly all of every head, and others underflow
    lens = [400]
    ev = qsa.Evictor(_cache(lens, 512, 0, seed=10), 8)
    ev.cache.k_blocks.mul_(16.0)
    q = (4 * torch.randn((1, 24, 128), generator=torch.Generator().manual_seed(11))) \
        .to(torch.bfloat16).to(DEV)
    idx, cnt = _selection(lens, 64, seed=12)
    before = _np(ev.mass)
    ev.accumulate(q, torch.from_numpy(idx).to(DEV), torch.from_numpy(cnt).to(DEV))
    keys = np.stack([_np(ev.cache.kv_rows(0, g, 400)[0]) for g in range(2)])
    w = oracle_evict.block_weights(_np(q[0]), keys, 400, idx[0, :cnt[0]])
    got = _np(ev.mass)[0][list(idx[0, :cnt[0]]) + [99]]
    # logits up to 64 times larger: their errors are as much larger (64 * 9.2e-5)
    assert np.all(np.abs(got - w) <= 6e-3 * w + 1e-30) and before.sum() == 0


def test_weights_bad_selections_are_left_out_and_recorded():
    lens = [200, 200, 200]
    ev = qsa.Evictor(_cache(lens, 256, 0, seed=13), 8)
    q = torch.randn((3, 24, 128), generator=torch.Generator().manual_seed(14)) \
        .to(torch.bfloat16).to(DEV)
    # row 0: a repeat, a block after the own one, a negative one; row 1: count above topk
    idx = torch.tensor([[1, 5, 5, 7, 60, -4], [0, 1, 2, 3, 4, 5], [0, 1, 2, 3, 4, 5]],
                       dtype=torch.int32)
    cnt = torch.tensor([6, 9, 2], dtype=torch.int32)
    before = _np(ev.mass)
    ev.accumulate(q, idx.to(DEV), cnt.to(DEV))
    status, site = ev.device_error()
    assert status == "QSA_ERR_DEVICE" and site in (300, 301)
    good = idx.numpy().copy()
    good[0, :3] = [1, 5, 7]
    _check_weights(ev, lens, q, good, np.array([3, 0, 2]), before, skip=(1,))


def _mass(shape, seed, kind):
    g = torch.Generator().manual_seed(seed)
    m = torch.exp(-9 * torch.rand(shape, generator=g))
    m.masked_fill_(torch.rand(shape, generator=g) < 0.3, 0.0)
    if kind == "ties":
        m = torch.randint(0, 3, shape, generator=g).float()
    elif kind == "zero":
        m.zero_()
    elif kind == "odd":
        m[..., ::5] = float("nan")
        m[..., 1::7] = float("inf")
        m[..., 2::7] = -0.0
        m[..., 3::7] = -1.5
    return m


def _check_evict(lens, capacity, page, keep, sinks, recent, kind="plain", seed=40):
    cache = _cache(lens, capacity, page, seed)
    B, nblk = len(lens), cache.capacity // 4
    mass = _mass((B, nblk), seed + 1, kind)
    for b, n in enumerate(lens):
        mass[b, (n + 3) // 4:] = 0.0
    ev = qsa.Evictor(cache, keep, sinks, recent, mass=mass.to(DEV))
    rows = [[cache.kv_rows(b, g, n) for g in range(2)] for b, n in enumerate(lens)]
    rows = [[(k.clone(), v.clone()) for k, v in r] for r in rows]
    kbar = [cache.kbar_rows(b, n // 4).clone() for b, n in enumerate(lens)]
    partial = cache.kbar_partial.clone()
    pools = [x.clone() for x in (cache.k_blocks, cache.v_blocks, cache.kbar)]
    kept = ev.evict(with_kept=True)
    torch.cuda.synchronize()
    assert ev.device_error() == ("QSA_OK", 0)
    kept = kept.cpu().numpy()
    for b, n in enumerate(lens):
        nb, tail = divmod(n, 4)
        want = oracle_evict.kept_blocks(mass[b].numpy(), nb, keep, sinks, recent)
        assert list(kept[b, :len(want)]) == want and np.all(kept[b, len(want):] == -1)
        m = n if nb <= keep else 4 * keep + tail
        assert cache.h_len[b] == m and int(cache.len[b]) == m
        tok = torch.tensor([4 * i + j for i in want for j in range(4)]
                           + list(range(4 * nb, n)), dtype=torch.long, device=DEV)
        for g in range(2):
            k, v = cache.kv_rows(b, g, m)
            assert torch.equal(k, rows[b][g][0][tok]) and torch.equal(v, rows[b][g][1][tok])
        at = torch.tensor(want, dtype=torch.long, device=DEV)
        assert torch.equal(cache.kbar_rows(b, len(want)), kbar[b][at])
        if nb > keep:
            new = torch.zeros(nblk)
            old = want + ([nb] if tail else [])
            new[:len(old)] = mass[b][old]
        else:
            new = mass[b]
        assert torch.equal(torch.nan_to_num(ev.mass[b].cpu(), nan=-7.0),
                           torch.nan_to_num(new, nan=-7.0))
    assert torch.equal(cache.kbar_partial, partial)
    return cache, pools


@pytest.mark.parametrize("page", PAGES)
@pytest.mark.parametrize("lens,keep,sinks,recent", [
    ([8], 1, 0, 0), ([9], 1, 0, 0), ([1, 3, 4, 7], 1, 0, 0), ([2047, 2046, 2045, 2044], 100, 4, 16),
    ([3000, 12, 1000, 401], 100, 1, 1), ([4096], 512, 512, 0), ([4096], 512, 0, 512),
    ([4095], 1022, 1, 2), ([4093, 17], 3, 1, 1)])
def test_evict(lens, keep, sinks, recent, page):
    _check_evict(lens, 4096, page, keep, sinks, recent)


@pytest.mark.parametrize("kind", ["ties", "zero", "odd"])
@pytest.mark.parametrize("page", PAGES)
def test_evict_equal_and_odd_weights(kind, page):
    _check_evict([4001, 2500, 333], 4096, page, 200, 2, 9, kind=kind)


def test_evict_long_row_and_many_rows():
    _check_evict([100001], 100004, 0, 9000, 4, 100, seed=50)
    _check_evict([600 + 7 * i for i in range(70)], 1536, 512, 100, 1, 8, seed=51)


@pytest.mark.parametrize("kind", ["plain", "ties", "zero"])
def test_evict_row_over_a_cluster(kind):
    # rows of 40,001 blocks: several CTAs each, parts that start at odd places, a short row beside
    _check_evict([160007, 40], 160012, 0, 20001, 3, 77, kind=kind, seed=52)


def test_evict_keeps_nearly_all_or_nearly_nothing():
    _check_evict([60003], 60004, 512, 14999, 0, 0, seed=53)
    _check_evict([60003], 60004, 0, 1, 0, 1, seed=54)
    _check_evict([60003], 60004, 0, 17, 16, 0, seed=55)


def test_evict_twice_in_a_row():
    # the second cut finds the first one's lengths, weights and flags
    cache = _cache([6001, 300, 2000], 6004, 0, seed=56)
    mass = _mass((3, 1501), 57, "plain").to(DEV)
    keys = [cache.kv_rows(b, 0, 6000)[0].clone() for b in range(3)]
    first = qsa.Evictor(cache, 700, 1, 5, mass=mass)
    k1 = first.evict(with_kept=True).cpu().numpy()
    second = qsa.Evictor(cache, 300, 0, 2, mass=mass)
    k2 = second.evict(with_kept=True).cpu().numpy()
    torch.cuda.synchronize()
    assert first.device_error() == second.device_error() == ("QSA_OK", 0)
    assert cache.h_len == [1201, 300, 1200] and cache.len.tolist() == cache.h_len
    for b in (0, 2):
        old = [k1[b, i] if k1[b, i] >= 0 else i for i in k2[b] if i >= 0]
        tok = torch.tensor([4 * i + j for i in old for j in range(4)], device=DEV)
        assert torch.equal(cache.kv_rows(b, 0, 1200)[0], keys[b][tok])


def test_evict_touches_nothing_else():
    # blocks behind the new length and other sequences' pages keep their bytes
    cache, pools = _check_evict([1000, 50], 1024, 0, 60, 1, 4)
    for now, old in zip((cache.k_blocks, cache.v_blocks), pools):
        assert torch.equal(now[1], old[1]) and torch.equal(now[0][:, 60:], old[0][:, 60:])
    assert torch.equal(cache.kbar[0][60:], pools[2][0][60:])
    cache, pools = _check_evict([1000, 50], 1024, 512, 60, 1, 4)
    used = {int(x) for x in cache.page_table[0]}
    for now, old in zip((cache.k_blocks, cache.v_blocks, cache.kbar), pools):
        for p in set(range(cache.pool_pages)) - used:
            assert torch.equal(now[p], old[p])


def test_evict_lengths_out_of_range_are_recorded():
    cache = _cache([400, 300], 512, 0, seed=60)
    ev = qsa.Evictor(cache, 10)
    cache.len[0] = 1000
    k = cache.k_blocks.clone()
    ev.evict()
    assert ev.device_error() == ("QSA_ERR_DEVICE", 310)
    assert int(cache.len[0]) == 1000 and torch.equal(cache.k_blocks[0], k[0])
    assert int(cache.len[1]) == 40


def test_evict_length_inside_the_block_behind_the_capacity():
    # 512 tokens fit: 513 would have an incomplete block of their own behind the last row's end
    for length in (511, 512, 513, 515):
        cache = _cache([300, 400], 512, 0, seed=65)
        ev = qsa.Evictor(cache, 10)
        cache.len[1] = length
        k = cache.k_blocks.clone()
        ev.evict()
        assert int(cache.len[0]) == 40
        if length <= 512:
            assert ev.device_error() == ("QSA_OK", 0)
            assert int(cache.len[1]) == 40 + length % 4
        else:
            assert ev.device_error() == ("QSA_ERR_DEVICE", 310)
            assert int(cache.len[1]) == length and torch.equal(cache.k_blocks[1], k[1])


def test_evict_bad_page_is_not_followed():
    cache = _cache([1000], 1024, 512, seed=61)
    other = [p for p in range(cache.pool_pages) if p not in cache.page_table.flatten().tolist()]
    cache.page_table[0, 1] = cache.pool_pages + 5
    before = cache.k_blocks.clone()
    ev = qsa.Evictor(cache, 100, 0, 0)
    ev.mass[0, 100:250] = 1.0
    ev.evict()
    status, site = ev.device_error()
    assert status == "QSA_ERR_DEVICE" and site in (311, 312)
    for p in other:
        assert torch.equal(cache.k_blocks[p], before[p])


def test_evict_in_a_graph_on_another_stream():
    cache = _cache([2000, 1500], 2048, 0, seed=62)
    mass = _mass((2, 512), 63, "plain").to(DEV)
    ev = qsa.Evictor(cache, 300, 2, 5, mass=mass)
    twin = _cache([2000, 1500], 2048, 0, seed=62)
    ev2 = qsa.Evictor(twin, 300, 2, 5, mass=mass.clone())
    ev2.evict()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        ev.evict()
    g.replay()
    g.replay()      # nothing left to cut
    torch.cuda.synchronize()
    for name in ("k_blocks", "v_blocks", "kbar", "len"):
        assert torch.equal(getattr(cache, name), getattr(twin, name)), name
    assert torch.equal(ev.mass, ev2.mass)


def test_binding_refusals():
    cache = _cache([40, 30], 64, 0, seed=64)
    with pytest.raises(qsa.QSAError):
        qsa.Evictor(cache, 4, 3, 2)
    with pytest.raises(ValueError):
        qsa.Evictor(cache, 4, mass=torch.zeros((2, 15), device=DEV))
    ev = qsa.Evictor(cache, 4)
    q = torch.zeros((2, 24, 128), dtype=torch.bfloat16, device=DEV)
    i = torch.zeros((2, 4), dtype=torch.int32, device=DEV)
    with pytest.raises(ValueError):
        ev.accumulate(q[:1], i, i[:, 0].contiguous())
    with pytest.raises(TypeError):
        ev.accumulate(q, i.long(), i[:, 0].contiguous())


# ---- together: a small hybrid stack decodes with a bounded cache --------------------------------
@pytest.mark.parametrize("page", PAGES)
def test_hybrid_decode_with_a_bounded_cache(page):
    """Delta-rule layers fed a prompt in pieces, then decode steps of both kinds of layer; the
    attention's cache is cut whenever it passes 96 blocks.  Every step's attention output must
    equal the decode of a fresh cache that holds the kept tokens only, and the delta-rule
    outputs the oracle's."""
    B, heads, key_heads, steps = 2, 4, 2, 48
    lens = [380, 371]
    cache = _cache(lens, 512, page, seed=70)
    ev, dec = qsa.Evictor(cache, 64, 1, 8), qsa.Decoder(cache, 32)
    toks = [[(cache.kv_rows(b, 0, n), cache.kv_rows(b, 1, n)) for b, n in enumerate(lens)]][0]
    hist = [[torch.stack([t[g][i] for g in range(2)], 1).clone() for i in range(2)] for t in toks]
    live = [list(range(n)) for n in lens]            # original tokens still in the cache
    spec = W.small_decode_spec(batch=B, context=lens, capacity=512, topk=32, steps=steps, seed=70)
    _, _, ki = W.decode_context(spec)
    kidx = [ki[b, :n].to(DEV) for b, n in enumerate(lens)]
    # the prompt of the delta-rule layer in two pieces
    total = 150 + steps
    w = W.gated_deltanet([total] * B, heads, seed=71)
    q, k, v, la, be = (x.view(B, total, *x.shape[1:]).to(DEV)
                       for x in (w.q[:, :key_heads].contiguous(), w.k[:, :key_heads].contiguous(),
                                 w.v, w.log_alpha, w.beta))
    states = torch.zeros((B, heads, 128, 128), device=DEV)
    outs = [[] for _ in range(B)]
    for a, b_ in ((0, 100), (100, 150)):
        piece = [x[:, a:b_].reshape(B * (b_ - a), *x.shape[2:]).contiguous() for x in (q, k, v, la, be)]
        o = qsa.gated_deltanet_extend(*piece, [0, b_ - a, 2 * (b_ - a)], states)
        for b in range(B):
            outs[b].append(o[b * (b_ - a):(b + 1) * (b_ - a)])
    cuts = 0
    for s in range(steps):
        st = {n: x.to(DEV) for n, x in W.decode_step(spec, s).items()}
        x = [y[:, 150 + s:151 + s].contiguous() for y in (q, k, v, la, be)]
        o = qsa.gated_deltanet_step(*x, states)
        cache.append(st["k"], st["v"], st["k_idx"])
        for b in range(B):
            outs[b].append(o[b])
            live[b].append(hist[b][0].shape[0])
            hist[b][0] = torch.cat([hist[b][0], st["k"][b]])
            hist[b][1] = torch.cat([hist[b][1], st["v"][b]])
            kidx[b] = torch.cat([kidx[b], st["k_idx"][b]])
        got, idx, cnt = dec.run(st["q"], st["q_idx"], st["w"], with_selection=True)
        ev.accumulate(st["q"], idx, cnt)
        if s % 11 == 0:
            assert cache.h_len == [len(x) for x in live]
            fresh = qsa.KVCache(B, 512, DEV)
            n = max(len(x) for x in live)
            pad = lambda y, i: torch.nn.functional.pad(  # noqa: E731
                y[torch.tensor(i, device=DEV)], (0, 0) * (y.dim() - 1) + (0, n - len(i)))
            fresh.append(*(torch.stack([pad(h, i) for h, i in zip(y, live)]).contiguous()
                           for y in ([h[0] for h in hist], [h[1] for h in hist], kidx)),
                         counts=[len(x) for x in live])
            want, widx, _ = qsa.Decoder(fresh, 32).run(st["q"], st["q_idx"], st["w"],
                                                       with_selection=True)
            assert torch.equal(idx, widx) and torch.equal(got, want)
        if max(cache.h_len) // 4 > 96:
            kept = ev.evict(with_kept=True).cpu().tolist()
            cuts += 1
            for b in range(B):
                nb = len(live[b]) // 4
                if nb > 64:
                    live[b] = [live[b][4 * i + j] for i in kept[b] for j in range(4)] \
                        + live[b][4 * nb:]
    torch.cuda.synchronize()
    assert cuts >= 1 and ev.device_error() == dec.device_error() == ("QSA_OK", 0)
    for b in range(B):
        ref, ref_state = gated_delta_rule(*(_np(x[b]) for x in (q, k, v, la, be)),
                                          np.zeros((heads, 128, 128)))
        tol = 2.0 ** -8 * np.abs(ref) + (512 * 2.0 ** -24 + 2.0 ** -10) * 2.0
        assert np.all(np.abs(_np(torch.cat(outs[b])) - ref) <= tol)
        assert np.abs(_np(states[b]) - ref_state).max() <= 512 * 2.0 ** -24 * 2.0

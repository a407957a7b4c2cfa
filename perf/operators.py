"""Workloads of the operators that serve a hybrid stack's two kinds of memory while it decodes:
the Gated DeltaNet layers' recurrent state and the sparse attention layers' KV cache.

* ``extend``: the gated delta rule over packed sequences, in chunks, each sequence entered with
  and leaving its state in a slot of a pool (a prompt that arrives in pieces).
* ``step``: the same rule token by token for a batch of decoding sequences (one new token each,
  or a short drafted run of which `counts[b]` tokens are taken).
* ``weights``: the attention weight that one decode step gives to every selected 4-token block,
  summed over the 24 query heads and added to the cache's running weights.
* ``evict``: each cached sequence keeps its `keep` blocks of largest running weight (the first
  `sinks` and last `recent` ones always), compacted in place.

``run`` computes each in plain torch operations, or, where ``own`` is true, through this
package's entry points.
"""
from __future__ import annotations

import math

import torch

own = False

DEV = "cuda"
D = 128                       # head width of the delta rule and of the attention
HEADS, KV_HEADS, GROUP = 24, 2, 12
BLOCK, IDX_DIM, TOPK = 4, 64, 512
CHUNK = 64
MIN_LOG_ALPHA = -87.0         # a smaller log gate counts as this (alpha of about 1.6e-38)


# ---- the cases -----------------------------------------------------------------------------
def listed():
    return [
        # the repository's own Gated DeltaNet workload: a batch of full prompts
        dict(name="extend_8x8192_h16", op="extend", lens="8192 " * 7 + "8192", heads=16, key_heads=16,
             reset=0, lo=0.9),
        # one long prompt alone, two value heads to a key head: few rows, a long axis
        dict(name="extend_1x65536_h32", op="extend", lens="65536", heads=32, key_heads=16, reset=0,
             lo=0.9),
        # pieces of ragged prompts around the chunk's length, with gates that reset the state
        dict(name="extend_ragged_h4", op="extend", lens="1 63 64 65 200 1000 37", heads=4,
             key_heads=2, reset=29, lo=0.5),
        # two pieces of a few hundred tokens in a mixed batch
        dict(name="extend_2x513_h32", op="extend", lens="513 390", heads=32, key_heads=16, reset=0,
             lo=0.9),
        # one sequence, one token: the smallest call, all latency
        dict(name="step_1x1_h32", op="step", batch=1, n=1, counted=False, heads=32, key_heads=16),
        # the decode batch of the repository's 256K workload, one token each
        dict(name="step_64x1_h32", op="step", batch=64, n=1, counted=False, heads=32, key_heads=16),
        # drafted runs of up to five tokens, some rejected (counts 0..5), some rows padding
        dict(name="step_24x5_h16", op="step", batch=24, n=5, counted=True, heads=16, key_heads=16),
        # one long conversation
        dict(name="weights_b1_64k", op="weights", batch=1, context=65533, page=0),
        # a decode batch on a paged cache
        dict(name="weights_b64_32k_paged", op="weights", batch=64, context=32766, page=4096),
        # a short cache cut to half
        dict(name="evict_b1_8k", op="evict", batch=1, context=8191, page=0, keep=1024, sinks=1,
             recent=32),
        # a batch of long caches cut to half their length
        dict(name="evict_b16_64k", op="evict", batch=16, context=65535, page=0, keep=8192, sinks=4,
             recent=128),
        # the longest context on a paged cache cut to a quarter
        dict(name="evict_b1_1m_paged", op="evict", batch=1, context=1048574, page=4096, keep=65536,
             sinks=4, recent=512),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["extend", "step", "weights", "evict"])
    if op in ("extend", "step"):
        key_heads = rng.choice([1, 2, 3, 4, 6, 8, 16])
        heads = key_heads * rng.choice([1, 2, 4])
    if op == "extend":
        n = rng.randint(1, 9)
        most = max(1, 65536 * 32 // heads // 2 // n)
        lens = [_log_int(rng, 1, min(most, 65536)) for _ in range(n)]
        return dict(op=op, lens=" ".join(map(str, lens)), heads=heads, key_heads=key_heads,
                    reset=rng.choice([0, 0, rng.randint(5, 200)]), lo=rng.choice([0.3, 0.7, 0.9, 0.99]))
    if op == "step":
        n = rng.choice([1, 1, rng.randint(2, 16)])
        return dict(op=op, batch=_log_int(rng, 1, max(1, 8192 // heads)), n=n,
                    counted=n > 1 and rng.random() < 0.7, heads=heads, key_heads=key_heads)
    if op == "weights":
        batch = _log_int(rng, 1, 64)
        return dict(op=op, batch=batch, context=_log_int(rng, 5, min(262144, 2097152 // batch)),
                    page=rng.choice([0, 512, 4096]))
    batch = _log_int(rng, 1, 16)
    context = _log_int(rng, 200, min(1048575, 1048576 // batch))
    keep = max(1, int(context // BLOCK * rng.uniform(0.1, 0.9)))
    return dict(op=op, batch=batch, context=context, page=rng.choice([0, 512, 4096]), keep=keep,
                sinks=min(keep // 4, rng.choice([0, 1, 4])), recent=min(keep // 4, rng.choice([0, 32, 300])))


# ---- inputs --------------------------------------------------------------------------------
def _unit_rows(shape, g):
    x = torch.randn(shape, generator=g, device=DEV)
    return (x / x.norm(dim=-1, keepdim=True).clamp_min(1e-6)).to(torch.bfloat16)


def _delta_inputs(rows, heads, key_heads, g, lo, reset):
    """Unit-norm queries and keys, gates alpha ~ U(lo, 1) (alpha = 0 every `reset` tokens)."""
    la = torch.log(lo + (1 - lo) * torch.rand((rows, heads), generator=g, device=DEV))
    if reset:
        la[::reset] = float("-inf")
    return dict(q=_unit_rows((rows, key_heads, D), g), k=_unit_rows((rows, key_heads, D), g),
                v=torch.randn((rows, heads, D), generator=g, device=DEV).to(torch.bfloat16),
                log_alpha=la, beta=torch.rand((rows, heads), generator=g, device=DEV))


def _cache(case, g):
    """A filled cache of `batch` sequences whose lengths fall a little short of `context`, in the
    library's blocked layout (paged: a shuffled page table over a shared pool)."""
    B, ctx, page = case["batch"], case["context"], case["page"]
    lens = [max(1, ctx - (37 * i) % max(1, ctx // 2)) for i in range(B)]
    unit = page or BLOCK
    cap = (ctx + 1 + unit - 1) // unit * unit
    pages, nb = (B * cap // page, page // BLOCK) if page else (B, cap // BLOCK)
    s = dict(lens=lens, cap=cap, pages=pages, nb=nb)
    s["k_blocks"] = torch.randn((pages, KV_HEADS, nb, BLOCK, D), generator=g, device=DEV, dtype=torch.bfloat16)
    s["v_blocks"] = torch.randn((pages, KV_HEADS, nb, BLOCK, D), generator=g, device=DEV, dtype=torch.bfloat16)
    s["kbar"] = torch.randn((pages, nb, IDX_DIM), generator=g, device=DEV, dtype=torch.bfloat16)
    s["len"] = torch.tensor(lens, dtype=torch.int32, device=DEV)
    s["table"] = (torch.randperm(pages, generator=g, device=DEV).to(torch.int32).view(B, cap // page)
                  if page else None)
    if own:
        import block_sparse_attention_40_b200 as qsa
        dev = s["len"].device
        c = (qsa.PagedKVCache(B, cap, page, pages, s["table"], dev, zero=False) if page
             else qsa.KVCache(B, cap, dev, zero=False))
        c.k_blocks, c.v_blocks, c.kbar, c.len = s["k_blocks"], s["v_blocks"], s["kbar"], s["len"]
        c.h_len = list(lens)
        s["cache"] = c
    return s


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    op = case["op"]
    if op == "extend":
        lens = [int(x) for x in case["lens"].split()]
        s = _delta_inputs(sum(lens), case["heads"], case["key_heads"], g, case["lo"], case["reset"])
        slots = len(lens) + 1
        s["states"] = torch.randn((slots, case["heads"], D, D), generator=g, device=DEV) * 0.3
        s["slots"] = torch.randperm(slots, generator=g, device=DEV)[:len(lens)].to(torch.int32)
        s["lens"] = lens
        s["cu"] = torch.tensor([0] + torch.tensor(lens).cumsum(0).tolist(), dtype=torch.int32)
        if own:
            import block_sparse_attention_40_b200 as qsa
            s["plan"] = qsa.DeltaExtend(s["cu"], case["heads"], DEV, key_heads=case["key_heads"])
    elif op == "step":
        B, n, H = case["batch"], case["n"], case["heads"]
        s = _delta_inputs(B * n, H, case["key_heads"], g, 0.9, 0)
        s = {k: x.view(B, n, *x.shape[1:]) for k, x in s.items()}
        s["states"] = torch.randn((B + 3, H, D, D), generator=g, device=DEV) * 0.3
        s["slots"] = torch.randperm(B + 3, generator=g, device=DEV)[:B].to(torch.int32)
        s["counts"] = None
        if case["counted"]:
            s["counts"] = torch.randint(0, n + 1, (B,), generator=g, device=DEV, dtype=torch.int32)
            s["slots"][3::8] = -1        # rows of a padded batch
        s["out"] = torch.zeros((B, n, H, D), dtype=torch.bfloat16, device=DEV)
    else:
        s = _cache(case, g)
        B, nblk = case["batch"], s["cap"] // BLOCK
        if op == "weights":
            s["q"] = torch.randn((B, HEADS, D), generator=g, device=DEV).to(torch.bfloat16)
            # a decode step's selection: up to TOPK complete blocks before the query's own
            cand = (s["len"].long() - 1) // BLOCK
            cnt = cand.clamp_max(TOPK)
            score = torch.rand((B, nblk), generator=g, device=DEV)
            score.masked_fill_(torch.arange(nblk, device=DEV) >= cand[:, None], -1.0)
            idx = torch.full((B, TOPK), nblk, dtype=torch.int64, device=DEV)
            k = min(TOPK, nblk)
            idx[:, :k] = score.topk(k, dim=1).indices
            idx.masked_fill_(torch.arange(TOPK, device=DEV) >= cnt[:, None], nblk)
            idx = idx.sort(dim=1).values
            s["idx"] = idx.masked_fill(idx == nblk, -1).to(torch.int32)
            s["cnt"] = cnt.to(torch.int32)
            s["mass"] = 0.05 * torch.rand((B, nblk), generator=g, device=DEV)
            keep, sinks, recent = 1, 0, 0
        else:
            # running weights fall off over four decades; many blocks were never attended
            m = torch.exp(-9.0 * torch.rand((B, nblk), generator=g, device=DEV))
            m.masked_fill_(torch.rand((B, nblk), generator=g, device=DEV) < 0.3, 0.0)
            used = (s["len"].long() + BLOCK - 1) // BLOCK
            s["mass0"] = m.masked_fill_(torch.arange(nblk, device=DEV) >= used[:, None], 0.0)
            s["mass"] = m.clone()
            s["len0"] = s["len"].clone()
            s["keep"], s["sinks"], s["recent"] = case["keep"], case["sinks"], case["recent"]
            keep, sinks, recent = case["keep"], case["sinks"], case["recent"]
        if own:
            import block_sparse_attention_40_b200 as qsa
            s["evictor"] = qsa.Evictor(s["cache"], keep, sinks, recent, mass=s["mass"])
    s["op"] = op
    return s


# ---- one pass ------------------------------------------------------------------------------
def run(s):
    op = s["op"]
    if op == "extend":
        if own:
            out = s["plan"].run(s["q"], s["k"], s["v"], s["log_alpha"], s["beta"], s["states"],
                                slots=s["slots"])
        else:
            out = _plain_extend(s)
        return dict(out=out, states=s["states"])
    if op == "step":
        if own:
            import block_sparse_attention_40_b200 as qsa
            qsa.gated_deltanet_step(s["q"], s["k"], s["v"], s["log_alpha"], s["beta"], s["states"],
                                    slots=s["slots"], counts=s["counts"], out=s["out"])
        else:
            _plain_step(s)
        return dict(out=s["out"], states=s["states"])
    if op == "weights":
        if own:
            s["evictor"].accumulate(s["q"], s["idx"], s["cnt"])
        else:
            _plain_weights(s)
        return s["mass"]
    # every pass cuts the same cache again: its lengths and weights (a small part of it) are set
    # back first, on either side
    s["len"].copy_(s["len0"])
    s["mass"].copy_(s["mass0"])
    if own:
        s["cache"].h_len = list(s["lens"])
        kept = s["evictor"].evict(with_kept=True)
    else:
        kept = _plain_evict(s)
    return dict(kept=kept, len=s["len"], mass=s["mass"], k=s["k_blocks"], v=s["v_blocks"], kbar=s["kbar"])


# ---- the plain forms -----------------------------------------------------------------------
def _plain_extend(s):
    """The rule in chunks of 64 tokens, all sequences padded to the longest.  Per chunk entered
    with state S (g: running log gate):  U = T (V - e^g K S^T),  T = (I + diag(beta) A)^-1
    diag(beta), A_tj = e^(g_t - g_j) k_t.k_j (j < t);  O = e^g Q S^T + M U, M_tj = e^(g_t - g_j)
    q_t.k_j (j <= t);  S <- e^(g_C) S + (e^(g_C - g) U)^T K."""
    lens, H = s["lens"], s["v"].shape[1]
    S, rep = len(lens), H // s["k"].shape[1]
    nc = max(1, (max(lens) + CHUNK - 1) // CHUNK)
    L = nc * CHUNK
    pos = torch.arange(L, device=DEV)
    n = torch.tensor(lens, device=DEV)
    live = pos < n[:, None]                                            # [S, L]
    row = (s["cu"][:-1].to(DEV).long()[:, None] + pos).clamp_max(sum(lens) - 1)

    def chunks(x, heads_rep):                                          # [S, H, nc, 64, ...]
        x = x[row].float()
        x = x * live.view(S, L, *([1] * (x.dim() - 2)))
        x = x.repeat_interleave(heads_rep, dim=2)
        return x.movedim(2, 1).reshape(S, H, nc, CHUNK, *x.shape[3:]).contiguous()

    q, k, v = chunks(s["q"], rep), chunks(s["k"], rep), chunks(s["v"], 1)
    beta = chunks(s["beta"], 1)
    g = chunks(s["log_alpha"].clamp_min(MIN_LOG_ALPHA), 1).double().cumsum(3)   # 64 bits: far resets
    diff = g[..., :, None] - g[..., None, :]
    low = torch.ones((CHUNK, CHUNK), dtype=torch.bool, device=DEV).tril()
    dec = torch.exp(diff.masked_fill(~low, float("-inf"))).float()
    del diff
    A = (k @ k.transpose(-1, -2)) * dec * beta[..., None]
    A = A.tril(-1)
    M = (q @ k.transpose(-1, -2)) * dec
    del dec
    T = torch.diag_embed(beta)
    for t in range(1, CHUNK):                                          # forward substitution
        T[..., t, :] -= (A[..., t, None, :t] @ T[..., :t, :])[..., 0, :]
    del A
    eg = torch.exp(g).float()
    ec = torch.exp(g[..., -1:] - g).float()
    gc = torch.exp(g[..., -1]).float()
    sl = s["slots"].long()
    state = s["states"][sl]                                            # [S, H, v, k]
    out = torch.empty_like(v)
    for c in range(nc):
        kc = k[:, :, c]
        u = T[:, :, c] @ (v[:, :, c] - eg[:, :, c, :, None] * (kc @ state.transpose(-1, -2)))
        out[:, :, c] = eg[:, :, c, :, None] * (q[:, :, c] @ state.transpose(-1, -2)) + M[:, :, c] @ u
        state = gc[:, :, c, None, None] * state + (ec[:, :, c, :, None] * u).transpose(-1, -2) @ kc
    s["states"][sl] = state
    out = out.view(S, H, L, D).movedim(1, 2)[live]
    return out.to(torch.bfloat16)


def _plain_step(s):
    B, n, H = s["beta"].shape
    rep = H // s["k"].shape[2]
    slots = s["slots"].long()
    rows = slots >= 0
    state = s["states"][slots.clamp_min(0)]
    a = torch.exp(s["log_alpha"].clamp_min(MIN_LOG_ALPHA))
    for t in range(n):
        on = rows if s["counts"] is None else rows & (s["counts"] > t)
        q, k = (s[x][:, t].float().repeat_interleave(rep, dim=1) for x in "qk")
        new = a[:, t, :, None, None] * state
        u = s["beta"][:, t, :, None] * (s["v"][:, t].float() - (new * k[:, :, None, :]).sum(-1))
        new = new + u[..., None] * k[:, :, None, :]
        o = (new * q[:, :, None, :]).sum(-1).to(torch.bfloat16)
        state = torch.where(on[:, None, None, None], new, state)
        s["out"][:, t] = torch.where(on[:, None, None], o, s["out"][:, t])
    at = torch.where(rows, slots, s["states"].shape[0])
    wide = torch.cat([s["states"], s["states"][:1]])                   # padding writes behind the pool
    wide[at] = state
    s["states"].copy_(wide[:-1])


def _pool_blocks(s, blk):
    """(pool page, block inside it) of logical blocks `blk` [B, n]."""
    b = torch.arange(blk.shape[0], device=DEV)[:, None]
    if s["table"] is None:
        return b.expand_as(blk), blk
    return s["table"].long()[b, blk // s["nb"]], blk % s["nb"]


def _plain_weights(s, dtype=torch.float32):
    B = s["q"].shape[0]
    idx = s["idx"].long()
    pos = s["len"].long() - 1
    blk = torch.cat([idx.clamp_min(0), (pos // BLOCK)[:, None]], dim=1)         # [B, n]
    page, at = _pool_blocks(s, blk)
    keys = s["k_blocks"][page, :, at].to(dtype)                                 # [B, n, 2, 4, 128]
    q = s["q"].to(dtype).view(B, KV_HEADS, GROUP, D)
    logit = torch.einsum("bghd,bngtd->bghnt", q, keys) / math.sqrt(D)
    tok = blk[..., None] * BLOCK + torch.arange(BLOCK, device=DEV)
    dead = (tok > pos[:, None, None]) | torch.cat([idx < 0, torch.zeros_like(idx[:, :1], dtype=torch.bool)],
                                                  dim=1)[..., None]
    logit = logit.masked_fill(dead[:, None, None], float("-inf"))
    logit = logit - logit.amax(dim=(3, 4), keepdim=True)
    p = torch.exp(logit)
    p = p / p.sum(dim=(3, 4), keepdim=True)
    w = p.sum(dim=(1, 2, 4))                                                    # [B, n]
    mass = s["mass"] if dtype == torch.float32 else s["mass"].to(dtype)
    live = torch.where(dead.all(-1), torch.zeros_like(w), w)
    return mass.scatter_add_(1, blk, live)


def _plain_evict(s):
    keep, sinks, recent = s["keep"], s["sinks"], s["recent"]
    mass, n = s["mass"], s["len"].long()
    B, nblk = mass.shape
    nb, tail = n // BLOCK, n % BLOCK
    i = torch.arange(nblk, device=DEV)
    key = mass.masked_fill((i < sinks) | (i >= (nb - recent)[:, None]), float("inf"))
    key = key.masked_fill(i >= nb[:, None], float("-inf"))
    order = key.sort(dim=1, descending=True, stable=True).indices
    cut = nb > keep
    k = min(keep, nblk)
    kept = order[:, :k].sort(dim=1).values
    j = torch.arange(k, device=DEV)
    kept = torch.where(cut[:, None], kept, j)
    said = torch.where(j < nb[:, None], kept, -1).to(torch.int32)
    if k < keep:
        said = torch.cat([said, said.new_full((B, keep - k), -1)], dim=1)
    # the incomplete last block follows the kept ones
    m = min(k + 1, nblk)
    src = torch.arange(m, device=DEV).expand(B, m).clone()
    src[:, :k] = kept
    if m > k:
        src[:, k] = torch.where(cut & (tail > 0), nb, src[:, k])
    old = s["mass"].clone()
    (fp, fa), (tp, ta) = _pool_blocks(s, src), _pool_blocks(s, torch.arange(m, device=DEV).expand(B, m))
    for x in (s["k_blocks"], s["v_blocks"]):
        x[tp, :, ta] = x[fp, :, fa]
    tp, ta, fp, fa = (y[:, :k] for y in (tp, ta, fp, fa))              # compressed keys: whole blocks
    s["kbar"][tp, ta] = s["kbar"][fp, fa]
    s["mass"][:, :m] = torch.gather(old, 1, src)
    end = k + (tail > 0).long()
    s["mass"].masked_fill_(cut[:, None] & (i >= end[:, None]), 0.0)
    s["len"].copy_(torch.where(cut, BLOCK * keep + tail, n))
    return said


# ---- 64 bits, from the definitions ---------------------------------------------------------
def _rule(state, q, k, v, a, beta):
    """One token: S <- a S + beta (v - a S k) k^T, o = S q; state [..., v, k] in 64 bits."""
    state = state * a[..., None, None]
    u = beta[..., None] * (v - torch.matmul(state, k[..., None])[..., 0])
    state = state + u[..., None] * k[..., None, :]
    return state, torch.matmul(state, q[..., None])[..., 0]


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "extend":
        H, rep = case["heads"], case["heads"] // case["key_heads"]
        lens, cu = s["lens"], s["cu"].tolist()
        order = sorted(range(len(lens)), key=lambda i: -lens[i])       # live ones stay in front
        sl = s["slots"].long()[order]
        state = s["states"][sl].double()
        a = torch.exp(s["log_alpha"].double().clamp_min(MIN_LOG_ALPHA))
        out = torch.empty((cu[-1], H, D), dtype=torch.float64, device=DEV)
        first = torch.tensor([cu[i] for i in order], device=DEV)
        for t in range(max(lens)):
            live = sum(lens[i] > t for i in order)
            r = first[:live] + t
            q, k = (s[x][r].double().repeat_interleave(rep, dim=1) for x in "qk")
            state[:live], out[r] = _rule(state[:live], q, k, s["v"][r].double(), a[r], s["beta"][r].double())
        states = s["states"].double()
        states[sl] = state
        return dict(out=out, states=states)
    if op == "step":
        B, n, H = s["beta"].shape
        rep = H // s["k"].shape[2]
        slots = s["slots"].tolist()
        counts = [n] * B if s["counts"] is None else s["counts"].tolist()
        states, out = s["states"].double(), s["out"].double()
        for t in range(n):
            on = [b for b in range(B) if slots[b] >= 0 and counts[b] > t]
            if on:
                at = torch.tensor([slots[b] for b in on], device=DEV)
                r = torch.tensor(on, device=DEV)
                q, k = (s[x][r, t].double().repeat_interleave(rep, dim=1) for x in "qk")
                states[at], out[r, t] = _rule(states[at], q, k, s["v"][r, t].double(),
                                              torch.exp(s["log_alpha"][r, t].double()), s["beta"][r, t].double())
        return dict(out=out, states=states)
    if op == "weights":
        mass = s["mass"].double()
        for b, n in enumerate(s["lens"]):
            own_blk = (n - 1) // BLOCK
            blocks = s["idx"][b, : int(s["cnt"][b])].long().tolist() + [own_blk]
            blk = torch.tensor(blocks, device=DEV)
            if s["table"] is None:
                keys = s["k_blocks"][b][:, blk]
            else:
                keys = s["k_blocks"][s["table"][b].long()[blk // s["nb"]], :, blk % s["nb"]].transpose(0, 1)
            keys = keys.double().reshape(KV_HEADS, -1, D)[:, : 4 * (len(blocks) - 1) + n - 4 * own_blk]
            for g in range(KV_HEADS):
                q = s["q"][b, GROUP * g: GROUP * (g + 1)].double()
                p = torch.softmax(q @ keys[g].T / D ** 0.5, dim=1).sum(0)
                p = torch.nn.functional.pad(p, (0, 4 * len(blocks) - p.numel())).view(-1, BLOCK).sum(1)
                mass[b, blk] += p
        return mass
    # the moved keys and values are copies: only the choice, the lengths and the weights are computed
    keep = case["keep"]
    kept = torch.full((case["batch"], keep), -1, dtype=torch.int32)
    mass, lens = s["mass0"].cpu().double(), []
    for b, n in enumerate(s["lens"]):
        nb, tail = divmod(n, BLOCK)
        if nb <= keep:
            kept[b, :nb] = torch.arange(nb, dtype=torch.int32)
            lens.append(n)
            continue
        row = mass[b].tolist()
        middle = sorted(range(case["sinks"], nb - case["recent"]), key=lambda i: (-row[i], i))
        mine = sorted(list(range(case["sinks"])) + middle[: keep - case["sinks"] - case["recent"]]
                      + list(range(nb - case["recent"], nb)))
        kept[b] = torch.tensor(mine, dtype=torch.int32)
        new = [row[i] for i in mine] + ([row[nb]] if tail else [])
        mass[b] = torch.tensor(new + [0.0] * (mass.shape[1] - len(new)), dtype=torch.float64)
        lens.append(BLOCK * keep + tail)
    return dict(kept=kept, len=torch.tensor(lens, dtype=torch.int32), mass=mass, k=None, v=None, kbar=None)


# ---- what a pass cannot do without -----------------------------------------------------------
def work(case):
    op = case["op"]
    if op in ("extend", "step"):
        H, Hk = case["heads"], case["key_heads"]
        if op == "extend":
            lens = [int(x) for x in case["lens"].split()]
            tokens, seqs = sum(lens), len(lens)
        else:
            tokens, seqs = case["batch"] * case["n"], case["batch"]
            if case["counted"]:          # half of the drafted tokens, seven rows of eight
                tokens, seqs = tokens * 7 // 16, seqs * 7 // 8
        state = seqs * H * D * D * 4
        rows = tokens * (2 * Hk * D * 2 + 2 * H * D * 2 + 2 * H * 4)
        return dict(bytes=2 * state + rows, flops=6 * D * D * tokens * H)
    B, ctx = case["batch"], case["context"]
    lens = [max(1, ctx - (37 * i) % max(1, ctx // 2)) for i in range(B)]
    if op == "weights":
        blocks = sum(min(TOPK, (n - 1) // BLOCK) + 1 for n in lens)
        return dict(bytes=blocks * (KV_HEADS * BLOCK * D * 2 + 4 + 8) + B * HEADS * D * 2,
                    flops=blocks * BLOCK * HEADS * D * 2)
    moved = sum(case["keep"] - case["sinks"] for n in lens if n // BLOCK > case["keep"])
    rows = sum(n // BLOCK for n in lens)
    return dict(bytes=rows * 4 + case["keep"] * B * 4 + moved * 2 * (2 * KV_HEADS * BLOCK * D * 2 + IDX_DIM * 2 + 4),
                flops=rows)

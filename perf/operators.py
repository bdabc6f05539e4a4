"""The block-selected attention, cached attention and cache eviction operators as measured work.

Each case is one call that a program makes: the plain form in elementary torch operations, or (`own`)
the library's entry points. Kinds:

  select   block means of the keys and the blocks that every query selects (a prefill's first half)
  forward  the whole prefill call: pool, select, attention over the selected blocks
  train    the same with its backward pass
  decode   one token per sequence over a cache: last block's mean, selection, attention over the selected blocks
  weigh    one token per sequence over the whole cache, adding each slot's softmax weight to the running sums
  evict    a cache brought back to `keep` slots per head by those sums
"""
import math

import torch

own = False

_NEG = float("-inf")


def listed():
    return [
        # the first chunk of a short prompt, small heads: launch latency counts
        dict(name="select_small", kind="select", B=1, H=12, Hkv=2, N=1024, Nk=1024, d=64, block=64, n_sel=8, causal=True, topics=True),
        # a long document at fine blocks: 1024 blocks to choose from
        dict(name="select_long", kind="select", B=1, H=24, Hkv=4, N=65536, Nk=65536, d=128, block=64, n_sel=16, causal=True, topics=True),
        # a chunk of a prompt whose earlier part is in the cache, ragged sizes, three heads a group
        dict(name="forward_chunk", kind="forward", B=2, H=12, Hkv=4, N=333, Nk=1999, d=64, block=64, n_sel=8, causal=True, topics=False),
        # prefill of a long document, eight heads a group
        dict(name="forward_long", kind="forward", B=1, H=16, Hkv=2, N=32760, Nk=32760, d=128, block=64, n_sel=16, causal=True, topics=True),
        # bidirectional video tokens, as many key heads as query heads, larger blocks
        dict(name="forward_video", kind="forward", B=1, H=12, Hkv=12, N=16380, Nk=16380, d=128, block=128, n_sel=16, causal=False, topics=True),
        # a right-padded training batch of odd lengths
        dict(name="train_ragged", kind="train", B=3, H=8, Hkv=2, N=1500, Nk=1500, d=64, block=64, n_sel=6, causal=True, topics=True, ragged=True),
        # training on long sequences
        dict(name="train_long", kind="train", B=1, H=16, Hkv=4, N=16384, Nk=16384, d=128, block=64, n_sel=16, causal=True, topics=True),
        # one user's next token
        dict(name="decode_one", kind="decode", B=1, H=24, Hkv=8, cap=8192, d=128, block=64, n_sel=16),
        # a full serving batch over long caches
        dict(name="decode_batch", kind="decode", B=48, H=40, Hkv=8, cap=32768, d=128, block=64, n_sel=32),
        # a batch over bounded caches, with the running sums of what its tokens attended to
        dict(name="weigh_batch", kind="weigh", B=24, H=40, Hkv=8, cap=8192, d=128),
        # each step of a bounded cache: one slot too many
        dict(name="evict_one", kind="evict", B=32, Hkv=8, cap=2049, d=128, keep=2048, sink=4, recent=64),
        # after a prompt: half of every cache goes
        dict(name="evict_half", kind="evict", B=16, Hkv=8, cap=8192, d=128, keep=4096, sink=4, recent=256),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["select", "forward", "forward", "train", "train", "decode", "decode", "weigh", "weigh", "evict"])
    d = rng.choice([64, 128])
    Hkv = rng.choice([1, 2, 3, 4, 8])
    H = Hkv * rng.choice([1, 2, 3, 4, 5, 6, 8])
    if kind in ("select", "forward", "train"):
        block = rng.choice([64, 64, 128, 192, 256, 512])
        n_sel = rng.randint(2, 16) if block <= 128 else rng.randint(2, 6)
        top = {"select": 32768, "forward": 20000, "train": 10000}[kind]
        Nk = _log(rng, 100, top)
        B = rng.randint(1, 3) if Nk < 3000 else 1
        while H > 16 and Nk > 3000:
            Hkv, H = max(1, Hkv // 2), max(1, Hkv // 2) * (H // Hkv)
        c = dict(kind=kind, B=B, H=H, Hkv=Hkv, N=Nk, Nk=Nk, d=d, block=block, n_sel=n_sel, causal=rng.random() < 0.75, topics=rng.random() < 0.7)
        if c["causal"] and kind != "train" and rng.random() < 0.3:
            c["N"] = _log(rng, 1, Nk)
        if kind == "train" and B > 1 and c["causal"]:
            c["ragged"] = rng.random() < 0.5
        return c
    B, cap = _log(rng, 1, 32), _log(rng, 200, 32768)
    while B * Hkv * cap > 4_000_000:
        B, cap = max(1, B // 2), max(200, cap * 2 // 3)
    if kind == "decode":
        return dict(kind=kind, B=B, H=H, Hkv=Hkv, cap=cap, d=d, block=rng.choice([64, 64, 128, 256]), n_sel=rng.randint(2, 32))
    if kind == "weigh":
        return dict(kind=kind, B=B, H=H, Hkv=Hkv, cap=cap, d=d)
    keep = cap - 1 if rng.random() < 0.4 else max(20, int(cap * rng.uniform(0.2, 0.9)))
    return dict(kind=kind, B=B, Hkv=Hkv, cap=cap, d=d, keep=keep, sink=rng.randint(0, 4), recent=rng.randint(1, max(1, keep // 3)))


def _q_start(c):
    return c["Nk"] - c["N"]


def _lengths(c):
    """Right-padded lengths of a ragged batch: the first sequence is full."""
    if not c.get("ragged"):
        return None
    return [max(1, c["Nk"] - 1 - (b * 389) % c["Nk"]) if b else c["Nk"] for b in range(c["B"])]


# ----------------------------------------------------------------------------- inputs


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _qkv(g, B, H, Hkv, N, Nk, d, topics):
    """Keys and queries that share topics over runs of tokens (neighbouring queries mostly want the same
    blocks, as in text and video), or independent normals."""
    k, v, q = _randn(g, B, Hkv, Nk, d), _randn(g, B, Hkv, Nk, d), _randn(g, B, H, N, d)
    if topics:
        C = 48
        cen = _randn(g, B, Hkv, C, d) * 0.6
        tk = torch.randint(C, (B, Hkv, (Nk + 39) // 40), generator=g, device="cuda").repeat_interleave(40, -1)[..., :Nk]
        tq = torch.randint(C, (B, Hkv, (N + 95) // 96), generator=g, device="cuda").repeat_interleave(96, -1)[..., :N]
        k += cen.gather(2, tk.unsqueeze(-1).expand(-1, -1, -1, d))
        q += cen.gather(2, tq.unsqueeze(-1).expand(-1, -1, -1, d)).repeat_interleave(H // Hkv, 1)
    return q.bfloat16(), k.bfloat16(), v.bfloat16()


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda").manual_seed(seed)
    s = dict(case=c)
    if c["kind"] in ("select", "forward", "train"):
        s["q"], s["k"], s["v"] = _qkv(g, c["B"], c["H"], c["Hkv"], c["N"], c["Nk"], c["d"], c["topics"])
        ln = _lengths(c)
        s["lengths"] = None if ln is None else torch.tensor(ln, dtype=torch.int32, device="cuda")
        if c["kind"] == "train":
            s["do"] = _randn(g, c["B"], c["H"], c["N"], c["d"]).bfloat16()
            for n in "qkv":
                s[n].requires_grad_(True)
        return s
    B, Hkv, cap, d = c["B"], c["Hkv"], c["cap"], c["d"]
    if c["kind"] == "evict":
        s["k"], s["v"] = _randn(g, B, Hkv, cap, d).bfloat16(), _randn(g, B, Hkv, cap, d).bfloat16()
        # a few slots hold most of the weight
        s["w0"] = _randn(g, B, Hkv, cap).mul_(1.5).exp_()
        s["p0"] = torch.argsort(torch.rand(B, Hkv, cap, generator=g, device="cuda"), -1).int()
        s["l0"] = torch.full((B,), cap, dtype=torch.int32, device="cuda")
        s["weight"], s["pos"], s["lengths"] = s["w0"].clone(), s["p0"].clone(), s["l0"].clone()
        return s
    s["q"], s["k"], s["v"] = _qkv(g, B, c["H"], Hkv, 1, cap, d, True)
    # sequences between half and all of the cache
    s["lengths"] = cap - torch.randint(cap // 2, (B,), generator=g, device="cuda").int()
    if c["kind"] == "decode":
        # the means as the earlier tokens left them
        s["pool"] = _pool(s["k"], c["block"], s["lengths"])
    else:
        s["weight"] = torch.rand(B, Hkv, cap, generator=g, device="cuda")
    return s


# ----------------------------------------------------------------------------- plain forms


def _pool(k, block, lengths):
    """Mean of each block's valid keys: summed in 64 bits, since a selection hangs on it, rounded once."""
    B, Hkv, Nk, d = k.shape
    nb = -(-Nk // block)
    ln = torch.full((B,), Nk, device=k.device) if lengths is None else lengths.long()
    ok = torch.arange(Nk, device=k.device)[None, :] < ln[:, None]
    x = torch.zeros(B, Hkv, nb * block, d, dtype=torch.float64, device=k.device)
    x[:, :, :Nk] = torch.where(ok[:, None, :, None], k.detach().double(), 0.0)
    n = (ln[:, None] - torch.arange(nb, device=k.device)[None, :] * block).clamp(0, block)
    return (x.view(B, Hkv, nb, block, d).sum(3) / n.clamp(min=1)[:, None, :, None]).float()


def _select(q, pool, c, pos, ln):
    """The n_sel best blocks of each query, ascending, -1 behind them. Scores in 64 bits: neighbours in the
    order can be close."""
    B, H, N, d = q.shape
    Hkv, nb = pool.shape[1], pool.shape[2]
    qs = q.detach().double().view(B, Hkv, H // Hkv, N, d).sum(2)
    s = qs @ pool.double().transpose(-1, -2)
    blk = torch.arange(nb, device=q.device)
    cur = torch.div(pos, c["block"], rounding_mode="floor")[:, None, :, None]  # [B,1,N,1]
    if c.get("causal", True):
        forced = (blk == cur) | (blk < 1)
        there = (blk <= cur) & (pos >= 0)[:, None, :, None] & (pos < ln[:, None])[:, None, :, None]
    else:
        forced = blk < 1
        there = (blk * c["block"] < ln[:, None])[:, None, None, :]
    s = torch.where(forced, float("inf"), s)
    s = torch.where(there, s, _NEG)
    n = c["n_sel"]
    val, idx = torch.sort(s, dim=-1, descending=True, stable=True)
    idx = torch.where(val[..., :n] == _NEG, nb, idx[..., :n]).sort(-1)[0]
    out = torch.full((B, Hkv, N, n), -1, dtype=torch.int32, device=q.device)
    out[..., : idx.shape[-1]] = torch.where(idx == nb, -1, idx).int()
    return out


def _mask(idx, block, Nk, lim):
    """[B,Hkv,1,n,Nk]: the keys of each query's selected blocks below its limit."""
    nb = -(-Nk // block)
    m = torch.zeros(*idx.shape[:3], nb + 1, dtype=torch.bool, device=idx.device)
    m.scatter_(3, torch.where(idx < 0, nb, idx).long(), True)
    m = m[..., :nb].repeat_interleave(block, -1)[..., :Nk]
    return (m & (torch.arange(Nk, device=idx.device) < lim[:, None, :, None]))[:, :, None]


def _attend(q, k, v, idx, c, lim, do=None):
    """Attention over the selected blocks, and with `do` its gradient; queries in pieces, for memory alone."""
    B, H, N, d = q.shape
    Hkv, Nk = k.shape[1], k.shape[2]
    G, scale = H // Hkv, 1.0 / math.sqrt(d)
    kf, vf = k.detach().float()[:, :, None], v.detach().float()[:, :, None]
    qf = q.detach().float().view(B, Hkv, G, N, d)
    o = torch.zeros(B, Hkv, G, N, d, device=q.device)
    lse = torch.zeros(B, Hkv, G, N, device=q.device)
    if do is not None:
        dof = do.float().view(B, Hkv, G, N, d)
        dq, dk, dv = torch.zeros_like(qf), torch.zeros_like(kf), torch.zeros_like(vf)
    step = max(64, (1 << 29) // (B * H * Nk))
    for a in range(0, N, step):
        z = slice(a, a + step)
        m = _mask(idx[:, :, z], c["block"], Nk, lim[:, z])
        s = torch.where(m, qf[:, :, :, z] @ kf.transpose(-1, -2) * scale, _NEG)
        top = s.amax(-1, keepdim=True).clamp(min=-3e38)
        p = torch.exp(s - top)
        l = p.sum(-1, keepdim=True)
        lse[:, :, :, z] = torch.where(l > 0, torch.log(l) + top, _NEG)[..., 0]
        p /= torch.where(l > 0, l, 1.0)
        o[:, :, :, z] = p @ vf
        if do is not None:
            g = dof[:, :, :, z]
            dv += (p.transpose(-1, -2) @ g).sum(2, keepdim=True)
            ds = p * (g @ vf.transpose(-1, -2) - (g * o[:, :, :, z]).sum(-1, keepdim=True)) * scale
            dq[:, :, :, z] = ds @ kf
            dk += (ds.transpose(-1, -2) @ qf[:, :, :, z]).sum(2, keepdim=True)
    o, lse = o.view(B, H, N, d).to(q.dtype), lse.view(B, H, N)
    if do is None:
        return o, lse
    return o, lse, dq.view(B, H, N, d).to(q.dtype), dk[:, :, 0].to(k.dtype), dv[:, :, 0].to(v.dtype)


def _positions(c, q, lengths, at_end=False):
    B, N = q.shape[0], q.shape[2]
    Nk = c.get("Nk", c.get("cap"))
    ln = torch.full((B,), Nk, device=q.device) if lengths is None else lengths.long()
    if at_end:
        pos = (ln - N)[:, None] + torch.arange(N, device=q.device)
    else:
        pos = (_q_start(c) + torch.arange(N, device=q.device))[None].expand(B, N)
    lim = torch.where((pos >= 0) & (pos < ln[:, None]), pos + 1, 0) if c.get("causal", True) else ln[:, None].expand(B, N)
    return pos, ln, lim


def _plain(s):
    c = s["case"]
    kind = c["kind"]
    if kind == "evict":
        return _evict(s)
    q, k, v = s["q"], s["k"], s["v"]
    pos, ln, lim = _positions(c, q, s["lengths"], at_end=kind in ("decode", "weigh"))
    if kind == "weigh":
        B, H, _, d = q.shape
        Hkv, cap = c["Hkv"], c["cap"]
        ok = (torch.arange(cap, device=q.device) < ln[:, None])[:, None, None, :]
        x = (q.float().view(B, Hkv, H // Hkv, d) @ k.float().transpose(-1, -2)) / math.sqrt(d)
        x = torch.where(ok, x, _NEG)
        top = x.amax(-1, keepdim=True)
        p = torch.exp(x - top)
        l = p.sum(-1, keepdim=True)
        p = p / l
        s["weight"] += p.sum(2)
        return dict(o=(p @ v.float()).view(B, H, 1, d).to(q.dtype), lse=(torch.log(l) + top).view(B, H, 1), weight=s["weight"])
    if kind == "decode":
        # the last block's mean, anew
        last = torch.div(ln - 1, c["block"], rounding_mode="floor")
        rows = last[:, None] * c["block"] + torch.arange(c["block"], device=q.device)
        ok = rows < ln[:, None]
        rows = rows.clamp(max=c["cap"] - 1)[:, None, :, None].expand(-1, c["Hkv"], -1, c["d"])
        x = torch.where(ok[:, None, :, None], k.gather(2, rows).double(), 0.0).sum(2) / ok.sum(1)[:, None, None]
        s["pool"].scatter_(2, last[:, None, None, None].expand(-1, c["Hkv"], 1, c["d"]), x.float()[:, :, None])
        idx = _select(q, s["pool"], c, pos, ln)
        # the selected blocks' keys and values, side by side
        at = (idx.clamp(min=0).long()[..., None] * c["block"] + torch.arange(c["block"], device=q.device)).flatten(2)
        ok = (idx >= 0)[..., None].expand(-1, -1, -1, -1, c["block"]).flatten(2) & (at < ln[:, None, None])
        at = at.clamp(max=c["cap"] - 1)[..., None].expand(-1, -1, -1, c["d"])
        kk, vv = k.gather(2, at).float(), v.gather(2, at).float()
        B, H, _, d = q.shape
        x = q.float().view(B, c["Hkv"], -1, d) @ kk.transpose(-1, -2) / math.sqrt(d)
        x = torch.where(ok[:, :, None], x, _NEG)
        top = x.amax(-1, keepdim=True)
        p = torch.exp(x - top)
        l = p.sum(-1, keepdim=True)
        return dict(o=(p @ vv / l).view(B, H, 1, d).to(q.dtype), lse=(torch.log(l) + top).view(B, H, 1), idx=idx, pool=s["pool"])
    pool = _pool(k, c["block"], s["lengths"])
    idx = _select(q, pool, c, pos, ln)
    if kind == "select":
        return dict(pool=pool, idx=idx)
    if kind == "forward":
        o, lse = _attend(q, k, v, idx, c, lim)
        return dict(o=o, lse=lse, idx=idx)
    o, _, dq, dk, dv = _attend(q, k, v, idx, c, lim, s["do"])
    return dict(o=o, dq=dq, dk=dk, dv=dv)


def _evict(s):
    """Keeps the `keep` best slots: protected ones, then by weight, ties to the lower slot. The i-th evicted
    slot below `keep` takes the i-th kept one at or above it. The bookkeeping is set back first, so that
    every pass makes the same moves."""
    c = s["case"]
    k, v, w, pos, keep = s["k"], s["v"], s["weight"], s["pos"], c["keep"]
    w.copy_(s["w0"]), pos.copy_(s["p0"]), s["lengths"].copy_(s["l0"])
    B, Hkv, cap, d = k.shape
    seen = pos.amax(-1, keepdim=True) + 1
    safe = (pos < c["sink"]) | (pos >= seen - c["recent"])
    order = torch.where(safe, float("inf"), w).sort(dim=-1, descending=True, stable=True)[1]
    kept = torch.zeros(B, Hkv, cap, dtype=torch.bool, device=k.device).scatter_(-1, order[..., :keep], True)
    m = min(keep, cap - keep)
    slot = torch.arange(cap, device=k.device)
    hole = torch.where(~kept & (slot < keep), slot, cap).sort(-1)[0][..., :m]
    src = torch.where(kept & (slot >= keep), slot, cap).sort(-1)[0][..., :m]
    # where there is no move left, the last slot (never a hole) is written onto itself
    hole, src = hole.clamp(max=cap - 1), src.clamp(max=cap - 1)
    at, to = src[..., None].expand(-1, -1, -1, d), hole[..., None].expand(-1, -1, -1, d)
    k.scatter_(2, to, k.gather(2, at)), v.scatter_(2, to, v.gather(2, at))
    w.scatter_(2, hole, w.gather(2, src)), pos.scatter_(2, hole, pos.gather(2, src))
    s["lengths"].clamp_(max=keep)
    return dict(k=k, v=v, weight=w, pos=pos, lengths=s["lengths"])


# ----------------------------------------------------------------------------- the library's calls


def _cfg(c):
    import free_sparse_attention_head_b200 as svoo
    causal = c.get("causal", True)
    return svoo.BlockConfig(block=c["block"], n_sel=c["n_sel"], sink=1, local=1 if causal else 0, causal=causal)


def _own(s):
    import free_sparse_attention_head_b200 as svoo
    c = s["case"]
    kind = c["kind"]
    if kind == "evict":
        s["weight"].copy_(s["w0"]), s["pos"].copy_(s["p0"]), s["lengths"].copy_(s["l0"])
        svoo.cache_evict(s["k"], s["v"], s["weight"], s["pos"], s["lengths"], c["keep"], sink=c["sink"], recent=c["recent"])
        return {n: s[n] for n in ("k", "v", "weight", "pos", "lengths")}
    if kind == "weigh":
        o, lse = svoo.cache_attn(s["q"], s["k"], s["v"], s["lengths"], weight=s["weight"])
        return dict(o=o, lse=lse, weight=s["weight"])
    cfg = _cfg(c)
    if kind == "decode":
        svoo.block_pool(s["k"], cfg, lengths=s["lengths"], pool=s["pool"], last=1)
        idx = svoo.block_select(s["q"], s["pool"], cfg, c["cap"], lengths=s["lengths"], q_start=-1)
        o, lse = svoo.cache_attn(s["q"], s["k"], s["v"], s["lengths"], idx=idx, cfg=cfg)
        return dict(o=o, lse=lse, idx=idx, pool=s["pool"])
    if kind == "select":
        pool = svoo.block_pool(s["k"], cfg, lengths=s["lengths"])
        return dict(pool=pool, idx=svoo.block_select(s["q"], pool, cfg, c["Nk"], lengths=s["lengths"]))
    o, aux = svoo.block_attention(s["q"], s["k"], s["v"], cfg, lengths=s["lengths"])
    if kind == "forward":
        return dict(o=o, lse=aux["lse"], idx=aux["idx"])
    dq, dk, dv = torch.autograd.grad(o, (s["q"], s["k"], s["v"]), s["do"])
    return dict(o=o.detach(), dq=dq, dk=dk, dv=dv)


def run(state):
    return _own(state) if own else _plain(state)


# ----------------------------------------------------------------------------- work


def _keys_attended(c):
    """Selected keys over all query rows of one (batch, head), and candidate blocks over all rows, averaged
    over the batch."""
    keys = cands = 0
    block, n = c["block"], c["n_sel"]
    for L in _lengths(c) or [c["Nk"]] * c["B"]:
        if not c["causal"]:
            nb = -(-L // block)
            keys += c["N"] * min(L, n * block)
            cands += c["N"] * nb
            continue
        for p in range(_q_start(c), min(_q_start(c) + c["N"], L)):
            cur = p // block
            keys += min(n - 1, cur) * block + p % block + 1
            cands += cur + 1
    return keys, cands


def work(case):
    c = case
    d = c["d"]
    if c["kind"] == "evict":
        slots = c["B"] * c["Hkv"] * c["cap"]
        # a slot is moved when it is kept from behind `keep`: about (1 - keep/cap) of the kept ones
        moved = c["B"] * c["Hkv"] * c["keep"] * (1 - c["keep"] / c["cap"])
        return dict(bytes=24 * slots + moved * (8 * d + 16), flops=0)
    if c["kind"] in ("decode", "weigh"):
        L = c["cap"] * 0.75  # lengths are even between half and all
        rows = c["B"] * c["Hkv"] * (L if c["kind"] == "weigh" else min(L, c["n_sel"] * c["block"]))
        by = rows * 4 * d + 4 * c["B"] * c["H"] * d
        fl = rows * 4 * d * (c["H"] // c["Hkv"])
        if c["kind"] == "weigh":
            return dict(bytes=by + 8 * rows, flops=fl)
        nb = L / c["block"]
        return dict(bytes=by + c["B"] * c["Hkv"] * (nb * 4 * d + c["block"] * 2 * d), flops=fl + 2 * d * nb * c["B"] * c["Hkv"])
    keys, cands = _keys_attended(c)
    q, k = 2 * c["B"] * c["H"] * c["N"] * d, 2 * c["B"] * c["Hkv"] * c["Nk"] * d
    idx = 4 * c["B"] * c["Hkv"] * c["N"] * c["n_sel"]
    pick = 2 * d * cands * c["Hkv"]
    if c["kind"] == "select":
        return dict(bytes=q + k + 2 * k // c["block"] + idx, flops=pick)
    if c["kind"] == "forward":
        return dict(bytes=2 * q + 2 * k + idx, flops=pick + 4 * d * keys * c["H"])
    return dict(bytes=4 * q + 4 * k, flops=pick + 14 * d * keys * c["H"])


# ----------------------------------------------------------------------------- 64 bits


def exact(case, seed):
    """From the definitions, in 64 bits: one sequence and key head at a time, each query with its own keys."""
    c = case
    s = prepare(c, seed)
    if c["kind"] == "evict":
        return None
    B, Hkv, d = c["B"], c["Hkv"], c["d"]
    G = s["q"].shape[1] // Hkv
    N, Nk = s["q"].shape[2], s["k"].shape[2]
    lens = [Nk] * B if s["lengths"] is None else s["lengths"].tolist()
    q, k, v = (s[n].detach() for n in "qkv")
    dev, f64 = q.device, torch.float64
    o = torch.zeros(B, Hkv, G, N, d, dtype=f64, device=dev)
    lse = torch.full((B, Hkv, G, N), _NEG, dtype=f64, device=dev)
    served = c["kind"] in ("decode", "weigh")
    if c["kind"] == "weigh":
        weight = s["weight"].double()
    else:
        block, n, causal = c["block"], c["n_sel"], c.get("causal", True)
        nb = -(-Nk // block)
        pool = torch.zeros(B, Hkv, nb, d, dtype=f64, device=dev)
    if c["kind"] == "train":
        do = s["do"].view(B, Hkv, G, N, d)
        dq, dk, dv = torch.zeros_like(o), torch.zeros(B, Hkv, Nk, d, dtype=f64, device=dev), torch.zeros(B, Hkv, Nk, d, dtype=f64, device=dev)
    for b in range(B):
        L = lens[b]
        for h in range(Hkv):
            K, V = k[b, h, :L].double(), v[b, h, :L].double()
            Q = q.view(B, Hkv, G, N, d)[b, h].double()
            if c["kind"] == "weigh":
                x = Q[:, 0] @ K.T / math.sqrt(d)
                lse[b, h, :, 0] = x.logsumexp(-1)
                p = torch.exp(x - lse[b, h])
                o[b, h, :, 0] = p @ V
                weight[b, h, :L] += p.sum(0)
                continue
            for j in range(-(-L // block) if c["kind"] == "select" or L < 4 * block else 0):
                pool[b, h, j] = K[j * block:(j + 1) * block].mean(0)
            if L >= 4 * block and c["kind"] != "select":
                full = L // block
                pool[b, h, :full] = K[:full * block].view(full, block, d).mean(1)
                if L % block:
                    pool[b, h, full] = K[full * block:].mean(0)
            if c["kind"] == "select":
                continue
            # selections are made on the means as they are kept, in 32 bits
            sc_all = Q.sum(0) @ pool[b, h].float().double().T
            first = L - N if served else _q_start(c)
            for a in range(0, N, 256):
                rows = torch.arange(a, min(a + 256, N), device=dev)
                p_ = rows + first
                if causal:
                    rows = rows[(p_ >= 0) & (p_ < L)]
                    if not len(rows):
                        continue
                    p_ = rows + first
                lim = p_ + 1 if causal else torch.full_like(p_, L)
                sc = sc_all[rows].clone()
                j = torch.arange(nb, device=dev)
                sc[:, 0] = float("inf")
                if causal:
                    sc[j[None] == (p_ // block)[:, None]] = float("inf")
                sc[j[None] * block >= lim[:, None]] = _NEG
                val, at = sc.topk(min(n, nb), -1)
                keys = (at[..., None] * block + torch.arange(block, device=dev)).flatten(1)
                ok = (val > _NEG)[..., None].expand(-1, -1, block).flatten(1) & (keys < lim[:, None])
                keys = torch.where(ok, keys, 0)
                kk, vv = K[keys], V[keys]
                x = torch.einsum("grd,rkd->rgk", Q[:, rows], kk) / math.sqrt(d)
                x = torch.where(ok[:, None], x, _NEG)
                ls = x.logsumexp(-1, keepdim=True)
                p = torch.exp(x - ls)
                oo = p @ vv
                lse[b, h][:, rows] = ls[..., 0].T
                o[b, h][:, rows] = oo.transpose(0, 1)
                if c["kind"] == "train":
                    g = do[b, h][:, rows].double().transpose(0, 1)
                    ds = p * (g @ vv.transpose(-1, -2) - (g * oo).sum(-1, keepdim=True)) / math.sqrt(d)
                    dq[b, h][:, rows] = (ds @ kk).transpose(0, 1)
                    add = lambda to, x: to.index_add_(0, keys.flatten(), torch.where(ok[..., None], x, 0.0).flatten(0, 1))  # noqa: E731
                    add(dv[b, h], torch.einsum("rgk,rgd->rkd", p, g))
                    add(dk[b, h], torch.einsum("rgk,grd->rkd", ds, Q[:, rows]))
    H = Hkv * G
    o, lse = o.view(B, H, N, d), lse.view(B, H, N)
    if c["kind"] == "select":
        return dict(pool=pool, idx=None)
    if c["kind"] == "weigh":
        return dict(o=o, lse=lse, weight=weight)
    if c["kind"] == "train":
        return dict(o=o, dq=dq.view(B, H, N, d), dk=dk, dv=dv)
    if served:
        return dict(o=o, lse=lse, idx=None, pool=pool)
    return dict(o=o, lse=lse, idx=None)

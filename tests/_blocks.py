"""The block-selected attention, cached attention and eviction written out in fp64 with plain loops over
sequences, heads and queries: the reference of the tests."""
import math

import torch

F64 = torch.float64


def pool(k, block, lengths=None):
    B, Hkv, Nk, d = k.shape
    nb = -(-Nk // block)
    out = torch.zeros(B, Hkv, nb, d, dtype=F64)
    for b in range(B):
        L = Nk if lengths is None else int(lengths[b])
        for c in range(-(-L // block)):
            out[b, :, c] = k[b, :, c * block:min(L, (c + 1) * block)].to(F64).mean(1)
    return out


def positions(Nq, Nk, L, q_start):
    first = Nk - Nq if q_start is None else (L - Nq if q_start == -1 else q_start)
    return [first + i for i in range(Nq)]


def select(q, pooled, cfg, Nk, lengths=None, q_start=None):
    """Scores from the fp32 means in fp64, stable order."""
    B, H, Nq, d = q.shape
    Hkv = pooled.shape[1]
    out = torch.full((B, Hkv, Nq, cfg.n_sel), -1, dtype=torch.int32)
    for b in range(B):
        L = Nk if lengths is None else int(lengths[b])
        pos = positions(Nq, Nk, L, q_start)
        for hk in range(Hkv):
            s = q[b].view(Hkv, H // Hkv, Nq, d)[hk].to(F64).sum(0) @ pooled[b, hk].float().to(F64).T
            for i, p in enumerate(pos):
                if cfg.causal and not 0 <= p < L:
                    continue
                nc = p // cfg.block + 1 if cfg.causal else -(-L // cfg.block)
                row = s[i, :nc].tolist()
                forced = set(range(min(cfg.sink, nc))) | set(range(max(0, nc - cfg.local), nc))
                rest = sorted((c for c in range(nc) if c not in forced), key=lambda c: (-row[c], c))
                got = sorted(list(forced) + rest[:max(0, cfg.n_sel - len(forced))])
                out[b, hk, i, :len(got)] = torch.tensor(got, dtype=torch.int32)
    return out


def attn(q, k, v, idx, cfg, lengths=None, q_start=None, scale=None, grad_o=None):
    """o, lse, and with grad_o the formula's dq, dk, dv. Garbage behind a sequence is never touched."""
    B, H, Nq, d = q.shape
    Hkv, Nk = k.shape[1], k.shape[2]
    G = H // Hkv
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    o = torch.zeros(B, H, Nq, d, dtype=F64)
    lse = torch.full((B, H, Nq), -math.inf, dtype=F64)
    dq, dk, dv = torch.zeros_like(o), torch.zeros(k.shape, dtype=F64), torch.zeros(v.shape, dtype=F64)
    for b in range(B):
        L = Nk if lengths is None else int(lengths[b])
        pos = positions(Nq, Nk, L, q_start)
        for hk in range(Hkv):
            for i, p in enumerate(pos):
                lim = (p + 1 if 0 <= p < L else 0) if cfg.causal else L
                keys = [c * cfg.block + r for c in idx[b, hk, i].tolist() if c >= 0 for r in range(cfg.block)
                        if c * cfg.block + r < lim]
                if not keys:
                    continue
                K, V = k[b, hk, keys].to(F64), v[b, hk, keys].to(F64)
                rows = slice(hk * G, hk * G + G)
                Q = q[b, rows, i].to(F64)
                x = Q @ K.T * scale
                ls = x.logsumexp(-1, keepdim=True)
                P = torch.exp(x - ls)
                o[b, rows, i], lse[b, rows, i] = P @ V, ls[:, 0]
                if grad_o is not None:
                    g = grad_o[b, rows, i].to(F64)
                    ds = P * (g @ V.T - (g * (P @ V)).sum(-1, keepdim=True)) * scale
                    dq[b, rows, i] = ds @ K
                    dk[b, hk].index_add_(0, torch.tensor(keys), ds.T @ Q)
                    dv[b, hk].index_add_(0, torch.tensor(keys), P.T @ g)
    return (o, lse) if grad_o is None else (o, lse, dq, dk, dv)


def evict(weight, pos, length, keep, sink, recent):
    """One head: the (hole, source) moves."""
    if length <= keep:
        return []
    newest = max(pos[:length])
    safe = [pos[i] < sink or pos[i] > newest - recent for i in range(length)]
    w = [-math.inf if math.isnan(x) else x for x in weight[:length]]
    order = sorted(range(length), key=lambda i: (not safe[i], -w[i] if not safe[i] else 0.0, math.isnan(weight[i]) and not safe[i], i))
    kept = set(order[:keep])
    return list(zip([i for i in range(keep) if i not in kept], [i for i in range(keep, length) if i in kept]))

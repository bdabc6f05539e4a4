"""Calls of the block-selected attention whose row tiles would visit nearly every block (many queries a tile,
blocks of 128 keys and more): they go by key blocks over lists of queries. Checked on a B200 against dense masked
attention in fp64, head by head.

Tolerances. P is rounded to bf16 before the second product (at most u = 2^-8 of it), its sum is not: numerator and
denominator differ by at most u of the weights, so |o - o64| <= u max|V| + u |o| and with the output's own rounding
below 2 u max|V| + u |o|; parts and their sum are fp32, far below that.
"""
import math

import pytest
import torch

import free_sparse_attention_head_b200 as svoo

pytestmark = pytest.mark.gpu

U = torch.finfo(torch.bfloat16).eps / 2   # half a bf16 step: 2^-8


def dense(q, k, v, idx, cfg, length, pos):
    """One head in fp64: q [N, d], idx [N, n_sel], pos the queries' positions."""
    Nk = k.shape[0]
    seen = torch.zeros(q.shape[0], -(-Nk // cfg.block) + 1, dtype=torch.bool, device="cuda")
    seen.scatter_(1, idx.long().where(idx >= 0, torch.tensor(seen.shape[1] - 1, device="cuda")), True)
    m = seen[:, :-1].repeat_interleave(cfg.block, 1)[:, :Nk]
    lim = torch.where((pos >= 0) & (pos < length), pos + 1, 0) if cfg.causal else torch.full_like(pos, length)
    m &= torch.arange(Nk, device="cuda")[None] < lim[:, None]
    s = (q.double() @ k.double().T / math.sqrt(q.shape[1])).masked_fill(~m, -math.inf)
    lse = s.logsumexp(-1)
    p = torch.exp(s - lse.where(lse > -math.inf, torch.zeros_like(lse))[:, None])
    return p @ v.double().masked_fill(~m.any(0)[:, None], 0), lse


CASES = [
    # B, H, Hkv, Nq, Nk, d, block, n_sel, sink, local, causal, lengths, q_start
    (1, 64, 64, 2048, 2048, 64, 128, 3, 1, 0, False, None, None),
    (2, 32, 32, 2001, 2001, 128, 128, 3, 1, 0, False, [2001, 1930], None),
    (1, 64, 32, 1900, 3911, 64, 128, 3, 0, 1, True, None, None),
    (2, 48, 48, 1000, 4999, 128, 256, 2, 1, 1, True, [4999, 700], -1),
    (1, 48, 48, 2048, 2600, 128, 256, 2, 1, 0, False, None, None),   # the last block's second half holds no key
    (1, 24, 24, 2048, 5700, 64, 512, 2, 0, 1, True, None, None),
    (3, 40, 40, 1100, 1300, 64, 128, 2, 0, 0, False, [0, 1, 1299], 0),
]


@pytest.mark.parametrize("case", CASES, ids=str)
def test_lists_against_fp64(case):
    B, H, Hkv, Nq, Nk, d, block, n_sel, sink, local, causal, lengths, q_start = case
    g = torch.Generator(device="cuda").manual_seed(5)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda").bfloat16()  # noqa: E731
    q, k, v = r(B, H, Nq, d), r(B, Hkv, Nk, d), r(B, Hkv, Nk, d)
    cfg = svoo.BlockConfig(block=block, n_sel=n_sel, sink=sink, local=local, causal=causal)
    ln = None if lengths is None else torch.tensor(lengths, dtype=torch.int32, device="cuda")
    for b, L in enumerate(lengths or []):  # what lies behind a sequence may hold anything
        k[b, :, L:], v[b, :, L:] = math.nan, math.nan
    pool = svoo.block_pool(k, cfg, ln)
    idx = svoo.block_select(q, pool, cfg, Nk, ln, q_start)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    # a workspace that held something else: no part is read that was not written
    size = svoo._ws_bytes("svoo_block_attn_workspace_size", B, H, Hkv, Nq, Nk, Nk, d, block, n_sel, sink, local,
                          int(causal), Nk - Nq if q_start is None else q_start)
    assert size >= B * H * Nq * n_sel * block // 128 * d * 4   # the parts' place: the call goes by lists
    ws = torch.full((size,), 0x41, dtype=torch.uint8, device="cuda")
    o, lse = svoo.block_attn(q, k, v, idx, cfg, ln, q_start, workspace=ws, dev_err=err)
    again, lse2 = svoo.block_attn(q, k, v, idx, cfg, ln, q_start)
    assert torch.equal(o, again) and torch.equal(lse, lse2) and int(err) == 0
    for b in range(B):
        L = Nk if lengths is None else lengths[b]
        first = Nk - Nq if q_start is None else (L - Nq if q_start == -1 else q_start)
        pos = first + torch.arange(Nq, device="cuda")
        K, V = k[b].clone(), v[b].clone()
        K[:, L:], V[:, L:] = 0, 0
        for h in range(0, H, 7):
            hk = h // (H // Hkv)
            o64, l64 = dense(q[b, h], K[hk], V[hk], idx[b, hk], cfg, L, pos)
            fin = torch.isfinite(l64)
            assert torch.equal(torch.isfinite(lse[b, h]), fin)
            assert ((lse[b, h].double() - l64)[fin].abs() <= 2e-5 * (1 + l64[fin].abs())).all()
            tol = 2 * U * (float(V[hk].abs().max()) if L else 0.0) + U * o64.abs() + 1e-6
            assert ((o[b, h].double() - o64)[fin].abs() <= tol[fin]).all()
            assert (o[b, h][~fin] == 0).all()


def test_selections_of_the_caller():
    """Slots that end early, no slot at all, blocks behind the query; a list out of order is reported and ends there."""
    H, N, Nk, d = 48, 2048, 4096, 64
    g = torch.Generator(device="cuda").manual_seed(6)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda").bfloat16()  # noqa: E731
    q, k, v = r(1, H, N, d), r(1, H, Nk, d), r(1, H, Nk, d)
    cfg = svoo.BlockConfig(block=128, n_sel=3, sink=0, local=0, causal=False)
    idx = torch.rand(1, H, N, 32, generator=g, device="cuda").argsort(-1)[..., :3].sort(-1).values.int()
    idx[:, :, ::5, 2] = -1
    idx[:, :, 1::5, 1:] = -1
    idx[:, :, 2::5] = -1
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    for causal in (False, True):
        cfg.causal, cfg.local = causal, int(causal)
        o, lse = svoo.block_attn(q, k, v, idx.contiguous(), cfg, dev_err=err)
        assert int(err) == 0
        for h in (0, 17, 47):
            o64, l64 = dense(q[0, h], k[0, h], v[0, h], idx[0, h], cfg, Nk, Nk - N + torch.arange(N, device="cuda"))
            fin = torch.isfinite(l64)
            assert torch.equal(torch.isfinite(lse[0, h]), fin)
            tol = 2 * U * float(v[0, h].abs().max()) + U * o64.abs() + 1e-6
            assert ((o[0, h].double() - o64)[fin].abs() <= tol[fin]).all()
            assert (o[0, h][~fin] == 0).all()
    cfg.causal, cfg.local = False, 0
    idx[0, 3, 7] = torch.tensor([5, 2, 9], dtype=torch.int32, device="cuda")
    bad, _ = svoo.block_attn(q, k, v, idx.contiguous(), cfg, dev_err=err)
    assert int(err) != 0
    idx[0, 3, 7] = torch.tensor([5, -1, -1], dtype=torch.int32, device="cuda")
    good, _ = svoo.block_attn(q, k, v, idx.contiguous(), cfg)
    assert torch.equal(bad, good)

"""Block-selected attention against its fp64 definition on a B200: block means, selection, forward,
gradient; head layouts, odd sizes, padded batches, rows without keys.

Tolerances. A rounding to bf16 is off by at most u = eps / 2 = 2^-8 of the value. P is rounded before the
second product and divided by the sum of the rounded P, so the weights move by at most u each and still sum to
one: |o - o64| <= 2 u max|V| + u |o| (the output's own rounding), fp32 sums far below that. The gradient's
terms (P, dS, delta from the rounded o) are rounded once or twice, with errors of both signs: 4 u of the value
plus 4 u of the largest value, and 2 u in the 2-norm, where they add like squares.
"""
import math

import pytest
import torch

import _blocks as ref
import free_sparse_attention_head_b200 as svoo

pytestmark = pytest.mark.gpu

U = torch.finfo(torch.bfloat16).eps / 2   # half a bf16 step: 2^-8


def make(B, H, Hkv, Nq, Nk, d, seed=0, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: (torch.randn(*s, generator=g) * scale).bfloat16()  # noqa: E731
    return r(B, H, Nq, d), r(B, Hkv, Nk, d), r(B, Hkv, Nk, d)


def lens(t):
    return None if t is None else torch.tensor(t, dtype=torch.int32, device="cuda")


def check_out(o, lse, o64, l64, vmax):
    o, lse = o.double().cpu(), lse.double().cpu()
    assert torch.equal(torch.isinf(lse), torch.isinf(l64))
    fin = torch.isfinite(l64)
    assert ((lse - l64)[fin].abs() <= 2e-5 * (1 + l64[fin].abs())).all()
    # numerator and denominator see the same rounded P: at most 2 u of the weights move, times the spread of V
    tol = 2 * U * vmax + U * o64.abs() + 1e-6
    assert ((o - o64).abs() <= tol).all(), float(((o - o64).abs() - tol).max())
    assert (o[~fin] == 0).all()


CASES = [
    # B, H, Hkv, Nq, Nk, d, block, n_sel, sink, local, causal, lengths, q_start
    (1, 1, 1, 1, 1, 64, 64, 1, 0, 1, True, None, None),
    (1, 2, 1, 64, 64, 128, 64, 2, 1, 1, True, None, None),
    (2, 6, 2, 130, 130, 64, 64, 2, 0, 2, True, None, None),
    (1, 8, 1, 257, 257, 128, 64, 3, 1, 1, True, None, None),
    (2, 4, 4, 300, 300, 64, 64, 3, 1, 1, True, [300, 77], None),
    (3, 5, 1, 191, 191, 128, 64, 2, 1, 1, True, [0, 64, 191], None),
    (1, 4, 2, 33, 513, 64, 128, 3, 1, 1, True, None, None),
    (2, 4, 2, 7, 400, 128, 64, 4, 1, 2, True, [3, 400], -1),
    (1, 3, 3, 200, 450, 64, 192, 2, 1, 0, False, None, None),
    (2, 12, 4, 129, 321, 128, 64, 3, 0, 0, False, [0, 200], 0),
    (1, 40, 1, 50, 700, 64, 64, 5, 1, 1, True, None, None),
    (1, 128, 1, 3, 200, 64, 64, 2, 1, 1, True, None, None),
    (1, 2, 2, 150, 1100, 64, 1024, 2, 1, 1, True, None, None),
]


def config(block, n_sel, sink, local, causal):
    return svoo.BlockConfig(block=block, n_sel=n_sel, sink=sink, local=local, causal=causal)


@pytest.mark.parametrize("case", CASES)
def test_pool_and_selection_are_those_of_fp64(case):
    B, H, Hkv, Nq, Nk, d, block, n_sel, sink, local, causal, lengths, q_start = case
    q, k, _ = make(B, H, Hkv, Nq, Nk, d)
    cfg = config(block, n_sel, sink, local, causal)
    pool = svoo.block_pool(k.cuda(), cfg, lens(lengths))
    want = ref.pool(k, block, lengths)
    # fp64 sums on both sides, one rounding to fp32
    assert ((pool.double().cpu() - want).abs() <= torch.finfo(torch.float32).eps * want.abs()).all()
    idx = svoo.block_select(q.cuda(), pool, cfg, Nk, lens(lengths), q_start)
    assert torch.equal(idx.cpu(), ref.select(q, pool.cpu(), cfg, Nk, lengths, q_start))


@pytest.mark.parametrize("case", CASES)
def test_forward(case):
    B, H, Hkv, Nq, Nk, d, block, n_sel, sink, local, causal, lengths, q_start = case
    q, k, v = make(B, H, Hkv, Nq, Nk, d, seed=1)
    cfg = config(block, n_sel, sink, local, causal)
    o, aux = svoo.block_attention(q.cuda(), k.cuda(), v.cuda(), cfg, lens(lengths), q_start)
    svoo.check_device_errors(aux["dev_err"])
    o64, l64 = ref.attn(q, k, v, aux["idx"].cpu(), cfg, lengths, q_start)
    check_out(o, aux["lse"], o64, l64, float(v.float().abs().max()))


@pytest.mark.parametrize("case", CASES)
def test_gradient(case):
    B, H, Hkv, Nq, Nk, d, block, n_sel, sink, local, causal, lengths, q_start = case
    q, k, v = make(B, H, Hkv, Nq, Nk, d, seed=2)
    g = make(B, H, Hkv, Nq, Nk, d, seed=3)[0]
    cfg = config(block, n_sel, sink, local, causal)
    qc, kc, vc = (t.cuda().requires_grad_(True) for t in (q, k, v))
    o, aux = svoo.block_attention(qc, kc, vc, cfg, lens(lengths), q_start)
    got = torch.autograd.grad(o, (qc, kc, vc), g.cuda())
    svoo.check_device_errors(aux["dev_err"])
    _, _, *want = ref.attn(q, k, v, aux["idx"].cpu(), cfg, lengths, q_start, grad_o=g)
    for name, x, y in zip(("dq", "dk", "dv"), got, want):
        x = x.double().cpu()
        assert torch.isfinite(x).all(), name
        tol = 4 * U * y.abs() + 4 * U * float(y.abs().max()) + 1e-6
        assert ((x - y).abs() <= tol).all(), (name, float((x - y).abs().max()), float(y.abs().max()))
        if float(y.norm()) > 0:
            assert float((x - y).norm() / y.norm()) <= 2 * U, (name, float((x - y).norm() / y.norm()))


@pytest.mark.parametrize("kind", ["plain", "rising", "ties", "equal", "zero", "close", "far"])
@pytest.mark.parametrize("shape", [(1, 3, 1, 1000, 64, 64, 6), (1, 4, 2, 700, 128, 64, 12), (2, 2, 2, 3000, 64, 64, 44),
                                   (1, 2, 1, 65 * 64, 64, 64, 60)])
def test_selection_of_many_queries(shape, kind):
    """Orders of scores that a streaming choice can trip over: rising along the sequence, few distinct blocks,
    all equal, differences below fp32's, magnitudes far apart."""
    B, H, Hkv, N, d, block, n_sel = shape
    q, k, _ = make(B, H, Hkv, N, N, d, seed=11)
    nb = -(-N // block)
    g = torch.Generator().manual_seed(12)
    base = torch.randn(B, Hkv, 1, d, generator=g)
    if kind == "rising":  # the mean grows along the queries' common direction
        q = (q.float() * 0.1 + base.repeat_interleave(H // Hkv, 1)).bfloat16()
        k = (k.float() * 0.01 + base * torch.arange(N)[:, None] / N).bfloat16()
    if kind in ("ties", "equal"):
        n = 3 if kind == "ties" else 1
        rows = torch.randn(B, Hkv, n, d, generator=g)
        which = torch.randint(n, (nb,), generator=g).repeat_interleave(block)[:N]
        k = rows[:, :, which].bfloat16()
    if kind == "zero":
        k = torch.zeros_like(k)
    if kind == "close":  # one key of each block in its last bit off a common block
        k = torch.randn(B, Hkv, block, d, generator=g).bfloat16().repeat(1, 1, nb, 1)[:, :, :N].clone()
        k.view(torch.int16)[:, :, ::block, ::7] ^= torch.randint(2, k[:, :, ::block, ::7].shape, generator=g, dtype=torch.int16)
    if kind == "far":
        k = (k.float() * 10.0 ** torch.randint(-6, 7, (B, Hkv, nb, 1), generator=g).repeat_interleave(block, 2)[:, :, :N]).bfloat16()
    cfg = svoo.BlockConfig(block=block, n_sel=n_sel, sink=1, local=2)
    pool = svoo.block_pool(k.cuda(), cfg)
    idx = svoo.block_select(q.cuda(), pool, cfg, N)
    assert torch.equal(idx.cpu(), ref.select(q, pool.cpu(), cfg, N))

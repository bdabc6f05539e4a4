"""Single-token attention over a cache, its running weights, and eviction, against fp64 and plain-loop
definitions on a B200. Tolerances as in test_gpu_blocks.py; weights are fp32 sums of fp32 terms."""
import math

import pytest
import torch

import _blocks as ref
import free_sparse_attention_head_b200 as svoo
from test_gpu_blocks import check_out, lens, make

pytestmark = pytest.mark.gpu

CACHES = [
    # B, H, Hkv, cap, d, lengths
    (1, 1, 1, 1, 64, [1]),
    (2, 6, 2, 100, 128, [100, 37]),
    (3, 8, 1, 513, 64, [0, 64, 513]),
    (2, 40, 8, 1000, 128, [999, 65]),
    (1, 17, 1, 700, 64, [641]),
    (1, 128, 1, 200, 128, [190]),
    (1, 2, 2, 9000, 64, [8777]),
    (5, 3, 3, 130, 128, [1, 63, 64, 65, 130]),
]


def fill_behind(t, lengths, value):
    """What lies behind a sequence: anything."""
    for b, L in enumerate(lengths):
        t[b, :, L:] = value
    return t


@pytest.mark.parametrize("garbage", [float("nan"), float("inf")])
@pytest.mark.parametrize("case", CACHES)
def test_whole_cache_and_weights(case, garbage):
    B, H, Hkv, cap, d, lengths = case
    q, k, v = make(B, H, Hkv, 1, cap, d, seed=4, scale=1.2)
    k, v = fill_behind(k, lengths, garbage), fill_behind(v, lengths, garbage)
    cfg = svoo.BlockConfig(block=64, n_sel=-(-cap // 64), sink=0, local=0, causal=False)
    idx = ref.select(q, torch.zeros(B, Hkv, -(-cap // 64), d), cfg, cap, lengths)
    o64, l64 = ref.attn(q, k, v, idx, cfg, lengths)
    vmax = max(float(v[b, :, :L].float().abs().max()) for b, L in enumerate(lengths) if L)
    w0 = torch.rand(B, Hkv, cap, generator=torch.Generator().manual_seed(5))
    weight = w0.cuda()
    o, lse = svoo.cache_attn(q.cuda(), k.cuda(), v.cuda(), lens(lengths), weight=weight)
    check_out(o, lse, o64, l64, vmax)
    plain = svoo.cache_attn(q.cuda(), k.cuda(), v.cuda(), lens(lengths))
    assert torch.equal(plain[0], o) and torch.equal(plain[1], lse)
    got = weight.double().cpu()
    for b, L in enumerate(lengths):
        assert torch.equal(got[b, :, L:], w0[b, :, L:].double())
        if not L:
            continue
        x = q[b].double().view(Hkv, H // Hkv, d) @ k[b, :, :L].double().transpose(-1, -2) / math.sqrt(d)
        p = torch.softmax(x, -1).sum(1)
        want = w0[b, :, :L].double() + p
        # scores to 2e-6 of their size in fp32 (d terms), so weights to 1e-5; the sum to one fp32 step
        assert ((got[b, :, :L] - want).abs() <= 2e-5 * p + 2.0 ** -23 * want).all()


@pytest.mark.parametrize("case", [
    (1, 4, 2, 100, 64, 64, 1, [100]), (3, 8, 2, 700, 128, 64, 4, [700, 0, 129]), (2, 5, 1, 2000, 64, 256, 3, [1999, 300]),
    (2, 24, 8, 1500, 128, 128, 40, [1500, 700]), (1, 2, 1, 5000, 64, 1024, 2, [4097])])
def test_selected_slots_step(case):
    """A token's whole step: the last block's mean anew, selection, attention over the selected blocks."""
    B, H, Hkv, cap, d, block, n_sel, lengths = case
    q, k, v = make(B, H, Hkv, 1, cap, d, seed=6)
    k, v = fill_behind(k, lengths, float("nan")), fill_behind(v, lengths, float("nan"))
    cfg = svoo.BlockConfig(block=block, n_sel=n_sel, sink=min(1, n_sel - 1), local=1)
    before = [max(0, L - 1) for L in lengths]
    pool = svoo.block_pool(k.cuda(), cfg, lens(before))
    svoo.block_pool(k.cuda(), cfg, lens(lengths), pool=pool, last=1)
    want = ref.pool(k, block, lengths)
    assert ((pool.double().cpu() - want).abs() <= torch.finfo(torch.float32).eps * want.abs()).all()
    idx = svoo.block_select(q.cuda(), pool, cfg, cap, lens(lengths), q_start=-1)
    assert torch.equal(idx.cpu(), ref.select(q, pool.cpu(), cfg, cap, lengths, -1))
    o, lse = svoo.cache_attn(q.cuda(), k.cuda(), v.cuda(), lens(lengths), idx=idx, cfg=cfg)
    o64, l64 = ref.attn(q, k, v, idx.cpu(), cfg, lengths, -1)
    check_out(o, lse, o64, l64, max(float(v[b, :, :L].float().abs().max()) for b, L in enumerate(lengths) if L))


EVICTIONS = [
    # B, Hkv, cap, d, keep, sink, recent, lengths, kind of weights
    (1, 1, 2, 64, 1, 0, 1, [2], "random"),
    (2, 3, 100, 128, 40, 4, 8, [100, 39], "random"),
    (3, 2, 1025, 64, 1024, 2, 16, [1025, 1024, 0], "random"),
    (1, 2, 3000, 128, 100, 0, 0, [2999], "ties"),
    (2, 1, 2100, 64, 2000, 4, 1996, [2100, 2050], "random"),
    (1, 4, 500, 64, 250, 1, 9, [500], "zeros"),
    (1, 1, 300, 64, 77, 2, 3, [300], "nan"),
    (1, 2, 5000, 64, 2500, 4, 100, [4999], "random"),
    (2, 1, 17000, 64, 16000, 4, 100, [17000, 16500], "random"),
    (1, 1, 17000, 64, 3000, 0, 10, [16999], "ties"),
]


@pytest.mark.parametrize("case", EVICTIONS)
def test_eviction_makes_the_defined_moves(case):
    B, Hkv, cap, d, keep, sink, recent, lengths, kind = case
    _, k, v = make(B, 1 * Hkv, Hkv, 1, cap, d, seed=7)
    g = torch.Generator().manual_seed(8)
    w = torch.randn(B, Hkv, cap, generator=g).exp()
    if kind == "ties":
        w = torch.randint(3, (B, Hkv, cap), generator=g).float()
    if kind == "zeros":
        w = torch.zeros_like(w) * torch.where(torch.rand(B, Hkv, cap, generator=g) < 0.5, -1.0, 1.0)
    if kind == "nan":
        w[..., ::3] = math.nan
    pos = torch.argsort(torch.rand(B, Hkv, cap, generator=g), -1).int()
    for b, L in enumerate(lengths):
        w[b, :, L:] = math.inf  # never looked at
        pos[b, :, L:] = 1 << 30
    want = [t.clone() for t in (k, v, w, pos)]
    for b, L in enumerate(lengths):
        for h in range(Hkv):
            for to, src in ref.evict(w[b, h].tolist(), pos[b, h].tolist(), L, keep, sink, recent):
                for t in want:
                    t[b, h, to] = t[b, h, src]
    got = [t.cuda() for t in (k, v, w, pos)]
    ln = lens(lengths)
    svoo.cache_evict(*got, ln, keep, sink=sink, recent=recent)
    for x, y in zip(got, want):
        assert torch.equal(x.cpu().view(torch.int16 if x.dtype == torch.bfloat16 else torch.int32),
                           y.view(torch.int16 if y.dtype == torch.bfloat16 else torch.int32))
    assert ln.tolist() == [min(L, keep) for L in lengths]


def test_serving_steps_together():
    """Tokens appended to a bounded cache: attention with weights, eviction, attention over what is left,
    against a model of the cache kept on the CPU."""
    B, H, Hkv, d, keep, cap = 2, 4, 2, 64, 96, 97
    g = torch.Generator().manual_seed(9)
    r = lambda *s: torch.randn(*s, generator=g).bfloat16()  # noqa: E731
    k, v = r(B, Hkv, cap, d), r(B, Hkv, cap, d)
    start = [90, 96]
    pos = torch.arange(cap, dtype=torch.int32).repeat(B, Hkv, 1)
    kc, vc, pc = k.cuda(), v.cuda(), pos.cuda().contiguous()
    wc, ln = torch.zeros(B, Hkv, cap, device="cuda"), lens(start)
    seen = list(start)
    for step in range(12):
        nk, nv, q = r(B, Hkv, d), r(B, Hkv, d), r(B, H, 1, d)
        L = ln.tolist()
        for b in range(B):
            kc[b, :, L[b]], vc[b, :, L[b]], pc[b, :, L[b]], wc[b, :, L[b]] = nk[b].cuda(), nv[b].cuda(), seen[b], 0.0
            seen[b] += 1
        ln += 1
        before = [t.cpu() for t in (kc, vc, wc, pc)]
        L = ln.tolist()
        o, lse = svoo.cache_attn(q.cuda(), kc, vc, ln, weight=wc)
        cfg = svoo.BlockConfig(block=64, n_sel=2, sink=0, local=0, causal=False)
        idx = ref.select(q, torch.zeros(B, Hkv, 2, d), cfg, cap, L)
        o64, l64 = ref.attn(q, before[0], before[1], idx, cfg, L)
        check_out(o, lse, o64, l64, float(before[1].float().abs().max()))
        added = (wc.cpu() - before[2]).double().sum(-1)
        assert ((added - H // Hkv).abs() <= 1e-4).all()  # a softmax's weights sum to one a head
        now = [t.cpu() for t in (kc, vc, wc, pc)]
        svoo.cache_evict(kc, vc, wc, pc, ln, keep, sink=2, recent=8)
        for b in range(B):
            for h in range(Hkv):
                for to, src in ref.evict(now[2][b, h].tolist(), now[3][b, h].tolist(), L[b], keep, 2, 8):
                    for t in now:
                        t[b, h, to] = t[b, h, src]
        for x, y in zip((kc, vc, wc, pc), now):
            assert torch.equal(x.cpu(), y)
        assert ln.tolist() == [min(x, keep) for x in L]
    # the positions that stay are distinct and hold the first and the last ones
    for b in range(B):
        for h in range(Hkv):
            p = pc[b, h, :keep].tolist()
            assert len(set(p)) == keep and {0, 1} <= set(p) and set(range(seen[b] - 8, seen[b])) <= set(p)

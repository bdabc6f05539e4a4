"""The block-selected attention, cached attention and eviction in the ways that a program uses them: padded
batches with garbage in the padding, views into longer buffers, selections from elsewhere, streams, graphs,
repeated calls, long caches, refusals. Tolerances as in test_gpu_blocks.py."""
import math

import pytest
import torch

import _blocks as ref
import free_sparse_attention_head_b200 as svoo
from test_gpu_blocks import U, check_out, lens, make

pytestmark = pytest.mark.gpu


def close(got, want, name=""):
    got, want = got.double().cpu(), want.double().cpu()
    assert torch.isfinite(got).all(), name
    tol = 4 * U * want.abs() + 4 * U * float(want.abs().max()) + 1e-6
    assert ((got - want).abs() <= tol).all(), (name, float((got - want).abs().max()))


@pytest.mark.parametrize("garbage", [math.nan, math.inf])
def test_padding_may_hold_anything(garbage):
    """Right-padded batch: what lies behind a sequence, in q, k, v and the incoming gradient, reaches nothing."""
    B, H, Hkv, N, d, lengths = 3, 6, 2, 270, 64, [270, 130, 1]
    q, k, v = make(B, H, Hkv, N, N, d, seed=21)
    g = make(B, H, Hkv, N, N, d, seed=22)[0]
    for t in (q, k, v, g):
        for b, L in enumerate(lengths):
            t[b, :, L:] = garbage
    cfg = svoo.BlockConfig(block=64, n_sel=3)
    qc, kc, vc = (t.cuda().requires_grad_(True) for t in (q, k, v))
    o, aux = svoo.block_attention(qc, kc, vc, cfg, lens(lengths))
    got = torch.autograd.grad(o, (qc, kc, vc), g.cuda())
    svoo.check_device_errors(aux["dev_err"])
    assert torch.isfinite(o).all()
    o64, l64, *want = ref.attn(q, k, v, aux["idx"].cpu(), cfg, lengths, grad_o=g)
    vmax = max(float(v[b, :, :L].float().abs().max()) for b, L in enumerate(lengths))
    check_out(o.detach(), aux["lse"], o64, l64, vmax)
    for name, x, y in zip(("dq", "dk", "dv"), got, want):
        close(x, y, name)
        for b, L in enumerate(lengths):
            assert (x[b, :, L:] == 0).all(), name


def test_keys_as_a_view_of_a_longer_buffer():
    B, H, Hkv, Nq, Nk, cap, d = 2, 4, 2, 90, 200, 333, 128
    q, k, v = make(B, H, Hkv, Nq, cap, d, seed=23)
    g = make(B, H, Hkv, Nq, cap, d, seed=24)[0]
    k[:, :, Nk:], v[:, :, Nk:] = math.nan, math.nan
    kb, vb = k.cuda(), v.cuda()
    cfg = svoo.BlockConfig(block=64, n_sel=3)
    o, aux = svoo.block_attention(q.cuda(), kb[:, :, :Nk], vb[:, :, :Nk], cfg)
    o2, aux2 = svoo.block_attention(q.cuda(), kb[:, :, :Nk].contiguous(), vb[:, :, :Nk].contiguous(), cfg)
    assert torch.equal(o, o2) and torch.equal(aux["idx"], aux2["idx"]) and torch.equal(aux["pool"], aux2["pool"])
    grads = svoo.block_attn_backward(q.cuda(), kb[:, :, :Nk], vb[:, :, :Nk], o, aux["lse"], g.cuda(), aux["idx"], cfg)
    _, _, *want = ref.attn(q, k[:, :, :Nk], v[:, :, :Nk], aux["idx"].cpu(), cfg, grad_o=g)
    for name, x, y in zip(("dq", "dk", "dv"), grads, want):
        assert x.is_contiguous() and x.shape == y.shape
        close(x, y, name)
    # one sequence's single head: no stride tells the capacity of a batch of one
    one, _ = svoo.block_attention(q[:1, :2].cuda(), kb[:1, :1, :Nk], vb[:1, :1, :Nk], cfg)
    assert torch.equal(one, o[:1, :2])


def test_a_selection_from_elsewhere():
    """Blocks that hide behind the query, lists that end early, and entries that no selection has."""
    B, H, Hkv, N, d = 1, 2, 1, 300, 64
    q, k, v = make(B, H, Hkv, N, N, d, seed=25)
    g = make(B, H, Hkv, N, N, d, seed=26)[0]
    cfg = svoo.BlockConfig(block=64, n_sel=4)
    idx = torch.full((B, Hkv, N, 4), -1, dtype=torch.int32)
    gen = torch.Generator().manual_seed(27)
    for t in range(N):
        n = int(torch.randint(5, (1,), generator=gen))
        idx[0, 0, t, :n] = torch.randperm(5, generator=gen)[:n].sort()[0].int()
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    args = (q.cuda(), k.cuda(), v.cuda())
    o, lse = svoo.block_attn(*args, idx.cuda(), cfg, dev_err=err)
    grads = svoo.block_attn_backward(*args, o, lse, g.cuda(), idx.cuda(), cfg, dev_err=err)
    svoo.check_device_errors(err)
    o64, l64, *want = ref.attn(q, k, v, idx, cfg, grad_o=g)
    check_out(o, lse, o64, l64, float(v.float().abs().max()))
    for name, x, y in zip(("dq", "dk", "dv"), grads, want):
        close(x, y, name)
    # a list ends at an entry that is out of range or not above the one before it, and says so
    bad, cut = idx.clone(), idx.clone()
    for t, row in ((70, [0, 5, 1, 2]), (71, [1, 1, 2, 3]), (72, [-7, 0, 1, 2]), (73, [0, 1, 1 << 30, 3]), (74, [2, 0, 1, 3])):
        bad[0, 0, t] = torch.tensor(row, dtype=torch.int32)
        n = {70: 1, 71: 1, 72: 0, 73: 2, 74: 1}[t]
        cut[0, 0, t] = torch.tensor(row[:n] + [-1] * (4 - n), dtype=torch.int32)
    o, lse = svoo.block_attn(*args, bad.cuda(), cfg, dev_err=err)
    assert int(err.item()) == 4
    o2, lse2 = svoo.block_attn(*args, cut.cuda(), cfg)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    err.zero_()
    for x, y in zip(svoo.block_attn_backward(*args, o, lse, g.cuda(), bad.cuda(), cfg, dev_err=err),
                    svoo.block_attn_backward(*args, o, lse, g.cuda(), cut.cuda(), cfg)):
        assert torch.equal(x, y)
    assert int(err.item()) == 4


@pytest.mark.parametrize("case", [
    (1, 2, 1, 700, 64, 64, 11, 33),     # more slots than lanes
    (1, 1, 1, 80 * 64, 64, 64, 80, 70),  # more than the streaming selection chooses
    (1, 2, 1, 200, 64, 64, 4, 200),     # more slots than blocks
])
def test_many_slots(case):
    B, H, Hkv, Nk, d, block, _, n_sel = case
    Nq = 70
    q, k, v = make(B, H, Hkv, Nq, Nk, d, seed=28)
    g = make(B, H, Hkv, Nq, Nk, d, seed=29)[0]
    cfg = svoo.BlockConfig(block=block, n_sel=n_sel, sink=1, local=2)
    qc, kc, vc = (t.cuda().requires_grad_(True) for t in (q, k, v))
    o, aux = svoo.block_attention(qc, kc, vc, cfg)
    assert torch.equal(aux["idx"].cpu(), ref.select(q, aux["pool"].cpu(), cfg, Nk))
    got = torch.autograd.grad(o, (qc, kc, vc), g.cuda())
    o64, l64, *want = ref.attn(q, k, v, aux["idx"].cpu(), cfg, grad_o=g)
    check_out(o.detach(), aux["lse"], o64, l64, float(v.float().abs().max()))
    for name, x, y in zip(("dq", "dk", "dv"), got, want):
        close(x, y, name)


def test_long_lists_are_cut_and_joined():
    """Blocks that every query keeps: their lists are longer than one piece of the gradient's work."""
    B, H, Hkv, N, d = 1, 16, 2, 3000, 64
    q, k, v = make(B, H, Hkv, N, N, d, seed=30)
    g = make(B, H, Hkv, N, N, d, seed=31)[0]
    cfg = svoo.BlockConfig(block=64, n_sel=4, sink=2)
    args = [t.cuda() for t in (q, k, v)]
    o, aux = svoo.block_attention(*args, cfg)
    got = svoo.block_attn_backward(*args, o, aux["lse"], g.cuda(), aux["idx"], cfg)
    again = svoo.block_attn_backward(*args, o, aux["lse"], g.cuda(), aux["idx"], cfg)
    for x, y in zip(got, again):
        assert torch.equal(x, y)  # every sum in a fixed order
    # the same in fp64 on the GPU, through a mask
    m = torch.zeros(B, Hkv, N, 48, dtype=torch.bool, device="cuda")
    m.scatter_(3, torch.where(aux["idx"] < 0, 47, aux["idx"]).long(), True)
    m[..., 47] = False
    m = m.repeat_interleave(64, -1)[..., :N] & torch.ones(N, N, dtype=torch.bool, device="cuda").tril()
    q64, k64, v64, g64 = (t.cuda().double() for t in (q, k, v, g))
    k8, v8 = (t.repeat_interleave(8, 1) for t in (k64, v64))
    s = torch.where(m.repeat_interleave(8, 1), q64 @ k8.transpose(-1, -2) / 8, -math.inf)
    p = torch.softmax(s, -1)
    o64 = p @ v8
    close(o, o64, "o")
    ds = p * (g64 @ v8.transpose(-1, -2) - (g64 * o64).sum(-1, keepdim=True)) / 8
    close(got[0], ds @ k8, "dq")
    close(got[1], (ds.transpose(-1, -2) @ q64).view(B, Hkv, 8, N, d).sum(2), "dk")
    close(got[2], (p.transpose(-1, -2) @ g64).view(B, Hkv, 8, N, d).sum(2), "dv")


def test_large_scores():
    """Maxima that grow by hundreds along the keys, and scores far apart: rescaling, no overflow."""
    B, H, Hkv, N, d = 1, 2, 1, 512, 64
    q, k, v = make(B, H, Hkv, N, N, d, seed=32)
    k = (k.float() * torch.linspace(0.1, 40, N)[:, None]).bfloat16()
    cfg = svoo.BlockConfig(block=64, n_sel=8, scale=1.0)
    o, aux = svoo.block_attention(q.cuda(), k.cuda(), v.cuda(), cfg)
    o64, l64 = ref.attn(q, k, v, aux["idx"].cpu(), cfg, scale=1.0)
    check_out(o, aux["lse"], o64, l64, float(v.float().abs().max()))


def test_other_streams():
    B, H, Hkv, N, d = 1, 4, 2, 500, 64
    q, k, v = (t.cuda() for t in make(B, H, Hkv, N, N, d, seed=33))
    cfg = svoo.BlockConfig(block=64, n_sel=3)
    want, aux = svoo.block_attention(q, k, v, cfg)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    outs = []
    for s in (s1, s2, s1, s2):  # two calls at once, each with its own workspace
        with torch.cuda.stream(s):
            outs.append(svoo.block_attention(q, k, v, cfg)[0])
    pool = svoo.block_pool(k, cfg, stream=s1)
    idx = svoo.block_select(q, pool, cfg, N, stream=s1)
    outs.append(svoo.block_attn(q, k, v, idx, cfg, stream=s1)[0])
    torch.cuda.synchronize()
    for o in outs:
        assert torch.equal(o, want)


def test_prefill_and_decoding_steps_in_graphs():
    """Captured once, replayed on new contents of the same buffers."""
    B, H, Hkv, cap, d = 2, 4, 2, 300, 64
    cfg = svoo.BlockConfig(block=64, n_sel=3)
    qs, ks, vs = (t.cuda() for t in make(B, H, Hkv, 200, 200, d, seed=34))
    q1, k1, v1 = (t.cuda() for t in make(B, H, Hkv, 1, cap, d, seed=35))
    ln = lens([200, 130])
    pool = svoo.block_pool(k1, cfg, ln)
    weight = torch.zeros(B, Hkv, cap, device="cuda")
    pos = torch.arange(cap, dtype=torch.int32, device="cuda").repeat(B, Hkv, 1).contiguous()

    def prefill():
        return svoo.block_attention(qs, ks, vs, cfg)[0]

    def step():
        svoo.block_pool(k1, cfg, ln, pool=pool, last=1)
        idx = svoo.block_select(q1, pool, cfg, cap, ln, q_start=-1)
        return svoo.cache_attn(q1, k1, v1, ln, idx=idx, cfg=cfg)[0], svoo.cache_attn(q1, k1, v1, ln, weight=weight)[0]

    prefill(), step()
    torch.cuda.synchronize()
    g1, g2 = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g1):
        o1 = prefill()
    with torch.cuda.graph(g2):
        o2, o3 = step()
    for seed in (36, 37):
        a, b, c = make(B, H, Hkv, 200, 200, d, seed=seed)
        qs.copy_(a), ks.copy_(b), vs.copy_(c)
        a, b, c = make(B, H, Hkv, 1, cap, d, seed=seed + 10)
        q1.copy_(a), k1.copy_(b), v1.copy_(c)
        ln += 1
        pool.copy_(svoo.block_pool(k1, cfg, ln))
        before = weight.clone()
        g1.replay(), g2.replay()
        got = [o1.clone(), o2.clone(), o3.clone(), weight.clone()]
        weight.copy_(before)
        want = [prefill(), *step(), weight]
        for x, y in zip(got, want):
            assert torch.equal(x, y)
    g3 = torch.cuda.CUDAGraph()
    svoo.cache_evict(k1.clone(), v1.clone(), weight.clone(), pos.clone(), ln.clone(), 100, 2, 8)
    with torch.cuda.graph(g3):
        svoo.cache_evict(k1, v1, weight, pos, ln, 100, sink=2, recent=8)
    other = [t.clone() for t in (k1, v1, weight, pos, ln)]
    g3.replay()
    svoo.cache_evict(*other, 100, sink=2, recent=8)
    for x, y in zip((k1, v1, weight, pos, ln), other):
        assert torch.equal(x, y)
    assert ln.tolist() == [100, 100]


def test_training_step_in_a_graph():
    B, H, Hkv, N, d = 1, 4, 2, 260, 64
    cfg = svoo.BlockConfig(block=64, n_sel=3)
    q, k, v = (t.cuda().requires_grad_(True) for t in make(B, H, Hkv, N, N, d, seed=40))
    g = make(B, H, Hkv, N, N, d, seed=41)[0].cuda()

    def step():
        o, _ = svoo.block_attention(q, k, v, cfg)
        return torch.autograd.grad(o, (q, k, v), g)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        grads = step()
    with torch.no_grad():
        for t, new in zip((q, k, v), make(B, H, Hkv, N, N, d, seed=42)):
            t.copy_(new)
    graph.replay()
    torch.cuda.synchronize()
    for x, y in zip(grads, step()):
        assert torch.equal(x, y)


def test_gradient_in_a_training_program():
    """Through other operations, shared leaves and a gradient that is no dense tensor; the selection is a constant."""
    B, H, Hkv, N, d = 1, 4, 1, 200, 64
    cfg = svoo.BlockConfig(block=64, n_sel=2)
    x = make(B, H, Hkv, N, N, d, seed=43)[0].float().cuda().requires_grad_(True)
    q = x.bfloat16()
    kv = q.mean(1, keepdim=True)
    o, aux = svoo.block_attention(q, kv, kv, cfg)
    assert not aux["lse"].requires_grad and not aux["pool"].requires_grad
    o.sum(2).float().sum().backward()  # an expanded gradient
    assert x.grad is not None and torch.isfinite(x.grad).all()
    qf, kf = q.detach().cpu(), kv.detach().cpu()
    _, _, dq, dk, dv = ref.attn(qf, kf, kf, aux["idx"].cpu(), cfg, grad_o=torch.ones_like(qf))
    want = dq + (dk + dv) / H
    # the three gradients rounded to bf16, and once more where autograd adds them
    close(x.grad, want, "x")
    with torch.no_grad():
        assert torch.equal(svoo.block_attention(q, kv, kv, cfg)[0], o)
    a, b = q.detach().requires_grad_(True), kv.detach().requires_grad_(True)
    o, _ = svoo.block_attention(a, b, b, cfg)
    (ga,) = torch.autograd.grad(o.float().sum(), a, create_graph=True)
    with pytest.raises(RuntimeError):
        ga.float().sum().backward()


def test_cache_longer_than_32_bit_offsets():
    """The last head of a cache of more than 2^32 bytes."""
    B, H, Hkv, cap, d = 1, 18, 18, 1 << 20, 128
    k = torch.zeros(B, Hkv, cap, d, dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    gen = torch.Generator(device="cuda").manual_seed(44)
    k[0, -1] = torch.randn(cap, d, generator=gen, device="cuda").bfloat16()
    v[0, -1] = torch.randn(cap, d, generator=gen, device="cuda").bfloat16()
    q = torch.randn(B, H, 1, d, generator=gen, device="cuda").bfloat16()
    ln = lens([cap - 3])
    weight = torch.zeros(B, Hkv, cap, device="cuda")
    o, lse = svoo.cache_attn(q, k, v, ln, weight=weight)
    s = (q[0, -1, 0].double() @ k[0, -1, :cap - 3].double().T) / math.sqrt(d)
    p = torch.softmax(s, -1)
    check_out(o[:, -1:], lse[:, -1:], (p @ v[0, -1, :cap - 3].double())[None, None, None].cpu(),
              s.logsumexp(-1)[None, None, None].cpu(), float(v[0, -1].abs().max()))
    # equal scores of zero: 2^20 - 3 equal weights
    assert abs(float(lse[0, 0, 0]) - math.log(cap - 3)) <= 2e-5 * 14
    assert float((weight[0, -1, :cap - 3].double() - p).abs().max()) <= 2e-5 * float(p.max())
    cfg = svoo.BlockConfig(block=1024, n_sel=8)
    pool = svoo.block_pool(k, cfg, ln)
    mean = k[0, -1, -1024:-3].double().mean(0)
    assert ((pool[0, -1, -1].double() - mean).abs() <= 2.0 ** -23 * mean.abs()).all()
    idx = svoo.block_select(q, pool, cfg, cap, ln, q_start=-1)
    assert torch.equal(idx[:, -1:].cpu(), ref.select(q[:, -1:].cpu(), pool[:, -1:].cpu(), cfg, cap, [cap - 3], -1))
    del k, v
    torch.cuda.empty_cache()


def test_refusals():
    q, k, v = (t.cuda() for t in make(2, 4, 2, 1, 128, 64, seed=50))
    cfg = svoo.BlockConfig(block=64, n_sel=2)
    ln, w = lens([128, 100]), torch.zeros(2, 2, 128, device="cuda")
    pos = torch.zeros(2, 2, 128, dtype=torch.int32, device="cuda")
    pool = svoo.block_pool(k, cfg)
    idx = svoo.block_select(q, pool, cfg, 128)
    half, long = k.half(), ln.long()
    for call in (
        lambda: svoo.block_attention(q.float(), k, v, cfg),
        lambda: svoo.block_attention(q, half, half, cfg),
        lambda: svoo.block_attention(q, k, v[:, :, :64], cfg),
        lambda: svoo.block_attention(q.transpose(1, 2), k, v, cfg),
        lambda: svoo.block_attention(q, k.transpose(-1, -2).contiguous().transpose(-1, -2), v, cfg),
        lambda: svoo.block_attention(q, k[:1], v[:1], cfg),
        lambda: svoo.block_attention(q, k, v, cfg, lengths=long),
        lambda: svoo.block_attention(q, k, v, cfg, lengths=ln[:1]),
        lambda: svoo.block_attention(q, k, v, cfg, lengths=ln.cpu()),
        lambda: svoo.block_attention(q[:, :3].contiguous(), k, v, cfg),
        lambda: svoo.block_attention(q, k, v, svoo.BlockConfig(block=100)),
        lambda: svoo.block_attention(q, k, v, svoo.BlockConfig(n_sel=1)),
        lambda: svoo.block_attention(q, k, v, svoo.BlockConfig(causal=False)),
        lambda: svoo.block_attention(q, k, v, svoo.BlockConfig(n_sel=2, scale=-1.0)),
        lambda: svoo.block_attention(q, k, v, cfg, q_start=-2),
        lambda: svoo.block_pool(k, cfg, last=1),
        lambda: svoo.block_pool(k, cfg, pool=pool[:, :, :1]),
        lambda: svoo.block_select(q, pool[:, :, :1].contiguous(), cfg, 128),
        lambda: svoo.block_attn(q, k, v, idx.long(), cfg),
        lambda: svoo.block_attn(q, k, v, idx[..., :1].contiguous(), cfg),
        lambda: svoo.cache_attn(torch.cat([q, q], 2), k, v, ln),
        lambda: svoo.cache_attn(q, k, v, ln, idx=idx),
        lambda: svoo.cache_attn(q, k, v, ln, idx=idx, cfg=cfg, weight=w),
        lambda: svoo.cache_attn(q, k, v, ln, weight=w[..., :64]),
        lambda: svoo.cache_attn(q, k[:, :, :64], v[:, :, :64], ln, weight=w),
        lambda: svoo.cache_attn(q, k, v, ln, weight=w, workspace=torch.empty(16, dtype=torch.uint8, device="cuda")),
        lambda: svoo.cache_evict(k, v, w, pos, ln, 0),
        lambda: svoo.cache_evict(k, v, w, pos, ln, 10, sink=8, recent=3),
        lambda: svoo.cache_evict(k, v, w, pos.long(), ln, 10),
        lambda: svoo.cache_evict(k[:, :, :64], v[:, :, :64], w[..., :64], pos[..., :64], ln, 10),
        lambda: svoo.cache_evict(k, v, w, pos, ln, 10, workspace=torch.empty(8, dtype=torch.uint8, device="cuda")),
    ):
        with pytest.raises(svoo.SvooError):
            call()
    torch.cuda.synchronize()  # nothing was launched that could have gone wrong
    assert ln.tolist() == [128, 100] and not w.any()
    # what has nothing to do, does it
    none, aux = svoo.block_attention(q[:, :, :0], k, v, cfg)
    assert none.shape == (2, 4, 0, 64) and aux["idx"].shape == (2, 2, 0, 2)
    for x in svoo.block_attn_backward(q[:, :, :0], k, v, none, aux["lse"], none, aux["idx"], cfg)[1:]:
        assert x.shape == k.shape and not x.any()
    z = lens([0, 0])
    o, lse = svoo.cache_attn(q, k, v, z, weight=w)
    assert not o.any() and torch.isinf(lse).all() and not w.any()
    svoo.cache_evict(k, v, w, pos, z, 5)
    assert z.tolist() == [0, 0]

"""Calls at the edges of what the block-selected attention and the cache calls document. Tolerances as in
test_gpu_blocks.py."""
import math
import threading

import pytest
import torch

import _blocks as ref
import free_sparse_attention_head_b200 as svoo
from test_gpu_blocks import check_out, lens, make
from test_gpu_blocks_use import close

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("first,Nk", [(100, 900), (937, 63), (10, 990)])
def test_keys_as_a_view_that_begins_inside_its_buffer(first, Nk):
    """The buffer ends with the view's last row; what lies before it holds garbage."""
    B, H, Hkv, cap, d = 2, 8, 4, 1000, 128
    q, k, v = make(B, H, Hkv, 130, cap, d, seed=51)
    k[:, :, :first], v[:, :, :first] = math.nan, math.nan
    g = make(B, H, Hkv, 130, cap, d, seed=52)[0].cuda()
    kb, vb, qc = k.cuda(), v.cuda(), q.cuda()
    kc, vc = kb[:, :, first:first + Nk].contiguous(), vb[:, :, first:first + Nk].contiguous()
    kb, vb = kb[:, :, first:first + Nk], vb[:, :, first:first + Nk]
    cfg = svoo.BlockConfig(block=64, n_sel=4)
    one = qc[:, :, :1].contiguous()
    for keys in ((kb, vb), (kc, vc)):
        o, aux = svoo.block_attention(qc, *keys, cfg, q_start=max(0, Nk - 130))
        got = [o, aux["lse"], aux["idx"], aux["pool"]]
        got += svoo.block_attn_backward(qc, *keys, o, aux["lse"], g, aux["idx"], cfg, q_start=max(0, Nk - 130))
        got += svoo.cache_attn(one, *keys)
        idx = svoo.block_select(one, aux["pool"], cfg, Nk)
        got += svoo.cache_attn(one, *keys, lens([Nk, Nk - 5]), idx=idx, cfg=cfg)
        if keys[0] is kb:
            want = got
    for x, y in zip(got, want):
        assert torch.equal(x, y) and torch.isfinite(x[x > -math.inf].float()).all()


def test_another_stream_owns_the_workspace(monkeypatch):
    """stream=: while that stream still has work before the call, nothing that the current stream allocates lies in
    the call's workspace or results, and filling it changes no result."""
    B, H, Hkv, N, d = 1, 16, 16, 5504, 64
    gen = torch.Generator(device="cuda").manual_seed(53)
    r = lambda *s: torch.randn(*s, generator=gen, device="cuda").bfloat16()  # noqa: E731
    q, k, v, g, one = r(B, H, N, d), r(B, Hkv, N, d), r(B, Hkv, N, d), r(B, H, N, d), r(B, H, 1, d)
    fine = svoo.BlockConfig(block=64, n_sel=4)                                        # selection of 86 blocks
    cfg = svoo.BlockConfig(block=128, n_sel=4, sink=1, local=0, causal=False)        # attention by key blocks
    w0 = torch.rand(B, Hkv, N, generator=gen, device="cuda")
    fine_pool, pool = svoo.block_pool(k, fine), svoo.block_pool(k, cfg)
    idx = svoo.block_select(q, pool, cfg, N)
    o, lse = svoo.block_attn(q, k, v, idx, cfg)
    pos = torch.arange(N, device="cuda").int().repeat(B, Hkv, 1)
    wide = svoo.BlockConfig(block=64, n_sel=64)
    idx1 = svoo.block_select(one, fine_pool, wide, N)
    calls = dict(
        pool=lambda **kw: [svoo.block_pool(k, cfg, **kw)],
        select=lambda **kw: [svoo.block_select(q, fine_pool, fine, N, **kw)],
        attn=lambda **kw: list(svoo.block_attn(q, k, v, idx, cfg, **kw)),
        backward=lambda **kw: list(svoo.block_attn_backward(q, k, v, o, lse, g, idx, cfg, **kw)),
        whole=lambda **kw: list(svoo.cache_attn(one, k, v, **kw)),
        selected=lambda **kw: list(svoo.cache_attn(one, k, v, idx=idx1, cfg=wide, **kw)),
    )

    def weigh(**kw):
        w = kw.pop("w")
        return [*svoo.cache_attn(one, k, v, weight=w, **kw), w]

    def evict(**kw):
        state = kw.pop("state")
        svoo.cache_evict(*state, 3000, sink=4, recent=100, **kw)
        return list(state)

    torch.full((1,), 0xFF, dtype=torch.uint8, device="cuda")   # a kernel's first launch may wait for the device
    side = torch.cuda.Stream()
    for name in (*calls, "weigh", "evict"):
        if name == "weigh":
            run = lambda kw, w: weigh(w=w, **kw)  # noqa: E731
            mine = [(w0.clone(),) for _ in range(2)]
        elif name == "evict":
            run = lambda kw, *st: evict(state=st, **kw)  # noqa: E731
            mine = [(k.clone(), v.clone(), w0.clone(), pos.clone(), lens([N])) for _ in range(2)]
        else:
            run = lambda kw: calls[name](**kw)  # noqa: E731
            mine = [(), ()]
        want = [t.clone() for t in run({}, *mine[0])]
        torch.cuda.synchronize()
        sizes = []
        empty = torch.empty

        def noting(*a, **kw):
            t = empty(*a, **kw)
            if t.is_cuda:
                sizes.append((t.data_ptr(), t.numel() * t.element_size()))
            return t

        with torch.cuda.stream(side):
            torch.cuda._sleep(800_000_000)     # some tenths of a second: the call's kernels have not begun
        monkeypatch.setattr(svoo.torch, "empty", noting)
        got = run({"stream": side}, *mine[1])
        monkeypatch.setattr(svoo.torch, "empty", empty)
        assert not side.query(), "the stream was to be busy"
        made = list(sizes)
        if name in ("select", "attn", "backward", "whole", "weigh", "evict"):
            assert made, name
        later = [torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda") for _, n in made for _ in range(3)]
        assert not side.query(), "the stream was to be busy"
        for at, n in made:
            for t in later:
                assert t.data_ptr() + t.numel() <= at or at + n <= t.data_ptr(), (name, n)
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(got, want)), name
        del later, got


def test_a_stream_of_no_device_of_the_tensors():
    k = torch.zeros(1, 1, 64, 64, dtype=torch.bfloat16)
    with pytest.raises(svoo.SvooError):
        svoo.block_pool(k, svoo.BlockConfig(), stream=torch.cuda.Stream())


def test_another_stream_in_a_graph():
    q, k, v = (t.cuda() for t in make(1, 4, 2, 200, 5000, 64, seed=54))
    cfg = svoo.BlockConfig(block=64, n_sel=4)

    def calls(side):
        side.wait_stream(torch.cuda.current_stream())
        pool = svoo.block_pool(k, cfg, stream=side)
        idx = svoo.block_select(q, pool, cfg, 5000, stream=side)
        o, lse = svoo.block_attn(q, k, v, idx, cfg, stream=side)
        out = (o, lse, *svoo.block_attn_backward(q, k, v, o, lse, q, idx, cfg, stream=side))
        torch.cuda.current_stream().wait_stream(side)
        return out

    warm = torch.cuda.Stream()
    calls(warm)
    torch.cuda.synchronize()
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(graph):
        out = calls(side)
    for seed in (55, 56):
        for t, new in zip((q, k, v), make(1, 4, 2, 200, 5000, 64, seed=seed)):
            t.copy_(new)
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in out]
        want = calls(warm)
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(got, want))


def test_two_host_threads_with_different_shapes():
    """Kernels of different shared-memory needs, called at the same time from two threads with their own streams."""
    def work(Nk, n_sel, block, seed):
        q, k, v, g = (t.cuda() for t in (*make(1, 2, 2, 200, Nk, 64, seed=seed), make(1, 2, 2, 200, Nk, 64, seed=seed + 1)[0]))
        cfg = svoo.BlockConfig(block=block, n_sel=n_sel)
        one = q[:, :, :1].contiguous()

        def call():
            pool = svoo.block_pool(k, cfg)
            idx = svoo.block_select(q, pool, cfg, Nk)
            o, lse = svoo.block_attn(q, k, v, idx, cfg)
            tok = svoo.block_select(one, pool, cfg, Nk)
            return (idx, o, lse, tok, *svoo.block_attn_backward(q, k, v, o, lse, g, idx, cfg),
                    *svoo.cache_attn(one, k, v, idx=tok, cfg=cfg))
        return call, call()

    jobs = [work(300, 2, 64, 57), work(60000, 30, 64, 58)]
    torch.cuda.synchronize()
    wrong = []

    def loop(call, want):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(60):
                    got = call()
                    torch.cuda.current_stream().synchronize()
                    if not all(torch.equal(x, y) for x, y in zip(got, want)):
                        wrong.append("results differ")
        except Exception as e:  # noqa: BLE001
            wrong.append(repr(e))

    threads = [threading.Thread(target=loop, args=j) for j in jobs]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong, wrong[:3]


@pytest.mark.parametrize("case", [
    # H, Hkv, Nq, Nk, d, block, n_sel: lists of a row tile's blocks that fit beside the tiles, and that do not
    (1, 1, 150, 200_000, 128, 64, 32),
    (1, 1, 150, 262_144, 128, 64, 32),        # the gradient's
    (2, 2, 300, 524_288 - 5, 128, 64, 64),    # the forward call's too
    (2, 1, 140, 360_000, 128, 128, 128),
    (1, 1, 200, 600_001, 64, 64, 200),
    (1, 1, 9, 1 << 20, 128, 1024, 256),
], ids=str)
def test_long_sequences_of_few_heads(case):
    H, Hkv, Nq, Nk, d, block, n_sel = case
    gen = torch.Generator(device="cuda").manual_seed(59)
    r = lambda *s: torch.randn(*s, generator=gen, device="cuda").bfloat16()  # noqa: E731
    q, k, v, g = r(1, H, Nq, d), r(1, Hkv, Nk, d), r(1, Hkv, Nk, d), r(1, H, Nq, d)
    cfg = svoo.BlockConfig(block=block, n_sel=n_sel)
    qc, kc, vc = (t.clone().requires_grad_(True) for t in (q, k, v))
    o, aux = svoo.block_attention(qc, kc, vc, cfg)
    got = torch.autograd.grad(o, (qc, kc, vc), g)
    svoo.check_device_errors(aux["dev_err"])
    q, k, v, g = (t.cpu() for t in (q, k, v, g))
    idx = aux["idx"].cpu()
    assert torch.equal(idx, ref.select(q, aux["pool"].cpu(), cfg, Nk))
    o64, l64, *want = ref.attn(q, k, v, idx, cfg, grad_o=g)
    check_out(o.detach(), aux["lse"], o64, l64, float(v.float().abs().max()))
    for name, x, y in zip(("dq", "dk", "dv"), got, want):
        close(x, y, name)


@pytest.mark.parametrize("Nq", [201, 202, 500])
def test_more_queries_than_keys(Nq):
    """Not causal: every query sees all keys; a causal call says where its queries are."""
    Nk, lengths = 200, [200, 130]
    q, k, v = make(2, 4, 2, Nq, Nk, 64, seed=60)
    g = make(2, 4, 2, Nq, Nk, 64, seed=61)[0]
    cfg = svoo.BlockConfig(block=64, n_sel=2, sink=1, local=0, causal=False)
    qc, kc, vc = (t.cuda().requires_grad_(True) for t in (q, k, v))
    o, aux = svoo.block_attention(qc, kc, vc, cfg, lens(lengths))
    got = torch.autograd.grad(o, (qc, kc, vc), g.cuda())
    assert torch.equal(aux["idx"].cpu(), ref.select(q, aux["pool"].cpu(), cfg, Nk, lengths, 0))
    o64, l64, *want = ref.attn(q, k, v, aux["idx"].cpu(), cfg, lengths, 0, grad_o=g)
    check_out(o.detach(), aux["lse"], o64, l64, float(v.float().abs().max()))
    for name, x, y in zip(("dq", "dk", "dv"), got, want):
        close(x, y, name)
    causal = svoo.BlockConfig(block=64, n_sel=2)
    args = [t.detach() for t in (qc, kc, vc)]
    with pytest.raises(svoo.SvooError):
        svoo.block_attention(*args, causal, lens(lengths))
    with pytest.raises(svoo.SvooError):
        svoo.block_select(args[0], aux["pool"], causal, Nk, lens(lengths))
    for q_start in (-1, 0):   # the queries before the first token, or behind the last, see nothing
        o, aux = svoo.block_attention(*args, causal, lens(lengths), q_start)
        assert torch.equal(aux["idx"].cpu(), ref.select(q, aux["pool"].cpu(), causal, Nk, lengths, q_start))
        o64, l64 = ref.attn(q, k, v, aux["idx"].cpu(), causal, lengths, q_start)
        check_out(o, aux["lse"], o64, l64, float(v.float().abs().max()))


@pytest.mark.parametrize("Nq", [1, 7, 40, 64, 200])      # both selection kernels, one to 32 queries a CTA
@pytest.mark.parametrize("G,d,block,n_sel", [(3, 64, 64, 6), (4, 128, 64, 12), (16, 64, 128, 5)])
def test_selection_of_heads_that_cancel(Nq, G, d, block, n_sel):
    """A group's sum is small beside its heads: fp32 additions of them are off by more than the scores' own bound."""
    Hkv, Nk = 2, 6000
    q, k, _ = make(1, G * Hkv, Hkv, Nq, Nk, d, seed=62)
    q = q.view(1, Hkv, G, Nq, d).clone()
    q[:, :, 0] *= 2.0 ** 17
    q[:, :, 2] = -q[:, :, 0]
    q = q.view(1, Hkv * G, Nq, d)
    for causal in (True, False):
        cfg = svoo.BlockConfig(block=block, n_sel=n_sel, sink=1, local=int(causal), causal=causal)
        pool = svoo.block_pool(k.cuda(), cfg)
        idx = svoo.block_select(q.cuda(), pool, cfg, Nk)
        assert torch.equal(idx.cpu(), ref.select(q, pool.cpu(), cfg, Nk))


@pytest.mark.parametrize("q_exp,k_exp", [(70, 0), (0, 70), (70, 70), (-80, 0), (0, -80), (-70, -50), (120, -100), (-120, 110)])
@pytest.mark.parametrize("Nq", [1, 40, 200])
def test_selection_far_from_one(Nq, q_exp, k_exp):
    """Norms whose squares, or scores that themselves, are outside fp32: blocks a few keys' last bits apart."""
    Hkv, G, d, block, Nk = 2, 2, 64, 64, 3000
    gen = torch.Generator().manual_seed(63)
    q, _, _ = make(1, G * Hkv, Hkv, Nq, 1, d, seed=64)
    k = torch.randn(1, Hkv, block, d, generator=gen).bfloat16().repeat(1, 1, 47, 1)[:, :, :Nk].clone()
    k.view(torch.int16)[:, :, ::block, ::7] ^= torch.randint(2, k[:, :, ::block, ::7].shape, generator=gen, dtype=torch.int16)
    q, k = q * 2.0 ** q_exp, k * 2.0 ** k_exp   # powers of two: no rounding
    for causal in (True, False):
        cfg = svoo.BlockConfig(block=block, n_sel=9, sink=1, local=int(causal), causal=causal)
        pool = svoo.block_pool(k.cuda(), cfg)
        idx = svoo.block_select(q.cuda(), pool, cfg, Nk)
        assert torch.equal(idx.cpu(), ref.select(q, pool.cpu(), cfg, Nk))


def test_forward_mode_gradients_are_refused():
    q, k, v = (t.cuda() for t in make(1, 2, 1, 70, 70, 64, seed=65))
    cfg = svoo.BlockConfig(n_sel=2)
    want, _ = svoo.block_attention(q, k, v, cfg)
    with torch.autograd.forward_ad.dual_level():
        for grad in (False, True):
            dual = torch.autograd.forward_ad.make_dual(v.clone().requires_grad_(grad), torch.ones_like(v))
            with pytest.raises(svoo.SvooError, match="forward-mode"):
                svoo.block_attention(q, k, dual, cfg)
        assert torch.equal(svoo.block_attention(q, k, v, cfg)[0], want)


@pytest.mark.parametrize("last", [1, 2, 5, 6, 100])
def test_renewed_means_leave_the_others(last):
    """The last blocks that hold keys are renewed, all others stay, also where more are asked for than there are."""
    lengths, block, Nk = [300, 64, 1, 0, 130], 64, 300
    _, k, _ = make(5, 2, 2, 1, Nk, 64, seed=66)
    cfg = svoo.BlockConfig(block=block)
    pool = torch.full((5, 2, 5, 64), 7.0, device="cuda")
    svoo.block_pool(k.cuda(), cfg, lens(lengths), pool=pool, last=last)
    want = ref.pool(k, block, lengths).float()
    for b, L in enumerate(lengths):
        n = -(-L // block)
        for c in range(5):
            if max(0, n - last) <= c < n:
                assert ((pool[b, :, c].cpu() - want[b, :, c]).abs() <= 2.0 ** -23 * want[b, :, c].abs()).all()
            else:
                assert (pool[b, :, c] == 7.0).all(), (b, c)


@pytest.mark.parametrize("bad", [lambda: torch.zeros(1, dtype=torch.int32), lambda: torch.zeros(1, dtype=torch.int64, device="cuda"),
                                 lambda: torch.zeros(0, dtype=torch.int32, device="cuda")])
def test_error_words_that_are_none(bad):
    q, k, v = (t.cuda() for t in make(1, 2, 1, 70, 70, 64, seed=67))
    cfg, err = svoo.BlockConfig(n_sel=2), bad()
    pool = svoo.block_pool(k, cfg)
    idx = svoo.block_select(q, pool, cfg, 70)
    o, lse = svoo.block_attn(q, k, v, idx, cfg)
    one = q[:, :, :1].contiguous()
    for call in (lambda: svoo.block_select(q, pool, cfg, 70, dev_err=err), lambda: svoo.block_attn(q, k, v, idx, cfg, dev_err=err),
                 lambda: svoo.block_attn_backward(q, k, v, o, lse, q, idx, cfg, dev_err=err),
                 lambda: svoo.block_attention(q, k, v, cfg, dev_err=err), lambda: svoo.cache_attn(one, k, v, dev_err=err),
                 lambda: svoo.cluster(q, k, svoo.Config(n_qc=4, n_kc=4), dev_err=err)):
        with pytest.raises(svoo.SvooError, match="dev_err"):
            call()
    torch.cuda.synchronize()


def test_tensors_written_in_place_are_known_to_autograd():
    """A backward pass over a cache that was cut since says so, instead of using the moved rows."""
    B, H, Hkv, N, d = 1, 4, 2, 200, 64
    q, k, v = (t.cuda() for t in make(B, H, Hkv, N, N, d, seed=68))
    cfg = svoo.BlockConfig(n_sel=3)
    w, pos = torch.rand(B, Hkv, N, device="cuda"), torch.arange(N, device="cuda").int().repeat(B, Hkv, 1)
    ln = lens([N])
    q.requires_grad_(True)
    for n in range(3):
        o, _ = svoo.block_attention(q, k, v, cfg, ln)
        if n == 0:
            o.float().sum().backward()   # nothing was written
            continue
        if n == 1:
            svoo.cache_evict(k, v, w, pos, ln, 150)
        else:
            svoo.block_attn(q.detach(), k, v, svoo.block_select(q.detach(), svoo.block_pool(k, cfg), cfg, N), cfg, out=o.detach())
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            o.float().sum().backward()
    one = q.detach()[:, :, :1].contiguous()
    pool = svoo.block_pool(k, cfg)
    idx = svoo.block_select(one, pool, cfg, N)
    before = [t._version for t in (w, pool, idx)]
    svoo.cache_attn(one, k, v, weight=w)
    svoo.block_pool(k, cfg, pool=pool, last=1)
    svoo.block_select(one, pool, cfg, N, idx=idx)
    assert [t._version for t in (w, pool, idx)] == [x + 1 for x in before]
    with torch.inference_mode():   # tensors without versions
        caches = [t.clone() for t in (k, v, w, pos, lens([N]))]
        svoo.cache_attn(one, *caches[:2], weight=caches[2])
    svoo.cache_evict(*caches, 100)
    assert caches[4].tolist() == [100]


@pytest.mark.parametrize("G,cap,d", [(128, 768 * 64, 64), (128, 767 * 64 + 5, 128), (120, 820 * 64 + 1, 64)])
def test_joining_runs_of_large_groups(G, cap, d):
    """The joining kernel's factors, one per head and run, take about the 48 KB that need no leave."""
    gen = torch.Generator(device="cuda").manual_seed(69)
    q, k, v = (torch.randn(1, h, n, d, generator=gen, device="cuda").bfloat16() for h, n in ((G, 1), (1, cap), (1, cap)))
    w = torch.zeros(1, 1, cap, device="cuda")
    o, lse = svoo.cache_attn(q, k, v, weight=w)
    s = q[0, :, 0].double() @ k[0, 0].double().T / math.sqrt(d)
    p = torch.softmax(s, -1)
    check_out(o, lse, (p @ v[0, 0].double())[None, :, None].cpu(), s.logsumexp(-1)[None, :, None].cpu(), float(v.abs().max()))
    assert ((w[0, 0].double() - p.sum(0)).abs() <= 2e-5 * p.sum(0)).all()


@pytest.mark.parametrize("kind", ["zero k", "zero q", "equal", "three", "close", "far"])
@pytest.mark.parametrize("Nq,d,n_sel,nb", [(1, 64, 12, 300), (5, 128, 100, 260), (40, 64, 30, 200), (40, 128, 80, 1500),
                                           (70, 64, 80, 300), (200, 128, 16, 130), (70, 64, 16, 2000), (70, 64, 20, 5000)])
def test_selection_with_many_equal_scores(Nq, d, n_sel, nb, kind):
    """More blocks at the border than either kernel's list holds, up to all of them: the lowest ones win."""
    B, Hkv, G, block = 1, 2, 2, 64
    gen = torch.Generator(device="cuda").manual_seed(70)
    Nk = nb * block
    q = torch.randn(B, Hkv * G, Nq, d, generator=gen, device="cuda").bfloat16()
    k = torch.zeros(B, Hkv, Nk, d, dtype=torch.bfloat16, device="cuda")
    rows = torch.randn(B, Hkv, block, d, generator=gen, device="cuda").bfloat16()
    if kind != "zero k":
        k += rows.repeat(1, 1, nb, 1)
    if kind == "zero q":
        q.zero_()
    if kind == "three":    # three kinds of blocks
        which = torch.randint(3, (nb,), generator=gen, device="cuda").repeat_interleave(block)
        k = (k.float() * torch.tensor([1.0, 1.5, 0.25], device="cuda")[which][:, None]).bfloat16()
    if kind == "close":    # one key in its last bits
        k.view(torch.int16)[:, :, ::block, ::7] ^= torch.randint(2, k[:, :, ::block, ::7].shape, generator=gen,
                                                                  device="cuda", dtype=torch.int16)
    if kind == "far":      # norms out of fp32's range, no two blocks alike
        q, k = q * 2.0 ** 70, (torch.randn(k.shape, generator=gen, device="cuda") * 2.0 ** 70).bfloat16()
    for causal in (True, False):
        cfg = svoo.BlockConfig(block=block, n_sel=n_sel, sink=1, local=int(causal), causal=causal)
        pool = svoo.block_pool(k, cfg)
        idx = svoo.block_select(q, pool, cfg, Nk)
        assert torch.equal(idx.cpu(), ref.select(q.cpu(), pool.cpu(), cfg, Nk))


@pytest.mark.parametrize("Nq,n_sel", [(1, 16), (40, 16), (4096, 16)])
def test_equal_scores_take_no_ages(Nq, n_sel):
    """Keys of zeros, as a program warms up with: slower than others, not by hundreds of times."""
    H, Hkv, d, Nk = 16, 4, 128, 32768
    gen = torch.Generator(device="cuda").manual_seed(71)
    q = torch.randn(1, H, Nq, d, generator=gen, device="cuda").bfloat16()
    k = torch.randn(1, Hkv, Nk, d, generator=gen, device="cuda").bfloat16()
    cfg = svoo.BlockConfig(block=64, n_sel=n_sel)
    took = []
    for keys in (k, torch.zeros_like(k)):
        pool, best = svoo.block_pool(keys, cfg), math.inf
        for _ in range(4):
            a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            torch.cuda._sleep(2_000_000)     # the host is ahead
            a.record()
            svoo.block_select(q, pool, cfg, Nk)
            b.record()
            torch.cuda.synchronize()
            best = min(best, a.elapsed_time(b))
        took.append(best)
    print(f"{Nq} queries: {took[0] * 1e3:.1f} us, equal scores {took[1] * 1e3:.1f} us")
    assert took[1] <= 60 * took[0]

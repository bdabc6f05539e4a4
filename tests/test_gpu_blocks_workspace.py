"""What workspaces and outputs hold before a call reaches no result: every operator of the block-selected attention
and of the cache, with its workspace and outputs filled beforehand, against a call of its own, bit for bit."""
import math
import threading

import pytest
import torch

import free_sparse_attention_head_b200 as svoo

pytestmark = pytest.mark.gpu


def rand(seed, *shape):
    return torch.randn(*shape, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda").bfloat16()


def filled(what, *args, byte):
    n = svoo._ws_bytes(what, *args)
    return torch.full((max(n, 256),), byte, dtype=torch.uint8, device="cuda")


SHAPES = [
    # B, H, Hkv, Nq, Nk, d, block, n_sel, sink, local, causal, lengths
    (2, 6, 3, 700, 700, 64, 64, 4, 1, 1, True, [700, 133]),       # one CTA a row tile or a few shares
    (1, 8, 2, 90, 1500, 128, 64, 8, 1, 1, True, None),            # shares
    (2, 4, 1, 333, 1111, 128, 192, 3, 1, 0, False, [1, 1000]),
    (1, 4, 4, 2100, 2100, 128, 256, 3, 1, 1, True, None),
    (1, 6, 3, 7446, 7446, 64, 256, 6, 1, 0, False, None),         # by key blocks
]


@pytest.mark.parametrize("byte", [0x41, 0xFF, 0x00])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_attention(shape, byte):
    B, H, Hkv, Nq, Nk, d, block, n_sel, sink, local, causal, lengths = shape
    q, k, v, g = rand(1, B, H, Nq, d), rand(2, B, Hkv, Nk, d), rand(3, B, Hkv, Nk, d), rand(4, B, H, Nq, d)
    ln = None if lengths is None else torch.tensor(lengths, dtype=torch.int32, device="cuda")
    cfg = svoo.BlockConfig(block=block, n_sel=n_sel, sink=sink, local=local, causal=causal)
    args = (B, H, Hkv, Nq, Nk, Nk, d, block, n_sel, sink, local, int(causal), Nk - Nq)
    pool = svoo.block_pool(k, cfg, ln, pool=torch.zeros(B, Hkv, -(-Nk // block), d, device="cuda"))
    idx = svoo.block_select(q, pool, cfg, Nk, ln)
    o, lse = svoo.block_attn(q, k, v, idx, cfg, ln)
    grads = svoo.block_attn_backward(q, k, v, o, lse, g, idx, cfg, ln)
    idx2 = svoo.block_select(q, pool, cfg, Nk, ln, idx=torch.full_like(idx, 77),
                             workspace=filled("svoo_block_select_workspace_size", *args, byte=byte))
    o2, lse2 = svoo.block_attn(q, k, v, idx, cfg, ln, out=torch.full_like(o, math.nan),
                               workspace=filled("svoo_block_attn_workspace_size", *args, byte=byte))
    again = svoo.block_attn_backward(q, k, v, o, lse, g, idx, cfg, ln,
                                     workspace=filled("svoo_block_attn_backward_workspace_size", *args, byte=byte))
    assert torch.equal(idx, idx2) and torch.equal(o, o2) and torch.equal(lse, lse2)
    assert all(torch.equal(x, y) for x, y in zip(grads, again))


@pytest.mark.parametrize("byte", [0x41, 0xFF, 0x00])
@pytest.mark.parametrize("B,H,Hkv,cap,d", [(1, 8, 8, 3000, 128), (5, 20, 4, 900, 64), (2, 32, 1, 5000, 128)])
def test_cache(B, H, Hkv, cap, d, byte):
    q, k, v = rand(1, B, H, 1, d), rand(2, B, Hkv, cap, d), rand(3, B, Hkv, cap, d)
    ln = torch.tensor([cap - 41 * b for b in range(B)], dtype=torch.int32, device="cuda")
    cfg = svoo.BlockConfig(block=64, n_sel=8, sink=1, local=1)
    pool = svoo.block_pool(k, cfg, ln)
    idx = svoo.block_select(q, pool, cfg, cap, ln, -1)
    sel = (B, H, Hkv, 1, cap, cap, d, 64, 8, 1, 1, 1, 0)
    whole = svoo._block_args(q, k, v, svoo._WHOLE, ln, 0)
    w0 = torch.rand(B, Hkv, cap, device="cuda")
    for args, kw in ((sel, dict(idx=idx, cfg=cfg)), (whole, {}), (whole, dict(weight=1))):
        got = []
        for ws in (None, filled("svoo_cache_attn_workspace_size", *args, "idx" in kw, "weight" in kw, byte=byte)):
            w = w0.clone()
            o = torch.full_like(q, math.nan)
            _, lse = svoo.cache_attn(q, k, v, ln, out=o, workspace=ws, **{**kw, **({"weight": w} if "weight" in kw else {})})
            got.append((o, lse, w))
        assert all(torch.equal(x, y) for x, y in zip(*got))
        assert torch.isfinite(got[0][0].float()).all()
    got = []
    for ws in (None, filled("svoo_cache_evict_workspace_size", B, Hkv, cap, 400, byte=byte)):
        state = k.clone(), v.clone(), w0.clone(), torch.arange(cap, device="cuda").int().repeat(B, Hkv, 1), ln.clone()
        svoo.cache_evict(*state, 400, sink=2, recent=30, workspace=ws)
        got.append(state)
    assert all(torch.equal(x, y) for x, y in zip(*got))


def test_first_call_of_a_host_thread():
    """A thread that has made no CUDA call before: forward, gradient, selection, cache, and the gradient by autograd,
    whose own thread may be such a one."""
    q, k, v, g = rand(1, 1, 4, 300, 64), rand(2, 1, 2, 300, 64), rand(3, 1, 2, 300, 64), rand(4, 1, 4, 300, 64)
    one = q[:, :, :1].contiguous()
    cfg = svoo.BlockConfig(n_sel=3)
    pool = svoo.block_pool(k, cfg)
    idx = svoo.block_select(q, pool, cfg, 300)
    o, lse = svoo.block_attn(q, k, v, idx, cfg)
    calls = dict(select=lambda: (svoo.block_select(q, pool, cfg, 300),), attn=lambda: svoo.block_attn(q, k, v, idx, cfg),
                 grad=lambda: svoo.block_attn_backward(q, k, v, o, lse, g, idx, cfg), cache=lambda: svoo.cache_attn(one, k, v))

    def leaves():
        x = [t.detach().clone().requires_grad_(True) for t in (q, k, v)]
        return torch.autograd.grad(svoo.block_attention(*x, cfg)[0], x, g)

    calls["autograd"] = leaves
    for name, call in calls.items():
        want, got = call(), []
        torch.cuda.synchronize()
        t = threading.Thread(target=lambda: got.append(call()))
        t.start()
        t.join()
        assert got and all(torch.equal(x, y) for x, y in zip(want, got[0])), name


@pytest.mark.parametrize("shape", [SHAPES[1], SHAPES[4]], ids=["shares", "by key blocks"])
def test_captured_and_replayed(shape):
    """A graph with the forward call and its gradient, replayed over other inputs, and one token's calls."""
    B, H, Hkv, Nq, Nk, d, block, n_sel, sink, local, causal, _ = shape
    cfg = svoo.BlockConfig(block=block, n_sel=n_sel, sink=sink, local=local, causal=causal)
    q, k, v, g = rand(1, B, H, Nq, d), rand(2, B, Hkv, Nk, d), rand(3, B, Hkv, Nk, d), rand(4, B, H, Nq, d)
    one = rand(5, B, H, 1, d)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")

    def calls():
        pool = svoo.block_pool(k, cfg)
        idx = svoo.block_select(q, pool, cfg, Nk, dev_err=err)
        o, lse = svoo.block_attn(q, k, v, idx, cfg, dev_err=err)
        tok = svoo.block_select(one, pool, cfg, Nk, dev_err=err)
        return (o, lse, *svoo.block_attn_backward(q, k, v, o, lse, g, idx, cfg, dev_err=err),
                *svoo.cache_attn(one, k, v, idx=tok, cfg=cfg, dev_err=err), *svoo.cache_attn(one, k, v, dev_err=err))

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        calls()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = calls()
    for seed in (11, 12):
        for i, t in enumerate((q, k, v, g, one)):
            t.copy_(rand(seed * 10 + i, *t.shape))
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in out]
        assert all(torch.equal(x, y) for x, y in zip(got, calls()))
    assert int(err) == 0

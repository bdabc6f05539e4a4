"""The timeout path of the block-selected attention's and the cache's kernels, run on the GPU with the test-only
build libsvoo_stall.so: one wait on a barrier that nothing completes runs out after about 10 ms, the kernel sets its
bit in the error word and returns, and nothing of the call reaches what the caller keeps. No fault, no endless wait."""
import time

import pytest
import torch

import free_sparse_attention_head_b200 as svoo
from free_sparse_attention_head_b200 import build as svoo_build
from test_timeout_path import _stall_library

pytestmark = pytest.mark.gpu

TIMEOUT = 1 << 0    # error word bit: an attention pipeline wait ran out
BAD_LIST = 1 << 2   # ... a list of blocks that is none


@pytest.fixture(scope="module", autouse=True)
def built():
    svoo_build.build()
    svoo.load()


def rand(seed, *shape):
    return torch.randn(*shape, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda").bfloat16()


def stalled(call, err, others=0):
    """The call through the stalling library: it comes back, with the bit set (and at most those of others)."""
    with _stall_library():
        t0 = time.perf_counter()
        out = call()
        torch.cuda.synchronize()
        took = time.perf_counter() - t0
    assert int(err.item()) & ~others == TIMEOUT
    assert took < 20.0
    return out


# one run a head, runs that are a cluster, runs that a second kernel joins
@pytest.mark.parametrize("B,H,Hkv,cap,d", [(2, 4, 2, 60, 64), (5, 20, 4, 900, 64), (1, 8, 8, 3000, 128)])
def test_running_weights_outlive_a_timeout(B, H, Hkv, cap, d):
    q, k, v = rand(1, B, H, 1, d), rand(2, B, Hkv, cap, d), rand(3, B, Hkv, cap, d)
    w0 = torch.rand(B, Hkv, cap, device="cuda")
    want = w0.clone()
    o, lse = svoo.cache_attn(q, k, v, weight=want)
    err, w = torch.zeros(1, dtype=torch.int32, device="cuda"), w0.clone()
    args = svoo._block_args(q, k, v, svoo._WHOLE, None, 0)
    # scores and parts that were never written: large, and not even numbers
    for byte in (0x41, 0xFF):
        err.zero_()
        n = svoo._ws_bytes("svoo_cache_attn_workspace_size", *args, False, True)
        ws = torch.full((n,), byte, dtype=torch.uint8, device="cuda")
        stalled(lambda: svoo.cache_attn(q, k, v, weight=w, workspace=ws, dev_err=err), err)
        assert torch.equal(w, w0)
        # while the bit stands, later calls leave the weights alone too
        svoo.cache_attn(q, k, v, weight=w, workspace=ws, dev_err=err)
        assert torch.equal(w, w0)
    err.zero_()
    o2, lse2 = svoo.cache_attn(q, k, v, weight=w, dev_err=err)
    assert int(err.item()) == 0
    assert torch.equal(w, want) and torch.equal(o, o2) and torch.equal(lse, lse2)


def config(block=64, n_sel=4, causal=True):
    return svoo.BlockConfig(block=block, n_sel=n_sel, sink=1, local=int(causal), causal=causal)


SHAPES = {
    # B, H, Hkv, Nq, Nk, d, config
    "means made in the kernel": (1, 4, 2, 300, 2000, 64, config()),
    "means split before": (1, 4, 2, 300, 6000, 128, config(n_sel=12)),
    "a cluster a tile": (1, 4, 2, 100, 3000, 128, config(n_sel=16)),
    "many tiles": (2, 16, 8, 1500, 1500, 64, config()),
    "by key blocks": (1, 64, 64, 2048, 2048, 64, config(block=128, n_sel=3, causal=False)),
}


@pytest.mark.parametrize("name", SHAPES)
def test_calls_come_back_and_recover(name):
    B, H, Hkv, Nq, Nk, d, cfg = SHAPES[name]
    q, k, v, g = rand(1, B, H, Nq, d), rand(2, B, Hkv, Nk, d), rand(3, B, Hkv, Nk, d), rand(4, B, H, Nq, d)
    one = rand(5, B, H, 1, d)
    pool = svoo.block_pool(k, cfg)
    idx = svoo.block_select(q, pool, cfg, Nk)
    tok = svoo.block_select(one, pool, cfg, Nk)
    o, lse = svoo.block_attn(q, k, v, idx, cfg)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")

    def calls(err):
        return dict(
            select=lambda: (svoo.block_select(q, pool, cfg, Nk, dev_err=err),),
            attn=lambda: svoo.block_attn(q, k, v, idx, cfg, dev_err=err),
            backward=lambda: svoo.block_attn_backward(q, k, v, o, lse, g, idx, cfg, dev_err=err),
            cache=lambda: svoo.cache_attn(one, k, v, idx=tok, cfg=cfg, dev_err=err),
            whole=lambda: svoo.block_attention(q, k, v, cfg, dev_err=err)[:1])

    want = {n: f() for n, f in calls(None).items()}
    for n, f in calls(err).items():
        # the attention of a selection that was never written may find that it is none, and say so
        others = BAD_LIST if n == "whole" else 0
        stalled(f, err, others)
        f()   # the bit stands: the work is skipped, and the call comes back
        torch.cuda.synchronize()
        assert int(err.item()) & ~others == TIMEOUT
        err.zero_()
    # without an error word every CTA gives up by itself (the gradient's second kernel, too)
    with _stall_library():
        for f in (list(calls(None).values()) if name != "by key blocks" else []):
            t0 = time.perf_counter()
            f()
            torch.cuda.synchronize()
            assert time.perf_counter() - t0 < 20.0
    for n, f in calls(err).items():
        assert all(torch.equal(x, y) for x, y in zip(f(), want[n])), n
    assert int(err.item()) == 0

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

TIMEOUT = 1 << 0   # error word bit: an attention pipeline wait ran out


@pytest.fixture(scope="module", autouse=True)
def built():
    svoo_build.build()
    svoo.load()


def rand(seed, *shape):
    return torch.randn(*shape, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda").bfloat16()


def stalled(call, err):
    """The call through the stalling library: it comes back, with the bit set."""
    with _stall_library():
        t0 = time.perf_counter()
        out = call()
        torch.cuda.synchronize()
        took = time.perf_counter() - t0
    assert int(err.item()) == TIMEOUT
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

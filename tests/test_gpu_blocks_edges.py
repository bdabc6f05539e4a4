"""Calls at the edges of what the block-selected attention and the cache calls document. Tolerances as in
test_gpu_blocks.py."""
import math

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

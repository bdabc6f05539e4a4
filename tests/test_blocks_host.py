"""The block-selected attention, cached attention and eviction calls on the host: argument checks that fail
before any launch, workspace sizes, and the gradient formula of the tests' reference against differences.
No GPU."""
import ctypes
import itertools
import os
import re

import pytest
import torch

import _blocks as ref
import free_sparse_attention_head_b200 as svoo
from free_sparse_attention_head_b200 import build as svoo_build

HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "svoo.h")
INVALID, WORKSPACE, UNSUPPORTED = 1, 2, 3
GOOD = dict(B=2, H=8, Hkv=2, Nq=100, Nk=300, cap=320, d=64, block=64, n_sel=4, sink=1, local=1, causal=1, q_start=200)


@pytest.fixture(scope="module")
def lib():
    svoo_build.build()
    return svoo.load()


def shape(**change):
    return ctypes.pointer(svoo.BlockShape(**{**GOOD, **change}))


def test_shape_fields_are_the_headers():
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    body = re.search(r"typedef struct \{([^}]*)\} svoo_block_shape;", text).group(1)
    names = [n.strip() for line in re.findall(r"int ([^;]+);", body) for n in line.split(",")]
    assert names == [f for f, _ in svoo.BlockShape._fields_]


BAD = [dict(B=0), dict(H=0), dict(Hkv=0), dict(Hkv=3), dict(H=258, Hkv=2), dict(Nq=-1), dict(Nk=0), dict(cap=299),
       dict(cap=(1 << 20) + 1), dict(d=96), dict(d=0), dict(block=0), dict(block=63), dict(block=96), dict(block=1088),
       dict(n_sel=0), dict(n_sel=257), dict(sink=-1), dict(local=-1), dict(sink=5), dict(sink=2, local=3),
       dict(local=0), dict(causal=0), dict(causal=2), dict(q_start=-2), dict(B=70000, H=1, Hkv=1),
       dict(B=4096, H=8, Hkv=8, cap=1 << 20, Nk=1 << 20)]


@pytest.mark.parametrize("bad", BAD)
def test_bad_shapes_are_refused_before_any_launch(lib, bad):
    s, x, n = shape(**bad), 0x1000, 1 << 40
    assert lib.svoo_block_select_workspace_size(s) == 0
    assert lib.svoo_block_attn_workspace_size(s) == 0
    assert lib.svoo_block_attn_backward_workspace_size(s) == 0
    assert lib.svoo_block_pool(s, x, None, 0, x, None) == INVALID
    assert lib.svoo_block_select(s, x, x, None, x, x, n, None, None) == INVALID
    assert lib.svoo_block_attn(s, x, x, x, x, None, 0.1, x, x, x, n, None, None) == INVALID
    assert lib.svoo_block_attn_backward(s, x, x, x, x, x, x, x, None, 0.1, x, x, x, x, n, None, None) == INVALID
    one = shape(**{**bad, "Nq": bad.get("Nq", 1)})
    assert lib.svoo_cache_attn_workspace_size(one, 0, 1) == 0
    assert lib.svoo_cache_attn(one, x, x, x, None, None, 0.1, None, x, x, x, n, None, None) == INVALID


def test_null_and_misaligned_pointers_are_refused(lib):
    s, one, n = shape(), shape(Nq=1), 1 << 40
    calls = [
        (lib.svoo_block_pool, [s, 0x1000, None, 0, 0x1000, None], (1, 4), 16),
        (lib.svoo_block_select, [s, 0x1000, 0x1000, None, 0x1000, 0x1000, n, None, None], (1, 2, 4), 4),
        (lib.svoo_block_attn, [s] + [0x1000] * 4 + [None, 0.1] + [0x1000] * 3 + [n, None, None], (1, 2, 3, 4, 7, 8), 4),
        (lib.svoo_block_attn_backward, [s] + [0x1000] * 7 + [None, 0.1] + [0x1000] * 4 + [n, None, None],
         (1, 2, 3, 4, 5, 6, 7, 10, 11, 12, 13), 4),
        (lib.svoo_cache_attn, [one] + [0x1000] * 3 + [None, None, 0.1, None] + [0x1000] * 3 + [n, None, None],
         (1, 2, 3, 8, 9), 4),
    ]
    for fn, args, needed, _ in calls:
        for i in needed:
            for value in (None, 0x1001):
                bad = list(args)
                bad[i] = value
                assert fn(*bad) == INVALID, (fn.__name__, i, value)
    for scale in (0.0, -1.0, float("nan"), float("inf")):
        assert lib.svoo_block_attn(s, *[0x1000] * 4, None, scale, *[0x1000] * 3, n, None, None) == INVALID
        assert lib.svoo_cache_attn(one, *[0x1000] * 3, None, None, scale, None, *[0x1000] * 3, n, None, None) == INVALID
    assert lib.svoo_block_pool(s, 0x1000, None, -1, 0x1000, None) == INVALID
    assert lib.svoo_cache_attn(s, *[0x1000] * 3, None, None, 0.1, None, *[0x1000] * 3, n, None, None) == INVALID  # Nq > 1


def test_workspaces(lib):
    x = 0x1000
    s = shape()
    assert lib.svoo_block_select_workspace_size(s) == 0     # up to 64 blocks need none
    longer = shape(Nk=5000, cap=5000)
    need = lib.svoo_block_select_workspace_size(longer)
    assert need > 0
    assert lib.svoo_block_select(longer, x, x, None, x, x, need - 1, None, None) == WORKSPACE
    assert lib.svoo_block_select(longer, x, x, None, x, None, 0, None, None) == WORKSPACE
    # row tiles need none; by key blocks (here: 16 heads of their own, 3 of 32 blocks of 128 keys) the parts do
    assert lib.svoo_block_attn_workspace_size(s) == 0
    lists = shape(B=1, H=16, Hkv=16, Nq=8192, Nk=4096, cap=4096, block=128, n_sel=3, sink=1, local=0, causal=0, q_start=0)
    need = lib.svoo_block_attn_workspace_size(lists)
    assert need > 16 * 8192 * 3 * 64 * 4
    assert lib.svoo_block_attn(lists, x, x, x, x, None, 0.1, x, x, x, need - 1, None, None) == WORKSPACE
    assert lib.svoo_block_attn(lists, x, x, x, x, None, 0.1, x, x, None, 0, None, None) == WORKSPACE
    need = lib.svoo_block_attn_backward_workspace_size(s)
    assert lib.svoo_block_attn_backward(s, x, x, x, x, x, x, x, None, 0.1, x, x, x, x, need - 1, None, None) == WORKSPACE
    one = shape(Nq=1, cap=4096, Nk=4096)
    assert all(lib.svoo_cache_attn_workspace_size(one, selected, 1) > 0 for selected in (0, 1))
    assert lib.svoo_cache_attn_workspace_size(one, 1, 0) == 0   # few runs of slots join among themselves
    many = shape(B=1, H=1, Hkv=1, Nq=1, cap=1 << 16, Nk=1 << 16)
    assert lib.svoo_cache_attn_workspace_size(many, 0, 0) > 0
    need = lib.svoo_cache_attn_workspace_size(one, 0, 1)
    assert lib.svoo_cache_attn(one, x, x, x, None, None, 0.1, x, x, x, x, need - 1, None, None) == WORKSPACE
    assert lib.svoo_cache_attn(one, x, x, x, None, x, 0.1, x, x, x, x, need, None, None) == UNSUPPORTED
    # a long sequence's gradient stays far below its scores
    big = shape(B=1, H=16, Hkv=2, Nq=1 << 17, Nk=1 << 17, cap=1 << 17, d=128, n_sel=16, q_start=0)
    assert 0 < lib.svoo_block_attn_backward_workspace_size(big) < 1 << 30
    # no queries: nothing to do
    empty = shape(Nq=0)
    n = 1 << 40
    assert lib.svoo_block_select(empty, x, x, None, x, x, n, None, None) == 0
    assert lib.svoo_block_attn(empty, x, x, x, x, None, 0.1, x, x, x, n, None, None) == 0


def test_eviction_arguments(lib):
    x, n = 0x1000, 1 << 40
    good = (2, 4, 100, 64, 40, 4, 8)
    need = lib.svoo_cache_evict_workspace_size(2, 4, 100, 40)
    assert need > 0
    assert lib.svoo_cache_evict(*good, x, x, x, x, x, x, need - 1, None) == WORKSPACE
    for i, v in [(0, 0), (1, 0), (2, 0), (2, (1 << 20) + 1), (3, 80), (4, 0), (5, -1), (6, -1), (5, 41), (6, 37)]:
        bad = list(good)
        bad[i] = v
        assert lib.svoo_cache_evict(*bad, x, x, x, x, x, x, n, None) == INVALID, (i, v)
    for i in range(6):
        for value in (None, 0x1001):
            p = [x] * 6
            p[i] = value
            assert lib.svoo_cache_evict(*good, *p, n, None) == INVALID
    # a cache that cannot hold more than `keep` needs no work
    assert lib.svoo_cache_evict(2, 4, 40, 64, 40, 4, 8, x, x, x, x, x, x, n, None) == 0


def test_tensors_off_the_gpu_are_refused():
    q, k = torch.zeros(1, 2, 4, 64, dtype=torch.bfloat16), torch.zeros(1, 1, 64, 64, dtype=torch.bfloat16)
    cfg = svoo.BlockConfig()
    for call in (lambda: svoo.block_attention(q, k, k, cfg), lambda: svoo.block_pool(k, cfg),
                 lambda: svoo.block_select(q, torch.zeros(1, 1, 1, 64), cfg, 64),
                 lambda: svoo.cache_attn(q[:, :, :1], k, k),
                 lambda: svoo.cache_evict(k, k, torch.zeros(1, 1, 64), torch.zeros(1, 1, 64, dtype=torch.int32),
                                          torch.zeros(1, dtype=torch.int32), 8)):
        with pytest.raises(svoo.SvooError):
            call()


@pytest.mark.parametrize("causal", [True, False])
def test_reference_gradient_against_differences(causal):
    """The formula that the GPU tests compare with, against central differences of the reference's own output."""
    g = torch.Generator().manual_seed(1)
    B, H, Hkv, N, d = 1, 2, 1, 70, 64
    q, k, v, w = (torch.randn(B, h, N, d, generator=g, dtype=torch.float64) * 0.5 for h in (H, Hkv, Hkv, H))
    cfg = svoo.BlockConfig(block=64, n_sel=2, sink=0, local=2 if causal else 0, causal=causal)
    idx = torch.tensor([[[[0, 1] if (t >= 64 or not causal) and t % 3 else [0, -1] for t in range(N)]]], dtype=torch.int32)
    _, _, *grads = ref.attn(q, k, v, idx, cfg, grad_o=w)
    loss = lambda: float((ref.attn(q, k, v, idx, cfg)[0] * w).sum())  # noqa: E731
    h = 1e-5
    for t, grad in zip((q, k, v), grads):
        flat = t.view(-1)
        for i in torch.randint(flat.numel(), (6,), generator=g).tolist():
            keep = float(flat[i])
            flat[i] = keep + h
            up = loss()
            flat[i] = keep - h
            down = loss()
            flat[i] = keep
            # central differences: h^2 and 1e-16 / h, both below 1e-9 here
            assert abs((up - down) / (2 * h) - float(grad.view(-1)[i])) <= 1e-7

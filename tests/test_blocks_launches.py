"""What the block-selected attention and the cache calls ask of the CUDA runtime, checked without a GPU."""
import random

import pytest
import torch

from _host_launches import Host, shape


@pytest.fixture(scope="module")
def host(tmp_path_factory):
    return Host(str(tmp_path_factory.mktemp("host")))


@pytest.mark.parametrize("first,Nk", [(0, 1000), (100, 900), (10, 990), (1, 64), (0, 63), (937, 63)])
@pytest.mark.parametrize("B,Hkv", [(1, 1), (1, 4), (2, 1), (2, 4)])
def test_maps_of_keys_end_with_their_last_row(host, B, Hkv, first, Nk):
    """A view may begin inside its buffer (cap 1000 rows a head): a tensor map over whole tiles must not reach
    behind the view's last row, where the allocation may end."""
    cap, d = 1000, 64
    view = torch.empty(B, Hkv, cap, d)[:, :, first:first + Nk]
    last = sum((n - 1) * s for n, s in zip(view.shape, view.stride()))   # element that the view ends with
    rows = last // d + 1
    fields = dict(B=B, H=2 * Hkv, Hkv=Hkv, Nk=Nk, cap=cap, d=d, block=64, n_sel=2, sink=0, local=1, causal=1)
    for call, Nq in ((host.attn, 200), (host.backward, 200), (host.cache, 1)):
        assert call(shape(**fields, Nq=Nq, q_start=0)) == 0
        of_keys = [m for m in host.maps if m[0] in (0x20000, 0x30000)]
        assert {m[0] for m in of_keys} == {0x20000, 0x30000}
        for _, n, cols, _ in of_keys:
            assert (n, cols) == (rows, d)
    # by key blocks
    lists = dict(B=1, H=16, Hkv=16, Nq=8192, Nk=4000, cap=4096, d=64, block=128, n_sel=3, sink=1, local=0, causal=0, q_start=0)
    assert host.attn(shape(**lists)) == 0
    assert any("block_list_kernel" in x.kernel for x in host.launches)
    assert [m[1] for m in host.maps] == [15 * 4096 + 4000] * 2


SHAPES = [   # small to large lists and rows of scores, many and few queries, both head dimensions
    dict(B=B, H=H, Hkv=Hkv, Nq=Nq, Nk=Nk, cap=Nk, d=d, block=block, n_sel=n_sel, sink=0, local=1, causal=1, q_start=0)
    for B, H, Hkv, Nq, Nk, block, n_sel in [(1, 1, 1, 1, 64, 64, 2), (2, 8, 2, 40, 5000, 64, 4), (1, 2, 2, 300, 60000, 64, 16),
                                             (1, 64, 1, 20, 250000, 64, 70), (1, 4, 2, 3000, 90000, 128, 30),
                                             (3, 6, 6, 7, 1 << 19, 64, 100)] for d in (64, 128)]


def calls_of(host, s):
    f = dict(s)
    one = shape(**{**f, "Nq": 1})
    return [lambda: host.select(shape(**f)), lambda: host.attn(shape(**f)), lambda: host.backward(shape(**f)),
            lambda: host.select(one), lambda: host.cache(one), lambda: host.cache(one, idx=0x40000),
            lambda: host.cache(one, weight=0x40000)]


def test_leave_for_shared_memory_is_the_same_in_every_call(host):
    """It is a state of the function: a call that gave less could take it from another thread's, before its launch."""
    given = {}
    for s in SHAPES:
        for call in calls_of(host, s):
            call()
            for kernel, most in host.allowed:
                given.setdefault(kernel, set()).add(most)
    assert len(given) > 10
    assert {k: v for k, v in given.items() if len(v) > 1} == {}


def test_a_refused_call_leaves_no_error_behind(host):
    """The runtime's last error is the next launch check's to find, whoever makes it."""
    for s in SHAPES[:4]:
        for call in calls_of(host, s):
            host.lib.fake_refuse(1)
            try:
                assert call() != 0
                assert host.lib.fake_last_error() == 0
            finally:
                host.lib.fake_refuse(0)
            host.lib.fake_refuse(2)
            try:
                assert call() != 0
                assert host.lib.fake_last_error() == 0
            finally:
                host.lib.fake_refuse(0)
            call()


def draw(rng):
    """A shape from all that svoo_block_shape allows, extremes first."""
    d, block = rng.choice([64, 128]), rng.choice([64, 64, 128, 192, 1024])
    Hkv = rng.choice([1, 2, 5])
    G = rng.choice([1, 1, 2, 3, 8, 40, 128])
    Nk = rng.choice([1 << 20, 1 << 20, 262144, 360000, rng.randint(1, 1 << 20), rng.randint(1, 5000)])
    n_sel = rng.choice([256, 128, 64, 48, 32, 16, rng.randint(1, 256)])
    causal = rng.randint(0, 1)
    sink = rng.randint(0, min(2, n_sel - causal))
    return dict(B=rng.randint(1, 2), H=Hkv * G, Hkv=Hkv, Nq=rng.choice([1, 7, 63, 200, 5000]), Nk=Nk, cap=Nk, d=d, block=block,
                n_sel=n_sel, sink=sink, local=causal, causal=causal, q_start=rng.choice([-1, 0, Nk - 1]))


def test_every_shape_of_the_documented_range_is_launched(host):
    rng = random.Random(1)
    shapes = [dict(B=1, H=1, Hkv=1, Nq=200, Nk=Nk, cap=Nk, d=128, block=block, n_sel=n_sel, sink=1, local=1, causal=1, q_start=-1)
              for Nk, block, n_sel in [(262144, 64, 32), (360000, 128, 32), (524288, 64, 64), (1 << 20, 64, 256),
                                       (1 << 20, 1024, 256), (1 << 20, 64, 16)]]
    for s in shapes + [draw(rng) for _ in range(400)]:
        for call in calls_of(host, s):
            assert call() == 0, s
            assert not any(x.bad for x in host.launches), s


def test_clusters_never_share_an_sm_three_at_a_time(host):
    """A CTA of the forward call's clusters holds half of an SM's tensor memory until its whole cluster is through: a
    third on the SM would wait for some there, and clusters that wait for each other that way would never end."""
    seen = 0
    for d in (64, 128):
        for Nq, Nk, n_sel in [(333, 1999, 8), (20, 300, 4), (64, 5000, 30), (700, 700, 16), (1, 9000, 64)]:
            s = shape(B=1, H=4, Hkv=2, Nq=Nq, Nk=Nk, cap=Nk, d=d, block=64, n_sel=n_sel, sink=0, local=1, causal=1, q_start=-1)
            assert host.attn(s) == 0
            for x in host.launches:
                if "block_attn_kernel" in x.kernel and x.grid[2] > 1:
                    seen += 1
                    assert 3 * (x.smem + 1024) > 228 * 1024 and not x.bad
    assert seen >= 8


def test_misaligned_lengths_and_error_words_are_refused(host):
    """Optional addresses are checked like the others: kernels read and write 32-bit words there."""
    x, n, odd = 0x10000, 1 << 60, 0x10002
    s = dict(B=2, H=4, Hkv=2, Nq=100, Nk=300, cap=300, d=64, block=64, n_sel=4, sink=1, local=1, causal=1, q_start=0)
    many, one = shape(**s), shape(**{**s, "Nq": 1})

    def calls(lengths, err):
        yield host("svoo_block_select", many, x, x, lengths, x, x, n, err, None)
        yield host("svoo_block_attn", many, x, x, x, x, lengths, 0.1, x, x, x, n, err, None)
        yield host("svoo_block_attn_backward", many, x, x, x, x, x, x, x, lengths, 0.1, x, x, x, x, n, err, None)
        yield host("svoo_cache_attn", one, x, x, x, lengths, None, 0.1, None, x, x, x, n, err, None)
        if err is None:
            yield host("svoo_block_pool", many, x, lengths, 0, x, None)

    assert all(status == 0 for status in calls(None, None)) and all(status == 0 for status in calls(x, x))
    assert all(status == 1 and not host.launches for status in calls(odd, None))
    assert all(status == 1 and not host.launches for status in calls(None, odd))


@pytest.mark.parametrize("G", [112, 126, 127, 128])
@pytest.mark.parametrize("selected", [False, True])
def test_joining_runs_of_large_groups(host, G, selected):
    """A factor per head and run: about 48 KB, beside what the kernel declares for itself."""
    for B in (1, 2):
        for tiles in range(300, 1200, 4):
            s = dict(B=B, H=G, Hkv=1, Nq=1, Nk=64 * tiles, cap=64 * tiles, d=128, block=64, n_sel=16, sink=0, local=1, causal=1, q_start=0)
            if selected:
                s.update(Nk=832, cap=832, block=1024, n_sel=tiles // 16)
            assert host.cache(shape(**s), idx=0x40000 if selected else None) == 0, (B, tiles)

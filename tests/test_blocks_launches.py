"""What the block-selected attention and the cache calls ask of the CUDA runtime, checked without a GPU."""
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

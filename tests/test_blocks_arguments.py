"""Arguments that the Python entry points settle themselves, without a GPU."""
import pytest
import torch
import torch.autograd.forward_ad as fwd

import free_sparse_attention_head_b200 as svoo


def test_positions_of_the_queries():
    """-1 is the C call's word for the end of every sequence: no default may come out as it by arithmetic."""
    first = svoo._first_position
    assert first(None, 300, 100, True) == 200 and first(None, 300, 300, True) == 0
    for Nq in (301, 302, 1000):
        with pytest.raises(svoo.SvooError):
            first(None, 300, Nq, True)
        assert first(None, 300, Nq, False) == 0    # positions mean nothing
    for given in (-1, 0, 7):
        assert first(given, 300, 301, True) == first(given, 300, 301, False) == given


@pytest.mark.parametrize("which", range(3))
def test_forward_mode_gradients_are_refused(which):
    """A tangent would be lost without a word: the autograd function is passed by where nothing requires a gradient."""
    ts = [torch.zeros(1, 2, 4, 64, dtype=torch.bfloat16) for _ in range(3)]
    with fwd.dual_level():
        assert not svoo._has_tangent(*ts)
        ts[which] = fwd.make_dual(ts[which], torch.ones_like(ts[which]))
        assert svoo._has_tangent(*ts)
        with pytest.raises(svoo.SvooError, match="forward-mode"):
            svoo.block_attention(*ts, svoo.BlockConfig())
    assert not svoo._has_tangent(*ts)


def test_the_error_word_is_checked():
    """Kernels write to its address: an address of the host, of another device or of nothing may not reach them."""
    dev = torch.device("cuda", 0)
    for bad in (torch.zeros(1, dtype=torch.int32), torch.zeros(0, dtype=torch.int32, device="meta"), 4096, [0]):
        with pytest.raises(svoo.SvooError, match="dev_err"):
            svoo._err_at(bad, dev)
        with pytest.raises(svoo.SvooError, match="dev_err"):
            svoo._err_buf(bad, dev)
    meta = torch.device("meta")
    for bad in (torch.zeros(1, dtype=torch.int64, device=meta), torch.zeros(0, dtype=torch.int32, device=meta)):
        with pytest.raises(svoo.SvooError, match="dev_err"):
            svoo._err_at(bad, meta)
    good = torch.zeros(2, dtype=torch.int32, device=meta)
    assert svoo._err_buf(good, meta) is good and svoo._err_at(None, dev) is None

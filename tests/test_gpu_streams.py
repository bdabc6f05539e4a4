"""stream=: a call runs as if that stream were current. While the stream still has work before the call, nothing
that the current stream allocates may lie in what the call made for itself, and filling it changes no result."""
import pytest
import torch

import free_sparse_attention_head_b200 as svoo
import workload
from _parity import qkv_tensors

pytestmark = pytest.mark.gpu


def flat(x):
    return [t for t in svoo._tensors(x) if t.is_cuda]


@pytest.mark.parametrize("path", ["clustered", "steps", "stripes"])
def test_calls_on_another_stream(path, monkeypatch):
    w = workload.get("tiny")
    qd, kd, vd = qkv_tensors(*workload.make_qkv(w), w.B, w.H)
    cfg = svoo.Config(n_qc=w.n_qc, n_kc=w.n_kc, iters=w.iters, block_q=w.block_q)
    keep = torch.from_numpy(w.keep_ratios()).cuda()
    sh = svoo.make_shape(qd, w.n_text)
    params = svoo.psa_params([(7, 0, None, 3, 0, 5)] * (w.B * w.H), "cuda")

    def run(stream=None):
        kw = {} if stream is None else {"stream": stream}
        if path == "clustered":
            return svoo.sparse_attention(qd, kd, vd, keep, cfg, n_text=w.n_text, **kw)
        if path == "stripes":
            return svoo.psa_attention(qd, kd, vd, w.grid, w.cell, params, n_text=w.n_text, **kw)
        cl = svoo.cluster(qd, kd, cfg, n_text=w.n_text, **kw)
        plan = svoo.build_mask(sh, cl, keep, cfg, **kw)
        rows = svoo.permute(qd, kd, vd, cl["k_assign"], plan, **kw)
        return svoo.sparse_attn(*rows, plan, **kw), cl, plan

    want = [t.clone() for t in flat(run())]
    torch.full((1,), 0xFF, dtype=torch.uint8, device="cuda")   # a kernel's first launch may wait for the device
    torch.cuda.synchronize()
    made, real = [], {n: getattr(torch, n) for n in ("empty", "zeros", "empty_like")}

    def noting(f):
        def call(*a, **kw):
            t = f(*a, **kw)
            if t.is_cuda:
                made.append((t.data_ptr(), t.numel() * t.element_size()))
            return t
        return call

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        torch.cuda._sleep(800_000_000)     # some tenths of a second: the call's kernels have not begun
    for n, f in real.items():
        monkeypatch.setattr(svoo.torch, n, noting(f))
    got = run(side)
    monkeypatch.undo()
    assert not side.query(), "the stream was to be busy"
    assert made
    later = [torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda") for _, n in made for _ in range(3)]
    assert not side.query(), "the stream was to be busy"
    for at, n in made:
        for t in later:
            assert t.data_ptr() + t.numel() <= at or at + n <= t.data_ptr(), n
    torch.cuda.synchronize()
    got = flat(got)
    assert len(got) == len(want) and all(torch.equal(x, y) for x, y in zip(got, want))

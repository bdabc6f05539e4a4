"""Python binding of libsvoo (online QK co-clustered block-sparse attention, sm_100a).

Argument marshalling only: every step runs in the library's CUDA kernels
(`csrc/`, C ABI in `include/svoo.h`). PyTorch provides device memory and the
current CUDA stream. If the compiled library is missing or no CUDA device is
present, calls raise; there is no CPU fallback. stream= runs a call as if that
stream were current: what the call reads must be ready there, and stay allocated
until the stream has used it; workspaces and results made inside are the stream's.

Typical use (all tensors on one CUDA device, bf16 [B, H, N, d]):

    import free_sparse_attention_head_b200 as svoo
    cfg = svoo.Config(n_qc=256, n_kc=256, iters=10, block_q=128)
    out, plan = svoo.sparse_attention(q, k, v, keep, cfg)
"""
from __future__ import annotations

import ctypes
import dataclasses
import functools
import math
import os
from typing import Optional

import torch

__all__ = [
    "Config", "Shape", "Plan", "load", "lib_path", "cluster", "cluster_step", "build_mask",
    "permute", "sparse_attn", "sparse_attention", "check_device_errors", "workspace_sizes",
    "SvooError", "CLUSTER_WARM", "CLUSTER_IDENTITY", "PSA_INF", "psa_config", "psa_params",
    "psa_mask", "psa_attention", "snr_top_p", "cluster_outputs",
    "BlockConfig", "BlockShape", "block_pool", "block_select", "block_attn", "block_attn_backward",
    "block_attention", "cache_attn", "cache_evict",
]

_HERE = os.path.dirname(os.path.abspath(__file__))
_LIB_PATH = os.path.join(_HERE, "libsvoo.so")
_lib = None


class SvooError(RuntimeError):
    pass


class Shape(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int), ("H", ctypes.c_int), ("N", ctypes.c_int), ("d", ctypes.c_int),
                ("n_text", ctypes.c_int)]


class BlockShape(ctypes.Structure):
    _fields_ = [(f, ctypes.c_int) for f in ("B", "H", "Hkv", "Nq", "Nk", "cap", "d", "block", "n_sel",
                                            "sink", "local", "causal", "q_start")]


_PLAN_FIELDS = ["kmask", "q_label", "q_sizes", "stats", "q_perm", "q_off", "k_perm", "k_off",
                "tiles", "tile_count", "units", "unit_count"]


class _CPlan(ctypes.Structure):
    _fields_ = [(f, ctypes.c_void_p) for f in _PLAN_FIELDS]


_P = ctypes.c_void_p
_I = ctypes.c_int
_F = ctypes.c_float
_SZ = ctypes.c_size_t
_SP = ctypes.POINTER(Shape)
_PP = ctypes.POINTER(_CPlan)
_BP = ctypes.POINTER(BlockShape)

_SIGS = {
    "svoo_status_string": (ctypes.c_char_p, [_I]),
    "svoo_version": (_I, []),
    "svoo_plan_counts": (_I, [_SP, _I, _I, _I, ctypes.POINTER(ctypes.c_int64)]),
    "svoo_cluster_workspace_size": (_SZ, [_SP, _I, _I]),
    "svoo_cluster": (_I, [_SP, _P, _P, _I, _I, _I, _I, _P, _P, _P, _P, _P, _P, _P, _SZ, _P, _P]),
    "svoo_cluster_step": (_I, [_SP, _P, _I, _P, _P, _P, _P, _P, _I, _P, _SZ, _P, _P]),
    "svoo_cluster_step_static": (_I, [_SP, _P, _I, _P, _P, _P, _P, _P, _I, _P, _P]),
    "svoo_mask_workspace_size": (_SZ, [_SP, _I, _I]),
    "svoo_build_mask": (_I, [_SP, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _F, _PP, _P, _SZ,
                             _P, _P]),
    "svoo_permute": (_I, [_SP, _P, _P, _P, _P, _I, _I, _I, _PP, _P, _P, _P, _P, _P]),
    "svoo_sparse_attn": (_I, [_SP, _P, _P, _P, _PP, _I, _I, _I, _F, _P, _P, _P]),
    "svoo_psa_block_count": (_I, [_I, _I, _I, _I, _I, _I]),
    "svoo_psa_mask": (_I, [_SP, _I, _I, _I, _I, _I, _I, _P, _I, _PP, _P, _P, _P]),
    "svoo_snr_top_p": (_I, [_I, _I, ctypes.c_double, ctypes.c_double, ctypes.c_double, _P]),
    "svoo_block_pool": (_I, [_BP, _P, _P, _I, _P, _P]),
    "svoo_block_select_workspace_size": (_SZ, [_BP]),
    "svoo_block_select": (_I, [_BP, _P, _P, _P, _P, _P, _SZ, _P, _P]),
    "svoo_block_attn_workspace_size": (_SZ, [_BP]),
    "svoo_block_attn": (_I, [_BP, _P, _P, _P, _P, _P, _F, _P, _P, _P, _SZ, _P, _P]),
    "svoo_block_attn_backward_workspace_size": (_SZ, [_BP]),
    "svoo_block_attn_backward": (_I, [_BP, _P, _P, _P, _P, _P, _P, _P, _P, _F, _P, _P, _P, _P, _SZ, _P, _P]),
    "svoo_cache_attn_workspace_size": (_SZ, [_BP, _I, _I]),
    "svoo_cache_attn": (_I, [_BP, _P, _P, _P, _P, _P, _F, _P, _P, _P, _P, _SZ, _P, _P]),
    "svoo_cache_evict_workspace_size": (_SZ, [_I, _I, _I, _I]),
    "svoo_cache_evict": (_I, [_I, _I, _I, _I, _I, _I, _I, _P, _P, _P, _P, _P, _P, _SZ, _P]),
}

EXPORTS = tuple(_SIGS)


def lib_path() -> str:
    return _LIB_PATH


def load(path: Optional[str] = None):
    """Loads libsvoo.so (built by `free_sparse_attention_head_b200.build`)."""
    global _lib
    if _lib is None:
        p = path or _LIB_PATH
        if not os.path.exists(p):
            raise SvooError(f"{p} is missing: run `python -m free_sparse_attention_head_b200.build`")
        L = ctypes.CDLL(p)
        for name, (res, args) in _SIGS.items():
            fn = getattr(L, name)
            fn.restype = res
            fn.argtypes = args
        _lib = L
    return _lib


def _check(status: int, what: str):
    if status != 0:
        msg = load().svoo_status_string(status).decode()
        raise SvooError(f"{what}: {msg} (status {status})")


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream():
    return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)


def _under(stream, device, fn, *args):
    """A call with stream=: fn(*args) with that stream current, so that the workspaces and results made inside
    are the stream's own memory. The current stream's would be given to later work there while the
    kernels still use it. Results may be freed once the current stream has used them."""
    mine = torch.cuda.current_stream(device) if device.type == "cuda" else None
    if mine is None or stream.device != mine.device:
        raise SvooError(f"stream is one of {stream.device}: the tensors must live there")
    if stream == mine:
        return fn(*args)
    with torch.cuda.stream(stream):
        out = fn(*args)
    given = {id(t) for t in _tensors(args)}
    for t in _tensors(out):
        if id(t) not in given:
            t.record_stream(mine)
    return out


def _tensors(x):
    if isinstance(x, torch.Tensor):
        yield x
    elif isinstance(x, (tuple, list, dict, Plan)):
        for y in x.values() if isinstance(x, dict) else vars(x).values() if isinstance(x, Plan) else x:
            yield from _tensors(y)


def _need_cuda(*ts):
    for t in ts:
        if t is None:
            continue
        if not t.is_cuda:
            raise SvooError("tensors must live on a CUDA device")
        if not t.is_contiguous():
            raise SvooError("tensors must be contiguous")


@dataclasses.dataclass
class Config:
    n_qc: int = 256
    n_kc: int = 256
    iters: int = 10
    block_q: int = 128
    select_mode: int = 0          # 0 keep ratio, 1 top-p
    merge_rounds: int = 2
    scale: Optional[float] = None  # default 1/sqrt(d)
    metric: int = 0               # 0 QK interaction (co-clustering), 1 identity (independent)


def make_shape(q: torch.Tensor, n_text: int = 0) -> Shape:
    if q.dim() != 4:
        raise SvooError("q/k/v must be [B, H, N, d]")
    B, H, N, d = q.shape
    return Shape(B, H, N, d, n_text)


class Plan:
    """Device buffers of one call's sparse plan (see svoo_plan in include/svoo.h)."""

    def __init__(self, shape: Shape, cfg: Config, device):
        counts = (ctypes.c_int64 * 12)()
        _check(load().svoo_plan_counts(ctypes.byref(shape), cfg.n_qc, cfg.n_kc, cfg.block_q, counts),
               "svoo_plan_counts")
        self.shape = shape
        self.cfg = cfg
        self.kmask = torch.zeros(counts[0], dtype=torch.int64, device=device)
        ints = {}
        for i, f in enumerate(_PLAN_FIELDS[1:], start=1):
            ints[f] = torch.zeros(counts[i], dtype=torch.int32, device=device)
        self.__dict__.update(ints)
        self._c = _CPlan(*[t.data_ptr() for t in [self.kmask] + [ints[f] for f in _PLAN_FIELDS[1:]]])

    @property
    def c(self):
        return ctypes.byref(self._c)

    @property
    def BH(self) -> int:
        return self.shape.B * self.shape.H

    @property
    def Gq(self) -> int:
        return self.cfg.n_qc + (1 if self.shape.n_text > 0 else 0)

    @property
    def Gk(self) -> int:
        return self.cfg.n_kc + (1 if self.shape.n_text > 0 else 0)

    @property
    def W(self) -> int:
        return (self.Gk + 63) // 64

    @property
    def tile_cap(self) -> int:
        return (self.shape.N + self.cfg.block_q - 1) // self.cfg.block_q + self.Gq

    @property
    def unit_cap(self) -> int:
        return (self.shape.N + 255) // 256 + self.Gq

    def views(self) -> dict:
        """Per-head views of the plan arrays (still on the device)."""
        BH, N = self.BH, self.shape.N
        return dict(
            kmask=self.kmask.view(BH, self.Gq, self.W),
            q_label=self.q_label.view(BH, N),
            q_sizes=self.q_sizes.view(BH, self.Gq),
            stats=self.stats.view(BH, 8),
            q_perm=self.q_perm.view(BH, N),
            q_off=self.q_off.view(BH, self.Gq + 1),
            k_perm=self.k_perm.view(BH, N),
            k_off=self.k_off.view(BH, self.Gk + 1),
            tiles=self.tiles.view(BH, self.tile_cap, 4),
            tile_count=self.tile_count.view(BH),
            units=self.units.view(BH, self.unit_cap, 4),
            unit_count=self.unit_count.view(BH),
        )


def workspace_sizes(shape: Shape, cfg: Config) -> tuple:
    L = load()
    c = L.svoo_cluster_workspace_size(ctypes.byref(shape), cfg.n_qc, cfg.n_kc)
    m = L.svoo_mask_workspace_size(ctypes.byref(shape), cfg.n_qc, cfg.n_kc)
    if c == 0 or m == 0:
        raise SvooError("unsupported shape or cluster counts")
    return int(c), int(m)


def _error_word(dev_err, device):
    """The caller's error word, which kernels write to through its address."""
    if not isinstance(dev_err, torch.Tensor) or dev_err.dtype is not torch.int32 or dev_err.device != device or \
            dev_err.numel() < 1:
        raise SvooError(f"dev_err must be an int32 tensor on {device}")
    return dev_err


def _err_buf(dev_err, device):
    return torch.zeros(1, dtype=torch.int32, device=device) if dev_err is None else _error_word(dev_err, device)


def check_device_errors(dev_err: torch.Tensor):
    """Raises if the device error word has bits set (synchronises the stream)."""
    v = int(dev_err.item())
    if v:
        names = {1: "attention wait timeout", 2: "clustering wait timeout", 4: "plan out of range",
                 8: "cluster label out of range"}
        raise SvooError("device error: " + ", ".join(n for b, n in names.items() if v & b))


CLUSTER_WARM = 1
CLUSTER_IDENTITY = 2


def _cluster_flags(cfg: Config, warm) -> int:
    if cfg.metric not in (0, 1):
        raise SvooError(f"Config.metric must be 0 (QK interaction) or 1 (identity), not {cfg.metric}")
    return (CLUSTER_WARM if warm is not None else 0) | (CLUSTER_IDENTITY if cfg.metric == 1 else 0)


_CLUSTER_OUT = ("q_assign", "k_assign", "q_cent", "k_cent", "q_sizes", "k_sizes")


def cluster_outputs(shape: Shape, cfg: Config, device) -> dict:
    """Device output buffers of `cluster` for a shape, to be reused across calls."""
    BH, nv, d = shape.B * shape.H, shape.N - shape.n_text, shape.d
    return dict(
        q_assign=torch.empty(BH, nv, dtype=torch.int32, device=device),
        k_assign=torch.empty(BH, nv, dtype=torch.int32, device=device),
        q_cent=torch.empty(BH, cfg.n_qc, d, dtype=torch.float32, device=device),
        k_cent=torch.empty(BH, cfg.n_kc, d, dtype=torch.float32, device=device),
        q_sizes=torch.zeros(BH, cfg.n_qc, dtype=torch.int32, device=device),
        k_sizes=torch.zeros(BH, cfg.n_kc, dtype=torch.int32, device=device),
    )


def cluster(q, k, cfg: Config, n_text=0, warm=None, workspace=None, dev_err=None, stream=None,
            out: Optional[dict] = None):
    """Co-clusters the video tokens of every head; returns a dict of device tensors.

    `out` (from cluster_outputs) is written in place instead of allocating new
    outputs. warm = (q_cent, k_cent, k_sizes) starts from those centroids
    (SVOO_CLUSTER_WARM); they may be out's own tensors (the previous call's
    result), in which case nothing is copied."""
    if stream is not None:
        return _under(stream, q.device, cluster, q, k, cfg, n_text, warm, workspace, dev_err, None, out)
    _need_cuda(q, k)
    sh = make_shape(q, n_text)
    dev = q.device
    if workspace is None:
        workspace = torch.empty(workspace_sizes(sh, cfg)[0], dtype=torch.uint8, device=dev)
    if out is None:
        out = cluster_outputs(sh, cfg, dev)
    else:
        missing = [f for f in _CLUSTER_OUT if f not in out]
        if missing:
            raise SvooError(f"cluster(out=...) lacks {missing}")
        _need_cuda(*(out[f] for f in _CLUSTER_OUT))
    if warm is not None:
        for dst, src in zip(("q_cent", "k_cent", "k_sizes"), warm):
            if out[dst].data_ptr() != src.data_ptr():
                out[dst].copy_(src)
    err = _err_buf(dev_err, dev)
    _check(load().svoo_cluster(ctypes.byref(sh), _ptr(q), _ptr(k), cfg.n_qc, cfg.n_kc, cfg.iters,
                               _cluster_flags(cfg, warm), _ptr(out["q_assign"]), _ptr(out["k_assign"]),
                               _ptr(out["q_cent"]), _ptr(out["k_cent"]), _ptr(out["q_sizes"]),
                               _ptr(out["k_sizes"]), _ptr(workspace), workspace.numel(), _ptr(err),
                               _stream()), "svoo_cluster")
    out["dev_err"] = err
    return out


def cluster_step(x, cent, sizes, assign, metric_cent=None, metric_sizes=None, n_text=0,
                 workspace=None, dev_err=None, stream=None):
    """One assignment + update half-step (cent, sizes, assign are updated in place)."""
    if stream is not None:
        return _under(stream, x.device, cluster_step, x, cent, sizes, assign, metric_cent, metric_sizes, n_text,
                      workspace, dev_err)
    _need_cuda(x, cent, sizes, assign, metric_cent, metric_sizes)
    sh = make_shape(x, n_text)
    C = cent.shape[-2]
    mC = metric_cent.shape[-2] if metric_cent is not None else 0
    cfg = Config(n_qc=max(C, mC, 1), n_kc=max(C, mC, 1))
    if workspace is None:
        workspace = torch.empty(workspace_sizes(sh, cfg)[0], dtype=torch.uint8, device=x.device)
    err = _err_buf(dev_err, x.device)
    _check(load().svoo_cluster_step(ctypes.byref(sh), _ptr(x), C, _ptr(cent), _ptr(sizes),
                                    _ptr(assign), _ptr(metric_cent), _ptr(metric_sizes), mC,
                                    _ptr(workspace), workspace.numel(), _ptr(err), _stream()),
           "svoo_cluster_step")
    return err


def cluster_step_static(x, cent, sizes, assign, metric_cent=None, metric_sizes=None, n_text=0,
                        dev_err=None, stream=None):
    """cluster_step with the library's fixed device scratch instead of a
    workspace (for callers that may not allocate device memory)."""
    if stream is not None:
        return _under(stream, x.device, cluster_step_static, x, cent, sizes, assign, metric_cent, metric_sizes,
                      n_text, dev_err)
    _need_cuda(x, cent, sizes, assign, metric_cent, metric_sizes)
    sh = make_shape(x, n_text)
    C = cent.shape[-2]
    mC = metric_cent.shape[-2] if metric_cent is not None else 0
    err = _err_buf(dev_err, x.device)
    _check(load().svoo_cluster_step_static(ctypes.byref(sh), _ptr(x), C, _ptr(cent), _ptr(sizes),
                                           _ptr(assign), _ptr(metric_cent), _ptr(metric_sizes), mC,
                                           _ptr(err), _stream()), "svoo_cluster_step_static")
    return err


def build_mask(shape: Shape, cl: dict, keep: torch.Tensor, cfg: Config, plan: Optional[Plan] = None,
               workspace=None, dev_err=None, stream=None) -> Plan:
    """Pair masses, keep-ratio / top-p selection and tail merging into `plan`."""
    if stream is not None:
        return _under(stream, cl["q_cent"].device, build_mask, shape, cl, keep, cfg, plan, workspace, dev_err)
    dev = cl["q_cent"].device
    keep = keep.to(device=dev, dtype=torch.float32).contiguous()
    _need_cuda(keep, cl["q_cent"], cl["k_cent"], cl["q_sizes"], cl["k_sizes"], cl["q_assign"])
    if plan is None:
        plan = Plan(shape, cfg, dev)
    if workspace is None:
        workspace = torch.empty(workspace_sizes(shape, cfg)[1], dtype=torch.uint8, device=dev)
    scale = cfg.scale if cfg.scale is not None else 1.0 / math.sqrt(shape.d)
    err = _err_buf(dev_err, dev)
    _check(load().svoo_build_mask(ctypes.byref(shape), _ptr(cl["q_cent"]), _ptr(cl["k_cent"]),
                                  _ptr(cl["q_sizes"]), _ptr(cl["k_sizes"]), _ptr(cl["q_assign"]),
                                  _ptr(keep), cfg.n_qc, cfg.n_kc, cfg.select_mode, cfg.block_q,
                                  cfg.merge_rounds, scale, plan.c, _ptr(workspace),
                                  workspace.numel(), _ptr(err), _stream()), "svoo_build_mask")
    return plan


def permute(q, k, v, k_assign, plan: Plan, qp=None, kp=None, vp=None, dev_err=None, stream=None):
    """Cluster-order permutation, query tiles and gathered copies (qp, kp, vp)."""
    if stream is not None:
        return _under(stream, q.device, permute, q, k, v, k_assign, plan, qp, kp, vp, dev_err)
    _need_cuda(q, k, v, k_assign)
    qp = torch.empty_like(q) if qp is None else qp
    kp = torch.empty_like(k) if kp is None else kp
    vp = torch.empty_like(v) if vp is None else vp
    err = _err_buf(dev_err, q.device)
    cfg = plan.cfg
    _check(load().svoo_permute(ctypes.byref(plan.shape), _ptr(q), _ptr(k), _ptr(v), _ptr(k_assign),
                               cfg.n_qc, cfg.n_kc, cfg.block_q, plan.c, _ptr(qp), _ptr(kp), _ptr(vp),
                               _ptr(err), _stream()), "svoo_permute")
    return qp, kp, vp


def sparse_attn(qp, kp, vp, plan: Plan, out=None, dev_err=None, stream=None):
    """Block-sparse attention over the plan's kept tiles; returns O in token order."""
    if stream is not None:
        return _under(stream, qp.device, sparse_attn, qp, kp, vp, plan, out, dev_err)
    _need_cuda(qp, kp, vp)
    out = torch.empty_like(qp) if out is None else out
    cfg = plan.cfg
    scale = cfg.scale if cfg.scale is not None else 1.0 / math.sqrt(plan.shape.d)
    err = _err_buf(dev_err, qp.device)
    _check(load().svoo_sparse_attn(ctypes.byref(plan.shape), _ptr(qp), _ptr(kp), _ptr(vp), plan.c,
                                   cfg.n_qc, cfg.n_kc, cfg.block_q, scale, _ptr(out), _ptr(err),
                                   _stream()), "svoo_sparse_attn")
    return out


def sparse_attention(q, k, v, keep, cfg: Config, n_text=0, dev_err=None, stream=None):
    """The whole path: cluster -> mask + tail merge -> permute -> sparse attention."""
    if stream is not None:
        return _under(stream, q.device, sparse_attention, q, k, v, keep, cfg, n_text, dev_err)
    sh = make_shape(q, n_text)
    err = _err_buf(dev_err, q.device)
    cl = cluster(q, k, cfg, n_text=n_text, dev_err=err)
    plan = build_mask(sh, cl, keep, cfg, dev_err=err)
    qp, kp, vp = permute(q, k, v, cl["k_assign"], plan, dev_err=err)
    out = sparse_attn(qp, kp, vp, plan, dev_err=err)
    return out, dict(cl=cl, plan=plan, dev_err=err)


# --------------------------------------------------------------------------- static stripe mask

PSA_INF = 2 ** 31 - 1   # SVOO_PSA_INF: infinite stride, one diagonal band on that axis


def psa_params(per_head, device) -> torch.Tensor:
    """int32 [B*H, 6] device tensor from per-head (Tw, To, Ts, Sw, So, Ss) tuples;
    None or math.inf for an infinite stride."""
    rows = []
    for prm in per_head:
        if len(prm) != 6:
            raise SvooError("a PSA mask has six parameters (Tw, To, Ts, Sw, So, Ss)")
        rows.append([PSA_INF if (i in (2, 5) and (v is None or v == math.inf)) else int(v)
                     for i, v in enumerate(prm)])
    return torch.tensor(rows, dtype=torch.int32).to(device)


def psa_config(grid, block, block_q: int = 128, scale: Optional[float] = None) -> Config:
    """The Config of a stripe-mask plan: one group per PSABlock on each side."""
    nb = load().svoo_psa_block_count(*grid, *block)
    if nb < 1 or nb > 256:
        raise SvooError(f"PSABlock grid of {grid} by {block} has {nb} blocks (1..256 supported)")
    return Config(n_qc=nb, n_kc=nb, iters=1, block_q=block_q, scale=scale)


def psa_mask(shape: Shape, grid, block, params: torch.Tensor, cfg: Config,
             plan: Optional[Plan] = None, k_assign: Optional[torch.Tensor] = None, dev_err=None,
             stream=None):
    """Plan of the PSA stripe mask (svoo_psa_mask): returns (plan, k_assign)."""
    if stream is not None:
        return _under(stream, params.device, psa_mask, shape, grid, block, params, cfg, plan, k_assign, dev_err)
    _need_cuda(params)
    dev = params.device
    BH, nv = shape.B * shape.H, shape.N - shape.n_text
    if tuple(params.shape) != (BH, 6) or params.dtype != torch.int32 or not params.is_contiguous():
        raise SvooError("params must be a contiguous int32 [B*H, 6] tensor")
    if plan is None:
        plan = Plan(shape, cfg, dev)
    if k_assign is None:
        k_assign = torch.empty(BH, nv, dtype=torch.int32, device=dev)
    err = _err_buf(dev_err, dev)
    _check(load().svoo_psa_mask(ctypes.byref(shape), *grid, *block, _ptr(params), cfg.block_q, plan.c,
                                _ptr(k_assign), _ptr(err), _stream()), "svoo_psa_mask")
    return plan, k_assign


def psa_attention(q, k, v, grid, block, params: torch.Tensor, n_text=0, block_q: int = 128,
                  scale: Optional[float] = None, dev_err=None, stream=None):
    """The stripe-mask path: PSA plan -> permute -> sparse attention."""
    if stream is not None:
        return _under(stream, q.device, psa_attention, q, k, v, grid, block, params, n_text, block_q, scale,
                      dev_err)
    sh = make_shape(q, n_text)
    cfg = psa_config(grid, block, block_q, scale)
    err = _err_buf(dev_err, q.device)
    plan, k_assign = psa_mask(sh, grid, block, params, cfg, dev_err=err)
    qp, kp, vp = permute(q, k, v, k_assign, plan, dev_err=err)
    out = sparse_attn(qp, kp, vp, plan, dev_err=err)
    return out, dict(plan=plan, k_assign=k_assign, dev_err=err, cfg=cfg)


# --------------------------------------------------------------------------- SNR-guided top-p


def snr_top_p(steps: int, warmup: int = 0, p_min: float = 0.7, tau: float = 0.999,
              shift: float = 1.0):
    """Top-p of each of `steps` denoising calls (svoo_snr_top_p), as a float32
    numpy array; feed p[t] to build_mask with Config(select_mode=1)."""
    import numpy as np
    p = np.empty(int(steps), dtype=np.float32)
    _check(load().svoo_snr_top_p(int(steps), int(warmup), float(p_min), float(tau), float(shift),
                                 p.ctypes.data_as(ctypes.c_void_p)), "svoo_snr_top_p")
    return p


# --------------------------------------------------------------------------- block-selected attention


@dataclasses.dataclass
class BlockConfig:
    """How every query selects its key blocks (see svoo_block_shape in include/svoo.h)."""
    block: int = 64                # keys per block: a multiple of 64 up to 1024
    n_sel: int = 16                # blocks per query, forced ones included
    sink: int = 1                  # the first blocks, kept by every query
    local: int = 1                 # causal: the query's own block and the local - 1 before it
    causal: bool = True            # when False, local must be 0
    scale: Optional[float] = None  # default 1/sqrt(d)


# The calls below serve single tokens, where the host's own work counts: shapes and
# workspace sizes are looked up by their numbers, pointers go to ctypes as integers.


@functools.lru_cache(maxsize=1024)
def _bshape(*fields) -> "ctypes.Array":
    """BlockShape of its thirteen fields, as the pointer that the C calls take."""
    return ctypes.pointer(BlockShape(*fields))


def _dp(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def _err_at(dev_err, device):
    return None if dev_err is None else _error_word(dev_err, device).data_ptr()


def _call(what: str, t: torch.Tensor, *args):
    """Calls a C entry point with t's device current, on that device's current stream."""
    fn = getattr(_lib if _lib is not None else load(), what)
    dev = t.device.index
    st = torch._C._cuda_getCurrentRawStream(dev)
    if dev == torch._C._cuda_getDevice():
        status = fn(*args, st)
    else:
        with torch.cuda.device(dev):
            status = fn(*args, st)
    if status:
        _check(status, what)


def _written(*ts: torch.Tensor):
    """Tells autograd that the caller's tensors were written in place, so that a backward pass that had saved
    one of them says so instead of using what it holds now."""
    torch._C._increment_version(ts)    # (of torch.autograd.graph, without its look at the type)


def _need(what: str, dtype, device, shape, t: Optional[torch.Tensor]):
    """A dense tensor of that type, device and shape, or None."""
    if t is None or (t.dtype is dtype and t.shape == shape and t.device == device and t.is_contiguous()):
        return
    if not t.is_cuda:
        raise SvooError(f"{what} must live on a CUDA device")
    if t.dtype != dtype or t.device != device:
        raise SvooError(f"{what} must be {dtype} on {device}, not {t.dtype} on {t.device}")
    if tuple(t.shape) != tuple(shape):
        raise SvooError(f"{what} must have shape {tuple(shape)}, not {tuple(t.shape)}")
    raise SvooError(f"{what} must be contiguous")


def _queries(q: torch.Tensor):
    if q.dim() != 4 or q.dtype is not torch.bfloat16 or not q.is_cuda:
        raise SvooError("q must be a bf16 [B, H, N, d] tensor on a CUDA device")
    if not q.is_contiguous():
        raise SvooError("q must be contiguous")
    return q.shape


def _key_rows(what: str, t: torch.Tensor, device) -> int:
    """Rows from one head to the next of a bf16 [B, Hkv, Nk, d] tensor: contiguous, or the same Nk
    rows of every head of a longer contiguous buffer."""
    if t.dim() != 4 or t.dtype is not torch.bfloat16 or t.device != device or not t.is_cuda:
        raise SvooError(f"{what} must be a bf16 [B, Hkv, N, d] tensor on {device}")
    B, Hkv, Nk, d = t.shape
    if t.is_contiguous():
        return Nk
    s0, s1, s2, s3 = t.stride()
    cap = s1 // d if Hkv > 1 else s0 // (Hkv * d)
    if s3 != 1 or (s2 != d and Nk > 1) or cap < Nk or (Hkv > 1 and s1 != cap * d) or \
            (B > 1 and s0 != Hkv * cap * d):
        raise SvooError(f"{what} must be contiguous or the same rows of every head of a contiguous buffer")
    return cap


def _first_position(q_start: Optional[int], n_keys: int, Nq: int, causal) -> int:
    """q_start of a BlockShape: None is the last Nq of n_keys. (-1 means the last Nq of every sequence's own
    length there, so a position before the first is never passed on.) Without causality positions mean nothing."""
    if q_start is not None:
        return q_start
    if not causal:
        return 0
    if Nq > n_keys:
        raise SvooError(f"{Nq} queries cannot be the last of {n_keys} keys: pass q_start")
    return n_keys - Nq


def _block_args(q, k, v, cfg: BlockConfig, lengths, q_start):
    """The fields of a call's BlockShape, after checking its tensors."""
    B, H, Nq, d = _queries(q)
    dev = q.device
    cap = _key_rows("k", k, dev)
    if v.shape != k.shape or _key_rows("v", v, dev) != cap:
        raise SvooError("k and v must have the same shape and strides")
    Bk, Hkv, Nk, dk = k.shape
    if Bk != B or dk != d:
        raise SvooError("q, k and v must agree in batch and head dimension")
    _need("lengths", torch.int32, dev, (B,), lengths)
    return (B, H, Hkv, Nq, Nk, cap, d, cfg.block, cfg.n_sel, cfg.sink, cfg.local, 1 if cfg.causal else 0,
            _first_position(q_start, Nk, Nq, cfg.causal))


@functools.lru_cache(maxsize=1024)
def _ws_bytes(what: str, *args) -> int:
    """Bytes of a call's workspace (0 where the C side refuses the shape, as the call then does)."""
    fn = getattr(load(), what)
    if what == "svoo_cache_evict_workspace_size":
        return fn(*args)
    return fn(_bshape(*args[:13]), *args[13:])


def _workspace(workspace, device, what: str, *args):
    """(tensor to keep alive, address, bytes) of a call's workspace."""
    if workspace is None:
        n = _ws_bytes(what, *args)
        if n == 0:
            return None, None, 0
        workspace = torch.empty(n, dtype=torch.uint8, device=device)
        return workspace, workspace.data_ptr(), n
    if not workspace.is_cuda or workspace.device != device or not workspace.is_contiguous():
        raise SvooError(f"workspace must be a contiguous tensor on {device}")
    return workspace, workspace.data_ptr(), workspace.numel() * workspace.element_size()


def _block_scale(cfg: Optional[BlockConfig], d: int) -> float:
    return cfg.scale if cfg is not None and cfg.scale is not None else 1.0 / math.sqrt(d)


def block_pool(k, cfg: BlockConfig, lengths=None, pool=None, last: int = 0, stream=None) -> torch.Tensor:
    """Mean of the valid keys of every block of cfg.block keys: fp32 [B, Hkv, blocks, d].

    `pool` is written in place instead of a new tensor; with last > 0 only the last `last` blocks that
    hold keys of each sequence are renewed (after a token was appended, last=1)."""
    if stream is not None:
        return _under(stream, k.device, block_pool, k, cfg, lengths, pool, last)
    if k.dim() != 4 or not k.is_cuda:
        raise SvooError("k must be a bf16 [B, Hkv, N, d] tensor on a CUDA device")
    dev = k.device
    cap = _key_rows("k", k, dev)
    B, Hkv, Nk, d = k.shape
    nb = -(-Nk // cfg.block) if cfg.block > 0 else 0
    _need("lengths", torch.int32, dev, (B,), lengths)
    given = pool
    if pool is None:
        if last:
            raise SvooError("last renews blocks of an existing pool: pass it")
        pool = torch.empty(B, Hkv, nb, d, dtype=torch.float32, device=dev)
    else:
        _need("pool", torch.float32, dev, (B, Hkv, nb, d), pool)
    _call("svoo_block_pool", k, _bshape(B, Hkv, Hkv, 1, Nk, cap, d, cfg.block, 1, 0, 0, 0, 0),
          k.data_ptr(), _dp(lengths), last, pool.data_ptr())
    if given is not None:
        _written(given)
    return pool


def block_select(q, pool, cfg: BlockConfig, n_keys: int, lengths=None, q_start: Optional[int] = None,
                 idx=None, workspace=None, dev_err=None, stream=None) -> torch.Tensor:
    """The blocks that every query selects: int32 [B, Hkv, Nq, n_sel], ascending, -1 behind them.

    n_keys: key rows per head (an upper bound of lengths). q_start: position of query 0; None: the
    queries are the last Nq of n_keys (which cannot be fewer); -1: the last Nq of each sequence's
    lengths, of which a longer Nq has some before the first token: those select nothing. Not causal:
    positions mean nothing, and there may be more queries than keys."""
    if stream is not None:
        return _under(stream, q.device, block_select, q, pool, cfg, n_keys, lengths, q_start, idx, workspace, dev_err)
    B, H, Nq, d = _queries(q)
    dev = q.device
    nb = -(-n_keys // cfg.block) if cfg.block > 0 else 0
    Hkv = pool.shape[1] if pool.dim() == 4 else 0
    _need("pool", torch.float32, dev, (B, Hkv, nb, d), pool)
    _need("lengths", torch.int32, dev, (B,), lengths)
    given = idx
    if idx is None:
        idx = torch.empty(B, Hkv, Nq, max(cfg.n_sel, 0), dtype=torch.int32, device=dev)
    else:
        _need("idx", torch.int32, dev, (B, Hkv, Nq, cfg.n_sel), idx)
    args = (B, H, Hkv, Nq, n_keys, n_keys, d, cfg.block, cfg.n_sel, cfg.sink, cfg.local, 1 if cfg.causal else 0,
            _first_position(q_start, n_keys, Nq, cfg.causal))
    ws, ws_at, ws_n = _workspace(workspace, dev, "svoo_block_select_workspace_size", *args)
    _call("svoo_block_select", q, _bshape(*args), q.data_ptr(), pool.data_ptr(), _dp(lengths),
          idx.data_ptr(), ws_at, ws_n, _err_at(dev_err, dev))
    if given is not None:
        _written(given)
    return idx


def block_attn(q, k, v, idx, cfg: BlockConfig, lengths=None, q_start: Optional[int] = None, out=None,
               workspace=None, dev_err=None, stream=None):
    """Attention of every query over the blocks in idx; returns (o, lse). No gradient is recorded
    (block_attention records one)."""
    if stream is not None:
        return _under(stream, q.device, block_attn, q, k, v, idx, cfg, lengths, q_start, out, workspace, dev_err)
    args = _block_args(q, k, v, cfg, lengths, q_start)
    B, H, Hkv, Nq, _, _, d = args[:7]
    dev = q.device
    _need("idx", torch.int32, dev, (B, Hkv, Nq, cfg.n_sel), idx)
    _need("out", torch.bfloat16, dev, q.shape, out)
    return _run_attn(args, _block_scale(cfg, d), q, k, v, idx, lengths, out, workspace, dev_err)


def _run_attn(args, scale, q, k, v, idx, lengths, out, workspace, dev_err):
    dev, given = q.device, out
    out = torch.empty_like(q) if out is None else out
    lse = torch.empty(args[0], args[1], args[3], dtype=torch.float32, device=dev)
    ws, ws_at, ws_n = _workspace(workspace, dev, "svoo_block_attn_workspace_size", *args)
    _call("svoo_block_attn", q, _bshape(*args), q.data_ptr(), k.data_ptr(), v.data_ptr(), idx.data_ptr(),
          _dp(lengths), scale, out.data_ptr(), lse.data_ptr(), ws_at, ws_n, _err_at(dev_err, dev))
    if given is not None:
        _written(given)
    return out, lse


def block_attn_backward(q, k, v, o, lse, grad_o, idx, cfg: BlockConfig, lengths=None,
                        q_start: Optional[int] = None, workspace=None, dev_err=None, stream=None):
    """Gradient of block_attn: (dq, dk, dv), with idx, o and lse as block_attn had or gave them."""
    if stream is not None:
        return _under(stream, q.device, block_attn_backward, q, k, v, o, lse, grad_o, idx, cfg, lengths, q_start,
                      workspace, dev_err)
    args = _block_args(q, k, v, cfg, lengths, q_start)
    B, H, Hkv, Nq, _, _, d = args[:7]
    dev = q.device
    _need("idx", torch.int32, dev, (B, Hkv, Nq, cfg.n_sel), idx)
    _need("o", torch.bfloat16, dev, q.shape, o)
    _need("grad_o", torch.bfloat16, dev, q.shape, grad_o)
    _need("lse", torch.float32, dev, (B, H, Nq), lse)
    return _run_attn_backward(args, _block_scale(cfg, d), q, k, v, o, lse, grad_o, idx, lengths, workspace, dev_err)


def _run_attn_backward(args, scale, q, k, v, o, lse, grad_o, idx, lengths, workspace, dev_err):
    dev = q.device
    ws, ws_at, ws_n = _workspace(workspace, dev, "svoo_block_attn_backward_workspace_size", *args)
    dq = torch.empty_like(q)
    dk = torch.empty(k.shape, dtype=k.dtype, device=dev)
    dv = torch.empty(v.shape, dtype=v.dtype, device=dev)
    _call("svoo_block_attn_backward", q, _bshape(*args), q.data_ptr(), k.data_ptr(), v.data_ptr(),
          o.data_ptr(), lse.data_ptr(), grad_o.data_ptr(), idx.data_ptr(), _dp(lengths), scale,
          dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), ws_at, ws_n, _err_at(dev_err, dev))
    return dq, dk, dv


class _BlockAttn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, idx, args, scale, lengths, dev_err):
        o, lse = _run_attn(args, scale, q, k, v, idx, lengths, None, None, dev_err)
        ctx.save_for_backward(q, k, v, idx, lengths, o, lse)
        ctx.args = (args, scale, dev_err)    # an error word may be cleared between the two passes
        ctx.mark_non_differentiable(lse)
        ctx.set_materialize_grads(False)    # no zeros for lse
        return o, lse

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, grad_o, _):
        if grad_o is None:
            return (None,) * 8
        q, k, v, idx, lengths, o, lse = ctx.saved_tensors
        args, scale, dev_err = ctx.args
        _need("the incoming gradient", torch.bfloat16, q.device, q.shape, grad_o := grad_o.contiguous())
        dq, dk, dv = _run_attn_backward(args, scale, q, k, v, o, lse, grad_o, idx, lengths, None, dev_err)
        return dq, dk, dv, None, None, None, None, None


def _has_tangent(*ts) -> bool:
    """Whether forward-mode differentiation is under way and one of the tensors takes part."""
    ad = torch.autograd.forward_ad
    return ad._current_level >= 0 and any(ad.unpack_dual(t).tangent is not None for t in ts)


def block_attention(q, k, v, cfg: BlockConfig, lengths=None, q_start: Optional[int] = None, dev_err=None):
    """The whole path on the current stream: block means -> selection -> attention over the selected
    blocks. q: bf16 [B, H, Nq, d]; k, v: bf16 [B, Hkv, Nk, d]; lengths: int32 [B], the valid keys of a
    right-padded batch; q_start as in block_select. Differentiable in q, k and v (the selection is a
    constant of the gradient; the gradient's gradient and forward-mode gradients are not offered). fp32
    softmax and sums; P and dS in bf16 for the second products (svoo_block_attn_backward says which).
    Where neighbouring queries select nearly all blocks, blocks of 128 keys and multiples, a call takes
    a workspace of 4 * (d + 2) bytes for every query's 128 selected keys, up to 4.5 GB.
    Returns (o, dict(idx, lse, pool, dev_err))."""
    if _has_tangent(q, k, v):
        raise SvooError("block_attention has no forward-mode gradient")
    args = _block_args(q, k, v, cfg, lengths, q_start)
    scale = _block_scale(cfg, args[6])
    err = _err_buf(dev_err, q.device)
    pool = block_pool(k, cfg, lengths)
    idx = block_select(q, pool, cfg, args[4], lengths, q_start, dev_err=err)
    if torch.is_grad_enabled() and (q.requires_grad or k.requires_grad or v.requires_grad):
        o, lse = _BlockAttn.apply(q, k, v, idx, args, scale, lengths, err)
    else:
        o, lse = _run_attn(args, scale, q, k, v, idx, lengths, None, None, err)
    return o, dict(idx=idx, lse=lse, pool=pool, dev_err=err)


# --------------------------------------------------------------------------- single tokens over a cache


def cache_attn(q, k, v, lengths=None, idx=None, cfg: Optional[BlockConfig] = None, weight=None, out=None,
               workspace=None, dev_err=None, stream=None):
    """Attention of one token per sequence, q bf16 [B, H, 1, d], over the first lengths[b] slots of a
    cache, k and v bf16 [B, Hkv, cap, d]; returns (o, lse). No gradient is recorded.

    idx (from block_select, with its cfg): only the slots of the selected blocks. weight (fp32
    [B, Hkv, cap]): every valid slot's softmax weight, summed over the group's heads, is added to it."""
    if stream is not None:
        return _under(stream, q.device, cache_attn, q, k, v, lengths, idx, cfg, weight, out, workspace, dev_err)
    if q.dim() != 4 or q.shape[2] != 1:
        raise SvooError("q must be [B, H, 1, d]: one token per sequence")
    if idx is not None and cfg is None:
        raise SvooError("idx needs the BlockConfig that it was selected with")
    if idx is not None and weight is not None:
        raise SvooError("weights are summed over whole caches only: idx and weight exclude each other")
    args = _block_args(q, k, v, cfg if idx is not None else _WHOLE, lengths, 0)
    B, H, Hkv, _, Nk, cap, d = args[:7]
    dev = q.device
    if idx is not None:
        _need("idx", torch.int32, dev, (B, Hkv, 1, cfg.n_sel), idx)
    if weight is not None:
        if cap != Nk:
            raise SvooError("weights need k and v as whole buffers")
        _need("weight", torch.float32, dev, (B, Hkv, Nk), weight)
    _need("out", torch.bfloat16, dev, q.shape, out)
    ws, ws_at, ws_n = _workspace(workspace, dev, "svoo_cache_attn_workspace_size", *args, idx is not None, weight is not None)
    given = out
    out = torch.empty_like(q) if out is None else out
    lse = torch.empty(B, H, 1, dtype=torch.float32, device=dev)
    _call("svoo_cache_attn", q, _bshape(*args), q.data_ptr(), k.data_ptr(), v.data_ptr(), _dp(lengths),
          _dp(idx), _block_scale(cfg, d), _dp(weight), out.data_ptr(), lse.data_ptr(), ws_at, ws_n,
          _err_at(dev_err, dev))
    if given is not None:
        _written(given)
    if weight is not None:
        _written(weight)
    return out, lse


_WHOLE = BlockConfig()  # of a call without a selection


def cache_evict(k, v, weight, pos, lengths, keep: int, sink: int = 0, recent: int = 0, workspace=None,
                stream=None):
    """Brings every sequence of a cache with more than `keep` slots down to `keep`, in place (k, v, weight,
    pos and lengths; see svoo_cache_evict): the first `sink` and last `recent` positions stay, then the
    heaviest slots of each key head. Block means of the cache are to be made anew afterwards."""
    if stream is not None:
        return _under(stream, k.device, cache_evict, k, v, weight, pos, lengths, keep, sink, recent, workspace)
    if k.dim() != 4 or not k.is_cuda:
        raise SvooError("k must be a bf16 [B, Hkv, cap, d] tensor on a CUDA device")
    B, Hkv, cap, d = k.shape
    dev = k.device
    for what, t in (("k", k), ("v", v)):
        _need(what, torch.bfloat16, dev, (B, Hkv, cap, d), t)
    for what, t, dtype in (("weight", weight, torch.float32), ("pos", pos, torch.int32)):
        _need(what, dtype, dev, (B, Hkv, cap), t)
    _need("lengths", torch.int32, dev, (B,), lengths)
    ws, ws_at, ws_n = _workspace(workspace, dev, "svoo_cache_evict_workspace_size", B, Hkv, cap, keep)
    _call("svoo_cache_evict", k, B, Hkv, cap, d, keep, sink, recent, k.data_ptr(), v.data_ptr(),
          weight.data_ptr(), pos.data_ptr(), lengths.data_ptr(), ws_at, ws_n)
    _written(k, v, weight, pos, lengths)

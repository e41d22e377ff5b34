"""RIB windowed attention on B200 (sm_100a): Python binding of librib.so.

Every function here has the name of a C entry point of include/rib.h and only
marshals arguments: it checks devices / dtypes / contiguity, allocates
missing outputs with torch (PyTorch is the device-memory and stream
provider), passes raw pointers and the current CUDA stream, and raises
RibError on a non-zero status.  All arithmetic runs in the library's CUDA
kernels; there is no CPU or PyTorch fallback.

"Rank-Factorized Implicit Neural Bias: Scaling Super-Resolution Transformer
with FlashAttention" (arXiv 2603.06738): position tokens from a Fourier-
feature MLP on window coordinates are concatenated with the content tokens so
that the positional bias Qp Kp^T comes out of the attention dot product.
"""
from __future__ import annotations

import ctypes
from dataclasses import dataclass
from typing import Dict, Optional, Tuple

import torch

from . import _abi

try:   # the current stream's handle without a Stream object around it
    from torch._C import _cuda_getCurrentRawStream as _raw_stream
except ImportError:   # pragma: no cover - a torch build without it
    def _raw_stream(index):
        return torch.cuda.current_stream(index).cuda_stream

__all__ = [
    "RibError", "PositionMLP", "PositionMLPGrad", "PosTokenCache", "rib_pos_tokens",
    "rib_pos_tokens_bwd", "rib_pos_tokens_bwd_workspace", "rib_pos_tokens_bwd_noalloc",
    "rib_window_attn_fwd", "rib_window_attn_fwd_tf32", "rib_window_attn_bwd",
    "rib_window_attn_bwd_workspace",
    "rib_window_gather", "rib_window_scatter", "rib_last_status", "rib_status_string",
    "rib_set_wait_limit_ns", "rib_set_bwd_kernel", "rib_bwd_kernel_for", "rib_debug_wait_timeout", "rib_version", "library",
    "rib_trace_enable", "rib_trace_collect", "rib_debug_exp2", "ClaGate", "rib_cla_gate",
    "rib_window_attn_fwd_cla", "rib_cla_bwd", "rib_cla_bwd_workspace",
    "rib_layer_norm_fwd", "rib_layer_norm_bwd", "rib_layer_norm_bwd_workspace",
    "rib_linear_fwd", "rib_linear_bwd", "rib_linear_bwd_workspace",
    "GatedFfn", "rib_gated_ffn_fwd", "rib_gated_ffn_fwd_workspace",
    "rib_gated_ffn_bwd", "rib_gated_ffn_bwd_workspace",
]


class RibError(RuntimeError):
    def __init__(self, code: int, where: str):
        self.code = code
        super().__init__(f"{where}: {rib_status_string(code)} ({code})")


# Entry points that enqueue GPU work get an NVTX range named after them, so a
# profiler's timeline (ncu --nvtx, Nsight Systems) shows which call launched
# which kernels.  Without a tool attached a range costs well under a
# microsecond; where torch has no NVTX support the ranges are left out.
_NO_RANGE = ("_workspace", "rib_status_string", "rib_last_status", "rib_version",
             "rib_set_wait_limit_ns", "rib_trace_enable", "rib_trace_collect")


def _nvtx_calls():
    try:
        torch.cuda.nvtx.range_push("rib")
        torch.cuda.nvtx.range_pop()
        return torch.cuda.nvtx.range_push, torch.cuda.nvtx.range_pop
    except Exception:  # pragma: no cover - a torch build without NVTX
        return None


class _RangedLibrary:
    """librib.so with every work-enqueuing entry point wrapped in an NVTX
    range; other attributes are the ctypes library's own."""

    def __init__(self, cdll: ctypes.CDLL):
        self._cdll = cdll
        calls = _nvtx_calls()
        for name in _abi._SIGS:
            fn = getattr(cdll, name)
            if calls is not None and not any(t in name for t in _NO_RANGE):
                fn = self._ranged(name, fn, *calls)
            setattr(self, name, fn)

    @staticmethod
    def _ranged(name, fn, push, pop):
        def call(*args):
            push(name)
            try:
                return fn(*args)
            finally:
                pop()
        call.__name__ = name
        return call

    def __getattr__(self, name):
        return getattr(self._cdll, name)


_ranged_lib: Optional[_RangedLibrary] = None


def library() -> _RangedLibrary:
    """The loaded librib.so (raises if it is missing)."""
    global _ranged_lib
    if _ranged_lib is None:
        _ranged_lib = _RangedLibrary(_abi.load())
    return _ranged_lib


def _check(code: int, where: str) -> None:
    if code != _abi.RIB_OK:
        raise RibError(code, where)


def _stream(stream) -> ctypes.c_void_p:
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))


def _ptr(t: Optional[torch.Tensor], dtype=None, name="tensor") -> Optional[int]:
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    return t.data_ptr()


def _sizes(where: str, dev, **buffers) -> None:
    """Buffers handed to the library must hold exactly the elements the call
    reads or writes, on the device of the call's other tensors: the library
    takes bare pointers and can check neither.  buffers: name=(tensor or
    None, element count).  The library launches on the current CUDA device,
    so the call's tensors must live there (torch.cuda.set_device)."""
    if dev is not None and dev.type == "cuda" and dev.index != torch.cuda.current_device():
        raise RibError(_abi.RIB_ERR_ARG, f"{where}: tensors are on {dev}, the current device "
                       f"is cuda:{torch.cuda.current_device()}")
    for name, (t, n) in buffers.items():
        if t is None:
            continue
        if t.numel() != n:
            raise RibError(_abi.RIB_ERR_ARG,
                           f"{where}: {name} holds {t.numel()} elements, the call needs {n}")
        if t.device != dev:
            raise RibError(_abi.RIB_ERR_ARG, f"{where}: {name} is on {t.device}, not {dev}")


def _grad_sizes(dmlp: Optional["PositionMLPGrad"], mlp: Optional["PositionMLP"]):
    """Each position-MLP gradient sized like its weight."""
    if dmlp is None or mlp is None:
        return {}
    return {f"dmlp.{n}": (getattr(dmlp, n), getattr(mlp, n[:2] + n[3:]).numel())
            for n in ("q_dw1", "q_db1", "q_dw2", "q_db2", "k_dw1", "k_db1", "k_dw2", "k_db2")}


def _cla_sizes(cla: "ClaGate", C: int):
    return {"w_dw": (cla.w_dw, 9 * C), "b_dw": (cla.b_dw, C), "w_pw": (cla.w_pw, C * C),
            "b_pw": (cla.b_pw, C)}


def rib_status_string(code: int) -> str:
    return library().rib_status_string(int(code)).decode()


def rib_version() -> str:
    return library().rib_version().decode()


# ---------------------------------------------------------------- MLP weights

@dataclass
class PositionMLP:
    """Device fp32 weights of the two position MLPs (Linear layout [out][in])."""
    freqs: torch.Tensor
    q_w1: torch.Tensor
    q_b1: torch.Tensor
    q_w2: torch.Tensor
    q_b2: torch.Tensor
    k_w1: torch.Tensor
    k_b1: torch.Tensor
    k_w2: torch.Tensor
    k_b2: torch.Tensor
    heads: int
    rank: int

    @property
    def n_freq(self) -> int:
        return self.freqs.numel()

    @property
    def hidden(self) -> int:
        return self.q_w1.shape[0]

    @classmethod
    def from_params(cls, freqs, mlp_q, mlp_k, heads, rank, device="cuda"):
        """From host tensors (anything with w1, b1, w2, b2)."""
        f = lambda t: t.detach().to(device=device, dtype=torch.float32).contiguous()
        return cls(f(freqs), f(mlp_q.w1), f(mlp_q.b1), f(mlp_q.w2), f(mlp_q.b2),
                   f(mlp_k.w1), f(mlp_k.b1), f(mlp_k.w2), f(mlp_k.b2), heads, rank)

    def c_struct(self) -> _abi.rib_mlp_t:
        p = lambda t, n: _ptr(t, torch.float32, n)
        return _abi.rib_mlp_t(
            self.n_freq, p(self.freqs, "freqs"), self.hidden, self.heads, self.rank,
            p(self.q_w1, "q_w1"), p(self.q_b1, "q_b1"), p(self.q_w2, "q_w2"),
            p(self.q_b2, "q_b2"), p(self.k_w1, "k_w1"), p(self.k_b1, "k_b1"),
            p(self.k_w2, "k_w2"), p(self.k_b2, "k_b2"))

    def tensors(self) -> Tuple[torch.Tensor, ...]:
        """Every tensor the position tokens depend on."""
        return (self.freqs, self.q_w1, self.q_b1, self.q_w2, self.q_b2,
                self.k_w1, self.k_b1, self.k_w2, self.k_b2)

    def key(self) -> Tuple[int, ...]:
        """Addresses of those tensors (which storage the tokens come from)."""
        return tuple(t.data_ptr() for t in self.tensors())

    def versions(self) -> Tuple[int, ...]:
        """Their in-place modification counters (an optimizer step that
        updates the weights in place moves them on)."""
        return tuple(_tensor_version(t) for t in self.tensors())


def _tensor_version(t: torch.Tensor) -> int:
    try:
        return t._version
    except RuntimeError:  # an inference-mode tensor carries no version counter
        return -1


@dataclass
class PositionMLPGrad:
    q_dw1: torch.Tensor
    q_db1: torch.Tensor
    q_dw2: torch.Tensor
    q_db2: torch.Tensor
    k_dw1: torch.Tensor
    k_db1: torch.Tensor
    k_dw2: torch.Tensor
    k_db2: torch.Tensor

    @classmethod
    def empty_like(cls, mlp: PositionMLP):
        e = torch.empty_like
        return cls(e(mlp.q_w1), e(mlp.q_b1), e(mlp.q_w2), e(mlp.q_b2),
                   e(mlp.k_w1), e(mlp.k_b1), e(mlp.k_w2), e(mlp.k_b2))

    def c_struct(self) -> _abi.rib_mlp_grad_t:
        return _abi.rib_mlp_grad_t(*[_ptr(getattr(self, n), torch.float32, n) for n in (
            "q_dw1", "q_db1", "q_dw2", "q_db2", "k_dw1", "k_db1", "k_dw2", "k_db2")])

    def tensors(self) -> Dict[str, torch.Tensor]:
        return dict(self.__dict__)


# ---------------------------------------------------------------- entry points

def rib_pos_tokens(mlp: PositionMLP, window: int, qp=None, kp=None, qp_bf16=None,
                   kp_bf16=None, stream=None, with_bf16: bool = True):
    """Qp, Kp fp32 [heads][M][M][rank] (+ bf16 copies) for one window size."""
    shape = (mlp.heads, window, window, mlp.rank)
    dev = mlp.freqs.device
    qp = torch.empty(shape, device=dev, dtype=torch.float32) if qp is None else qp
    kp = torch.empty(shape, device=dev, dtype=torch.float32) if kp is None else kp
    if with_bf16:
        qp_bf16 = torch.empty(shape, device=dev, dtype=torch.bfloat16) if qp_bf16 is None else qp_bf16
        kp_bf16 = torch.empty(shape, device=dev, dtype=torch.bfloat16) if kp_bf16 is None else kp_bf16
    n = mlp.heads * int(window) ** 2 * mlp.rank
    _sizes("rib_pos_tokens", dev, qp=(qp, n), kp=(kp, n), qp_bf16=(qp_bf16, n),
           kp_bf16=(kp_bf16, n))
    c = mlp.c_struct()
    _check(library().rib_pos_tokens(
        ctypes.byref(c), int(window), _ptr(qp, torch.float32, "qp"), _ptr(kp, torch.float32, "kp"),
        _ptr(qp_bf16, torch.bfloat16, "qp_bf16"), _ptr(kp_bf16, torch.bfloat16, "kp_bf16"),
        _stream(stream)), "rib_pos_tokens")
    return qp, kp, qp_bf16, kp_bf16


def rib_pos_tokens_bwd_workspace(mlp: PositionMLP, window: int) -> int:
    c = mlp.c_struct()
    return int(library().rib_pos_tokens_bwd_workspace(ctypes.byref(c), int(window)))


def rib_pos_tokens_bwd(mlp: PositionMLP, window: int, dqp: torch.Tensor, dkp: torch.Tensor,
                       dmlp: Optional["PositionMLPGrad"] = None, workspace=None, stream=None):
    """Position-MLP gradients from dL/dQp, dL/dKp ([heads][M][M][rank] fp32)."""
    dmlp = PositionMLPGrad.empty_like(mlp) if dmlp is None else dmlp
    n = mlp.heads * int(window) ** 2 * mlp.rank
    _sizes("rib_pos_tokens_bwd", mlp.freqs.device, dqp=(dqp, n), dkp=(dkp, n),
           **_grad_sizes(dmlp, mlp))
    need = rib_pos_tokens_bwd_workspace(mlp, window)
    if workspace is None:
        workspace = torch.empty(max(need, 256), device=dqp.device, dtype=torch.uint8)
    c, cg = mlp.c_struct(), dmlp.c_struct()
    _check(library().rib_pos_tokens_bwd(
        ctypes.byref(c), int(window), _ptr(dqp, torch.float32, "dqp"),
        _ptr(dkp, torch.float32, "dkp"), ctypes.byref(cg), _ptr(workspace, None, "workspace"),
        workspace.numel() * workspace.element_size(), _stream(stream)), "rib_pos_tokens_bwd")
    return dmlp


def rib_pos_tokens_bwd_noalloc(mlp: PositionMLP, window: int, dqp: torch.Tensor,
                               dkp: torch.Tensor, dmlp: "PositionMLPGrad", stream=None):
    """rib_pos_tokens_bwd for callers that cannot allocate device memory at
    the point of the call (inside CUDA graph capture, under an allocator that
    owns all device memory, or where cudaMalloc's synchronisation is too
    costly).  The library's own static 24 MiB device scratch is used instead
    of a workspace; `dmlp` must be given (preallocated).  Calls that overlap
    on the GPU share that scratch and race; the first call on a device should
    precede any stream capture."""
    n = mlp.heads * int(window) ** 2 * mlp.rank
    _sizes("rib_pos_tokens_bwd_noalloc", mlp.freqs.device, dqp=(dqp, n), dkp=(dkp, n),
           **_grad_sizes(dmlp, mlp))
    c, cg = mlp.c_struct(), dmlp.c_struct()
    _check(library().rib_pos_tokens_bwd_noalloc(
        ctypes.byref(c), int(window), _ptr(dqp, torch.float32, "dqp"),
        _ptr(dkp, torch.float32, "dkp"), ctypes.byref(cg), _stream(stream)),
        "rib_pos_tokens_bwd_noalloc")
    return dmlp


def rib_window_attn_fwd(qkv: torch.Tensor, window: int, shift: int, qp_bf16=None,
                        kp_bf16=None, rank: int = 16, scale: float = 0.0, out=None, lse=None,
                        stream=None, region_mask: bool = False):
    """out bf16 [B][H][W][heads][d], lse fp32 [B][heads][H][W].

    region_mask: the optional shifted-window region mask
    (rib_window_attn_fwd_masked)."""
    B, H, W, three, heads, d = qkv.shape
    if three != 3:
        raise ValueError("qkv must be [B][H][W][3][heads][head_dim]")
    out = torch.empty((B, H, W, heads, d), device=qkv.device, dtype=torch.bfloat16) if out is None else out
    lse = torch.empty((B, heads, H, W), device=qkv.device, dtype=torch.float32) if lse is None else lse
    name = "rib_window_attn_fwd_masked" if region_mask else "rib_window_attn_fwd"
    nt = heads * int(window) ** 2 * int(rank)
    _sizes(name, qkv.device, out=(out, B * H * W * heads * d), lse=(lse, B * heads * H * W),
           qp_bf16=(qp_bf16 if rank > 0 else None, nt),
           kp_bf16=(kp_bf16 if rank > 0 else None, nt))
    _check(getattr(library(), name)(
        _ptr(qkv, torch.bfloat16, "qkv"), B, H, W, heads, d, int(window), int(shift),
        _ptr(qp_bf16, torch.bfloat16, "qp_bf16"), _ptr(kp_bf16, torch.bfloat16, "kp_bf16"),
        int(rank), float(scale), _ptr(out, torch.bfloat16, "out"),
        _ptr(lse, torch.float32, "lse"), _stream(stream)), name)
    return out, lse


def rib_window_attn_fwd_tf32(qkv: torch.Tensor, window: int, shift: int, qp=None, kp=None,
                             rank: int = 16, scale: float = 0.0, out=None, lse=None,
                             stream=None):
    """fp32 forward on the tf32 tensor cores: qkv fp32 [B][H][W][3][heads][d],
    qp/kp fp32 [heads][M][M][rank]; returns out fp32 [B][H][W][heads][d] and
    lse fp32 [B][heads][H][W]."""
    B, H, W, three, heads, d = qkv.shape
    if three != 3:
        raise ValueError("qkv must be [B][H][W][3][heads][head_dim]")
    out = torch.empty((B, H, W, heads, d), device=qkv.device, dtype=torch.float32) if out is None else out
    lse = torch.empty((B, heads, H, W), device=qkv.device, dtype=torch.float32) if lse is None else lse
    nt = heads * int(window) ** 2 * int(rank)
    name = "rib_window_attn_fwd_tf32"
    _sizes(name, qkv.device, out=(out, B * H * W * heads * d), lse=(lse, B * heads * H * W),
           qp=(qp if rank > 0 else None, nt), kp=(kp if rank > 0 else None, nt))
    _check(library().rib_window_attn_fwd_tf32(
        _ptr(qkv, torch.float32, "qkv"), B, H, W, heads, d, int(window), int(shift),
        _ptr(qp, torch.float32, "qp"), _ptr(kp, torch.float32, "kp"), int(rank), float(scale),
        _ptr(out, torch.float32, "out"), _ptr(lse, torch.float32, "lse"), _stream(stream)), name)
    return out, lse


@dataclass
class ClaGate:
    """Device fp32 weights of the convolutional local attention gate:
    depth-wise 3x3 (w_dw [C][3][3], b_dw [C]) then point-wise 1x1
    (w_pw [C_out][C_in], b_pw [C]) then a sigmoid."""
    w_dw: torch.Tensor
    b_dw: torch.Tensor
    w_pw: torch.Tensor
    b_pw: torch.Tensor

    @classmethod
    def from_params(cls, w_dw, b_dw, w_pw, b_pw, device="cuda"):
        f = lambda t: torch.as_tensor(t).detach().to(device=device, dtype=torch.float32).contiguous()
        return cls(f(w_dw), f(b_dw), f(w_pw), f(b_pw))

    @property
    def channels(self) -> int:
        return self.b_dw.numel()


def rib_cla_gate(x: torch.Tensor, cla: ClaGate, gate=None, stream=None) -> torch.Tensor:
    """G bf16 [B][H][W][C] = sigmoid(PW1x1(DW3x3(x))) for x bf16 [B][H][W][C]."""
    B, H, W, C = x.shape
    gate = torch.empty_like(x) if gate is None else gate
    _sizes("rib_cla_gate", x.device, gate=(gate, x.numel()), **_cla_sizes(cla, C))
    f32 = torch.float32
    _check(library().rib_cla_gate(
        _ptr(x, torch.bfloat16, "x"), B, H, W, C, _ptr(cla.w_dw, f32, "w_dw"),
        _ptr(cla.b_dw, f32, "b_dw"), _ptr(cla.w_pw, f32, "w_pw"), _ptr(cla.b_pw, f32, "b_pw"),
        _ptr(gate, torch.bfloat16, "gate"), _stream(stream)), "rib_cla_gate")
    return gate


def rib_window_attn_fwd_cla(qkv: torch.Tensor, window: int, shift: int, gate: torch.Tensor,
                            qp_bf16=None, kp_bf16=None, rank: int = 16, scale: float = 0.0,
                            out=None, out_gated=None, lse=None, stream=None):
    """(out, out_gated, lse): the attention output O, O * gate (gate bf16
    [B][H][W][heads*d]) and lse, from one forward launch."""
    B, H, W, three, heads, d = qkv.shape
    if three != 3:
        raise ValueError("qkv must be [B][H][W][3][heads][head_dim]")
    if tuple(gate.shape) not in ((B, H, W, heads * d), (B, H, W, heads, d)):
        raise ValueError("gate must be [B][H][W][heads*head_dim]")
    shape = (B, H, W, heads, d)
    out = torch.empty(shape, device=qkv.device, dtype=torch.bfloat16) if out is None else out
    out_gated = torch.empty(shape, device=qkv.device, dtype=torch.bfloat16) if out_gated is None else out_gated
    lse = torch.empty((B, heads, H, W), device=qkv.device, dtype=torch.float32) if lse is None else lse
    n_out, nt = B * H * W * heads * d, heads * int(window) ** 2 * int(rank)
    _sizes("rib_window_attn_fwd_cla", qkv.device, gate=(gate, n_out), out=(out, n_out),
           out_gated=(out_gated, n_out), lse=(lse, B * heads * H * W),
           qp_bf16=(qp_bf16 if rank > 0 else None, nt),
           kp_bf16=(kp_bf16 if rank > 0 else None, nt))
    _check(library().rib_window_attn_fwd_cla(
        _ptr(qkv, torch.bfloat16, "qkv"), B, H, W, heads, d, int(window), int(shift),
        _ptr(qp_bf16, torch.bfloat16, "qp_bf16"), _ptr(kp_bf16, torch.bfloat16, "kp_bf16"),
        int(rank), float(scale), _ptr(gate, torch.bfloat16, "gate"),
        _ptr(out, torch.bfloat16, "out"), _ptr(out_gated, torch.bfloat16, "out_gated"),
        _ptr(lse, torch.float32, "lse"), _stream(stream)), "rib_window_attn_fwd_cla")
    return out, out_gated, lse


def rib_cla_bwd_workspace(B: int, H: int, W: int, C: int) -> int:
    return int(library().rib_cla_bwd_workspace(B, H, W, C))


def rib_cla_bwd(x: torch.Tensor, cla: ClaGate, gate: torch.Tensor, out: torch.Tensor,
                dout_gated: torch.Tensor, dout=None, dx=None, workspace=None, stream=None):
    """Backward of O' = O * gate: returns dict(dout = dO' * G (the attention
    backward's input), dx, dw_dw, db_dw, dw_pw, db_pw).  out / dout_gated may be
    [B][H][W][heads][d] or [B][H][W][C]."""
    B, H, W, C = x.shape
    dev = x.device
    dout = torch.empty(out.shape, device=dev, dtype=torch.bfloat16) if dout is None else dout
    dx = torch.empty_like(x) if dx is None else dx
    g = {k: torch.empty_like(getattr(cla, k.replace("d", "", 1)))
         for k in ("dw_dw", "db_dw", "dw_pw", "db_pw")}
    n = x.numel()
    _sizes("rib_cla_bwd", dev, gate=(gate, n), out=(out, n), dout_gated=(dout_gated, n),
           dout=(dout, n), dx=(dx, n), **_cla_sizes(cla, C))
    need = rib_cla_bwd_workspace(B, H, W, C)
    if workspace is None:
        workspace = torch.empty(max(need, 256), device=dev, dtype=torch.uint8)
    bf, f32 = torch.bfloat16, torch.float32
    _check(library().rib_cla_bwd(
        _ptr(x, bf, "x"), B, H, W, C, _ptr(cla.w_dw, f32, "w_dw"), _ptr(cla.b_dw, f32, "b_dw"),
        _ptr(cla.w_pw, f32, "w_pw"), _ptr(gate, bf, "gate"), _ptr(out, bf, "out"),
        _ptr(dout_gated, bf, "dout_gated"), _ptr(dout, bf, "dout"), _ptr(dx, bf, "dx"),
        _ptr(g["dw_dw"], f32, "dw_dw"), _ptr(g["db_dw"], f32, "db_dw"),
        _ptr(g["dw_pw"], f32, "dw_pw"), _ptr(g["db_pw"], f32, "db_pw"),
        _ptr(workspace, None, "workspace"), workspace.numel() * workspace.element_size(),
        _stream(stream)), "rib_cla_bwd")
    return dict(dout=dout, dx=dx, **g)


def rib_window_attn_bwd_workspace(B, H, W, heads, head_dim, window, rank,
                                  mlp: Optional[PositionMLP] = None) -> int:
    c = mlp.c_struct() if mlp is not None else None
    return int(library().rib_window_attn_bwd_workspace(
        B, H, W, heads, head_dim, int(window), int(rank),
        ctypes.byref(c) if c is not None else None))


def rib_window_attn_bwd(qkv, out, dout, lse, window: int, shift: int, qp_bf16=None,
                        kp_bf16=None, rank: int = 16, scale: float = 0.0,
                        mlp: Optional[PositionMLP] = None, dqkv=None, dqp=None, dkp=None,
                        dmlp: Optional[PositionMLPGrad] = None, workspace=None, stream=None,
                        region_mask: bool = False):
    """Returns dict(dqkv, dqp, dkp, dmlp).  dmlp is computed when mlp is given.
    region_mask: as for rib_window_attn_fwd (rib_window_attn_bwd_masked)."""
    B, H, W, _, heads, d = qkv.shape
    dev = qkv.device
    dqkv = torch.empty_like(qkv) if dqkv is None else dqkv
    if rank > 0:
        pshape = (heads, window, window, rank)
        dqp = torch.empty(pshape, device=dev, dtype=torch.float32) if dqp is None else dqp
        dkp = torch.empty(pshape, device=dev, dtype=torch.float32) if dkp is None else dkp
    if mlp is not None and dmlp is None:
        dmlp = PositionMLPGrad.empty_like(mlp)
    name = "rib_window_attn_bwd_masked" if region_mask else "rib_window_attn_bwd"
    n_out, nt = B * H * W * heads * d, heads * int(window) ** 2 * int(rank)
    pos = rank > 0
    _sizes(name, dev, out=(out, n_out), dout=(dout, n_out), lse=(lse, B * heads * H * W),
           dqkv=(dqkv, qkv.numel()), qp_bf16=(qp_bf16 if pos else None, nt),
           kp_bf16=(kp_bf16 if pos else None, nt), dqp=(dqp if pos else None, nt),
           dkp=(dkp if pos else None, nt), **_grad_sizes(dmlp, mlp))
    need = rib_window_attn_bwd_workspace(B, H, W, heads, d, window, rank, mlp)
    if workspace is None:
        workspace = torch.empty(max(need, 256), device=dev, dtype=torch.uint8)
    c_mlp = mlp.c_struct() if mlp is not None else None
    c_dmlp = dmlp.c_struct() if (mlp is not None and dmlp is not None) else None
    _check(getattr(library(), name)(
        _ptr(qkv, torch.bfloat16, "qkv"), _ptr(out, torch.bfloat16, "out"),
        _ptr(dout, torch.bfloat16, "dout"), _ptr(lse, torch.float32, "lse"),
        B, H, W, heads, d, int(window), int(shift),
        _ptr(qp_bf16, torch.bfloat16, "qp_bf16"), _ptr(kp_bf16, torch.bfloat16, "kp_bf16"),
        int(rank), float(scale), _ptr(dqkv, torch.bfloat16, "dqkv"),
        _ptr(dqp, torch.float32, "dqp"), _ptr(dkp, torch.float32, "dkp"),
        ctypes.byref(c_mlp) if c_mlp is not None else None,
        ctypes.byref(c_dmlp) if c_dmlp is not None else None,
        _ptr(workspace, None, "workspace"), workspace.numel() * workspace.element_size(),
        _stream(stream)), name)
    return {"dqkv": dqkv, "dqp": dqp, "dkp": dkp, "dmlp": dmlp}


# ---------------------------------------------------------------- the layer's other operators

_ACTS = {"none": _abi.RIB_ACT_NONE, "gelu": _abi.RIB_ACT_GELU, "silu": _abi.RIB_ACT_SILU}
_DTYPES = {torch.bfloat16: _abi.RIB_DTYPE_BF16, torch.float32: _abi.RIB_DTYPE_F32}
_MAX_ROWS = 1 << 30


def _act(where: str, act: str) -> int:
    a = _ACTS.get(act)
    if a is None:
        raise RibError(_abi.RIB_ERR_ARG, f"{where}: act {act!r} is none of {', '.join(_ACTS)}")
    return a


def _dtype(where: str, name: str, dtype: torch.dtype) -> int:
    d = _DTYPES.get(dtype)
    if d is None:
        raise RibError(_abi.RIB_ERR_UNSUPPORTED, f"{where}: {name} is {dtype}, not bfloat16 or float32")
    return d


class _Call:
    """One call of a layer operator: its device, its stream and the checks of
    its tensors.  Small maps are bound by what happens on the host, so every
    tensor is looked at once.

    What a call allocates for itself (missing outputs, workspace) belongs to
    the stream that the call runs on, also when that is not torch's current
    one: memory of the current stream could still be in use by work queued
    there, and could be handed out again while the call runs."""
    __slots__ = ("where", "x", "device", "index", "rows", "channels", "stream", "side")

    def __init__(self, where: str, x: torch.Tensor, stream):
        self.where, self.x = where, x
        if x.dim() < 1 or x.shape[-1] == 0:
            raise RibError(_abi.RIB_ERR_ARG, f"{where}: x must be [..., channels]")
        self.channels = x.shape[-1]
        self.rows = x.numel() // self.channels
        if self.rows > _MAX_ROWS:
            raise RibError(_abi.RIB_ERR_UNSUPPORTED, f"{where}: {self.rows} rows, more than 2^30")
        self.device, self.index = x.device, x.get_device()
        self.side = None
        self.stream = 0
        if self.index >= 0:
            if self.index != torch.cuda.current_device():
                raise RibError(_abi.RIB_ERR_ARG, f"{where}: tensors are on {x.device}, the current "
                               f"device is cuda:{torch.cuda.current_device()}")
            self.stream = _raw_stream(self.index)
            if stream is not None:
                if not hasattr(stream, "cuda_stream"):
                    stream = torch.cuda.ExternalStream(int(stream), device=x.device)
                if stream.cuda_stream != self.stream:
                    self.side, self.stream = stream, stream.cuda_stream

    def empty(self, shape, dtype) -> torch.Tensor:
        if self.side is None:
            # sizes one by one: 1.5 us, where a tuple takes 2.3 and a torch.Size 3.0
            return torch.empty(*shape, dtype=dtype, device=self.device) if shape else \
                torch.empty((), dtype=dtype, device=self.device)
        with torch.cuda.stream(self.side):
            return torch.empty(shape, dtype=dtype, device=self.device)

    def output(self, given, shape, dtype) -> torch.Tensor:
        """An output, allocated if it was not given; the caller will use it on
        the current stream."""
        if given is not None:
            return given
        t = self.empty(shape, dtype)
        if self.side is None:
            return t
        t.record_stream(torch.cuda.current_stream())
        return t

    def like_x(self, given) -> torch.Tensor:
        if given is not None:
            return given
        if self.side is None:
            return torch.empty_like(self.x)   # a strided x is refused
        return self.output(None, self.x.shape, self.x.dtype)

    def ptr(self, name: str, t: Optional[torch.Tensor], n: int, dtype=None) -> Optional[int]:
        """Address of a buffer that has to hold exactly n elements of dtype on
        the call's device (the library takes bare pointers and can check
        neither); None for None."""
        if t is None:
            return None
        if t.numel() != n:
            raise RibError(_abi.RIB_ERR_ARG,
                           f"{self.where}: {name} holds {t.numel()} elements, the call needs {n}")
        if t.get_device() != self.index or (self.index < 0 and t.device != self.device):
            raise RibError(_abi.RIB_ERR_ARG,
                           f"{self.where}: {name} is on {t.device}, not {self.device}")
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
        if dtype is not None and t.dtype != dtype:
            raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
        return t.data_ptr()

    def workspace(self, given: Optional[torch.Tensor], need: int):
        """(address, bytes) of the workspace, allocated if it was not given.
        After the tensors' checks: the first thing that needs a CUDA tensor."""
        if self.index < 0:
            raise ValueError("x must be a CUDA tensor")
        if given is None:
            if need == 0:   # the library does not look at it
                return None, 0, None
            given = self.empty((need,), torch.uint8)
        return (self.ptr("workspace", given, given.numel()), given.numel() * given.element_size(),
                given)

    def run(self, *args) -> None:
        if self.index < 0:
            raise ValueError("x must be a CUDA tensor")
        code = getattr(library(), self.where)(*args, self.stream)
        if code != _abi.RIB_OK:
            raise RibError(code, self.where)


_BF16, _F32 = torch.bfloat16, torch.float32


def rib_layer_norm_fwd(x: torch.Tensor, gamma: Optional[torch.Tensor] = None,
                       beta: Optional[torch.Tensor] = None, eps: float = 1e-5, y=None, mean=None,
                       rstd=None, stream=None):
    """(y, mean, rstd): layer norm of x [..., C] (bf16 or fp32) over its last
    axis, y like x, mean and rstd fp32 [...].  gamma, beta fp32 [C] or None."""
    c = _Call("rib_layer_norm_fwd", x, stream)
    dtype, rows, C = x.dtype, c.rows, c.channels
    dt, n, lead = _dtype(c.where, "x", dtype), c.rows * c.channels, x.shape[:-1]
    y = c.like_x(y)
    mean, rstd = c.output(mean, lead, _F32), c.output(rstd, lead, _F32)
    c.run(c.ptr("x", x, n), dt, rows, C, c.ptr("gamma", gamma, C, _F32),
          c.ptr("beta", beta, C, _F32), float(eps), c.ptr("y", y, n, dtype),
          c.ptr("mean", mean, rows, _F32), c.ptr("rstd", rstd, rows, _F32))
    return y, mean, rstd


def rib_layer_norm_bwd_workspace(rows: int, C: int) -> int:
    return int(library().rib_layer_norm_bwd_workspace(int(rows), int(C)))


def rib_layer_norm_bwd(x: torch.Tensor, dy: torch.Tensor, mean: torch.Tensor, rstd: torch.Tensor,
                       gamma: Optional[torch.Tensor] = None, dres: Optional[torch.Tensor] = None,
                       dx=None, dgamma=None, dbeta=None, weight_grads: bool = True,
                       workspace=None, stream=None):
    """dict(dx, dgamma, dbeta) of rib_layer_norm_fwd.  dres: a second gradient
    of x (the residual path's), added to dx before its rounding.  Without
    weight_grads dgamma and dbeta are None."""
    c = _Call("rib_layer_norm_bwd", x, stream)
    dtype, rows, C = x.dtype, c.rows, c.channels
    dt, n = _dtype(c.where, "x", dtype), c.rows * c.channels
    dx = c.like_x(dx)
    if weight_grads:
        dgamma, dbeta = c.output(dgamma, (C,), _F32), c.output(dbeta, (C,), _F32)
    else:
        dgamma = dbeta = None
    args = (c.ptr("x", x, n), c.ptr("dy", dy, n, dtype), dt, rows, C,
            c.ptr("mean", mean, rows, _F32), c.ptr("rstd", rstd, rows, _F32),
            c.ptr("gamma", gamma, C, _F32), c.ptr("dres", dres, n, dtype),
            c.ptr("dx", dx, n, dtype), c.ptr("dgamma", dgamma, C, _F32),
            c.ptr("dbeta", dbeta, C, _F32))
    need = rib_layer_norm_bwd_workspace(rows, C) if weight_grads and workspace is None else 0
    ws, size, _keep = c.workspace(workspace, need)
    c.run(*args, ws, size)
    return {"dx": dx, "dgamma": dgamma, "dbeta": dbeta}


def _weight(where: str, w: torch.Tensor, K: int) -> int:
    if w.dim() != 2 or w.shape[1] != K:
        raise RibError(_abi.RIB_ERR_ARG, f"{where}: w must be [out][{K}], got {tuple(w.shape)}")
    return w.shape[0]


def rib_linear_fwd(x: torch.Tensor, w: torch.Tensor, bias: Optional[torch.Tensor] = None,
                   act: str = "none", residual: Optional[torch.Tensor] = None,
                   save_pre: bool = False, y=None, pre=None, stream=None):
    """(y, pre): y = act(x w^T + bias) + residual for x bf16 [..., K], w bf16
    [N][K], bias fp32 [N]; act "none", "gelu" (erf form) or "silu".  pre is
    the bf16 x w^T + bias that the backward of an activation needs, when
    save_pre (or a buffer for it) is given, else None."""
    c = _Call("rib_linear_fwd", x, stream)
    rows, K = c.rows, c.channels
    N, a = _weight(c.where, w, K), _act(c.where, act)
    shape, n = (*x.shape[:-1], N), c.rows * N
    y = c.output(y, shape, _BF16)
    pre = c.output(pre, shape, _BF16) if save_pre or pre is not None else None
    c.run(c.ptr("x", x, rows * K, _BF16), rows, K, c.ptr("w", w, N * K, _BF16), N,
          c.ptr("bias", bias, N, _F32), a, c.ptr("residual", residual, n, _BF16),
          c.ptr("pre", pre, n, _BF16), c.ptr("y", y, n, _BF16))
    return y, pre


def rib_linear_bwd_workspace(rows: int, K: int, N: int, act: str = "none") -> int:
    return int(library().rib_linear_bwd_workspace(int(rows), int(K), int(N),
                                                  _act("rib_linear_bwd_workspace", act)))


def rib_linear_bwd(x: torch.Tensor, w: torch.Tensor, dy: torch.Tensor, act: str = "none",
                   pre: Optional[torch.Tensor] = None, dx_add: Optional[torch.Tensor] = None,
                   with_dx: bool = True, with_dw: bool = True, with_db: bool = True, dx=None,
                   dw=None, db=None, dw_dtype: torch.dtype = torch.float32, workspace=None,
                   stream=None):
    """dict(dx, dw, db) of rib_linear_fwd for dy bf16 [..., N]; what is not
    wanted (with_dx, with_dw, with_db) is None.  dx_add: a second gradient of x,
    added to dx before its rounding.  dw is fp32 or bf16 (dw_dtype, or the type
    of the buffer given)."""
    c = _Call("rib_linear_bwd", x, stream)
    rows, K = c.rows, c.channels
    N, a = _weight(c.where, w, K), _act(c.where, act)
    if a != _abi.RIB_ACT_NONE and pre is None:
        raise RibError(_abi.RIB_ERR_ARG,
                       f"{c.where}: act {act!r} needs pre (rib_linear_fwd's, with save_pre)")
    dw_dtype = dw.dtype if dw is not None else dw_dtype
    dt = _dtype(c.where, "dw", dw_dtype)
    dx = c.like_x(dx) if with_dx else None
    dw = c.output(dw, (N, K), dw_dtype) if with_dw else None
    db = c.output(db, (N,), _F32) if with_db else None
    args = (c.ptr("x", x, rows * K, _BF16), rows, K, c.ptr("w", w, N * K, _BF16), N, a,
            c.ptr("pre", pre, rows * N, _BF16), c.ptr("dy", dy, rows * N, _BF16),
            c.ptr("dx_add", dx_add, rows * K, _BF16), c.ptr("dx", dx, rows * K, _BF16),
            c.ptr("dw", dw, N * K), dt, c.ptr("db", db, N, _F32))
    need = rib_linear_bwd_workspace(rows, K, N, act) if workspace is None else 0
    ws, size, _keep = c.workspace(workspace, need)
    c.run(*args, ws, size)
    return {"dx": dx, "dw": dw, "db": db}


@dataclass
class GatedFfn:
    """Device weights of the gated feed-forward block: w_in bf16
    [2][hidden][C] (the gate's projection, then the other), w_out bf16
    [C][hidden]; biases fp32 [2][hidden] and [C], or None."""
    w_in: torch.Tensor
    b_in: Optional[torch.Tensor]
    w_out: torch.Tensor
    b_out: Optional[torch.Tensor]

    @classmethod
    def from_params(cls, w_in, b_in, w_out, b_out, device="cuda"):
        def f(t, dtype):
            return None if t is None else torch.as_tensor(t).detach().to(
                device=device, dtype=dtype).contiguous()
        return cls(f(w_in, torch.bfloat16), f(b_in, torch.float32), f(w_out, torch.bfloat16),
                   f(b_out, torch.float32))

    @property
    def hidden(self) -> int:
        return self.w_in.shape[1]


def _ffn_hidden(where: str, ffn: GatedFfn, C: int) -> int:
    s, o = ffn.w_in.shape, ffn.w_out.shape
    if len(s) != 3 or s[0] != 2 or s[2] != C:
        raise RibError(_abi.RIB_ERR_ARG, f"{where}: w_in must be [2][hidden][{C}], got {tuple(s)}")
    if len(o) != 2 or o[0] != C or o[1] != s[1]:
        raise RibError(_abi.RIB_ERR_ARG, f"{where}: w_out must be [{C}][{s[1]}], got {tuple(o)}")
    return s[1]


def rib_gated_ffn_fwd_workspace(rows: int, C: int, hidden: int) -> int:
    return int(library().rib_gated_ffn_fwd_workspace(int(rows), int(C), int(hidden)))


def rib_gated_ffn_fwd(x: torch.Tensor, ffn: GatedFfn, act: str = "silu",
                      residual: Optional[torch.Tensor] = None, y=None, workspace=None,
                      stream=None) -> torch.Tensor:
    """y = (act(x Wg^T + bg) * (x Wu^T + bu)) Wo^T + b_out + residual for x
    bf16 [..., C]."""
    c = _Call("rib_gated_ffn_fwd", x, stream)
    rows, C, n = c.rows, c.channels, c.rows * c.channels
    H, a = _ffn_hidden(c.where, ffn, C), _act(c.where, act)
    y = c.like_x(y)
    args = (c.ptr("x", x, n, _BF16), rows, C, H, c.ptr("w_in", ffn.w_in, 2 * H * C, _BF16),
            c.ptr("b_in", ffn.b_in, 2 * H, _F32), c.ptr("w_out", ffn.w_out, C * H, _BF16),
            c.ptr("b_out", ffn.b_out, C, _F32), a, c.ptr("residual", residual, n, _BF16),
            c.ptr("y", y, n, _BF16))
    need = rib_gated_ffn_fwd_workspace(rows, C, H) if workspace is None else 0
    ws, size, _keep = c.workspace(workspace, need)
    c.run(*args, ws, size)
    return y


def rib_gated_ffn_bwd_workspace(rows: int, C: int, hidden: int) -> int:
    return int(library().rib_gated_ffn_bwd_workspace(int(rows), int(C), int(hidden)))


def rib_gated_ffn_bwd(x: torch.Tensor, ffn: GatedFfn, dy: torch.Tensor, act: str = "silu",
                      dx_add: Optional[torch.Tensor] = None, dx=None, dw_in=None, db_in=None,
                      dw_out=None, db_out=None, dw_dtype: torch.dtype = torch.float32,
                      workspace=None, stream=None):
    """dict(dx, dw_in, db_in, dw_out, db_out) of rib_gated_ffn_fwd, from x and dy
    alone (the residual's gradient is dy: pass it as dx_add where the
    residual is x itself).  db_in and db_out are formed where the block has
    that bias, else None; dw_in and dw_out are both fp32 or both bf16."""
    c = _Call("rib_gated_ffn_bwd", x, stream)
    rows, C, n = c.rows, c.channels, c.rows * c.channels
    H, a = _ffn_hidden(c.where, ffn, C), _act(c.where, act)
    if dw_in is not None:
        dw_dtype = dw_in.dtype
    elif dw_out is not None:
        dw_dtype = dw_out.dtype
    dt = _dtype(c.where, "dw_in / dw_out", dw_dtype)
    dx = c.like_x(dx)
    dw_in = c.output(dw_in, (2, H, C), dw_dtype)
    dw_out = c.output(dw_out, (C, H), dw_dtype)
    db_in = c.output(db_in, (2, H), _F32) if ffn.b_in is not None else None
    db_out = c.output(db_out, (C,), _F32) if ffn.b_out is not None else None
    c.ptr("b_out", ffn.b_out, C, _F32)   # its values are not needed, its size is
    args = (c.ptr("x", x, n, _BF16), rows, C, H, c.ptr("w_in", ffn.w_in, 2 * H * C, _BF16),
            c.ptr("b_in", ffn.b_in, 2 * H, _F32), c.ptr("w_out", ffn.w_out, C * H, _BF16), a,
            c.ptr("dy", dy, n, _BF16), c.ptr("dx_add", dx_add, n, _BF16), c.ptr("dx", dx, n, _BF16),
            c.ptr("dw_in", dw_in, 2 * H * C, dw_dtype), c.ptr("db_in", db_in, 2 * H, _F32),
            c.ptr("dw_out", dw_out, C * H, dw_dtype), c.ptr("db_out", db_out, C, _F32), dt)
    need = rib_gated_ffn_bwd_workspace(rows, C, H) if workspace is None else 0
    ws, size, _keep = c.workspace(workspace, need)
    c.run(*args, ws, size)
    return {"dx": dx, "dw_in": dw_in, "db_in": db_in, "dw_out": dw_out, "db_out": db_out}


def rib_window_gather(x: torch.Tensor, window: int, shift: int, out=None, stream=None):
    """x [B][H][W][C] -> [B][nW][M*M][C] (roll by -shift, partition)."""
    B, H, W, C = x.shape
    nW = (H // window) * (W // window)
    out = torch.empty((B, nW, window * window, C), device=x.device, dtype=x.dtype) if out is None else out
    _sizes("rib_window_gather", x.device, out=(out, B * nW * window * window * C))
    _check(library().rib_window_gather(
        _ptr(x, None, "x"), B, H, W, C, x.element_size(), int(window), int(shift),
        _ptr(out, x.dtype, "out"), _stream(stream)), "rib_window_gather")
    return out


def rib_window_scatter(xw: torch.Tensor, H: int, W: int, window: int, shift: int, out=None,
                       stream=None):
    """Inverse of rib_window_gather."""
    B, nW, N, C = xw.shape
    out = torch.empty((B, H, W, C), device=xw.device, dtype=xw.dtype) if out is None else out
    _sizes("rib_window_scatter", xw.device, out=(out, B * H * W * C))
    if (window > 0 and H % window == 0 and W % window == 0 and
            (nW, N) != ((H // window) * (W // window), window * window)):
        raise RibError(_abi.RIB_ERR_ARG, f"rib_window_scatter: xw is [B][{nW}][{N}][C], the "
                       f"{window}x{window} windows of a {H}x{W} map need "
                       f"[B][{(H // window) * (W // window)}][{window * window}][C]")
    _check(library().rib_window_scatter(
        _ptr(xw, None, "xw"), B, H, W, C, xw.element_size(), int(window), int(shift),
        _ptr(out, xw.dtype, "out"), _stream(stream)), "rib_window_scatter")
    return out


def rib_last_status() -> Tuple[int, int]:
    site = ctypes.c_int(0)
    code = library().rib_last_status(ctypes.byref(site))
    return int(code), int(site.value)


def rib_set_wait_limit_ns(limit_ns: int) -> None:
    _check(library().rib_set_wait_limit_ns(int(limit_ns)), "rib_set_wait_limit_ns")


def rib_set_bwd_kernel(which: int) -> None:
    """Form of the attention backward kernel, process-wide: _abi.RIB_BWD_AUTO
    (by window size), RIB_BWD_PER_ITEM or RIB_BWD_PERSISTENT."""
    _check(library().rib_set_bwd_kernel(int(which)), "rib_set_bwd_kernel")


def rib_bwd_kernel_for(window: int) -> int:
    """The backward form a call with this window size would use."""
    return int(library().rib_bwd_kernel_for(int(window)))


def rib_debug_exp2(x: torch.Tensor, stream=None) -> torch.Tensor:
    """2^x with the attention kernels' FMA-pipe exponential (test hook)."""
    y = torch.empty_like(x)
    _check(library().rib_debug_exp2(_ptr(x, torch.float32, "x"), _ptr(y, torch.float32, "y"),
                                    x.numel(), _stream(stream)), "rib_debug_exp2")
    return y


def rib_debug_wait_timeout(limit_ns: int, stream=None) -> None:
    _check(library().rib_debug_wait_timeout(int(limit_ns), _stream(stream)),
           "rib_debug_wait_timeout")


def rib_trace_enable(on: bool = True) -> None:
    _check(library().rib_trace_enable(1 if on else 0), "rib_trace_enable")


def rib_trace_collect() -> Dict[str, Tuple[int, float]]:
    """{kernel: (launches, total_ms)} of the launches traced since enabling."""
    entries = (_abi.rib_trace_entry_t * 32)()
    n = ctypes.c_int(0)
    _check(library().rib_trace_collect(ctypes.cast(entries, ctypes.c_void_p), 32,
                                       ctypes.byref(n)), "rib_trace_collect")
    return {entries[i].kernel.decode(): (int(entries[i].launches), float(entries[i].total_ms))
            for i in range(n.value)}


# ---------------------------------------------------------------- geometry cache

class PosTokenCache:
    """Qp/Kp per window geometry, computed once and reused across windows,
    batch entries and layers (they depend only on the geometry and the MLP).

    An entry is keyed by the window and the addresses of the MLP's tensors
    (frequencies, weights and biases), and holds references to them, so no
    other tensor can take those addresses while it lives.  It is recomputed
    when any of them has been modified in place since (an optimizer step),
    and replaced, not kept beside the new one."""

    def __init__(self):
        self._cache = {}

    def get(self, mlp: PositionMLP, window: int, stream=None):
        k = (mlp.key(), int(window))
        ver = mlp.versions()
        e = self._cache.get(k)
        if e is None or e[0] != ver:
            tokens = rib_pos_tokens(mlp, window, stream=stream)
            self._cache[k] = (ver, tokens, mlp.tensors())
            e = self._cache[k]
        return e[1]

    def clear(self):
        self._cache.clear()

    def __len__(self):
        return len(self._cache)

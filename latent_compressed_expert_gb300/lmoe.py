"""ctypes binding of liblmoe.so (include/lmoe.h): argument marshalling only.

Every step of the layer runs in the library's CUDA kernels; PyTorch provides device
memory and the current stream.  There is no CPU fallback: if the library is missing or
its CUDA calls fail, these functions raise.
"""
from __future__ import annotations

import ctypes
import os
import threading

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "_build", "liblmoe.so")

LMOE_OK = 0
LMOE_ERR_INVALID_ARG = 1
LMOE_ERR_UNSUPPORTED = 2
LMOE_ERR_CUDA = 3
LMOE_ERR_DEVICE_TIMEOUT = 4
LMOE_ERR_WORKSPACE_TOO_SMALL = 5

# Every symbol the header declares, with its ctypes signature.
_vp, _i, _f, _sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
_ll = ctypes.c_longlong


class Dims(ctypes.Structure):
    _fields_ = [("T", _i), ("d", _i), ("L", _i), ("E", _i), ("K", _i), ("I", _i), ("S", _i),
                ("Is", _i), ("c", _f), ("eps", _f), ("expert_fp8", _i)]


class Weights(ctypes.Structure):
    _fields_ = [(n, _vp) for n in ("w_down", "w_router", "w_gate", "w_value", "w_edown", "gamma",
                                   "w_up", "w_sgate", "w_svalue", "w_sdown")]


class IO(ctypes.Structure):
    _fields_ = [("tau_in", _vp), ("balance", _i), ("logits_in", _vp), ("logits_out", _vp),
                ("tau_out", _vp), ("idx_out", _vp), ("gate_out", _vp), ("counts_out", _vp),
                ("stage_events", ctypes.POINTER(_vp)), ("kernel_launches", _i),
                ("aux_stream", _vp), ("aux_events", _vp * 2), ("shared_sms", _i),
                ("phase", _i), ("cand_out", _vp), ("cand_k", _i),
                ("tau_ema", _vp), ("ema_beta", _f), ("ema_first", _i), ("load_stats", _vp),
                ("save_pre", _vp), ("save_pre_shared", _vp), ("y_f32_out", _vp),
                ("logit_bias", _vp)]


OVERLAP_MIN_T = 512  # LMOE_OVERLAP_MIN_T
FEW_MAX_TOKENS = 8  # LMOE_FEW_MAX_TOKENS
HOST_PIPE_MAX_DEPTH = 4  # LMOE_HOST_PIPE_MAX_DEPTH


class HostPipe(ctypes.Structure):
    _fields_ = [("depth", _i), ("max_tokens", _i), ("x_dev", _vp * HOST_PIPE_MAX_DEPTH),
                ("y_dev", _vp * HOST_PIPE_MAX_DEPTH), ("upload", _vp), ("compute", _vp),
                ("download", _vp), ("uploaded", _vp * HOST_PIPE_MAX_DEPTH),
                ("computed", _vp * HOST_PIPE_MAX_DEPTH),
                ("downloaded", _vp * HOST_PIPE_MAX_DEPTH), ("calls", ctypes.c_ulonglong)]

class LinearDesc(ctypes.Structure):
    _fields_ = [("M", _i), ("N", _i), ("K", _i), ("act", _i), ("type", _i), ("c", _f),
                ("x", _vp), ("ldx", _ll), ("x_scales", _vp), ("w", _vp), ("ldw", _ll),
                ("w_scales", _vp), ("bias", _vp), ("residual", _vp), ("ldr", _ll), ("y", _vp),
                ("ldy", _ll), ("pre", _vp), ("ldp", _ll), ("dev_flag", _vp)]


class LinearXentDesc(ctypes.Structure):
    _fields_ = [("M", _i), ("V", _i), ("K", _i), ("x", _vp), ("ldx", _ll), ("w", _vp),
                ("ldw", _ll), ("target", _vp), ("target_type", _i), ("loss", _vp), ("lse", _vp),
                ("dev_flag", _vp)]


class MuonDesc(ctypes.Structure):
    _fields_ = [("batch", _i), ("rows", _i), ("cols", _i), ("steps", _i), ("coeffs", _vp),
                ("eps", _f), ("grad", _vp), ("grad_type", _i), ("ldg", _ll), ("grad_stride", _ll),
                ("out", _vp), ("ldo", _ll), ("out_stride", _ll), ("momentum", _vp), ("ldm", _ll),
                ("momentum_stride", _ll), ("beta", _f), ("nesterov", _i), ("w", _vp), ("ldw", _ll),
                ("w_stride", _ll), ("master", _vp), ("ldmaster", _ll), ("master_stride", _ll),
                ("rate", _f), ("weight_decay", _f), ("scale", _f), ("dev_flag", _vp)]


MUON_MAX_STEPS = 64  # LMOE_MUON_MAX_STEPS

# enum lmoe_act
ACTS = {"none": 0, "silu": 1, "gelu": 2, "situ": 3}

# enum lmoe_type
BF16, E4M3, F32, I32, I64 = 0, 1, 2, 3, 4

# enum lmoe_phase
PHASE_ALL, PHASE_ROUTER, PHASE_EXPERTS = 0, 1, 2


# enum lmoe_stage
STAGES = ["latent_shared", "router", "thresholds", "route", "dispatch", "expert_gate_up",
          "expert_down", "combine", "output"]
NUM_STAGES = len(STAGES)


SIGNATURES = {
    "lmoe_packed_bytes": (_sz, [ctypes.POINTER(Dims)]),
    "lmoe_pack_weights": (_i, [ctypes.POINTER(Dims), ctypes.POINTER(Weights), _vp, _sz, _vp]),
    "lmoe_workspace_bytes": (_sz, [ctypes.POINTER(Dims)]),
    "lmoe_thresholds": (_i, [_vp, _i, _i, _i, _i, _vp, _vp]),
    "lmoe_threshold_candidates": (_i, [_vp, _i, _i, _i, _vp, _vp]),
    "lmoe_fair_share_rank": (_i, [ctypes.c_longlong, _i, _i]),
    "lmoe_quantize_e4m3": (_i, [_vp, ctypes.c_longlong, _i, _vp, _vp, _vp]),
    "lmoe_tau_ema": (_i, [_vp, _vp, _i, _f, _i, _vp]),
    "lmoe_packed_backward_bytes": (_sz, [ctypes.POINTER(Dims)]),
    "lmoe_pack_backward_weights": (_i, [ctypes.POINTER(Dims), ctypes.POINTER(Weights), _vp, _vp,
                                        _sz, _vp]),
    "lmoe_backward_workspace_bytes": (_sz, [ctypes.POINTER(Dims)]),
    "lmoe_backward": (_i, [ctypes.POINTER(Dims), _vp, _vp, _vp, _sz, _vp, _vp, _vp, _vp, _vp,
                           _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _sz, _vp]),
    "lmoe_routed_backward_workspace_bytes": (_sz, [ctypes.POINTER(Dims)]),
    "lmoe_routed_backward": (_i, [ctypes.POINTER(Dims), _vp, _vp, _vp, _sz, _vp, _vp, _vp, _vp,
                                  _vp, _vp, _vp, _vp, _sz, _vp]),
    "lmoe_ep_workspace_bytes": (_sz, [_i, _i, _i, _i]),
    "lmoe_ep_dispatch": (_i, [_vp, _i, _i, _i, _i, _vp, _i, _vp, _vp, _vp, _vp, _vp, _sz, _vp]),
    "lmoe_ep_combine": (_i, [_vp, _i, _i, _i, _i, _vp, _vp, _vp, _vp, _vp, _vp, _i, _vp, _vp,
                             _vp, _vp]),
    "lmoe_add_rmsnorm": (_i, [_vp, _ll, _vp, _ll, _vp, _ll, _i, _f, _vp, _ll, _i, _vp, _vp, _ll,
                              _vp, _vp]),
    "lmoe_add_rmsnorm_backward_workspace_bytes": (_sz, [_ll, _i]),
    "lmoe_add_rmsnorm_backward": (_i, [_vp, _ll, _vp, _ll, _vp, _vp, _vp, _ll, _ll, _i, _vp, _ll,
                                       _vp, _vp, _sz, _vp]),
    "lmoe_norm_last_device_error": (_i, []),
    "lmoe_linear_forward": (_i, [_vp, _vp]),
    "lmoe_linear_backward_workspace_bytes": (_sz, [_vp]),
    "lmoe_linear_backward": (_i, [_vp, _vp, _ll, _vp, _ll, _vp, _i, _vp, _vp, _sz, _vp]),
    "lmoe_linear_xent_workspace_bytes": (_sz, [_vp]),
    "lmoe_linear_xent_forward": (_i, [_vp, _vp, _sz, _vp]),
    "lmoe_linear_xent_backward_workspace_bytes": (_sz, [_vp]),
    "lmoe_linear_xent_backward": (_i, [_vp, _vp, _vp, _ll, _vp, _i, _vp, _sz, _vp]),
    "lmoe_muon_workspace_bytes": (_sz, [_vp]),
    "lmoe_orthogonalize": (_i, [_vp, _vp, _sz, _vp]),
    "lmoe_muon_update": (_i, [_vp, _vp, _sz, _vp]),
    "lmoe_few_workspace_bytes": (_sz, [ctypes.POINTER(Dims)]),
    "lmoe_forward_few": (_i, [ctypes.POINTER(Dims), _vp, _vp, _vp, _vp, _vp, _sz,
                              ctypes.POINTER(IO), _vp]),
    "lmoe_load_stats_update": (_i, [_vp, _i, _vp, _vp]),
    "lmoe_route": (_i, [_vp, _vp, _i, _i, _i, _vp, _vp, _vp, _vp]),
    "lmoe_forward": (_i, [ctypes.POINTER(Dims), _vp, _vp, _vp, _vp, _vp, _sz, ctypes.POINTER(IO),
                          _vp]),
    "lmoe_gemm_bf16": (_i, [_vp, _vp, _vp, _i, _i, _i, _vp, _vp]),
    "lmoe_gemm_wgrad_bf16": (_i, [_vp, _vp, _vp, _i, _i, _i, _vp, _vp]),
    "lmoe_forward_noalloc": (_i, [ctypes.POINTER(Dims), _vp, _vp, _vp, _vp, ctypes.POINTER(IO),
                                  _vp]),
    "lmoe_forward_host": (_i, [ctypes.POINTER(Dims), _vp, _vp, _i, _vp, _vp, _sz,
                               ctypes.POINTER(IO), ctypes.POINTER(HostPipe)]),
    "lmoe_noalloc_last_device_error": (_i, []),
    "lmoe_last_device_error": (_i, [_vp]),
    "lmoe_error_string": (ctypes.c_char_p, [_i]),
    "lmoe_version": (ctypes.c_char_p, []),
}

_lock = threading.Lock()
_lib = None


def load():
    """Load liblmoe.so (built by ``python -m latent_compressed_expert_gb300.build``)."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is not None:
            return _lib
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is not built; run "
                               "`python -m latent_compressed_expert_gb300.build` (needs nvcc)")
        lib = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in SIGNATURES.items():
            fn = getattr(lib, name)
            fn.restype = res
            fn.argtypes = args
        _lib = lib
        return lib


class LmoeError(RuntimeError):
    def __init__(self, code: int, what: str):
        msg = load().lmoe_error_string(code).decode()
        super().__init__(f"{what}: {msg} (status {code})")
        self.code = code


def _check(code: int, what: str):
    if code != LMOE_OK:
        raise LmoeError(code, what)


def _stream(stream=None):
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def _ptr(t):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("lmoe: tensors must be CUDA device tensors")
    if not t.is_contiguous():
        raise ValueError("lmoe: tensors must be contiguous")
    return ctypes.c_void_p(t.data_ptr())


def _expect(t, dtype, shape, name):
    if t.dtype != dtype or tuple(t.shape) != tuple(shape):
        raise ValueError(f"lmoe: {name} must be {dtype} {tuple(shape)}, got {t.dtype} "
                         f"{tuple(t.shape)}")


def make_dims(T, d, L, E, K, I, S, Is, c=100.0, eps=1e-6, expert_fp8=False) -> Dims:
    return Dims(T, d, L, E, K, I, S, Is, c, eps, 1 if expert_fp8 else 0)


def dims_of(shape, T=None, expert_fp8=False) -> Dims:
    """Dims from an object with T, d, L, E, K, I, S, Is (and optionally c, eps)."""
    return make_dims(shape.T if T is None else T, shape.d, shape.L, shape.E, shape.K, shape.I,
                     shape.S, shape.Is, getattr(shape, "c", 100.0), getattr(shape, "eps", 1e-6),
                     expert_fp8)


def packed_bytes(dims: Dims) -> int:
    return int(load().lmoe_packed_bytes(ctypes.byref(dims)))


SPLITK_BYTES = 12 << 20  # the optional split-K region of lmoe_workspace_bytes (T <= 128)
NOALLOC_SCRATCH_BYTES = 24 << 20  # LMOE_NOALLOC_SCRATCH_BYTES: lmoe_forward_noalloc's array


def workspace_base_bytes(dims: Dims) -> int:
    """The smallest workspace lmoe_forward accepts: lmoe_workspace_bytes less the optional
    split-K region of small batches."""
    full = workspace_bytes(dims)
    return full - SPLITK_BYTES if full and 0 < dims.T <= 128 else full


def workspace_bytes(dims: Dims) -> int:
    return int(load().lmoe_workspace_bytes(ctypes.byref(dims)))


def pack_weights(dims: Dims, w: dict, stream=None) -> torch.Tensor:
    """Repack a dict of unpacked weights (bf16 [out, in], gamma fp32) into one device
    buffer in the layout lmoe_forward reads."""
    D = dims
    bf = torch.bfloat16
    _expect(w["w_down"], bf, (D.L, D.d), "w_down")
    _expect(w["w_router"], bf, (D.E, D.L), "w_router")
    _expect(w["w_gate"], bf, (D.E, D.I, D.L), "w_gate")
    _expect(w["w_value"], bf, (D.E, D.I, D.L), "w_value")
    _expect(w["w_edown"], bf, (D.E, D.L, D.I), "w_edown")
    _expect(w["gamma"], torch.float32, (D.L,), "gamma")
    _expect(w["w_up"], bf, (D.d, D.L), "w_up")
    if D.S > 0:
        _expect(w["w_sgate"], bf, (D.S, D.Is, D.d), "w_sgate")
        _expect(w["w_svalue"], bf, (D.S, D.Is, D.d), "w_svalue")
        _expect(w["w_sdown"], bf, (D.S, D.d, D.Is), "w_sdown")
    nbytes = packed_bytes(D)
    if nbytes == 0:
        raise LmoeError(LMOE_ERR_UNSUPPORTED, "lmoe_packed_bytes")
    dev = w["w_down"].device
    packed = torch.empty(nbytes, dtype=torch.uint8, device=dev)
    W = Weights(*[_ptr(w.get(n)) for n, _ in Weights._fields_])
    _check(load().lmoe_pack_weights(ctypes.byref(D), ctypes.byref(W), _ptr(packed), nbytes,
                                    _stream(stream)), "lmoe_pack_weights")
    return packed


def thresholds(logits: torch.Tensor, K: int, k_rank: int = 0, stream=None) -> torch.Tensor:
    T, E = logits.shape
    _expect(logits, torch.float32, (T, E), "logits")
    tau = torch.empty(E, dtype=torch.float32, device=logits.device)
    _check(load().lmoe_thresholds(_ptr(logits), T, E, K, k_rank, _ptr(tau), _stream(stream)),
           "lmoe_thresholds")
    return tau


def quantize_e4m3(x: torch.Tensor, stream=None):
    """Per-row e4m3 codes (uint8) and fp32 scales of bf16 rows (lmoe_quantize_e4m3)."""
    rows, cols = x.shape
    _expect(x, torch.bfloat16, (rows, cols), "x")
    codes = torch.empty((rows, cols), dtype=torch.uint8, device=x.device)
    scales = torch.empty(rows, dtype=torch.float32, device=x.device)
    _check(load().lmoe_quantize_e4m3(_ptr(x), rows, cols, _ptr(codes), _ptr(scales),
                                     _stream(stream)), "lmoe_quantize_e4m3")
    return codes, scales


def tau_ema(tau_step: torch.Tensor, tau_ema_: torch.Tensor, beta: float, first: bool = False,
            stream=None) -> torch.Tensor:
    """Fold one step's thresholds into the streaming thresholds, in place (lmoe_tau_ema)."""
    E = tau_step.shape[0]
    _expect(tau_step, torch.float32, (E,), "tau_step")
    _expect(tau_ema_, torch.float32, (E,), "tau_ema")
    _check(load().lmoe_tau_ema(_ptr(tau_step), _ptr(tau_ema_), E, beta, 1 if first else 0,
                               _stream(stream)), "lmoe_tau_ema")
    return tau_ema_


class LoadStats:
    """64-bit per-expert load counters on the device (layout at lmoe_load_stats_update),
    updated by ``Layer.forward(load_stats=...)`` or ``update(counts)``."""

    def __init__(self, E: int, device):
        self.E = E
        self.acc = torch.zeros(4 + 4 * E, dtype=torch.int64, device=device)

    def update(self, counts: torch.Tensor, stream=None):
        _expect(counts, torch.int32, (self.E,), "counts")
        _check(load().lmoe_load_stats_update(_ptr(counts), self.E, _ptr(self.acc),
                                             _stream(stream)), "lmoe_load_stats_update")

    def summary(self) -> dict:
        a = self.acc.cpu().numpy().astype(float)
        E, steps = self.E, max(a[0], 1.0)
        mean = a[1] / steps / E                     # tokens per expert per step
        per = a[4:4 + E] / steps
        return {"steps": int(a[0]), "fair_share": mean,
                "mean_max_over_mean": a[2] / steps / mean if mean else None,
                "worst_max_over_mean": a[3] / mean if mean else None,
                "expert_cv": float(per.std() / per.mean()) if per.mean() else None,
                "idle_expert_steps": int(a[4 + 2 * E:4 + 3 * E].sum())}


def ep_dispatch(idx: torch.Tensor, E: int, R: int, rows: torch.Tensor | None = None,
                stream=None) -> dict:
    """Expert-parallel dispatch over R ranks (lmoe_ep_dispatch): pair offsets per rank, the
    token and slot mask of each pair, and (with rows, bf16 [T, W]) each pair's row."""
    T, K = idx.shape
    _expect(idx, torch.int32, (T, K), "idx")
    dev = idx.device
    pmax = T * min(K, R)
    W = 0
    if rows is not None:
        W = rows.shape[1]
        _expect(rows, torch.bfloat16, (T, W), "rows")
    ws_bytes = int(load().lmoe_ep_workspace_bytes(T, K, E, R))
    if ws_bytes == 0:
        raise LmoeError(LMOE_ERR_UNSUPPORTED, "lmoe_ep_workspace_bytes")
    d = {"ws": torch.empty(ws_bytes, dtype=torch.uint8, device=dev),
         "send_off": torch.empty(R + 1, dtype=torch.int32, device=dev),
         "send_tok": torch.empty(pmax, dtype=torch.int32, device=dev),
         "send_slots": torch.empty(pmax, dtype=torch.int32, device=dev),
         "send_rows": torch.empty((pmax, W), dtype=torch.bfloat16, device=dev) if W else None,
         "E": E, "R": R}
    _check(load().lmoe_ep_dispatch(_ptr(idx), T, K, E, R, _ptr(rows), W, _ptr(d["send_rows"]),
                                   _ptr(d["send_off"]), _ptr(d["send_tok"]), _ptr(d["send_slots"]),
                                   _ptr(d["ws"]), ws_bytes, _stream(stream)), "lmoe_ep_dispatch")
    return d


def ep_combine(idx: torch.Tensor, disp: dict, inv: torch.Tensor, gate: torch.Tensor,
               o: torch.Tensor, stream=None):
    """Expert-parallel combine (lmoe_ep_combine): (part bf16 [pairs, W], u fp32 [T, W])."""
    T, K = idx.shape
    W = o.shape[1]
    _expect(o, torch.bfloat16, (o.shape[0], W), "o")
    _expect(inv, torch.int32, (T, K), "inv")
    _expect(gate, torch.float32, (T, K), "gate")
    part = torch.empty((T * min(K, disp["R"]), W), dtype=torch.bfloat16, device=o.device)
    u = torch.empty((T, W), dtype=torch.float32, device=o.device)
    _check(load().lmoe_ep_combine(_ptr(idx), T, K, disp["E"], disp["R"], _ptr(disp["send_off"]),
                                  _ptr(disp["send_tok"]), _ptr(disp["send_slots"]), _ptr(inv),
                                  _ptr(gate), _ptr(o), W, _ptr(part), _ptr(u), _ptr(disp["ws"]),
                                  _stream(stream)), "lmoe_ep_combine")
    return part, u


def fair_share_rank(T: int, K: int, E: int) -> int:
    """The threshold's rank among a column's T scores (lmoe_fair_share_rank)."""
    k = int(load().lmoe_fair_share_rank(T, K, E))
    if k < 0:
        raise LmoeError(LMOE_ERR_INVALID_ARG, "lmoe_fair_share_rank")
    return k


def threshold_candidates(logits: torch.Tensor, k: int, stream=None) -> torch.Tensor:
    """[k, E] candidates this batch contributes to thresholds solved over several batches
    (lmoe_threshold_candidates)."""
    T, E = logits.shape
    _expect(logits, torch.float32, (T, E), "logits")
    cand = torch.empty((k, E), dtype=torch.float32, device=logits.device)
    _check(load().lmoe_threshold_candidates(_ptr(logits), T, E, k, _ptr(cand), _stream(stream)),
           "lmoe_threshold_candidates")
    return cand


def gather_candidates(cand: torch.Tensor, group=None) -> torch.Tensor:
    """All-gather every rank's [k, E] candidates into [world * k, E], rank order: the one
    exchange of a batch spread over ranks.  torch.distributed moves the bytes."""
    import torch.distributed as dist
    if not dist.is_initialized() or dist.get_world_size(group) == 1:
        return cand
    world = dist.get_world_size(group)
    parts = [torch.empty_like(cand) for _ in range(world)]
    dist.all_gather(parts, cand.contiguous(), group=group)
    return torch.cat(parts, dim=0)


def global_token_count(T: int, device, group=None) -> int:
    """Sum of the ranks' batch sizes."""
    import torch.distributed as dist
    if not dist.is_initialized():
        return T
    dev = device if dist.get_backend(group) == "nccl" else "cpu"
    t = torch.tensor([T], dtype=torch.int64, device=dev)
    dist.all_reduce(t, group=group)
    return int(t.item())


def route(logits: torch.Tensor, tau, K: int, want_scores: bool = False, stream=None):
    """Returns (idx int32 [T,K], gate fp32 [T,K]) and, with want_scores, scores [T,E]."""
    T, E = logits.shape
    _expect(logits, torch.float32, (T, E), "logits")
    if tau is not None:
        _expect(tau, torch.float32, (E,), "tau")
    dev = logits.device
    idx = torch.empty((T, K), dtype=torch.int32, device=dev)
    gate = torch.empty((T, K), dtype=torch.float32, device=dev)
    sc = torch.empty((T, E), dtype=torch.float32, device=dev) if want_scores else None
    _check(load().lmoe_route(_ptr(logits), _ptr(tau), T, E, K, _ptr(idx), _ptr(gate), _ptr(sc),
                             _stream(stream)), "lmoe_route")
    return (idx, gate, sc) if want_scores else (idx, gate)


def gemm_bf16(A: torch.Tensor, B: torch.Tensor, stream=None) -> torch.Tensor:
    """C = A . B^T (fp32) on the tcgen05 GEMM of the library."""
    M, Kd = A.shape
    N = B.shape[0]
    _expect(A, torch.bfloat16, (M, Kd), "A")
    _expect(B, torch.bfloat16, (N, Kd), "B")
    C = torch.empty((M, N), dtype=torch.float32, device=A.device)
    flag = torch.zeros(4, dtype=torch.int32, device=A.device)
    _check(load().lmoe_gemm_bf16(_ptr(A), _ptr(B), _ptr(C), M, N, Kd, _ptr(flag),
                                 _stream(stream)), "lmoe_gemm_bf16")
    return C, flag


def gemm_wgrad_bf16(A: torch.Tensor, B: torch.Tensor, stream=None) -> torch.Tensor:
    """C = A^T . B (fp32) over all rows of token-major A [T, M] and B [T, N], as the backward's
    weight gradients compute it."""
    T, M = A.shape
    N = B.shape[1]
    _expect(A, torch.bfloat16, (T, M), "A")
    _expect(B, torch.bfloat16, (T, N), "B")
    C = torch.empty((M, N), dtype=torch.float32, device=A.device)
    words = torch.zeros(4, dtype=torch.int32, device=A.device)
    _check(load().lmoe_gemm_wgrad_bf16(_ptr(A), _ptr(B), _ptr(C), M, N, T, _ptr(words),
                                       _stream(stream)), "lmoe_gemm_wgrad_bf16")
    return C, words


def last_device_error(workspace: torch.Tensor) -> int:
    return int(load().lmoe_last_device_error(_ptr(workspace)))


# The calls below run for microseconds on the device, so what the host does per call is kept
# small: each argument is looked at once, and the current stream is asked for as the raw handle.
_raw_stream = torch._C._cuda_getCurrentRawStream


def _expect_on(t, dtype, shape, dev, name):
    """_expect, and on device number dev."""
    _expect(t, dtype, shape, name)
    if t.get_device() != dev:
        raise ValueError(f"lmoe: {name} must be on CUDA device {dev}, not {t.device}")


def _rows(t, dtype, rows, cols, dev, name):
    """(address, distance between rows) of a [rows, cols] tensor on device number dev whose rows
    are contiguous."""
    if t.dtype is not dtype or t.shape != (rows, cols):
        _expect(t, dtype, (rows, cols), name)
    if t.get_device() != dev:
        raise ValueError(f"lmoe: {name} must be on CUDA device {dev}, not {t.device}")
    rs, cs = t.stride()
    if cs != 1 and cols > 1:
        raise ValueError(f"lmoe: the rows of {name} must be contiguous")
    return t.data_ptr(), rs if rows > 1 else cols


def _vector(t, n, dev, name):
    """Address of a contiguous fp32 [n] tensor on device number dev."""
    if t.dtype is not torch.float32 or t.shape != (n,):
        _expect(t, torch.float32, (n,), name)
    if t.get_device() != dev:
        raise ValueError(f"lmoe: {name} must be on CUDA device {dev}, not {t.device}")
    if n > 1 and t.stride(0) != 1:
        raise ValueError(f"lmoe: {name} must be contiguous")
    return t.data_ptr()


def _matrices(t, dtype, shape, dev, name):
    """(address, distance between rows, between matrices) of a tensor of the given shape, (rows, cols)
    or (batch, rows, cols), on device number dev, whose rows are contiguous."""
    if t.dtype is not dtype or t.shape != shape:
        _expect(t, dtype, shape, name)
    if t.get_device() != dev:
        raise ValueError(f"lmoe: {name} must be on CUDA device {dev}, not {t.device}")
    s = t.stride()
    if s[-1] != 1 and shape[-1] > 1:
        raise ValueError(f"lmoe: the rows of {name} must be contiguous")
    return (t.data_ptr(), s[-2] if shape[-2] > 1 else shape[-1],
            s[0] if len(shape) == 3 and shape[0] > 1 else shape[-2] * shape[-1])


def _on(dev):
    """Device dev's current stream, dev being the current device.  (A call on another stream makes
    that the current one first, so that what it allocates belongs to that stream too.)"""
    if dev != torch.cuda.current_device():
        raise ValueError(f"lmoe: tensors on CUDA device {dev}, but the current device is "
                         f"{torch.cuda.current_device()}")
    return _raw_stream(dev)


def _device_of(t, name):
    dev = t.get_device()
    if dev < 0:
        raise ValueError(f"lmoe: {name} must be a CUDA device tensor")
    return dev


def _add_rmsnorm(x, gamma, residual, eps, fp8, train, y, total):
    rows, cols = x.shape
    bf, f, device = torch.bfloat16, torch.float32, x.device
    dev = _device_of(x, "x")
    px, ldx = _rows(x, bf, rows, cols, dev, "x")
    pg = _vector(gamma, cols, dev, "gamma")
    pr = pt = ps = pi = None
    ldr = ldt = 0
    if residual is not None:
        pr, ldr = _rows(residual, bf, rows, cols, dev, "residual")
    # (without a residual total is x, unless y is written over it)
    if total is None and (residual is not None or (y is not None and y.data_ptr() == px)):
        total = torch.empty((rows, cols), dtype=bf, device=device)
        pt, ldt = total.data_ptr(), cols
    if total is not None and pt is None:
        pt, ldt = _rows(total, bf, rows, cols, dev, "total")
    if y is None:
        y = torch.empty((rows, cols), dtype=torch.uint8 if fp8 else bf, device=device)
        py, ldy = y.data_ptr(), cols
    else:
        py, ldy = _rows(y, bf, rows, cols, dev, "y")
    scales = rstd = None
    if fp8:
        scales = torch.empty(rows, dtype=f, device=device)
        ps = scales.data_ptr()
    if train:
        rstd = torch.empty(rows, dtype=f, device=device)
        pi = rstd.data_ptr()
    rc = load().lmoe_add_rmsnorm(px, ldx, pr, ldr, pg, rows, cols, eps, py, ldy,
                                 E4M3 if fp8 else BF16, ps, pt, ldt, pi, _on(dev))
    if rc:
        _check(rc, "lmoe_add_rmsnorm")
    return y, scales, x if total is None else total, rstd


def add_rmsnorm(x: torch.Tensor, gamma: torch.Tensor, residual: torch.Tensor | None = None,
                eps: float = 1e-6, train: bool = False, y=None, total=None, stream=None):
    """Residual addition with RMSNorm (lmoe_add_rmsnorm): x and residual [rows, cols] bf16
    (rows contiguous, at any stride), gamma [cols] fp32 -> (y, total), or with train
    (y, total, rstd) for add_rmsnorm_backward.  total is x + residual in bf16 (without a residual
    x itself, or a copy where y is written over x); ``y`` and ``total`` may be given, and may be
    x or residual."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return add_rmsnorm(x, gamma, residual, eps, train, y, total)
    y, _, total, rstd = _add_rmsnorm(x, gamma, residual, eps, False, train, y, total)
    return (y, total, rstd) if train else (y, total)


def add_rmsnorm_e4m3(x: torch.Tensor, gamma: torch.Tensor, residual: torch.Tensor | None = None,
                     eps: float = 1e-6, total=None, stream=None):
    """add_rmsnorm with y as e4m3 codes (uint8) and one fp32 scale per row:
    (codes, scales, total)."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return add_rmsnorm_e4m3(x, gamma, residual, eps, total)
    return _add_rmsnorm(x, gamma, residual, eps, True, False, None, total)[:3]


def add_rmsnorm_backward(dy: torch.Tensor, total: torch.Tensor, gamma: torch.Tensor,
                         rstd: torch.Tensor, dtotal: torch.Tensor | None = None,
                         want_dgamma: bool = True, dx=None, stream=None):
    """Gradients of add_rmsnorm (lmoe_add_rmsnorm_backward): dy, and dtotal (the gradient that
    reaches total itself, or None), [rows, cols] bf16 -> (dx bf16, dgamma fp32 or None); dx is
    the gradient of x and of residual.  ``norm_device_error`` reports a device-side wait that ran
    out (the gradients are then NaN)."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return add_rmsnorm_backward(dy, total, gamma, rstd, dtotal, want_dgamma, dx)
    rows, cols = dy.shape
    bf, f, device = torch.bfloat16, torch.float32, dy.device
    dev = _device_of(dy, "dy")
    pd, ldy = _rows(dy, bf, rows, cols, dev, "dy")
    pt, ldt = _rows(total, bf, rows, cols, dev, "total")
    pe, lde = (None, 0) if dtotal is None else _rows(dtotal, bf, rows, cols, dev, "dtotal")
    pg = _vector(gamma, cols, dev, "gamma")
    pi = _vector(rstd, rows, dev, "rstd")
    if dx is None:
        dx = torch.empty((rows, cols), dtype=bf, device=device)
    po, ldo = _rows(dx, bf, rows, cols, dev, "dx")
    lib = load()
    dgamma = pm = pw = None
    nb = 0
    if want_dgamma:
        dgamma = torch.empty(cols, dtype=f, device=device)
        nb = lib.lmoe_add_rmsnorm_backward_workspace_bytes(rows, cols)
        ws = torch.empty(nb, dtype=torch.uint8, device=device)
        pm, pw = dgamma.data_ptr(), ws.data_ptr()
    rc = lib.lmoe_add_rmsnorm_backward(pd, ldy, pt, ldt, pg, pi, pe, lde, rows, cols, po, ldo, pm,
                                       pw, nb, _on(dev))
    if rc:
        _check(rc, "lmoe_add_rmsnorm_backward")
    return dx, dgamma


def norm_device_error() -> int:
    """LMOE_OK, or LMOE_ERR_DEVICE_TIMEOUT if a device-side wait of an earlier add_rmsnorm_backward on
    the current device ran out; call after its stream has synchronised.  Clears the word."""
    return int(load().lmoe_norm_last_device_error())


class Linear:
    """A linear layer with a fused epilogue (lmoe_linear_forward / _backward):
    y = act(x w^T + bias) + residual.

    w [N, K] bf16, or e4m3 codes (uint8) with fp32 ``w_scales`` [N] (forward only); bias [N] fp32
    or None; act "none", "silu", "gelu" or "situ" (then w, bias and w_scales hold the N gate rows,
    then the N value rows, and c is the cap).  N must be a multiple of 8, K of 8 (e4m3: 16).

    The layer keeps references, not copies, and looks at them at each call: w, bias and w_scales may be
    updated in place, given other storage or replaced by tensors of the same sizes and type, on the
    same device; c may be changed, and bias taken away or added."""

    def __init__(self, w: torch.Tensor, bias: torch.Tensor | None = None, act: str = "none",
                 w_scales: torch.Tensor | None = None, c: float = 100.0):
        if act not in ACTS:
            raise ValueError(f"lmoe: unknown activation {act!r}")
        rows, K = w.shape
        if act == "situ" and rows % 2:
            raise ValueError("lmoe: a gated layer needs as many value rows as gate rows")
        self.fp8 = w.dtype is torch.uint8
        if self.fp8 != (w_scales is not None):
            raise ValueError("lmoe: e4m3 codes (uint8) and w_scales go together")
        self.w, self.bias, self.w_scales, self._act, self.c = w, bias, w_scales, act, c
        self.rows, self.K, self.N = rows, K, rows // 2 if act == "situ" else rows
        self.device, self._dev = w.device, _device_of(w, "w")
        self._dtype = torch.uint8 if self.fp8 else torch.bfloat16
        self._sizes = (self.N, K, ACTS[act], E4M3 if self.fp8 else BF16)
        self._weights()
        self.flag = torch.zeros(1, dtype=torch.int32, device=w.device)
        torch.cuda.current_stream(w.device).synchronize()  # before any stream of the caller's
        self._flag = self.flag.data_ptr()

    @property
    def act(self) -> str:
        return self._act

    def _weights(self):
        """(w, its row distance, scales, bias) as they are now."""
        pw, ldw = _rows(self.w, self._dtype, self.rows, self.K, self._dev, "w")
        pws = pb = None
        if self.fp8:
            if self.w_scales is None:
                raise ValueError("lmoe: e4m3 codes (uint8) and w_scales go together")
            pws = _vector(self.w_scales, self.rows, self._dev, "w_scales")
        elif self.w_scales is not None:
            raise ValueError("lmoe: e4m3 codes (uint8) and w_scales go together")
        if self.bias is not None:
            pb = _vector(self.bias, self.rows, self._dev, "bias")
        return pw, ldw, pws, pb

    def _desc(self, M, px, ldx, pxs, pr, ldr, py, ldy, pp, ldp):
        return ctypes.byref(LinearDesc(M, *self._sizes, self.c, px, ldx, pxs, *self._weights(), pr,
                                       ldr, py, ldy, pp, ldp, self._flag))

    def forward(self, x: torch.Tensor, residual: torch.Tensor | None = None,
                x_scales: torch.Tensor | None = None, train: bool = False, y=None, stream=None):
        """x [M, K] bf16 (or e4m3 codes with x_scales [M]), residual [M, N] bf16 -> y [M, N] bf16;
        with train, (y, pre), the bf16 pre-activations that ``backward`` needs (None without an
        activation).  Rows at any stride of whole 16 bytes.  ``y`` may be given (or be residual)."""
        if stream is not None:
            with torch.cuda.stream(stream):
                return self.forward(x, residual, x_scales, train, y)
        M, N, dev = x.shape[0], self.N, self._dev
        bf = torch.bfloat16
        px, ldx = _rows(x, self._dtype, M, self.K, dev, "x")
        pxs = pr = pp = pre = None
        ldr = 0
        if self.fp8:
            if x_scales is None:
                raise ValueError("lmoe: e4m3 rows need x_scales")
            pxs = _vector(x_scales, M, dev, "x_scales")
        elif x_scales is not None:
            raise ValueError("lmoe: x_scales belong to e4m3 rows")
        if residual is not None:
            pr, ldr = _rows(residual, bf, M, N, dev, "residual")
        if y is None:
            y = torch.empty((M, N), dtype=bf, device=self.device)
            py, ldy = y.data_ptr(), N
        else:
            py, ldy = _rows(y, bf, M, N, dev, "y")
        if train and self.act != "none":
            pre = torch.empty((M, self.rows), dtype=bf, device=self.device)
            pp = pre.data_ptr()
        rc = load().lmoe_linear_forward(self._desc(M, px, ldx, pxs, pr, ldr, py, ldy, pp, self.rows),
                                        _on(dev))
        if rc:
            _check(rc, "lmoe_linear_forward")
        return (y, pre) if train else y

    def backward(self, x: torch.Tensor, dy: torch.Tensor, pre: torch.Tensor | None = None,
                 dw_dtype=torch.float32, want_dx: bool = True, want_dw: bool = True,
                 stream=None) -> dict:
        """Gradients for the x and pre of a ``forward(train=True)``: dy [M, N] bf16 -> dx [M, K]
        bf16, dw (fp32, or bf16 with dw_dtype) and, when the layer has a bias, dbias fp32.  The
        residual's gradient is dy itself."""
        if stream is not None:
            with torch.cuda.stream(stream):
                return self.backward(x, dy, pre, dw_dtype, want_dx, want_dw)
        M, dev = dy.shape[0], self._dev
        bf, f = torch.bfloat16, torch.float32
        if self.fp8:
            raise LmoeError(LMOE_ERR_UNSUPPORTED, "lmoe_linear_backward")
        if dw_dtype not in (bf, f):
            raise ValueError("lmoe: dw_dtype must be torch.float32 or torch.bfloat16")
        px, ldx = _rows(x, bf, M, self.K, dev, "x")
        pd, ldd = _rows(dy, bf, M, self.N, dev, "dy")
        pp, ldp = None, 0
        if self.act != "none":
            if pre is None:
                raise ValueError("lmoe: this layer's backward needs the forward's pre")
            pp, ldp = _rows(pre, bf, M, self.rows, dev, "pre")
        dx = dw = db = pdx = pdw = pdb = None
        if want_dx:
            dx = torch.empty((M, self.K), dtype=bf, device=self.device)
            pdx = dx.data_ptr()
        if want_dw:
            dw = torch.empty((self.rows, self.K), dtype=dw_dtype, device=self.device)
            pdw = dw.data_ptr()
        if self.bias is not None:
            db = torch.empty(self.rows, dtype=f, device=self.device)
            pdb = db.data_ptr()
        lib = load()
        d = self._desc(M, px, ldx, None, None, 0, None, 0, pp, ldp)
        nb = lib.lmoe_linear_backward_workspace_bytes(d)
        ws = torch.empty(nb, dtype=torch.uint8, device=self.device)
        rc = lib.lmoe_linear_backward(d, pd, ldd, pdx, self.K, pdw, F32 if dw_dtype is f else BF16,
                                      pdb, ws.data_ptr(), nb, _on(dev))
        if rc:
            _check(rc, "lmoe_linear_backward")
        return {"dx": dx, "dw": dw, "dbias": db}

    def device_error(self) -> int:
        """LMOE_OK, or LMOE_ERR_DEVICE_TIMEOUT if a device-side wait of an earlier call ran out
        (its output is not valid); call after the stream has synchronised.  Clears the flag."""
        return last_device_error(self.flag)


class LinearCrossEntropy:
    """The softmax cross entropy of a linear head w [V, K] bf16 over V tokens, and its gradients,
    without logits in memory (lmoe_linear_xent_forward / _backward).  K must be a multiple of 8.

    Like ``Linear`` it keeps a reference to w and looks at it at each call: w may be updated in place
    or replaced by a tensor of the same size and type on the same device."""

    def __init__(self, w: torch.Tensor):
        self.w = w
        self.V, self.K = w.shape
        self.device, self._dev = w.device, _device_of(w, "w")
        _rows(w, torch.bfloat16, self.V, self.K, self._dev, "w")
        self.flag = torch.zeros(1, dtype=torch.int32, device=w.device)
        torch.cuda.current_stream(w.device).synchronize()  # before any stream of the caller's
        self._flag = self.flag.data_ptr()

    def _desc(self, x, target, loss, lse):
        dev, M = self._dev, x.shape[0]
        px, ldx = _rows(x, torch.bfloat16, M, self.K, dev, "x")
        pw, ldw = _rows(self.w, torch.bfloat16, self.V, self.K, dev, "w")
        if target.dtype not in (torch.int32, torch.int64):
            raise ValueError(f"lmoe: target must be torch.int32 or torch.int64, not {target.dtype}")
        _expect_on(target, target.dtype, (M,), dev, "target")
        if M > 1 and target.stride(0) != 1:
            raise ValueError("lmoe: target must be contiguous")
        return ctypes.byref(LinearXentDesc(
            M, self.V, self.K, px, ldx, pw, ldw, target.data_ptr(),
            I64 if target.dtype is torch.int64 else I32, loss, lse, self._flag))

    def forward(self, x: torch.Tensor, target: torch.Tensor, stream=None):
        """x [M, K] bf16 (rows at any stride of whole 16 bytes), target [M] int64 or int32 -> (loss,
        lse), both [M] fp32: of each row, the target's negative log-probability and the logarithm of
        the sum that it is divided by, which ``backward`` needs.  A row whose target is outside
        0 .. V-1 has loss 0."""
        if stream is not None:
            with torch.cuda.stream(stream):
                return self.forward(x, target)
        M = x.shape[0]
        loss = torch.empty(M, dtype=torch.float32, device=self.device)
        lse = torch.empty(M, dtype=torch.float32, device=self.device)
        d = self._desc(x, target, loss.data_ptr(), lse.data_ptr())
        lib = load()
        nb = lib.lmoe_linear_xent_workspace_bytes(d)
        ws = torch.empty(nb, dtype=torch.uint8, device=self.device)
        rc = lib.lmoe_linear_xent_forward(d, ws.data_ptr(), nb, _on(self._dev))
        if rc:
            _check(rc, "lmoe_linear_xent_forward")
        return loss, lse

    def backward(self, x: torch.Tensor, target: torch.Tensor, lse: torch.Tensor,
                 dloss: torch.Tensor, dw_dtype=torch.float32, want_dx: bool = True,
                 want_dw: bool = True, stream=None) -> dict:
        """Gradients for the x, target and lse of a ``forward``: dloss [M] fp32, the gradient of each
        row's loss -> dx [M, K] bf16, dw [V, K] (fp32, or bf16 with dw_dtype).  Rows without a target
        have none, whatever x, lse and dloss hold there."""
        if stream is not None:
            with torch.cuda.stream(stream):
                return self.backward(x, target, lse, dloss, dw_dtype, want_dx, want_dw)
        M, dev = x.shape[0], self._dev
        bf, f = torch.bfloat16, torch.float32
        if dw_dtype not in (bf, f):
            raise ValueError("lmoe: dw_dtype must be torch.float32 or torch.bfloat16")
        pg = _vector(dloss, M, dev, "dloss")
        d = self._desc(x, target, None, _vector(lse, M, dev, "lse"))
        dx = dw = pdx = pdw = None
        if want_dx:
            dx = torch.empty((M, self.K), dtype=bf, device=self.device)
            pdx = dx.data_ptr()
        if want_dw:
            dw = torch.empty((self.V, self.K), dtype=dw_dtype, device=self.device)
            pdw = dw.data_ptr()
        lib = load()
        nb = lib.lmoe_linear_xent_backward_workspace_bytes(d)
        ws = torch.empty(nb, dtype=torch.uint8, device=self.device)
        rc = lib.lmoe_linear_xent_backward(d, pg, pdx, self.K, pdw, F32 if dw_dtype is f else BF16,
                                           ws.data_ptr(), nb, _on(dev))
        if rc:
            _check(rc, "lmoe_linear_xent_backward")
        return {"dx": dx, "dw": dw}

    def device_error(self) -> int:
        """LMOE_OK, or LMOE_ERR_DEVICE_TIMEOUT if a device-side wait of an earlier call ran out
        (its output is not valid); call after the stream has synchronised.  Clears the flag."""
        return last_device_error(self.flag)


class Muon:
    """Orthogonalised updates of weights (lmoe_orthogonalize, lmoe_muon_update): Newton-Schulz
    iterations of ``steps`` steps with coefficients ``coeffs``, one triple for all of them or one for
    each.  Matrices are [rows, cols], or [batch, rows, cols] of which each is taken by itself (experts,
    heads), with contiguous rows at any distance: the gradients of ``Layer.backward_layer`` and
    ``Linear.backward`` go in as they are.  The object keeps no state of the weights: momentum is the
    caller's."""

    def __init__(self, beta: float = 0.95, nesterov: bool = True, weight_decay: float = 0.0,
                 steps: int = 5, coeffs=(3.4445, -4.7750, 2.0315), eps: float = 1e-7, device=None):
        c = torch.as_tensor(coeffs, dtype=torch.float32)
        if c.shape not in ((3,), (steps, 3)) or not 1 <= steps <= MUON_MAX_STEPS:
            raise ValueError(f"lmoe: 1 to {MUON_MAX_STEPS} steps, and a triple of coefficients for all "
                             "of them or for each")
        self.beta, self.nesterov, self.weight_decay = beta, nesterov, weight_decay
        self.steps, self.eps = steps, eps
        self._coeffs = (_f * (3 * steps))(*c.expand(steps, 3).flatten().tolist())
        self._coeffs_ptr = ctypes.cast(self._coeffs, _vp)
        self.device = torch.device("cuda", torch.cuda.current_device()) if device is None \
            else torch.device(device)
        self.flag = torch.zeros(1, dtype=torch.int32, device=self.device)
        self.device = self.flag.device
        torch.cuda.current_stream(self.device).synchronize()  # before any stream of the caller's
        self._dev, self._flag = self.flag.get_device(), self.flag.data_ptr()

    def _desc(self, grad):
        if grad.dtype not in (torch.bfloat16, torch.float32):
            raise ValueError(f"lmoe: grad must be torch.bfloat16 or torch.float32, not {grad.dtype}")
        shape = tuple(grad.shape)
        if len(shape) not in (2, 3):
            raise ValueError(f"lmoe: grad must be [rows, cols] or [batch, rows, cols], not {shape}")
        d = MuonDesc()
        d.batch, d.rows, d.cols = (1, *shape) if len(shape) == 2 else shape
        d.steps, d.coeffs, d.eps, d.dev_flag = self.steps, self._coeffs_ptr, self.eps, self._flag
        d.grad, d.ldg, d.grad_stride = _matrices(grad, grad.dtype, shape, self._dev, "grad")
        d.grad_type = F32 if grad.dtype is torch.float32 else BF16
        return d, shape

    def _call(self, name, d):
        lib, ref = load(), ctypes.byref(d)
        nb = lib.lmoe_muon_workspace_bytes(ref)
        ws = torch.empty(nb, dtype=torch.uint8, device=self.device)
        rc = getattr(lib, name)(ref, ws.data_ptr(), nb, _on(self._dev))
        if rc:
            _check(rc, name)

    def orthogonalize(self, grad: torch.Tensor, out=None, stream=None) -> torch.Tensor:
        """grad, bf16 or fp32 -> its orthogonalisation in bf16 (``out``, which may be grad itself)."""
        if stream is not None:
            with torch.cuda.stream(stream):
                return self.orthogonalize(grad, out)
        d, shape = self._desc(grad)
        if out is None:
            out = torch.empty(shape, dtype=torch.bfloat16, device=self.device)
        d.out, d.ldo, d.out_stride = _matrices(out, torch.bfloat16, shape, self._dev, "out")
        self._call("lmoe_orthogonalize", d)
        return out

    def update(self, w: torch.Tensor | None, grad: torch.Tensor, momentum: torch.Tensor,
               rate: float, scale: float = 1.0, master: torch.Tensor | None = None, stream=None):
        """One step, in place: momentum (fp32) = beta momentum + grad, then
        w = w (1 - rate weight_decay) - rate scale X, X the orthogonalisation of grad + beta momentum
        (or of momentum, without nesterov).  w is bf16; with an fp32 ``master`` that is what is updated,
        and w, or None, receives its rounding.  Rate and scale are numbers of the call: a graph that has
        captured it replays them, and is captured anew where a schedule changes them."""
        if stream is not None:
            with torch.cuda.stream(stream):
                return self.update(w, grad, momentum, rate, scale, master)
        d, shape = self._desc(grad)
        f = torch.float32
        d.momentum, d.ldm, d.momentum_stride = _matrices(momentum, f, shape, self._dev, "momentum")
        if w is None and master is None:
            raise ValueError("lmoe: an update needs w or master")
        if w is not None:
            d.w, d.ldw, d.w_stride = _matrices(w, torch.bfloat16, shape, self._dev, "w")
        if master is not None:
            d.master, d.ldmaster, d.master_stride = _matrices(master, f, shape, self._dev, "master")
        d.beta, d.nesterov, d.weight_decay = self.beta, int(self.nesterov), self.weight_decay
        d.rate, d.scale = rate, scale
        self._call("lmoe_muon_update", d)

    def device_error(self) -> int:
        """LMOE_OK, or LMOE_ERR_DEVICE_TIMEOUT if a device-side wait of an earlier call ran out
        (its output is not valid); call after the stream has synchronised.  Clears the flag."""
        return last_device_error(self.flag)


class Layer:
    """One Stable Latent MoE layer on the device: packed weights + a workspace sized for up
    to ``max_tokens`` tokens.  ``forward`` is one lmoe_forward call."""

    def __init__(self, shape, weights: dict, max_tokens: int | None = None, stream=None,
                 overlap: bool = False, shared_sms: int = 0, expert_fp8: bool = False):
        """overlap: run the shared experts on an auxiliary stream beside the routed path for
        batches of at least OVERLAP_MIN_T tokens (shared_sms SMs for them; 0 = a third).
        Off by default: the routed expert GEMMs are limited per SM, so the SMs lent to the
        shared experts slow them down more than the concurrency gains.
        expert_fp8: routed experts with e4m3 operands (weights quantised when packed)."""
        self.shape = shape
        self.expert_fp8 = expert_fp8
        self.max_tokens = shape.T if max_tokens is None else max_tokens
        self.dims = dims_of(shape, T=self.max_tokens, expert_fp8=expert_fp8)
        self.device = weights["w_down"].device
        self.packed = pack_weights(self.dims, weights, stream)
        self.ws_bytes = workspace_bytes(self.dims)
        self.workspace = torch.empty(self.ws_bytes, dtype=torch.uint8, device=self.device)
        self.few_ws = None  # forward_few's, allocated by its first call
        self.overlap = overlap
        self.shared_sms = shared_sms
        self.aux_stream = torch.cuda.Stream(device=self.device) if overlap else None
        self.aux_events = []
        if overlap:
            for _ in range(2):
                ev = torch.cuda.Event()
                ev.record(torch.cuda.current_stream(self.device))  # create the event now
                self.aux_events.append(ev)

    def forward(self, x: torch.Tensor, residual: torch.Tensor | None = None, y=None,
                tau: torch.Tensor | None = None, balance: bool = True,
                logits_in: torch.Tensor | None = None, debug: bool = False, stream=None,
                stage_events=None, phase: int = PHASE_ALL, cand_k: int = 0,
                tau_ema: torch.Tensor | None = None, ema_beta: float = 0.9,
                ema_first: bool = False, load_stats: "LoadStats | None" = None,
                train: bool = False, logit_bias: torch.Tensor | None = None):
        """One lmoe_forward call.  stage_events: optional list of NUM_STAGES + 1
        torch.cuda.Event(enable_timing=True) recorded at the stage boundaries.  After the
        call, ``self.last_kernel_launches`` holds the number of kernels it launched.
        phase: PHASE_ALL, or one half of the layer: PHASE_ROUTER (returns the [cand_k, E]
        threshold candidates when cand_k > 0, else None) then PHASE_EXPERTS (x gives the
        batch size only).  tau_ema: [E] streaming thresholds, updated in place with this
        batch's (ema_beta, ema_first) and routed against.  load_stats: a LoadStats that this
        step's per-expert counts are added to.  train: also keep the routed experts'
        pre-activations (lmoe_io.save_pre) for the next ``backward`` / ``backward_layer``
        (needs ``enable_backward``).  logit_bias: [E] fp32 added to the router logits the
        layer computes (lmoe_io.logit_bias)."""
        sh = self.shape
        T = x.shape[0]
        if T > self.max_tokens:
            raise ValueError(f"lmoe: {T} tokens exceed the workspace's {self.max_tokens}")
        _expect(x, torch.bfloat16, (T, sh.d), "x")
        if residual is not None:
            _expect(residual, torch.bfloat16, (T, sh.d), "residual")
        if y is None:
            y = torch.empty((T, sh.d), dtype=torch.bfloat16, device=x.device)
        dims = dims_of(sh, T=T, expert_fp8=self.expert_fp8)
        io = IO()
        io.balance = 1 if balance else 0
        io.phase = phase
        cand = None
        if phase == PHASE_ROUTER and cand_k > 0:
            cand = torch.empty((cand_k, sh.E), dtype=torch.float32, device=x.device)
            io.cand_out = _ptr(cand)
            io.cand_k = cand_k
        if self.overlap and T >= OVERLAP_MIN_T and T <= self.max_tokens:
            io.aux_stream = ctypes.c_void_p(self.aux_stream.cuda_stream)
            io.aux_events[0] = self.aux_events[0].cuda_event
            io.aux_events[1] = self.aux_events[1].cuda_event
            io.shared_sms = self.shared_sms
        dbg = {}
        if tau is not None:
            _expect(tau, torch.float32, (sh.E,), "tau")
            io.tau_in = _ptr(tau)
        if logits_in is not None:
            _expect(logits_in, torch.float32, (T, sh.E), "logits_in")
            io.logits_in = _ptr(logits_in)
        if logit_bias is not None:
            _expect(logit_bias, torch.float32, (sh.E,), "logit_bias")
            io.logit_bias = _ptr(logit_bias)
        if tau_ema is not None:
            _expect(tau_ema, torch.float32, (sh.E,), "tau_ema")
            io.tau_ema = _ptr(tau_ema)
            io.ema_beta = ema_beta
            io.ema_first = 1 if ema_first else 0
        if load_stats is not None:
            io.load_stats = _ptr(load_stats.acc)
        self._pre_rows = None
        if train:
            if getattr(self, "pre_buf", None) is None:
                raise RuntimeError("lmoe: forward(train=True) needs enable_backward() first")
            io.save_pre = _ptr(self.pre_buf)
            if self.pre_shared_buf is not None:
                io.save_pre_shared = _ptr(self.pre_shared_buf)
            self._pre_rows = T
        if debug:
            dev = x.device
            dbg["logits"] = torch.empty((T, sh.E), dtype=torch.float32, device=dev)
            dbg["tau"] = torch.empty(sh.E, dtype=torch.float32, device=dev)
            dbg["idx"] = torch.empty((T, sh.K), dtype=torch.int32, device=dev)
            dbg["gate"] = torch.empty((T, sh.K), dtype=torch.float32, device=dev)
            dbg["counts"] = torch.empty(sh.E, dtype=torch.int32, device=dev)
            if phase != PHASE_ROUTER:
                # the output before its bf16 store (y is this, rounded to nearest even)
                dbg["y_f32"] = torch.empty((T, sh.d), dtype=torch.float32, device=dev)
                io.y_f32_out = _ptr(dbg["y_f32"])
            io.logits_out = _ptr(dbg["logits"])
            io.tau_out = _ptr(dbg["tau"])
            io.idx_out = _ptr(dbg["idx"])
            io.gate_out = _ptr(dbg["gate"])
            io.counts_out = _ptr(dbg["counts"])
        if stage_events is not None:
            if len(stage_events) != NUM_STAGES + 1:
                raise ValueError(f"lmoe: need {NUM_STAGES + 1} stage events")
            handles = []
            for ev in stage_events:
                if not ev.cuda_event:      # torch creates its events lazily
                    ev.record(torch.cuda.current_stream() if stream is None else stream)
                handles.append(ev.cuda_event)
            arr = (_vp * len(handles))(*handles)
            io.stage_events = ctypes.cast(arr, ctypes.POINTER(_vp))
        _check(load().lmoe_forward(ctypes.byref(dims), _ptr(self.packed), _ptr(x), _ptr(residual),
                                   _ptr(y), _ptr(self.workspace), self.ws_bytes,
                                   ctypes.byref(io), _stream(stream)), "lmoe_forward")
        self.last_kernel_launches = io.kernel_launches
        if phase == PHASE_ROUTER:
            return (cand, dbg) if debug else cand
        return (y, dbg) if debug else y

    def forward_few(self, x: torch.Tensor, residual: torch.Tensor | None = None, y=None,
                    tau: torch.Tensor | None = None, logits_in: torch.Tensor | None = None,
                    logit_bias: torch.Tensor | None = None, debug: bool = False, stream=None):
        """The layer on at most FEW_MAX_TOKENS tokens in one kernel (lmoe_forward_few), routed
        against thresholds ``tau`` (e.g. a prefill batch's) or none.  Arguments and debug outputs
        (logits, idx, gate, y_f32) as ``forward``'s.  The first call allocates a workspace of its
        own for up to min(max_tokens, FEW_MAX_TOKENS) tokens; make it before capturing a graph."""
        if stream is not None:
            with torch.cuda.stream(stream):
                return self.forward_few(x, residual, y, tau, logits_in, logit_bias, debug)
        sh = self.shape
        T = x.shape[0]
        bf, f = torch.bfloat16, torch.float32
        lib = load()
        if self.few_ws is None:
            self._prepare_few(lib)
        if T >= len(self._few_dims):
            raise ValueError(f"lmoe: {T} tokens exceed forward_few's {len(self._few_dims) - 1}")
        dims = self._few_dims[T]
        dev = self.device.index
        _expect_on(x, bf, (T, sh.d), dev, "x")
        if residual is not None:
            _expect_on(residual, bf, (T, sh.d), dev, "residual")
        if y is None:
            y = torch.empty((T, sh.d), dtype=bf, device=self.device)
        else:
            _expect_on(y, bf, (T, sh.d), dev, "y")
        io = IO()
        if tau is not None:
            _expect_on(tau, f, (sh.E,), dev, "tau")
            io.tau_in = _ptr(tau)
        if logits_in is not None:
            _expect_on(logits_in, f, (T, sh.E), dev, "logits_in")
            io.logits_in = _ptr(logits_in)
        if logit_bias is not None:
            _expect_on(logit_bias, f, (sh.E,), dev, "logit_bias")
            io.logit_bias = _ptr(logit_bias)
        dbg = {}
        if debug:
            dbg = {"logits": torch.empty((T, sh.E), dtype=f, device=self.device),
                   "idx": torch.empty((T, sh.K), dtype=torch.int32, device=self.device),
                   "gate": torch.empty((T, sh.K), dtype=f, device=self.device),
                   "y_f32": torch.empty((T, sh.d), dtype=f, device=self.device)}
            io.logits_out, io.idx_out = _ptr(dbg["logits"]), _ptr(dbg["idx"])
            io.gate_out, io.y_f32_out = _ptr(dbg["gate"]), _ptr(dbg["y_f32"])
        st = _on(dev)
        _check(lib.lmoe_forward_few(ctypes.byref(dims), _ptr(self.packed), _ptr(x), _ptr(residual),
                                    _ptr(y), _ptr(self.few_ws), self.few_ws.numel(),
                                    ctypes.byref(io), st), "lmoe_forward_few")
        self.last_kernel_launches = io.kernel_launches
        return (y, dbg) if debug else y

    def _prepare_few(self, lib):
        """forward_few's sizes and workspace, once, whichever host thread comes first."""
        with _lock:
            if self.few_ws is not None:
                return
            dims = [dims_of(self.shape, T=t, expert_fp8=self.expert_fp8)
                    for t in range(min(self.max_tokens, FEW_MAX_TOKENS) + 1)]
            sizes = [int(lib.lmoe_few_workspace_bytes(ctypes.byref(D))) for D in dims]
            while len(sizes) > 1 and sizes[-1] == 0:  # operands too wide for an SM's shared memory
                sizes.pop()
            if sizes[-1] == 0:
                raise LmoeError(LMOE_ERR_UNSUPPORTED, "lmoe_few_workspace_bytes")
            if torch.cuda.is_current_stream_capturing():  # the graph's memory, zeroed at its replay
                raise ValueError("lmoe: forward_few's first call allocates its workspace: make it "
                                 "before capturing a graph")
            ws = torch.zeros(sizes[-1], dtype=torch.uint8, device=self.device)
            torch.cuda.current_stream(self.device).synchronize()  # before any stream uses it
            self._few_dims, self.few_ws = dims[:len(sizes)], ws  # few_ws last: it says that all is there

    def few_device_error(self) -> int:
        """device_error of forward_few's workspace (call after the stream has synchronised)."""
        return LMOE_OK if self.few_ws is None else last_device_error(self.few_ws)

    def forward_global(self, x: torch.Tensor, residual: torch.Tensor | None = None, y=None,
                       group=None, global_tokens: int | None = None, debug: bool = False,
                       stage_events=None):
        """The layer on this rank's part of a batch spread over the ranks of ``group``, with
        one set of Quantile-Balancing thresholds solved over the whole batch: router phase
        with candidates, all-gather of the candidates, lmoe_thresholds on them, experts
        phase.  Runs on the current stream (the collectives order against it)."""
        sh = self.shape
        T = x.shape[0]
        Tg = global_token_count(T, x.device, group) if global_tokens is None else global_tokens
        if Tg == 0:  # every rank's part is empty
            return self.forward(x, residual, y, debug=debug)
        k = fair_share_rank(Tg, sh.K, sh.E)
        r = self.forward(x, phase=PHASE_ROUTER, cand_k=k, debug=debug, stage_events=stage_events)
        launches = self.last_kernel_launches
        cand, dbg0 = r if debug else (r, None)
        tau = thresholds(gather_candidates(cand, group), sh.K, k_rank=k)
        out = self.forward(x, residual, y, tau=tau, phase=PHASE_EXPERTS, debug=debug,
                           stage_events=stage_events)
        self.last_kernel_launches += launches + 1
        if debug:
            out[1]["logits"] = dbg0["logits"]
            out[1]["candidates"] = cand
        return out

    def forward_host(self, x_host: torch.Tensor, y_host: torch.Tensor, x_dev: torch.Tensor,
                     y_dev: torch.Tensor, residual_from_x: bool = True, stream=None,
                     qb: str = "local", **kw):
        """End-to-end call from host memory: copy x (pinned host) to the device, run the
        layer, copy y back to pinned host memory; all on one stream, asynchronous.  Extra
        keyword arguments go to ``forward`` (tau, balance, logits_in), or, with
        qb="global", to ``forward_global`` (group, global_tokens)."""
        x_dev.copy_(x_host, non_blocking=True)
        resid = x_dev if residual_from_x else None
        if qb == "global":
            self.forward_global(x_dev, resid, y=y_dev, **kw)
        else:
            self.forward(x_dev, residual=resid, y=y_dev, stream=stream, **kw)
        y_host.copy_(y_dev, non_blocking=True)
        return y_host

    def device_error(self) -> int:
        return last_device_error(self.workspace)

    def enable_backward(self, weights: dict, stream=None):
        """Pack the transposed weights and allocate the scratch of ``backward`` and
        ``backward_layer``."""
        D = self.dims
        nb = int(load().lmoe_packed_backward_bytes(ctypes.byref(D)))
        if nb == 0:
            raise LmoeError(LMOE_ERR_UNSUPPORTED, "lmoe_packed_backward_bytes")
        self.packed_bwd = torch.empty(nb, dtype=torch.uint8, device=self.device)
        W = Weights(*[_ptr(weights.get(n)) for n, _ in Weights._fields_])
        _check(load().lmoe_pack_backward_weights(ctypes.byref(D), ctypes.byref(W),
                                                 _ptr(self.packed), _ptr(self.packed_bwd), nb,
                                                 _stream(stream)),
               "lmoe_pack_backward_weights")
        self.bwd_bytes = int(load().lmoe_backward_workspace_bytes(ctypes.byref(D)))
        # the routed pre-activations a training forward keeps (lmoe_io.save_pre)
        sh = self.shape
        self.pre_buf = torch.empty((self.max_tokens * sh.K, 2 * sh.I), dtype=torch.bfloat16,
                                   device=self.device)
        self.pre_shared_buf = None if sh.S == 0 else torch.empty(
            (self.max_tokens, 2 * sh.S * sh.Is), dtype=torch.bfloat16, device=self.device)
        self.bwd_ws = torch.empty(self.bwd_bytes, dtype=torch.uint8, device=self.device)

    def backward_launches(self, T: int) -> int:
        """Kernels one lmoe_routed_backward call for T tokens launches: combine backward, two
        dgamma passes, two grouped dgrad GEMMs (and the pre-activation GEMM when the last
        forward was not a training step), SiTU backward, slot sum, latent row gather, row
        map and two grouped weight-gradient GEMMs."""
        return 11 + (0 if getattr(self, "_pre_rows", None) == T else 1)

    def _saved_pre(self, T: int, shared: bool = False):
        """The routed (or shared) experts' pre-activations kept by the last forward, if it
        was a training step of T tokens; else None (the backward recomputes them)."""
        if getattr(self, "_pre_rows", None) != T:
            return None
        return _ptr(self.pre_shared_buf if shared else self.pre_buf)

    def backward(self, dz: torch.Tensor, stream=None) -> dict:
        """Gradients of the routed branch for the batch of the last ``forward`` call
        (lmoe_routed_backward): dz [T, L] fp32 -> dlat, dgate, dgamma, dw_gate, dw_value,
        dw_edown (fp32)."""
        sh = self.shape
        T = dz.shape[0]
        _expect(dz, torch.float32, (T, sh.L), "dz")
        dims = dims_of(sh, T=T, expert_fp8=self.expert_fp8)
        dev = dz.device
        f = torch.float32
        out = {"dlat": torch.empty((T, sh.L), dtype=f, device=dev),
               "dgate": torch.empty((T, sh.K), dtype=f, device=dev),
               "dgamma": torch.empty(sh.L, dtype=f, device=dev),
               "dw_gu": torch.empty((sh.E, 2 * sh.I, sh.L), dtype=f, device=dev),
               "dw_edown": torch.empty((sh.E, sh.L, sh.I), dtype=f, device=dev)}
        bwd_bytes = int(load().lmoe_routed_backward_workspace_bytes(ctypes.byref(dims)))
        _check(load().lmoe_routed_backward(
            ctypes.byref(dims), _ptr(self.packed), _ptr(self.packed_bwd), _ptr(self.workspace),
            self.ws_bytes, _ptr(dz), self._saved_pre(T), _ptr(out["dlat"]), _ptr(out["dgate"]), _ptr(out["dgamma"]),
            _ptr(out["dw_gu"]), _ptr(out["dw_edown"]), _ptr(self.bwd_ws), bwd_bytes,
            _stream(stream)), "lmoe_routed_backward")
        out["dw_gate"] = out["dw_gu"][:, :sh.I]
        out["dw_value"] = out["dw_gu"][:, sh.I:]
        return out

    def layer_backward_launches(self, T: int) -> int:
        """Kernels one lmoe_backward call launches: the routed branch's, plus the row map of
        dw_in, the dz GEMM, router backward and its GEMM, the dx GEMM and three
        weight-gradient GEMMs; with shared experts also the dhs GEMM and their SiTU backward,
        and their pre-activation GEMM unless the last forward was a training step."""
        shared = 0
        if self.shape.S > 0:
            shared = 2 + (0 if getattr(self, "_pre_rows", None) == T else 1)
        return self.backward_launches(T) + 8 + shared

    def backward_layer(self, x: torch.Tensor, dy: torch.Tensor, logits=None,
                       stream=None) -> dict:
        """Gradients of the whole layer for the batch of the last ``forward`` call
        (lmoe_backward): x [T, d] bf16 (that call's input), dy [T, d] bf16 ->
        dx (through the latent and the shared experts; the residual adds dy), dgamma and
        every weight's gradient, fp32, in the weights' own shapes (dw_up, dw_sdown and the
        shared gate/value gradients are views into the packed gradient buffers).  logits:
        the fp32 [T, E] logits the forward routed on, when it was given ``logits_in``."""
        sh = self.shape
        T = x.shape[0]
        _expect(x, torch.bfloat16, (T, sh.d), "x")
        _expect(dy, torch.bfloat16, (T, sh.d), "dy")
        if logits is not None:
            _expect(logits, torch.float32, (T, sh.E), "logits")
        dims = dims_of(sh, T=T, expert_fp8=self.expert_fp8)
        dev = x.device
        f = torch.float32
        S, Is, L, d = sh.S, sh.Is, sh.L, sh.d
        sw = S * Is
        out = {"dx": torch.empty((T, d), dtype=f, device=dev),
               "dgamma": torch.empty(L, dtype=f, device=dev),
               "dw_in": torch.empty((L + 2 * sw, d), dtype=f, device=dev),
               "dw_router": torch.empty((sh.E, L), dtype=f, device=dev),
               "dw_gu": torch.empty((sh.E, 2 * sh.I, L), dtype=f, device=dev),
               "dw_edown": torch.empty((sh.E, L, sh.I), dtype=f, device=dev),
               "dw_out": torch.empty((d, L + sw), dtype=f, device=dev)}
        bwd_bytes = int(load().lmoe_backward_workspace_bytes(ctypes.byref(dims)))
        _check(load().lmoe_backward(
            ctypes.byref(dims), _ptr(self.packed), _ptr(self.packed_bwd), _ptr(self.workspace),
            self.ws_bytes, _ptr(x), _ptr(logits), _ptr(dy), self._saved_pre(T),
            self._saved_pre(T, shared=True), _ptr(out["dx"]),
            _ptr(out["dgamma"]), _ptr(out["dw_in"]), _ptr(out["dw_router"]), _ptr(out["dw_gu"]),
            _ptr(out["dw_edown"]), _ptr(out["dw_out"]), _ptr(self.bwd_ws), bwd_bytes,
            _stream(stream)), "lmoe_backward")
        out["dw_down"] = out["dw_in"][:L]
        out["dw_sgate"] = out["dw_in"][L:L + sw].view(S, Is, d)
        out["dw_svalue"] = out["dw_in"][L + sw:].view(S, Is, d)
        out["dw_gate"] = out["dw_gu"][:, :sh.I]
        out["dw_value"] = out["dw_gu"][:, sh.I:]
        out["dw_up"] = out["dw_out"][:, :L]
        out["dw_sdown"] = out["dw_out"][:, L:].unflatten(1, (S, Is)).permute(1, 0, 2)
        return out


class HostPipeline:
    """The layer on batches that live in pinned host memory, overlapped across batches: each
    ``submit`` is one lmoe_forward_host call (the upload of x, the layer and the download of
    y on three streams, through one of ``depth`` device staging slots), so batch i + 1's
    upload and batch i - 1's download run while batch i computes.  The library orders every
    reuse of a slot with the pipe's events; this class owns the slots, streams and events.
    ``synchronize`` waits for every submitted batch."""

    def __init__(self, layer: "Layer", depth: int = 2):
        if not 1 <= depth <= HOST_PIPE_MAX_DEPTH:
            raise ValueError(f"lmoe: pipeline depth must be 1..{HOST_PIPE_MAX_DEPTH}")
        self.layer = layer
        self.depth = depth
        T, d = layer.max_tokens, layer.shape.d
        dev = layer.device
        self.x = [torch.empty((T, d), dtype=torch.bfloat16, device=dev) for _ in range(depth)]
        self.y = [torch.empty((T, d), dtype=torch.bfloat16, device=dev) for _ in range(depth)]
        self.up = torch.cuda.Stream(device=dev)
        self.compute = torch.cuda.Stream(device=dev)
        self.down = torch.cuda.Stream(device=dev)
        self.events = [[torch.cuda.Event() for _ in range(3)] for _ in range(depth)]
        for evs in self.events:  # torch creates its events lazily: record each once
            for ev in evs:
                ev.record(self.compute)
        self.compute.synchronize()
        p = HostPipe()
        p.depth, p.max_tokens = depth, T
        for k in range(depth):
            p.x_dev[k] = self.x[k].data_ptr()
            p.y_dev[k] = self.y[k].data_ptr()
            p.uploaded[k] = self.events[k][0].cuda_event
            p.computed[k] = self.events[k][1].cuda_event
            p.downloaded[k] = self.events[k][2].cuda_event
        p.upload = self.up.cuda_stream
        p.compute = self.compute.cuda_stream
        p.download = self.down.cuda_stream
        p.calls = 0
        self.pipe = p

    def submit(self, x_host: torch.Tensor, y_host: torch.Tensor, residual_from_x: bool = True,
               tau: torch.Tensor | None = None, balance: bool = True,
               logit_bias: torch.Tensor | None = None):
        """Enqueue one batch: x_host [T, d] bf16 pinned in, y_host pinned out."""
        layer, sh = self.layer, self.layer.shape
        T = x_host.shape[0]
        if T > layer.max_tokens:
            raise ValueError(f"lmoe: {T} tokens exceed the pipeline's {layer.max_tokens}")
        _expect(x_host, torch.bfloat16, (T, sh.d), "x_host")
        _expect(y_host, torch.bfloat16, (T, sh.d), "y_host")
        if x_host.is_cuda or y_host.is_cuda or not x_host.is_contiguous() or \
                not y_host.is_contiguous():
            raise ValueError("lmoe: x_host and y_host must be contiguous host tensors")
        io = IO()
        io.balance = 1 if balance else 0
        if tau is not None:
            _expect(tau, torch.float32, (sh.E,), "tau")
            io.tau_in = _ptr(tau)
        if logit_bias is not None:
            _expect(logit_bias, torch.float32, (sh.E,), "logit_bias")
            io.logit_bias = _ptr(logit_bias)
        dims = dims_of(sh, T=T, expert_fp8=layer.expert_fp8)
        _check(load().lmoe_forward_host(ctypes.byref(dims), _ptr(layer.packed),
                                        ctypes.c_void_p(x_host.data_ptr()),
                                        1 if residual_from_x else 0,
                                        ctypes.c_void_p(y_host.data_ptr()),
                                        _ptr(layer.workspace), layer.ws_bytes, ctypes.byref(io),
                                        ctypes.byref(self.pipe)), "lmoe_forward_host")
        layer.last_kernel_launches = io.kernel_launches

    def synchronize(self):
        for s in (self.up, self.compute, self.down):
            s.synchronize()

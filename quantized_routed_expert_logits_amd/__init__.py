"""Python binding of libstrata_moe (the MI355X routed-expert prompt MoE layer).

Argument marshalling only: every step of the layer runs in the library's HIP
kernels.  Tensors are torch tensors on the GPU (torch provides device memory
and streams); each function takes the same arguments as the C entry point of
the same name in include/strata_moe.h, with shapes taken from the tensors
where the C call takes sizes.  There is no CPU fallback: importing this
package fails loudly when the library has not been built.
"""
from __future__ import annotations

import contextlib
import ctypes
import os

import numpy as np
import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libstrata_moe.so")

OK = 0
EINVAL = -1
EUNSUPPORTED = -2
ENOMEM = -3
EHIP = -4
EDATA = -5
Q2_SYM = 1  # w = d * (q - 1.5)
Q2_0 = 2    # w = d * (q - 1), the pages' Q2_0 packs
FORMATS = {"q2_sym": Q2_SYM, "q2_0": Q2_0}
FLAG_NO_GEMV = 1        # every chunk to the MFMA kernels (no GEMV, also at decode-window sizes)
FLAG_PER_SLOT_Q8 = 2    # the GEMV's input rounded per routed slot in the q8_1 form (A/B arm)
FLAG_GEMV_ALWAYS = 4    # the GEMV takes chunks of <= 8 rows at any average rows per expert


class StrataMoeError(RuntimeError):
    def __init__(self, code: int, message: str):
        super().__init__(f"[{code}] {message}")
        self.code = code


if not os.path.exists(LIB_PATH):
    raise ImportError(
        f"{LIB_PATH} is missing: build it first (python -c 'import __graft_entry__ as g; g.build()')")

_lib = ctypes.CDLL(LIB_PATH)
_P = ctypes.c_void_p
_i64, _i32 = ctypes.c_int64, ctypes.c_int32


class ExpertsStruct(ctypes.Structure):
    _fields_ = [("n_expert", _i32), ("hidden", _i32), ("ffn", _i32), ("format", _i32),
                ("gate_up", _P), ("gate_up_stride", _i64), ("down", _P), ("down_stride", _i64),
                ("router_bias", _P), ("router_prepared", _P), ("shared_gate", _P), ("flags", _i32)]


class DebugStruct(ctypes.Structure):
    _fields_ = [(name, _P) for name in ("ids", "p", "offsets", "src", "slot", "qx", "sx", "qh", "sh")]


class AdaptersStruct(ctypes.Structure):
    _fields_ = [("n_adapter", _i32), ("rank", _i32), ("in_dim", _i32), ("out_dim", _i32), ("dtype", _i32),
                ("a", _P), ("b", _P), ("scale", _P), ("ranks", _P)]


class MxfpWeightsStruct(ctypes.Structure):
    _fields_ = [("n_expert", _i32), ("rows", _i32), ("cols", _i32), ("swiglu", _i32), ("packed", _P),
                ("stride", _i64)]


class NormStruct(ctypes.Structure):
    _fields_ = [("weight", _P), ("weight_offset", ctypes.c_double), ("eps", ctypes.c_double)]


class BranchStruct(ctypes.Structure):
    _fields_ = [("y", _P), ("y_stride", _i64), ("y_rows", _i64), ("y_dtype", _i32), ("K", _i32), ("slot", _P),
                ("p", _P), ("norm", ctypes.POINTER(NormStruct)), ("gate", _P), ("gate_row_stride", _i64),
                ("gate_col_stride", _i32), ("residual_scale", ctypes.c_double), ("block_scale", ctypes.c_double)]


def _sig(name, args, res=ctypes.c_int):
    f = getattr(_lib, name)
    f.argtypes = args
    f.restype = res
    return f


_sig("strata_moe_device_supported", [])
_sig("strata_moe_last_error", [], ctypes.c_char_p)
_sig("strata_moe_packed_bytes", [_i32, _i32, ctypes.POINTER(_i64), ctypes.POINTER(_i64)])
_sig("strata_moe_workspace_bytes", [_i64, _i32, ctypes.POINTER(ExpertsStruct), ctypes.POINTER(ctypes.c_size_t)])
_sig("strata_moe_set_workspace", [_P, ctypes.c_size_t])
_sig("strata_moe_router_prepared_bytes", [_i32, _i32, ctypes.POINTER(ctypes.c_size_t)])
_sig("strata_moe_prepare_router", [_P, _i32, _i32, _P, _P])
_sig("strata_moe_pack", [_P, _P, _P, _P, _i32, _i32, _i32, _i32, _P, _i64, _P, _i64, _P])
_sig("strata_moe_unpack", [_P, _i64, _P, _i64, _i32, _i32, _i32, _i32, _P, _P, _P, _P, _P])
_sig("strata_moe_prefill", [_P, _P, ctypes.POINTER(ExpertsStruct), _i64, _i32, _P, _P])
_sig("strata_moe_prefill_noalloc", [_P, _P, ctypes.POINTER(ExpertsStruct), _i64, _i32, _P, _P])
_sig("strata_moe_prefill_debug", [_P, _P, ctypes.POINTER(ExpertsStruct), _i64, _i32, _P,
                                  ctypes.POINTER(DebugStruct), _P])
_sig("strata_moe_route", [_P, _P, _P, _i64, _i32, _i32, _i32, _P, _P, _P])
_sig("strata_moe_group", [_P, _i64, _i32, _i32, _P, _P, _P, _P])
_sig("strata_moe_quantize", [_P, _i64, _i32, _P, _P, _P])
_sig("strata_moe_gate_up", [_P, _P, _P, _P, _i64, _i32, ctypes.POINTER(ExpertsStruct), _P, _P, _P])
_sig("strata_moe_down", [_P, _P, _P, _P, _P, _P, _i64, _i32, ctypes.POINTER(ExpertsStruct), _P, _P])
_sig("strata_moe_ring_bytes", [_i32, _i32, _i32, ctypes.POINTER(ctypes.c_size_t)])
_sig("strata_moe_ring_create", [_i32, _i32, _i32, _P, ctypes.c_size_t, _P, ctypes.POINTER(_P)])
_sig("strata_moe_ring_destroy", [_P])
_sig("strata_moe_prefill_streamed", [_P, _P, ctypes.POINTER(ExpertsStruct), _P, _i64, _i32, _P, _P])
_sig("strata_moe_adapt_workspace_bytes", [_i64, ctypes.POINTER(AdaptersStruct), ctypes.POINTER(ctypes.c_size_t)])
_sig("strata_moe_adapt", [_P, _i64, _P, ctypes.POINTER(AdaptersStruct), _i64, _P, _i64, _P, _i64, _P,
                          ctypes.c_size_t, _P])
_sig("strata_moe_decode_workspace_bytes", [_i64, _i32, ctypes.POINTER(ExpertsStruct), ctypes.POINTER(AdaptersStruct),
                                           ctypes.POINTER(ctypes.c_size_t)])
_sig("strata_moe_decode", [_P, _P, ctypes.POINTER(ExpertsStruct), _i64, _i32, ctypes.POINTER(AdaptersStruct), _P, _P,
                           _P, ctypes.c_size_t, _P])
_sig("strata_moe_mxfp_quantize", [_P, _i32, _i64, _i64, _i32, _P, _P, _P])
_sig("strata_moe_mxfp_dequantize", [_P, _P, _i64, _i32, _P, _i32, _i64, _P])
_sig("strata_moe_mxfp_packed_bytes", [_i32, _i32, _i32, ctypes.POINTER(_i64)])
_sig("strata_moe_mxfp_pack", [_P, _P, _i32, _i32, _i32, _i32, _i32, _P, _i64, _P])
_sig("strata_moe_mxfp_product", [_P, _P, _i64, ctypes.POINTER(MxfpWeightsStruct), _P, _P, _i64, _P, _i32, _i64, _P])
_sig("strata_moe_norm_before", [_P, _i32, _i64, _i64, _i32, ctypes.POINTER(NormStruct), _P, _P, _P, _P])
_sig("strata_moe_norm_after", [_P, _i32, _i64, _i64, _i32, ctypes.POINTER(BranchStruct), _P, _i64,
                               ctypes.POINTER(NormStruct), _P, _P, _P, _P])
_sig("strata_moe_timing", [ctypes.c_int, _i32])
_sig("strata_moe_timing_kinds", [])
_sig("strata_moe_timing_name", [ctypes.c_int], ctypes.c_char_p)
_sig("strata_moe_timing_read", [ctypes.POINTER(ctypes.c_double), ctypes.POINTER(_i32), ctypes.c_int])

EXPORTED = [
    "strata_moe_device_supported", "strata_moe_last_error", "strata_moe_packed_bytes",
    "strata_moe_workspace_bytes", "strata_moe_set_workspace", "strata_moe_router_prepared_bytes",
    "strata_moe_prepare_router", "strata_moe_pack", "strata_moe_unpack",
    "strata_moe_prefill", "strata_moe_prefill_debug", "strata_moe_route", "strata_moe_group",
    "strata_moe_quantize", "strata_moe_gate_up", "strata_moe_down", "strata_moe_timing",
    "strata_moe_timing_kinds", "strata_moe_timing_name", "strata_moe_timing_read",
    "strata_moe_ring_bytes", "strata_moe_ring_create", "strata_moe_ring_destroy", "strata_moe_prefill_streamed",
    "strata_moe_prefill_noalloc", "strata_moe_adapt_workspace_bytes", "strata_moe_adapt",
    "strata_moe_decode_workspace_bytes", "strata_moe_decode", "strata_moe_mxfp_quantize",
    "strata_moe_mxfp_dequantize", "strata_moe_mxfp_packed_bytes", "strata_moe_mxfp_pack", "strata_moe_mxfp_product",
    "strata_moe_norm_before", "strata_moe_norm_after",
]
NOALLOC_SCRATCH_BYTES = 512 << 20  # STRATA_MOE_NOALLOC_SCRATCH_BYTES
DECODE_MAX_TOKENS = 64             # STRATA_MOE_DECODE_MAX_TOKENS
ADAPTER_DTYPES = {torch.float32: 1, torch.float16: 2, torch.bfloat16: 3}  # STRATA_MOE_ADAPTER_*
ROW_DTYPES = {torch.float32: 1, torch.float16: 2, torch.bfloat16: 3}      # STRATA_MOE_F32, _F16, _BF16


def library() -> ctypes.CDLL:
    return _lib


def strata_moe_last_error() -> str:
    return _lib.strata_moe_last_error().decode()


def _check(rc: int, what: str):
    if rc != 0:
        raise StrataMoeError(rc, f"{what}: {strata_moe_last_error()}")


def _ptr(t):
    if t is None:
        return None
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError("expected a CUDA (HIP) torch tensor")
    if not t.is_contiguous():
        raise ValueError("expected a contiguous tensor")
    return ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def _dtype(t, dt, name):
    if t is not None and t.dtype != dt:
        raise TypeError(f"{name} must be {dt}, got {t.dtype}")


def _expect(t, name: str, shape: tuple, dt):
    """Host-side check of one tensor argument before the C call: the library
    takes raw pointers and trusts the sizes it is given, so a tensor of the
    wrong shape would send its kernels past the allocation."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch tensor")
    _dtype(t, dt, name)
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")


def _one_device(**tensors):
    """Every given tensor is a CUDA (HIP) tensor, all on one device."""
    devs = set()
    for name, t in tensors.items():
        if t is None:
            continue
        if not t.is_cuda:
            raise TypeError(f"{name} must be a CUDA (HIP) tensor")
        devs.add(t.device)
    if len(devs) > 1:
        raise ValueError(f"arguments are on different devices: {sorted(str(d) for d in devs)}")


def _check_layer_args(x, router_w, experts: "Experts", out):
    """x [T][H], router_w [H][E], out [T][H] (fp32), on the experts' device
    (streamed experts: their parameters' device; the blobs are in host memory)."""
    H, E = experts.hidden, experts.n_expert
    if not isinstance(x, torch.Tensor) or x.dim() != 2:
        raise ValueError("x must be a 2-D [T][H] tensor")
    T = x.shape[0]
    _expect(x, "x", (T, H), torch.float32)
    _expect(router_w, "router_w", (H, E), torch.float32)
    _expect(out, "out", (T, H), torch.float32)
    blobs = {} if getattr(experts, "streamed", False) else dict(gate_up=experts.gate_up, down=experts.down)
    _one_device(x=x, router_w=router_w, out=out, router_bias=experts.router_bias,
                router_prepared=experts.router_prepared, shared_gate=experts.shared_gate, **blobs)
    return T


# ------------------------------------------------------------------- queries
def strata_moe_device_supported() -> bool:
    return bool(_lib.strata_moe_device_supported())


def strata_moe_packed_bytes(hidden: int, ffn: int) -> tuple[int, int]:
    gu, dn = _i64(), _i64()
    _check(_lib.strata_moe_packed_bytes(hidden, ffn, ctypes.byref(gu), ctypes.byref(dn)), "strata_moe_packed_bytes")
    return gu.value, dn.value


def strata_moe_router_prepared_bytes(hidden: int, n_expert: int) -> int:
    b = ctypes.c_size_t()
    _check(_lib.strata_moe_router_prepared_bytes(hidden, n_expert, ctypes.byref(b)), "strata_moe_router_prepared_bytes")
    return b.value


def strata_moe_prepare_router(router_w: torch.Tensor, stream=None) -> torch.Tensor:
    """router_w [H][E] fp32 on the device -> its prepared form (a uint8 device tensor)."""
    _dtype(router_w, torch.float32, "router_w")
    H, E = router_w.shape
    prepared = torch.empty(strata_moe_router_prepared_bytes(H, E), dtype=torch.uint8, device=router_w.device)
    _check(_lib.strata_moe_prepare_router(_ptr(router_w), H, E, _ptr(prepared), _stream(stream)),
           "strata_moe_prepare_router")
    return prepared


def strata_moe_set_workspace(buf: torch.Tensor | None) -> None:
    if buf is None:
        _check(_lib.strata_moe_set_workspace(None, 0), "strata_moe_set_workspace")
    else:
        _check(_lib.strata_moe_set_workspace(_ptr(buf), buf.numel() * buf.element_size()), "strata_moe_set_workspace")


# ------------------------------------------------------------------- experts
class Experts:
    """A layer's packed experts in device memory (blobs owned by torch).

    shared=True adds a blob slot for the layer's shared expert at index
    n_expert (pack it like a routed expert); the layer runs it once its scalar
    gate vector is set (with_shared_gate)."""

    def __init__(self, n_expert: int, hidden: int, ffn: int, router_bias: torch.Tensor | None = None,
                 device: str | torch.device = "cuda", fmt: str = "q2_sym", shared: bool = False):
        if fmt not in FORMATS:
            raise ValueError(f"unknown weight format {fmt!r}; one of {sorted(FORMATS)}")
        self.n_expert, self.hidden, self.ffn, self.format = n_expert, hidden, ffn, FORMATS[fmt]
        self.shared = bool(shared)
        nb = n_expert + self.shared
        self.gate_up_stride, self.down_stride = strata_moe_packed_bytes(hidden, ffn)
        self.gate_up = torch.empty(nb * self.gate_up_stride, dtype=torch.uint8, device=device)
        self.down = torch.empty(nb * self.down_stride, dtype=torch.uint8, device=device)
        if router_bias is not None:
            _expect(router_bias, "router_bias", (n_expert,), torch.float32)
        self.router_bias = router_bias
        self.router_prepared = None
        self.shared_gate = None
        self.flags = 0
        self._restruct()

    def _restruct(self):
        self.struct = ExpertsStruct(self.n_expert, self.hidden, self.ffn, self.format, self.gate_up.data_ptr(),
                                    self.gate_up_stride, self.down.data_ptr(), self.down_stride,
                                    None if self.router_bias is None else self.router_bias.data_ptr(),
                                    None if self.router_prepared is None else self.router_prepared.data_ptr(),
                                    None if self.shared_gate is None else self.shared_gate.data_ptr(),
                                    getattr(self, "flags", 0))

    def with_flags(self, flags: int) -> "Experts":
        """The same blobs with other kernel-choice flags (FLAG_NO_GEMV, FLAG_PER_SLOT_Q8, FLAG_GEMV_ALWAYS)."""
        import copy

        other = copy.copy(self)
        other.flags = int(flags)
        other._restruct()
        return other

    def with_router_bias(self, router_bias: torch.Tensor | None) -> "Experts":
        """The same blobs with another router bias (or none)."""
        import copy

        if router_bias is not None:
            _expect(router_bias, "router_bias", (self.n_expert,), torch.float32)
        other = copy.copy(self)
        other.router_bias = router_bias
        other._restruct()
        return other

    def with_shared_gate(self, gate: torch.Tensor | None) -> "Experts":
        """The same blobs with the shared expert's scalar gate vector [H] fp32
        (None: the layer runs the routed experts only)."""
        import copy

        if gate is not None:
            if not self.shared:
                raise ValueError("these experts have no shared-expert blob (Experts(..., shared=True))")
            _dtype(gate, torch.float32, "shared_gate")
            if tuple(gate.shape) != (self.hidden,) or not gate.is_contiguous():
                raise ValueError(f"shared_gate must be a contiguous [{self.hidden}] tensor")
        other = copy.copy(self)
        other.shared_gate = gate
        other._restruct()
        return other

    def with_prepared_router(self, router_w: torch.Tensor | None, stream=None) -> "Experts":
        """The same blobs with router_w prepared once (strata_moe_prepare_router);
        the layer calls must then pass the same router_w.  None: prepare per call."""
        import copy

        if router_w is not None:
            _expect(router_w, "router_w", (self.hidden, self.n_expert), torch.float32)
        other = copy.copy(self)
        other.router_prepared = None if router_w is None else strata_moe_prepare_router(router_w, stream)
        other._restruct()
        return other

    def pack(self, e0: int, codes_gu, scales_gu, codes_d, scales_d, stream=None):
        """Pack experts [e0, e0 + len(codes_gu)) from canonical arrays (numpy
        or torch; copied to the device if needed)."""
        dev = self.gate_up.device

        def to_dev(a, dt):
            if isinstance(a, np.ndarray):
                a = torch.from_numpy(np.ascontiguousarray(a))
            return a.to(device=dev, dtype=dt).contiguous()

        cg, sg = to_dev(codes_gu, torch.uint8), to_dev(scales_gu.view(np.int16) if isinstance(scales_gu, np.ndarray)
                                                       else scales_gu, torch.int16)
        cd, sd = to_dev(codes_d, torch.uint8), to_dev(scales_d.view(np.int16) if isinstance(scales_d, np.ndarray)
                                                      else scales_d, torch.int16)
        ne = cg.shape[0]
        assert cg.shape == (ne, 2 * self.ffn, self.hidden) and cd.shape == (ne, self.hidden, self.ffn)
        strata_moe_pack(cg, sg, cd, sd, e0, e0 + ne, self.hidden, self.ffn, self.gate_up, self.gate_up_stride,
                        self.down, self.down_stride, stream)


def strata_moe_pack(codes_gu, scales_gu, codes_d, scales_d, e0, e1, hidden, ffn, gate_up, gate_up_stride, down,
                    down_stride, stream=None):
    _check(_lib.strata_moe_pack(_ptr(codes_gu), _ptr(scales_gu), _ptr(codes_d), _ptr(scales_d), e0, e1, hidden, ffn,
                                _ptr(gate_up), gate_up_stride, _ptr(down), down_stride, _stream(stream)),
           "strata_moe_pack")


def strata_moe_unpack(experts: Experts, e0: int, e1: int, stream=None):
    """Returns canonical (codes_gu, scales_gu, codes_d, scales_d) device tensors of experts [e0, e1)."""
    ne, H, I = e1 - e0, experts.hidden, experts.ffn
    dev = experts.gate_up.device
    cg = torch.empty((ne, 2 * I, H), dtype=torch.uint8, device=dev)
    sg = torch.empty((ne, 2 * I, H // 32), dtype=torch.int16, device=dev)
    cd = torch.empty((ne, H, I), dtype=torch.uint8, device=dev)
    sd = torch.empty((ne, H, I // 32), dtype=torch.int16, device=dev)
    _check(_lib.strata_moe_unpack(_ptr(experts.gate_up), experts.gate_up_stride, _ptr(experts.down),
                                  experts.down_stride, e0, e1, H, I, _ptr(cg), _ptr(sg), _ptr(cd), _ptr(sd),
                                  _stream(stream)), "strata_moe_unpack")
    return cg, sg, cd, sd


def strata_moe_workspace_bytes(T: int, K: int, experts: Experts) -> int:
    b = ctypes.c_size_t()
    _check(_lib.strata_moe_workspace_bytes(T, K, ctypes.byref(experts.struct), ctypes.byref(b)),
           "strata_moe_workspace_bytes")
    return b.value


# ---------------------------------------------------------- streamed experts
class HostExperts(Experts):
    """A layer's packed experts in pinned host memory, for the streamed layer:
    expert e's gate/up blob at e * S and its down blob right after it (S =
    one ring slot), the layout strata_moe_prefill_streamed reads.  Packing
    runs on `device` (the library's packer) and the result is copied here."""

    streamed = True

    def __init__(self, n_expert: int, hidden: int, ffn: int, router_bias: torch.Tensor | None = None,
                 device: str | torch.device = "cuda", fmt: str = "q2_sym", shared: bool = False):
        if fmt not in FORMATS:
            raise ValueError(f"unknown weight format {fmt!r}; one of {sorted(FORMATS)}")
        self.n_expert, self.hidden, self.ffn, self.format = n_expert, hidden, ffn, FORMATS[fmt]
        self.shared = bool(shared)
        self.device = torch.device(device)
        gu, dn = strata_moe_packed_bytes(hidden, ffn)
        self.gate_up_bytes, self.slot_bytes = gu, gu + dn
        self.gate_up_stride = self.down_stride = self.slot_bytes
        nb = n_expert + self.shared
        self.host = torch.empty(nb * self.slot_bytes, dtype=torch.uint8, pin_memory=True)
        self.gate_up = self.host
        self.down = self.host[gu:]
        if router_bias is not None:
            _expect(router_bias, "router_bias", (n_expert,), torch.float32)
        self.router_bias = router_bias
        self.router_prepared = None
        self.shared_gate = None
        self.flags = 0
        self._restruct()

    def pack(self, e0: int, codes_gu, scales_gu, codes_d, scales_d, stream=None):
        """Pack experts [e0, e0 + len(codes_gu)) from canonical arrays on the
        device, then copy the blobs into their host places."""
        ne = len(codes_gu)
        staging = torch.empty(ne * self.slot_bytes, dtype=torch.uint8, device=self.device)

        def to_dev(a, dt):
            if isinstance(a, np.ndarray):
                a = torch.from_numpy(np.ascontiguousarray(a))
            return a.to(device=self.device, dtype=dt).contiguous()

        as_i16 = lambda a: a.view(np.int16) if isinstance(a, np.ndarray) else a  # noqa: E731
        cg, sg = to_dev(codes_gu, torch.uint8), to_dev(as_i16(scales_gu), torch.int16)
        cd, sd = to_dev(codes_d, torch.uint8), to_dev(as_i16(scales_d), torch.int16)
        assert cg.shape == (ne, 2 * self.ffn, self.hidden) and cd.shape == (ne, self.hidden, self.ffn)
        strata_moe_pack(cg, sg, cd, sd, 0, ne, self.hidden, self.ffn, staging, self.slot_bytes,
                        staging[self.gate_up_bytes:], self.slot_bytes, stream)
        self.host[e0 * self.slot_bytes:(e0 + ne) * self.slot_bytes].copy_(staging)


class Ring:
    """A ring of n_slots device slots (torch memory) with a copy stream of its
    own (default priority) and the library's ring object over them."""

    def __init__(self, n_slots: int, hidden: int, ffn: int, device: str | torch.device = "cuda"):
        b = ctypes.c_size_t()
        _check(_lib.strata_moe_ring_bytes(n_slots, hidden, ffn, ctypes.byref(b)), "strata_moe_ring_bytes")
        self.n_slots, self.hidden, self.ffn = n_slots, hidden, ffn
        self.slots = torch.empty(b.value, dtype=torch.uint8, device=device)
        self.copy_stream = torch.cuda.Stream(device=device)
        h = _P()
        _check(_lib.strata_moe_ring_create(n_slots, hidden, ffn, _ptr(self.slots), b.value,
                                           ctypes.c_void_p(self.copy_stream.cuda_stream), ctypes.byref(h)),
               "strata_moe_ring_create")
        self.handle = h

    def close(self):
        if getattr(self, "handle", None) is not None and self.handle.value:
            _lib.strata_moe_ring_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:  # pragma: no cover (interpreter shutdown)
            pass


def strata_moe_prefill_streamed(x: torch.Tensor, router_w: torch.Tensor, experts: HostExperts, ring: Ring, K: int,
                                out: torch.Tensor, stream=None) -> torch.Tensor:
    if not isinstance(experts, HostExperts):
        raise TypeError("streamed experts live in pinned host memory: use HostExperts")
    T = _check_layer_args(x, router_w, experts, out)
    if ring.handle is None:
        raise ValueError("the ring is closed")
    if (ring.hidden, ring.ffn) != (experts.hidden, experts.ffn):
        raise ValueError("the ring was made for other expert sizes")
    if ring.slots.device != x.device:
        raise ValueError("the ring is on another device")
    _check(_lib.strata_moe_prefill_streamed(_ptr(x), _ptr(router_w), ctypes.byref(experts.struct), ring.handle, T, K,
                                            _ptr(out), _stream(stream)), "strata_moe_prefill_streamed")
    return out


# --------------------------------------------------------------------- layer
def strata_moe_prefill(x: torch.Tensor, router_w: torch.Tensor, experts: Experts, K: int, out: torch.Tensor,
                       stream=None) -> torch.Tensor:
    T = _check_layer_args(x, router_w, experts, out)
    _check(_lib.strata_moe_prefill(_ptr(x), _ptr(router_w), ctypes.byref(experts.struct), T, K, _ptr(out),
                                   _stream(stream)), "strata_moe_prefill")
    return out


def strata_moe_prefill_noalloc(x: torch.Tensor, router_w: torch.Tensor, experts: Experts, K: int, out: torch.Tensor,
                               stream=None) -> torch.Tensor:
    """strata_moe_prefill on the library's fixed scratch: no device allocation."""
    T = _check_layer_args(x, router_w, experts, out)
    _check(_lib.strata_moe_prefill_noalloc(_ptr(x), _ptr(router_w), ctypes.byref(experts.struct), T, K, _ptr(out),
                                           _stream(stream)), "strata_moe_prefill_noalloc")
    return out


def strata_moe_prefill_debug(x, router_w, experts: Experts, K: int, out, stream=None) -> dict:
    """The layer plus its intermediates (ids, p, offsets, src, slot, qx, sx, qh, sh) as device tensors."""
    _check_layer_args(x, router_w, experts, out)
    T, H = x.shape
    sh = experts.shared_gate is not None  # the shared expert: pair slot K of each token, expert n_expert
    Kg = K + sh
    E, I, n = experts.n_expert + sh, experts.ffn, x.shape[0] * Kg
    dev = x.device
    d = dict(ids=torch.empty((T, Kg), dtype=torch.int32, device=dev),
             p=torch.empty((T, Kg), dtype=torch.float32, device=dev),
             offsets=torch.empty(E + 1, dtype=torch.int32, device=dev),
             src=torch.empty(n, dtype=torch.int32, device=dev),
             slot=torch.empty(n, dtype=torch.int32, device=dev),
             qx=torch.empty((T, H), dtype=torch.int8, device=dev),
             sx=torch.empty((T, H // 32), dtype=torch.float32, device=dev),
             qh=torch.empty((n, I), dtype=torch.int8, device=dev),
             sh=torch.empty((n, I // 32), dtype=torch.float32, device=dev))
    dbg = DebugStruct(*[d[k].data_ptr() for k in ("ids", "p", "offsets", "src", "slot", "qx", "sx", "qh", "sh")])
    _check(_lib.strata_moe_prefill_debug(_ptr(x), _ptr(router_w), ctypes.byref(experts.struct), T, K, _ptr(out),
                                         ctypes.byref(dbg), _stream(stream)), "strata_moe_prefill_debug")
    d["out"] = out
    return d


# ------------------------------------------- adapters and the few-token layer
class Adapters:
    """Low-rank adapters of many requests beside a projection they share:
    adapter n adds scale[n] * b[n] @ (a[n] @ x[t]) to the rows of its requests.

    a [n][rank][in_dim] and b [n][out_dim][rank] of one dtype (float32,
    float16 or bfloat16); scale [n] float32 or None (1); ranks [n] int32 or
    None: adapter n uses its first ranks[n] rows of a and columns of b."""

    def __init__(self, a: torch.Tensor, b: torch.Tensor, scale: torch.Tensor | None = None,
                 ranks: torch.Tensor | None = None):
        if not isinstance(a, torch.Tensor) or not isinstance(b, torch.Tensor) or a.dim() != 3 or b.dim() != 3:
            raise ValueError("a must be [n][rank][in_dim] and b [n][out_dim][rank]")
        if a.dtype not in ADAPTER_DTYPES:
            raise TypeError(f"adapters must be one of {sorted(str(d) for d in ADAPTER_DTYPES)}, got {a.dtype}")
        n, rank, in_dim = a.shape
        _expect(b, "b", (n, b.shape[1], rank), a.dtype)
        if scale is not None:
            _expect(scale, "scale", (n,), torch.float32)
        if ranks is not None:
            _expect(ranks, "ranks", (n,), torch.int32)
        for name, t in (("a", a), ("b", b), ("scale", scale), ("ranks", ranks)):
            if t is not None and not t.is_contiguous():
                raise ValueError(f"{name} must be contiguous")
            if t is not None and t.device != a.device:
                raise ValueError("arguments are on different devices")
        self.a, self.b, self.scale, self.ranks = a, b, scale, ranks
        self.n_adapter, self.rank, self.in_dim, self.out_dim = n, rank, in_dim, b.shape[1]
        self.struct = AdaptersStruct(n, rank, in_dim, self.out_dim, ADAPTER_DTYPES[a.dtype], a.data_ptr(), b.data_ptr(),
                                     None if scale is None else scale.data_ptr(),
                                     None if ranks is None else ranks.data_ptr())


def strata_moe_adapt_workspace_bytes(T: int, adapters: Adapters) -> int:
    b = ctypes.c_size_t()
    _check(_lib.strata_moe_adapt_workspace_bytes(T, ctypes.byref(adapters.struct), ctypes.byref(b)),
           "strata_moe_adapt_workspace_bytes")
    return b.value


def _rows(t, name: str, T: int, width: int):
    """A [T][width] fp32 tensor with contiguous rows -> its row stride."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch tensor")
    _dtype(t, torch.float32, name)
    if t.dim() != 2 or t.shape[0] != T or t.shape[1] != width:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {(T, width)}")
    if T <= 1:
        if width > 1 and t.stride(1) != 1 and T == 1:
            raise ValueError(f"{name} must have contiguous rows")
        return width
    if (width > 1 and t.stride(1) != 1) or t.stride(0) < width:
        raise ValueError(f"{name} must have contiguous rows that do not overlap")
    return t.stride(0)


def _with_workspace(call, device, workspace, nbytes, stream):
    """call(workspace pointer, its bytes, stream) with the tensors' device
    current and the given workspace, or one allocated on the stream.

    A few-token call takes the GPU a few microseconds, so the common case goes
    past torch's context managers and stream objects (5 us of host time)."""
    index = device.index
    if torch.cuda.current_device() != index:
        with torch.cuda.device(device):
            return _with_workspace(call, device, workspace, nbytes, stream)
    raw = torch._C._cuda_getCurrentRawStream(index) if stream is None else stream.cuda_stream
    if workspace is None:
        with contextlib.nullcontext() if stream is None else torch.cuda.stream(stream):
            workspace = torch.empty(max(nbytes(), 1), dtype=torch.uint8, device=device)
    elif workspace.device != device:
        raise ValueError("the workspace is on another device")
    elif not workspace.is_contiguous():
        raise ValueError("expected a contiguous workspace")
    return call(workspace.data_ptr(), workspace.numel() * workspace.element_size(), raw)


def strata_moe_adapt(x: torch.Tensor, ids: torch.Tensor, adapters: Adapters, y: torch.Tensor, out: torch.Tensor,
                     workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """out[t] = y[t] + the adapter ids[t]'s rows of x[t] (ids[t] < 0: y[t]).  x, y and out may have padded rows;
    out may be y.  workspace: strata_moe_adapt_workspace_bytes() bytes for this call alone, or None to allocate it."""
    if not isinstance(x, torch.Tensor) or x.dim() != 2:
        raise ValueError("x must be a 2-D [T][in_dim] tensor")
    if not isinstance(adapters, Adapters):
        raise TypeError("adapters must be an Adapters object")
    T = x.shape[0]
    xs, ys, os_ = (_rows(t, n, T, w) for t, n, w in ((x, "x", adapters.in_dim), (y, "y", adapters.out_dim),
                                                     (out, "out", adapters.out_dim)))
    _expect(ids, "ids", (T,), torch.int32)
    _one_device(x=x, ids=ids, y=y, out=out, a=adapters.a)
    if not ids.is_contiguous():
        raise ValueError("ids must be contiguous")

    def call(ws, nbytes, st):
        _check(_lib.strata_moe_adapt(x.data_ptr(), xs, ids.data_ptr(), ctypes.byref(adapters.struct), T, y.data_ptr(),
                                     ys, out.data_ptr(), os_, ws, nbytes, st), "strata_moe_adapt")
        return out

    return _with_workspace(call, x.device, workspace, lambda: strata_moe_adapt_workspace_bytes(T, adapters), stream)


def strata_moe_decode_workspace_bytes(T: int, K: int, experts: Experts, adapters: Adapters | None = None) -> int:
    b = ctypes.c_size_t()
    _check(_lib.strata_moe_decode_workspace_bytes(T, K, ctypes.byref(experts.struct),
                                                  None if adapters is None else ctypes.byref(adapters.struct),
                                                  ctypes.byref(b)), "strata_moe_decode_workspace_bytes")
    return b.value


def strata_moe_decode(x: torch.Tensor, router_w: torch.Tensor, experts: Experts, K: int, out: torch.Tensor,
                      adapters: Adapters | None = None, adapter_ids: torch.Tensor | None = None,
                      workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """The layer for at most DECODE_MAX_TOKENS tokens, with the requests' adapters beside it if given.  workspace:
    strata_moe_decode_workspace_bytes() bytes for this call alone, or None to allocate it."""
    if getattr(experts, "streamed", False):
        raise TypeError("the few-token layer reads resident experts: use Experts")
    T = _check_layer_args(x, router_w, experts, out)
    if (adapters is None) != (adapter_ids is None):
        raise ValueError("adapters and adapter_ids come together")
    if adapters is not None:
        if not isinstance(adapters, Adapters):
            raise TypeError("adapters must be an Adapters object")
        _expect(adapter_ids, "adapter_ids", (T,), torch.int32)
        _one_device(x=x, adapter_ids=adapter_ids, a=adapters.a)

    def call(ws, nbytes, st):
        _check(_lib.strata_moe_decode(_ptr(x), _ptr(router_w), ctypes.byref(experts.struct), T, K,
                                      None if adapters is None else ctypes.byref(adapters.struct), _ptr(adapter_ids),
                                      _ptr(out), ws, nbytes, st), "strata_moe_decode")
        return out

    return _with_workspace(call, x.device, workspace,
                           lambda: strata_moe_decode_workspace_bytes(T, K, experts, adapters), stream)


# ------------------------------------- 4-bit floating point, norms of a block
# These calls take the GPU a few microseconds for a token, so their checks read
# each tensor's properties once and go past torch's context managers.
_Tensor = torch.Tensor
_get_device, _raw_stream = torch._C._cuda_getDevice, torch._C._cuda_getCurrentRawStream
_row_code = ROW_DTYPES.get


def _float_rows(t, name: str, rows: int | None = None, width: int | None = None) -> tuple[int, int, int, int]:
    """A [rows][width] fp32, fp16 or bf16 tensor with contiguous rows that do not overlap -> (rows, width, row
    stride, type code)."""
    if not isinstance(t, _Tensor):
        raise TypeError(f"{name} must be a torch tensor")
    code = _row_code(t.dtype)
    if code is None:
        raise TypeError(f"{name} must be one of {sorted(str(d) for d in ROW_DTYPES)}, got {t.dtype}")
    shape = t.shape
    if len(shape) != 2 or (rows is not None and shape[0] != rows) or (width is not None and shape[1] != width):
        want = "2-D" if rows is None and width is None else (rows, width)
        raise ValueError(f"{name} has shape {tuple(shape)}, expected {want}")
    n, w = shape
    if t.is_contiguous():
        return n, w, w, code
    stride, col = t.stride()
    if (w > 1 and n > 0 and col != 1) or (n > 1 and stride < w):
        raise ValueError(f"{name} must have contiguous rows that do not overlap")
    return n, w, stride if n > 1 else w, code


def _array(t, name: str, shape: tuple, dt, dev: int):
    """A contiguous tensor of this shape and type on device `dev`, or None -> its pointer."""
    if t is None:
        return None
    if not isinstance(t, _Tensor):
        raise TypeError(f"{name} must be a torch tensor")
    if t.dtype is not dt:
        raise TypeError(f"{name} must be {dt}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {shape}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if t.get_device() != dev:
        raise ValueError(f"{name} is on another device")
    return t.data_ptr()


def _same_device(t, name: str, dev: int):
    if t.get_device() != dev:
        raise ValueError(f"{name} is on another device")


def _run_on(dev: int, stream, fn, *args) -> None:
    """fn(*args, stream) with device `dev` current, on its current stream if none is given."""
    if dev < 0:
        raise TypeError(f"{fn.__name__} takes CUDA (HIP) tensors")
    st = _raw_stream(dev) if stream is None else stream.cuda_stream
    if _get_device() == dev:
        rc = fn(*args, st)
    else:
        with torch.cuda.device(dev):
            rc = fn(*args, st)
    if rc:
        _check(rc, fn.__name__)


def _new_bytes(shape: tuple, like: torch.Tensor, stream) -> torch.Tensor:
    """An output that the call allocates, on the stream that it runs on."""
    with contextlib.nullcontext() if stream is None else torch.cuda.stream(stream):
        return torch.empty(shape, dtype=torch.uint8, device=like.device)


def strata_moe_mxfp_quantize(x: torch.Tensor, codes: torch.Tensor | None = None, scales: torch.Tensor | None = None,
                             stream=None) -> tuple[torch.Tensor, torch.Tensor]:
    """x [rows][cols] (fp32, fp16 or bf16; rows may be padded) -> codes uint8 [rows][cols/2], two 4-bit values a
    byte, and scales uint8 [rows][cols/32], powers of two."""
    rows, cols, xs, code = _float_rows(x, "x")
    dev = x.get_device()
    if dev < 0:
        raise TypeError("x must be a CUDA (HIP) tensor")
    if codes is None:
        codes = _new_bytes((rows, cols // 2), x, stream)
    if scales is None:
        scales = _new_bytes((rows, cols // 32), x, stream)
    _run_on(dev, stream, _lib.strata_moe_mxfp_quantize, x.data_ptr(), code, xs, rows, cols,
            _array(codes, "codes", (rows, cols // 2), torch.uint8, dev),
            _array(scales, "scales", (rows, cols // 32), torch.uint8, dev))
    return codes, scales


def strata_moe_mxfp_dequantize(codes: torch.Tensor, scales: torch.Tensor, out: torch.Tensor,
                               stream=None) -> torch.Tensor:
    """The values that codes and scales stand for, into out [rows][cols] (fp32, fp16 or bf16; rows may be padded)."""
    rows, cols, os_, code = _float_rows(out, "out")
    dev = out.get_device()
    if codes is None or scales is None:
        raise TypeError("codes and scales must be torch tensors")
    _run_on(dev, stream, _lib.strata_moe_mxfp_dequantize, _array(codes, "codes", (rows, cols // 2), torch.uint8, dev),
            _array(scales, "scales", (rows, cols // 32), torch.uint8, dev), rows, cols, out.data_ptr(), code, os_)
    return out


def strata_moe_mxfp_packed_bytes(rows: int, cols: int, swiglu: bool = False) -> int:
    b = _i64()
    _check(_lib.strata_moe_mxfp_packed_bytes(rows, cols, int(swiglu), ctypes.byref(b)), "strata_moe_mxfp_packed_bytes")
    return b.value


class MxfpWeights:
    """n_expert packed 4-bit matrices [rows][cols] in device memory.  swiglu: a matrix is [gate; up] and the product
    gives silu(gate x) (up x) of rows / 2 values."""

    def __init__(self, n_expert: int, rows: int, cols: int, swiglu: bool = False,
                 device: str | torch.device = "cuda"):
        self.n_expert, self.rows, self.cols, self.swiglu = n_expert, rows, cols, bool(swiglu)
        self.n_out = rows // 2 if self.swiglu else rows
        self.stride = strata_moe_mxfp_packed_bytes(rows, cols, self.swiglu)
        if not 1 <= n_expert <= 1024:
            raise ValueError(f"n_expert {n_expert} outside [1, 1024]")
        self.packed = torch.empty(n_expert * self.stride, dtype=torch.uint8, device=device)
        self.struct = MxfpWeightsStruct(n_expert, rows, cols, int(self.swiglu), self.packed.data_ptr(), self.stride)

    def pack(self, e0: int, codes: torch.Tensor, scales: torch.Tensor, stream=None) -> "MxfpWeights":
        """Pack experts [e0, e0 + n) from codes [n][rows][cols/2] and scales [n][rows][cols/32]."""
        strata_moe_mxfp_pack(codes, scales, e0, self, stream)
        return self


def strata_moe_mxfp_pack(codes: torch.Tensor, scales: torch.Tensor, e0: int, weights: MxfpWeights, stream=None) -> None:
    if not isinstance(codes, _Tensor) or codes.dim() != 3:
        raise ValueError("codes must be [n][rows][cols/2]")
    if scales is None:
        raise TypeError("scales must be a torch tensor")
    n, dev = codes.shape[0], codes.get_device()
    if e0 < 0 or e0 + n > weights.n_expert:
        raise ValueError(f"experts [{e0}, {e0 + n}) outside [0, {weights.n_expert})")
    args = (_array(codes, "codes", (n, weights.rows, weights.cols // 2), torch.uint8, dev),
            _array(scales, "scales", (n, weights.rows, weights.cols // 32), torch.uint8, dev))
    _same_device(weights.packed, "weights", dev)
    _run_on(dev, stream, _lib.strata_moe_mxfp_pack, *args, e0, e0 + n, weights.rows, weights.cols, int(weights.swiglu),
            weights.packed.data_ptr(), weights.stride)


def strata_moe_mxfp_product(codes: torch.Tensor, scales: torch.Tensor, weights: MxfpWeights, out: torch.Tensor,
                            offsets: torch.Tensor | None = None, src: torch.Tensor | None = None,
                            stream=None) -> torch.Tensor:
    """out[r] = W_e x[src[r]] for the rows r of expert e, [offsets[e], offsets[e+1]).  codes, scales: x in 4 bits;
    out [rows][n_out] fp32, fp16 or bf16 (rows may be padded).  One expert needs no offsets; without src row r is
    x's row r; a row whose src is outside x is 0."""
    if not isinstance(weights, MxfpWeights):
        raise TypeError("weights must be an MxfpWeights object")
    if not isinstance(codes, _Tensor) or codes.dim() != 2:
        raise ValueError("codes must be [x_rows][cols/2]")
    if scales is None:
        raise TypeError("scales must be a torch tensor")
    x_rows = codes.shape[0]
    rows, _, os_, code = _float_rows(out, "out", None, weights.n_out)
    dev = out.get_device()
    args = (_array(codes, "codes", (x_rows, weights.cols // 2), torch.uint8, dev),
            _array(scales, "scales", (x_rows, weights.cols // 32), torch.uint8, dev), x_rows,
            ctypes.byref(weights.struct), _array(offsets, "offsets", (weights.n_expert + 1,), torch.int32, dev),
            _array(src, "src", (rows,), torch.int32, dev))
    _same_device(weights.packed, "weights", dev)
    _run_on(dev, stream, _lib.strata_moe_mxfp_product, *args, rows, out.data_ptr(), code, os_)
    return out


class Norm:
    """A root mean square norm: v / sqrt(mean(v^2) + eps) * (weight_offset + weight); weight [H] float32 or None.
    The weight's memory is read by each call; eps, the offset and which memory it is are fixed here."""

    def __init__(self, weight: torch.Tensor | None = None, eps: float = 1e-6, weight_offset: float = 0.0):
        self.width = self.device = None
        if weight is not None:
            if not isinstance(weight, _Tensor) or weight.dim() != 1:
                raise ValueError("weight must be a 1-D [H] tensor")
            _dtype(weight, torch.float32, "weight")
            if not weight.is_contiguous():
                raise ValueError("weight must be contiguous")
            self.width, self.device = weight.shape[0], weight.get_device()
        self.weight, self.eps, self.weight_offset = weight, eps, weight_offset
        self.struct = NormStruct(None if weight is None else weight.data_ptr(), weight_offset, eps)
        self.pointer = ctypes.pointer(self.struct)


def _norm(norm, name: str, H: int, dev: int):
    """A Norm for rows of H, or None -> the pointer to its struct."""
    if norm is None:
        return None
    if not isinstance(norm, Norm):
        raise TypeError(f"{name} must be a Norm object")
    if norm.weight is not None:
        if norm.width != H:
            raise ValueError(f"{name} has a weight of {norm.width} values for rows of {H}")
        if norm.device != dev:
            raise ValueError(f"{name} is on another device")
    return norm.pointer


def _norm_outputs(x, codes, scales, T: int, H: int, dev: int) -> tuple:
    if codes is None and scales is None:
        return _array(x, "x", (T, H), torch.float32, dev), None, None
    if codes is None or scales is None:
        raise ValueError("codes and scales come together")
    return (_array(x, "x", (T, H), torch.float32, dev), _array(codes, "codes", (T, H // 2), torch.uint8, dev),
            _array(scales, "scales", (T, H // 32), torch.uint8, dev))


def strata_moe_norm_before(h: torch.Tensor, norm: Norm, x: torch.Tensor | None = None,
                           codes: torch.Tensor | None = None, scales: torch.Tensor | None = None, stream=None) -> None:
    """x = norm(h): the layer's fp32 input from the residual stream h [T][H] (fp32, fp16 or bf16; rows may be
    padded), and with codes and scales (uint8, as strata_moe_mxfp_quantize) x in 4 bits."""
    if norm is None:
        raise TypeError("norm must be a Norm object")
    T, H, hs, code = _float_rows(h, "h")
    dev = h.get_device()
    _run_on(dev, stream, _lib.strata_moe_norm_before, h.data_ptr(), code, hs, T, H,
            _norm(norm, "norm", H, dev), *_norm_outputs(x, codes, scales, T, H, dev))


def strata_moe_norm_after(h: torch.Tensor, y: torch.Tensor, out: torch.Tensor, norm: Norm | None = None,
                          slot: torch.Tensor | None = None, p: torch.Tensor | None = None,
                          gate: torch.Tensor | None = None, residual_scale: float = 1.0, block_scale: float = 1.0,
                          next_norm: Norm | None = None, x: torch.Tensor | None = None,
                          codes: torch.Tensor | None = None, scales: torch.Tensor | None = None,
                          stream=None) -> torch.Tensor:
    """out = residual_scale h + block_scale gate norm(v), v[t] = y[t], or with slot and p [T][K] the sum over k of
    p[t][k] y[slot[t][k]].  gate: float32 [H], [T][1] or [T][H].  out may be h.  next_norm: also the next block's
    input x = next_norm(out) (x, codes and scales as in strata_moe_norm_before)."""
    T, H, hs, code = _float_rows(h, "h")
    dev = h.get_device()
    if out is h:
        os_ = hs
    else:
        _, _, os_, out_code = _float_rows(out, "out", T, H)
        if out_code != code:
            raise TypeError(f"out must be {h.dtype}, got {out.dtype}")
        _same_device(out, "out", dev)
    y_rows, _, ys, y_code = _float_rows(y, "y", None, H)
    _same_device(y, "y", dev)
    K, slots, weights = 0, None, None
    if (slot is None) != (p is None):
        raise ValueError("slot and p come together")
    if slot is not None:
        if not isinstance(slot, _Tensor) or slot.dim() != 2:
            raise ValueError("slot must be [T][K]")
        K = slot.shape[1]
        if K == 0:  # without memory the tensors would pass for None
            raise ValueError("slot must have at least one row of y a token")
        slots, weights = _array(slot, "slot", (T, K), torch.int32, dev), _array(p, "p", (T, K), torch.float32, dev)
    elif y_rows != T:
        raise ValueError(f"y has {y_rows} rows for {T} tokens")
    gates, grow, gcol = None, 0, 0
    if gate is not None:
        if not isinstance(gate, _Tensor):
            raise TypeError("gate must be a torch tensor")
        if gate.dtype is not torch.float32:
            raise TypeError(f"gate must be {torch.float32}, got {gate.dtype}")
        shape = gate.shape
        if shape != (H,) and shape != (T, 1) and shape != (T, H):
            raise ValueError(f"gate has shape {tuple(shape)}, expected {(H,)}, {(T, 1)} or {(T, H)}")
        stride = gate.stride()
        grow = stride[0] if len(shape) == 2 and T > 1 else 0
        gcol = stride[-1] if shape[-1] > 1 else 0
        if gcol not in (0, 1) or grow < 0:
            raise ValueError("gate must have contiguous or broadcast rows")
        _same_device(gate, "gate", dev)
        gates = gate.data_ptr()
    branch = BranchStruct(y.data_ptr(), ys, y_rows, y_code, K, slots, weights,
                          _norm(norm, "norm", H, dev), gates, grow, gcol, residual_scale, block_scale)
    _run_on(dev, stream, _lib.strata_moe_norm_after, h.data_ptr(), code, hs, T, H, ctypes.byref(branch),
            out.data_ptr(), os_, _norm(next_norm, "next_norm", H, dev), *_norm_outputs(x, codes, scales, T, H, dev))
    return out


# -------------------------------------------------------------- single steps
def strata_moe_route(x, router_w, bias, K: int, ids=None, p=None, stream=None):
    if not isinstance(x, torch.Tensor) or x.dim() != 2 or not isinstance(router_w, torch.Tensor) or router_w.dim() != 2:
        raise ValueError("x must be [T][H] and router_w [H][E]")
    T, H = x.shape
    E = router_w.shape[1]
    _expect(x, "x", (T, H), torch.float32)
    _expect(router_w, "router_w", (H, E), torch.float32)
    if bias is not None:
        _expect(bias, "bias", (E,), torch.float32)
    if ids is not None:
        _expect(ids, "ids", (T, K), torch.int32)
    if p is not None:
        _expect(p, "p", (T, K), torch.float32)
    _one_device(x=x, router_w=router_w, bias=bias, ids=ids, p=p)
    ids = torch.empty((T, K), dtype=torch.int32, device=x.device) if ids is None else ids
    p = torch.empty((T, K), dtype=torch.float32, device=x.device) if p is None else p
    _check(_lib.strata_moe_route(_ptr(x), _ptr(router_w), _ptr(bias), T, H, E, K, _ptr(ids), _ptr(p),
                                 _stream(stream)), "strata_moe_route")
    return ids, p


def strata_moe_group(ids, E: int, stream=None):
    if not isinstance(ids, torch.Tensor) or ids.dim() != 2:
        raise ValueError("ids must be a 2-D [T][K] tensor")
    _dtype(ids, torch.int32, "ids")
    _one_device(ids=ids)
    T, K = ids.shape
    dev = ids.device
    offsets = torch.empty(E + 1, dtype=torch.int32, device=dev)
    src = torch.empty(T * K, dtype=torch.int32, device=dev)
    slot = torch.empty(T * K, dtype=torch.int32, device=dev)
    _check(_lib.strata_moe_group(_ptr(ids), T, K, E, _ptr(offsets), _ptr(src), _ptr(slot), _stream(stream)),
           "strata_moe_group")
    return offsets, src, slot


def strata_moe_quantize(v, stream=None):
    if not isinstance(v, torch.Tensor) or v.dim() != 2:
        raise ValueError("v must be a 2-D [rows][cols] tensor")
    _dtype(v, torch.float32, "v")
    _one_device(v=v)
    rows, cols = v.shape
    codes = torch.empty((rows, cols), dtype=torch.int8, device=v.device)
    scales = torch.empty((rows, cols // 32), dtype=torch.float32, device=v.device)
    _check(_lib.strata_moe_quantize(_ptr(v), rows, cols, _ptr(codes), _ptr(scales), _stream(stream)),
           "strata_moe_quantize")
    return codes, scales


def strata_moe_gate_up(qx, sx, offsets, src, K: int, experts: Experts, stream=None):
    if not isinstance(qx, torch.Tensor) or qx.dim() != 2:
        raise ValueError("qx must be a 2-D [T][H] tensor")
    T = qx.shape[0]
    n, I, H, E = T * K, experts.ffn, experts.hidden, experts.n_expert
    _expect(qx, "qx", (T, H), torch.int8)
    _expect(sx, "sx", (T, H // 32), torch.float32)
    _expect(offsets, "offsets", (E + 1,), torch.int32)
    _expect(src, "src", (n,), torch.int32)
    _one_device(qx=qx, sx=sx, offsets=offsets, src=src, gate_up=experts.gate_up)
    qh = torch.empty((n, I), dtype=torch.int8, device=qx.device)
    sh = torch.empty((n, I // 32), dtype=torch.float32, device=qx.device)
    _check(_lib.strata_moe_gate_up(_ptr(qx), _ptr(sx), _ptr(offsets), _ptr(src), T, K, ctypes.byref(experts.struct),
                                   _ptr(qh), _ptr(sh), _stream(stream)), "strata_moe_gate_up")
    return qh, sh


def strata_moe_down(qh, sh, offsets, src, slot, p, experts: Experts, out, stream=None):
    if not isinstance(p, torch.Tensor) or p.dim() != 2:
        raise ValueError("p must be a 2-D [T][K] tensor")
    T, K = p.shape
    n, I, H, E = T * K, experts.ffn, experts.hidden, experts.n_expert
    _expect(qh, "qh", (n, I), torch.int8)
    _expect(sh, "sh", (n, I // 32), torch.float32)
    _expect(offsets, "offsets", (E + 1,), torch.int32)
    _expect(src, "src", (n,), torch.int32)
    _expect(slot, "slot", (n,), torch.int32)
    _expect(p, "p", (T, K), torch.float32)
    _expect(out, "out", (T, H), torch.float32)
    _one_device(qh=qh, sh=sh, offsets=offsets, src=src, slot=slot, p=p, out=out, down=experts.down)
    _check(_lib.strata_moe_down(_ptr(qh), _ptr(sh), _ptr(offsets), _ptr(src), _ptr(slot), _ptr(p), T, K,
                                ctypes.byref(experts.struct), _ptr(out), _stream(stream)), "strata_moe_down")
    return out


# -------------------------------------------------------------------- timing
def strata_moe_timing(enable: bool, max_calls: int = 0) -> None:
    _check(_lib.strata_moe_timing(int(enable), max_calls), "strata_moe_timing")


def strata_moe_timing_read() -> dict:
    """{kernel kind: (total ms, launches)} of the current timing session."""
    n = _lib.strata_moe_timing_kinds()
    ms = (ctypes.c_double * n)()
    cnt = (_i32 * n)()
    _check(_lib.strata_moe_timing_read(ms, cnt, n), "strata_moe_timing_read")
    return {_lib.strata_moe_timing_name(i).decode(): (ms[i], cnt[i]) for i in range(n)}

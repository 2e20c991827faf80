"""ctypes binding of libreplayssm (argument marshalling only).

Every function here has the name of a C entry point of include/replayssm.h
without the `replayssm_` prefix, takes torch tensors that already live on the
GPU, passes their data pointers and the current HIP stream, and raises
ReplaySSMError on a non-zero status. No computation happens in Python and there
is no fallback: if the library is missing, loading fails loudly.

torch is imported first on purpose: the library then binds to the HIP runtime
that torch already loaded (same SONAME), so torch's device pointers and
streams are valid in it.
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional

import torch

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libreplayssm.so")

MAMBA2, GDN, KDA = 0, 1, 2
FP32, FP32_HP_BF16_LP, BF16_SHARED = 0, 1, 2
PRECISIONS = {"fp32": FP32, "fp32_hp_bf16_lp": FP32_HP_BF16_LP, "bf16_shared": BF16_SHARED}
KINDS = {"mamba2": MAMBA2, "gdn": GDN, "kda": KDA}

OK, EINVAL, ENOTSUP, EHIP = 0, -1, -2, -3
TILES_AUTO, TILES_ONE, TILES_TWO = 0, 1, 2
(DEVERR_APPEND_OVERFLOW, DEVERR_PENDING, DEVERR_ACCEPT, DEVERR_CORRUPT, DEVERR_STALE, DEVERR_INDEX, DEVERR_RANGE) = \
    1, 2, 4, 8, 16, 32, 64
F32, BF16, F16 = 0, 1, 2
DTYPES = {"f32": F32, "bf16": BF16, "f16": F16}
TORCH_DTYPES = {F32: torch.float32, BF16: torch.bfloat16, F16: torch.float16}
NORM_L2, NORM_RMS = 0, 1
NORMS = {"l2": NORM_L2, "rms": NORM_RMS}
GATE_NONE, GATE_BEFORE, GATE_AFTER = 0, 1, 2
GATES = {"none": GATE_NONE, None: GATE_NONE, "before": GATE_BEFORE, "after": GATE_AFTER}
DELTA_BLOCK = 64
RAGGED_SEQS = 16384

_i32 = ctypes.c_int32
_i64 = ctypes.c_int64
_vp = ctypes.c_void_p


class Config(ctypes.Structure):
    _fields_ = [("kind", _i32), ("precision", _i32), ("B", _i32), ("H", _i32), ("dv", _i32),
                ("dk", _i32), ("L", _i32), ("T_max", _i32)]


class State(ctypes.Structure):
    _fields_ = [("hp", _vp), ("lp", _vp), ("ring_alpha", _vp), ("ring_beta", _vp), ("ring_k", _vp),
                ("ring_v", _vp), ("head", _vp), ("h", _vp), ("p", _vp), ("folded", _vp),
                ("arrive", _vp), ("err", _vp), ("ring_vraw", _vp)]


class Sizes(ctypes.Structure):
    _fields_ = [("C", _i32), ("alignment", _i32), ("hp_bytes", _i64), ("lp_bytes", _i64),
                ("ring_alpha_bytes", _i64), ("ring_beta_bytes", _i64), ("ring_k_bytes", _i64),
                ("ring_v_bytes", _i64), ("ptr_bytes", _i64), ("folded_bytes", _i64),
                ("err_bytes", _i64), ("ring_vraw_bytes", _i64)]


class ConvConfig(ctypes.Structure):
    _fields_ = [("B", _i32), ("D", _i32), ("W", _i32), ("T_max", _i32)]


class ConvState(ctypes.Structure):
    _fields_ = [("ring", _vp), ("start", _vp), ("pend", _vp), ("arrive", _vp), ("err", _vp)]


class RaggedConfig(ctypes.Structure):
    _fields_ = [("n_seqs", _i32), ("block", _i32), ("max_tokens", _i64)]


class Ragged(ctypes.Structure):
    _fields_ = [("cu_tokens", _vp), ("cu_blocks", _vp), ("token_seq", _vp), ("token_pos", _vp), ("block_seq", _vp),
                ("err", _vp)]


class QkNormConfig(ctypes.Structure):
    _fields_ = [("n_tokens", _i32), ("Hq", _i32), ("Hk", _i32), ("D", _i32), ("norm", _i32), ("rot", _i32),
                ("interleaved", _i32), ("rep", _i32), ("dtype", _i32), ("out_dtype", _i32), ("eps", ctypes.c_float),
                ("q_scale", ctypes.c_float), ("q_stride", _i64), ("k_stride", _i64)]


class DeltaConfig(ctypes.Structure):
    _fields_ = [("n_seqs", _i32), ("H", _i32), ("Hk", _i32), ("dk", _i32), ("dv", _i32), ("dtype", _i32),
                ("n_tokens", _i64), ("q_stride", _i64), ("k_stride", _i64), ("v_stride", _i64),
                ("scale", ctypes.c_float)]


class ConvPromptConfig(ctypes.Structure):
    _fields_ = [("n_seqs", _i32), ("D", _i32), ("W", _i32), ("silu", _i32), ("dtype", _i32), ("n_tokens", _i64),
                ("x_stride", _i64)]


class LinearConfig(ctypes.Structure):
    _fields_ = [("n_seqs", _i32), ("H", _i32), ("Hk", _i32), ("dk", _i32), ("dv", _i32), ("dtype", _i32),
                ("n_tokens", _i64), ("q_stride", _i64), ("k_stride", _i64), ("v_stride", _i64),
                ("scale", ctypes.c_float), ("segment", _i32)]


class GatedNormConfig(ctypes.Structure):
    _fields_ = [("n_tokens", _i32), ("groups", _i32), ("D", _i32), ("gate", _i32), ("shared", _i32), ("dtype", _i32),
                ("eps", ctypes.c_float), ("x_stride", _i64), ("z_stride", _i64)]


class ReplaySSMError(RuntimeError):
    def __init__(self, status: int, where: str, text: str):
        super().__init__(f"{where}: status {status} ({text})")
        self.status = status


# entry point name -> argument types (all return int, except the two string functions)
SIGNATURES = {
    "replayssm_get_sizes": [ctypes.POINTER(Config), ctypes.POINTER(Sizes)],
    "replayssm_init": [ctypes.POINTER(Config), ctypes.POINTER(State), _vp],
    "replayssm_pack_state": [ctypes.POINTER(Config), _vp, _vp, _vp, _vp],
    "replayssm_unpack_state": [ctypes.POINTER(Config), _vp, _vp, _vp, _vp],
    "replayssm_read_error": [ctypes.POINTER(State), ctypes.POINTER(_i32), _vp],
    "replayssm_append": [ctypes.POINTER(Config), ctypes.POINTER(State), ctypes.c_int, _vp, _vp, _vp, _vp, _vp],
    "replayssm_append_static": [ctypes.POINTER(Config), ctypes.POINTER(State), ctypes.c_int, _vp, _vp, _vp, _vp,
                                _vp],
    "replayssm_append_dt": [ctypes.POINTER(Config), ctypes.POINTER(State), ctypes.c_int, _vp, _vp, _vp, _vp, _vp,
                            _vp, _vp],
    "replayssm_decode": [ctypes.POINTER(Config), ctypes.POINTER(State), _vp, _vp, _vp],
    "replayssm_conv_sizes": [ctypes.POINTER(ConvConfig), ctypes.POINTER(_i64), ctypes.POINTER(_i64)],
    "replayssm_conv_init": [ctypes.POINTER(ConvConfig), ctypes.POINTER(ConvState), _vp],
    "replayssm_conv_step": [ctypes.POINTER(ConvConfig), ctypes.POINTER(ConvState), ctypes.c_int, _vp, _vp, _vp,
                            ctypes.c_int, ctypes.c_int, _vp, _vp],
    "replayssm_conv_accept": [ctypes.POINTER(ConvConfig), ctypes.POINTER(ConvState), _vp, _vp],
    "replayssm_verify": [ctypes.POINTER(Config), ctypes.POINTER(State), ctypes.c_int, _vp, _vp, _vp],
    "replayssm_decode_step": [ctypes.POINTER(Config), ctypes.POINTER(State), _vp, _vp, _vp, _vp, _vp, _vp, _vp],
    "replayssm_verify_step": [ctypes.POINTER(Config), ctypes.POINTER(State), ctypes.c_int, _vp, _vp, _vp, _vp, _vp,
                              _vp, _vp],
    "replayssm_accept": [ctypes.POINTER(Config), ctypes.POINTER(State), _vp, _vp],
    "replayssm_flush": [ctypes.POINTER(Config), ctypes.POINTER(State), _vp],
    "replayssm_eager_step": [ctypes.POINTER(Config), _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp],
    "replayssm_eager_verify": [ctypes.POINTER(Config), _vp, _vp, ctypes.c_int, _vp, _vp, _vp, _vp, _vp, _vp, _vp],
    "replayssm_eager_accept": [ctypes.POINTER(Config), _vp, _vp, ctypes.c_int, _vp],
    "replayssm_probe_read": [_vp, ctypes.c_int64, _vp, _vp],
    "replayssm_set_tiling": [ctypes.c_int],
    "replayssm_get_tiling": [],
    "replayssm_flush_selected": [ctypes.POINTER(Config), ctypes.POINTER(State), _vp, _vp],
    "replayssm_snapshot": [ctypes.POINTER(Config), ctypes.POINTER(State), ctypes.c_int, _vp, _vp, _vp],
    "replayssm_restore": [ctypes.POINTER(Config), ctypes.POINTER(State), ctypes.c_int, _vp, _vp, _vp],
    "replayssm_ragged_sizes": [ctypes.POINTER(RaggedConfig), ctypes.POINTER(_i64)],
    "replayssm_ragged_maps": [ctypes.POINTER(RaggedConfig), ctypes.POINTER(Ragged), _vp, _vp, _vp],
    "replayssm_qk_norm_sizes": [ctypes.POINTER(QkNormConfig), ctypes.POINTER(_i64)],
    "replayssm_qk_norm": [ctypes.POINTER(QkNormConfig)] + [_vp] * 9,
    "replayssm_qk_norm_backward": [ctypes.POINTER(QkNormConfig)] + [_vp] * 14,
    "replayssm_delta_step": [ctypes.POINTER(DeltaConfig), _vp, _vp, ctypes.c_int] + [_vp] * 10,
    "replayssm_delta_prompt": [ctypes.POINTER(DeltaConfig), ctypes.POINTER(Ragged)] + [_vp] * 11,
    "replayssm_delta_prompt_backward": [ctypes.POINTER(DeltaConfig), ctypes.POINTER(Ragged)] + [_vp] * 17,
    "replayssm_delta_sizes": [ctypes.POINTER(DeltaConfig), ctypes.POINTER(_i64), ctypes.POINTER(_i64)],
    "replayssm_conv_prompt_sizes": [ctypes.POINTER(ConvPromptConfig), ctypes.POINTER(_i64)],
    "replayssm_conv_prompt": [ctypes.POINTER(ConvPromptConfig), ctypes.POINTER(Ragged)] + [_vp] * 8,
    "replayssm_conv_prompt_backward": [ctypes.POINTER(ConvPromptConfig), ctypes.POINTER(Ragged)] + [_vp] * 13,
    "replayssm_conv_restore": [ctypes.POINTER(ConvConfig), ctypes.POINTER(ConvState), ctypes.c_int, _vp, _vp, _vp],
    "replayssm_linear_segment": [ctypes.POINTER(LinearConfig), ctypes.POINTER(_i32)],
    "replayssm_linear_sizes": [ctypes.POINTER(LinearConfig), ctypes.POINTER(_i64), ctypes.POINTER(_i64)],
    "replayssm_linear_step": [ctypes.POINTER(LinearConfig), _vp, _vp, ctypes.c_int] + [_vp] * 11,
    "replayssm_linear_prompt": [ctypes.POINTER(LinearConfig), ctypes.POINTER(Ragged)] + [_vp] * 12,
    "replayssm_linear_prompt_backward": [ctypes.POINTER(LinearConfig), ctypes.POINTER(Ragged)] + [_vp] * 19,
    "replayssm_gated_norm_sizes": [ctypes.POINTER(GatedNormConfig), ctypes.POINTER(_i64)],
    "replayssm_gated_norm": [ctypes.POINTER(GatedNormConfig)] + [_vp] * 5,
    "replayssm_gated_norm_backward": [ctypes.POINTER(GatedNormConfig)] + [_vp] * 9,
}
STRING_FUNCTIONS = {"replayssm_status_string": [ctypes.c_int], "replayssm_last_error": []}

_lib = None


def lib():
    """The loaded library; raises if it was not built (there is no fallback)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with `python -m ssm_decode_amd.build`")
        L = ctypes.CDLL(LIB_PATH)
        for name, args in SIGNATURES.items():
            fn = getattr(L, name)
            fn.argtypes = args
            fn.restype = ctypes.c_int
        for name, args in STRING_FUNCTIONS.items():
            fn = getattr(L, name)
            fn.argtypes = args
            fn.restype = ctypes.c_char_p
        _lib = L
    return _lib


def _check(status: int, where: str) -> None:
    if status != OK:
        raise ReplaySSMError(status, where, lib().replayssm_last_error().decode())


def _p(t: Optional[torch.Tensor]):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("tensor must be on the GPU")
    if not t.is_contiguous():
        raise ValueError("tensor must be contiguous")
    return t.data_ptr()


def _s(stream) -> Optional[int]:
    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else stream


def _f32(t):
    if t is not None and t.dtype != torch.float32:
        raise TypeError("float32 tensor expected")
    return _p(t)


def _i32t(t):
    if t.dtype != torch.int32:
        raise TypeError("int32 tensor expected")
    return _p(t)


def make_config(kind="mamba2", precision="fp32", B=1, H=1, dv=64, dk=128, L=16, T_max=1) -> Config:
    return Config(KINDS.get(kind, kind), PRECISIONS.get(precision, precision), B, H, dv, dk, L, T_max)


def get_sizes(cfg: Config) -> Sizes:
    out = Sizes()
    _check(lib().replayssm_get_sizes(ctypes.byref(cfg), ctypes.byref(out)), "get_sizes")
    return out


def status_string(status: int) -> str:
    return lib().replayssm_status_string(status).decode()


def last_error() -> str:
    return lib().replayssm_last_error().decode()


def init(cfg, st, stream=None):
    _check(lib().replayssm_init(ctypes.byref(cfg), ctypes.byref(st), _s(stream)), "init")


def pack_state(cfg, src, hp=None, lp=None, stream=None):
    _check(lib().replayssm_pack_state(ctypes.byref(cfg), _f32(src), _p(hp), _p(lp), _s(stream)), "pack_state")


def unpack_state(cfg, hp, lp, dst, stream=None):
    _check(lib().replayssm_unpack_state(ctypes.byref(cfg), _p(hp), _p(lp), _f32(dst), _s(stream)), "unpack_state")


def read_error(st, stream=None) -> int:
    v = _i32(0)
    _check(lib().replayssm_read_error(ctypes.byref(st), ctypes.byref(v), _s(stream)), "read_error")
    return int(v.value)


def append(cfg, st, T, alpha, k, v, beta=None, stream=None):
    _check(lib().replayssm_append(ctypes.byref(cfg), ctypes.byref(st), int(T), _f32(alpha), _f32(k),
                                  _f32(v), _f32(beta), _s(stream)), "append")


def append_static(cfg, st, T, alpha, k, v, beta=None, stream=None):
    _check(lib().replayssm_append_static(ctypes.byref(cfg), ctypes.byref(st), int(T), _f32(alpha), _f32(k),
                                         _f32(v), _f32(beta), _s(stream)), "append_static")


def append_dt(cfg, st, T, dt, A, dt_bias, k, v, beta=None, stream=None):
    _check(lib().replayssm_append_dt(ctypes.byref(cfg), ctypes.byref(st), int(T), _f32(dt), _f32(A), _f32(dt_bias),
                                     _f32(k), _f32(v), _f32(beta), _s(stream)), "append_dt")


def decode(cfg, st, q, out, stream=None):
    _check(lib().replayssm_decode(ctypes.byref(cfg), ctypes.byref(st), _f32(q), _f32(out), _s(stream)), "decode")


def verify(cfg, st, T, q, out, stream=None):
    _check(lib().replayssm_verify(ctypes.byref(cfg), ctypes.byref(st), int(T), _f32(q), _f32(out),
                                  _s(stream)), "verify")


def decode_step(cfg, st, alpha, k, v, beta, q, out, stream=None):
    _check(lib().replayssm_decode_step(ctypes.byref(cfg), ctypes.byref(st), _f32(alpha), _f32(k), _f32(v),
                                       _f32(beta), _f32(q), _f32(out), _s(stream)), "decode_step")


def verify_step(cfg, st, T, alpha, k, v, beta, q, out, stream=None):
    _check(lib().replayssm_verify_step(ctypes.byref(cfg), ctypes.byref(st), int(T), _f32(alpha), _f32(k),
                                       _f32(v), _f32(beta), _f32(q), _f32(out), _s(stream)), "verify_step")


def accept(cfg, st, accepted, stream=None):
    _check(lib().replayssm_accept(ctypes.byref(cfg), ctypes.byref(st), _i32t(accepted), _s(stream)), "accept")


def flush(cfg, st, stream=None):
    _check(lib().replayssm_flush(ctypes.byref(cfg), ctypes.byref(st), _s(stream)), "flush")


def eager_step(cfg, S, alpha, k, v, beta, q, out, stream=None):
    _check(lib().replayssm_eager_step(ctypes.byref(cfg), _f32(S), _f32(alpha), _f32(k), _f32(v),
                                      _f32(beta), _f32(q), _f32(out), _s(stream)), "eager_step")


def eager_verify(cfg, pool, slot, T, alpha, k, v, beta, q, out, stream=None):
    _check(lib().replayssm_eager_verify(ctypes.byref(cfg), _f32(pool), _i32t(slot), int(T), _f32(alpha),
                                        _f32(k), _f32(v), _f32(beta), _f32(q), _f32(out), _s(stream)),
           "eager_verify")


def eager_accept(cfg, slot, accepted, T, stream=None):
    _check(lib().replayssm_eager_accept(ctypes.byref(cfg), _i32t(slot), _i32t(accepted), int(T), _s(stream)),
           "eager_accept")


def flush_selected(cfg, st, select, stream=None):
    _check(lib().replayssm_flush_selected(ctypes.byref(cfg), ctypes.byref(st), _i32t(select), _s(stream)),
           "flush_selected")


def snapshot(cfg, st, seqs, dst, stream=None):
    _check(lib().replayssm_snapshot(ctypes.byref(cfg), ctypes.byref(st), int(seqs.numel()), _i32t(seqs), _f32(dst),
                                    _s(stream)), "snapshot")


def restore(cfg, st, seqs, src, stream=None):
    _check(lib().replayssm_restore(ctypes.byref(cfg), ctypes.byref(st), int(seqs.numel()), _i32t(seqs), _f32(src),
                                   _s(stream)), "restore")


def set_tiling(policy):
    """replayssm_set_tiling: TILES_AUTO, TILES_ONE or TILES_TWO (process-wide; results unchanged)."""
    _check(lib().replayssm_set_tiling(int(policy)), "set_tiling")


def get_tiling():
    return int(lib().replayssm_get_tiling())


def probe_read(src, sink, stream=None):
    """Enqueue one pass of the read-ceiling probe over `src` (a CUDA tensor); `sink` is one float32."""
    _check(lib().replayssm_probe_read(_p(src), ctypes.c_int64(src.numel() * src.element_size()), _f32(sink),
                                      _s(stream)), "probe_read")


class LayerState:
    """Device memory (torch tensors) for one layer's ReplaySSM state, plus the C struct.

    Memory plumbing only: sizes come from replayssm_get_sizes, and replayssm_init
    is called once on construction.
    """

    def __init__(self, cfg: Config, device="cuda", stream=None):
        self.cfg = cfg
        sz = get_sizes(cfg)
        self.C = sz.C
        B, H, dv, dk, C = cfg.B, cfg.H, cfg.dv, cfg.dk, sz.C
        f32, i32 = torch.float32, torch.int32
        self.hp = torch.zeros((B, H, dv * dk), dtype=f32, device=device) if sz.hp_bytes else None
        self.lp = torch.zeros((B, H, dv * dk), dtype=torch.int16, device=device) if sz.lp_bytes else None
        # a scalar gate per record, or (KDA) a gate row of dk channels
        self.ring_alpha = torch.zeros((B, H, C, dk) if cfg.kind == KDA else (B, H, C), dtype=f32, device=device)
        self.ring_beta = torch.zeros((B, H, C), dtype=f32, device=device) if sz.ring_beta_bytes else None
        self.ring_k = torch.zeros((B, H, C, dk), dtype=f32, device=device)
        self.ring_v = torch.zeros((B, H, C, dv), dtype=f32, device=device)
        self.head = torch.zeros(B, dtype=i32, device=device)
        self.h = torch.zeros(B, dtype=i32, device=device)
        self.p = torch.zeros(B, dtype=i32, device=device)
        self.folded = torch.zeros(B, dtype=torch.int64, device=device)
        self.arrive = torch.zeros(B, dtype=i32, device=device)
        self.err = torch.zeros(4, dtype=i32, device=device)
        self.ring_vraw = torch.zeros((B, H, C, dv), dtype=f32, device=device) if sz.ring_vraw_bytes else None
        self.struct = State(*[None if t is None else t.data_ptr() for t in (
            self.hp, self.lp, self.ring_alpha, self.ring_beta, self.ring_k, self.ring_v, self.head,
            self.h, self.p, self.folded, self.arrive, self.err, self.ring_vraw)])
        init(cfg, self.struct, stream)

    def import_state(self, S_logical: torch.Tensor, stream=None):
        """Set the checkpoint from logical [B, H, dv, dk] fp32 values (both copies as the mode needs)."""
        pack_state(self.cfg, S_logical.contiguous(), self.hp, self.lp, stream)

    def export_state(self, which: str = "hp", stream=None) -> torch.Tensor:
        """Logical [B, H, dv, dk] fp32 view of the fp32 ("hp") or bf16 ("lp") checkpoint."""
        cfg = self.cfg
        dst = torch.empty((cfg.B, cfg.H, cfg.dv, cfg.dk), dtype=torch.float32, device=self.ring_k.device)
        if which == "hp":
            unpack_state(cfg, self.hp, None, dst, stream)
        else:
            unpack_state(cfg, None, self.lp, dst, stream)
        return dst

    def tensors(self):
        """Every device tensor the layer's state holds."""
        return [t for t in (self.hp, self.lp, self.ring_alpha, self.ring_beta, self.ring_k, self.ring_v, self.head,
                            self.h, self.p, self.folded, self.arrive, self.err, self.ring_vraw) if t is not None]

    def pointers(self):
        return {"head": self.head.tolist(), "h": self.h.tolist(), "p": self.p.tolist(),
                "folded": self.folded.tolist()}


# ---- convolution input ring -------------------------------------------------

def make_conv_config(B, D, W=4, T_max=1) -> ConvConfig:
    return ConvConfig(int(B), int(D), int(W), int(T_max))


def conv_sizes(cfg: ConvConfig):
    ring, ptr = _i64(0), _i64(0)
    _check(lib().replayssm_conv_sizes(ctypes.byref(cfg), ctypes.byref(ring), ctypes.byref(ptr)), "conv_sizes")
    return int(ring.value), int(ptr.value)


def conv_init(cfg, st, stream=None):
    _check(lib().replayssm_conv_init(ctypes.byref(cfg), ctypes.byref(st), _s(stream)), "conv_init")


def conv_step(cfg, st, T, x, w, bias, silu, commit, y, stream=None):
    _check(lib().replayssm_conv_step(ctypes.byref(cfg), ctypes.byref(st), int(T), _f32(x), _f32(w), _f32(bias),
                                     int(bool(silu)), int(bool(commit)), _f32(y), _s(stream)), "conv_step")


def conv_accept(cfg, st, accepted, stream=None):
    _check(lib().replayssm_conv_accept(ctypes.byref(cfg), ctypes.byref(st), _i32t(accepted), _s(stream)),
           "conv_accept")


class ConvLayer:
    """Device memory (torch tensors) for one layer's convolution input ring, plus the C struct;
    replayssm_conv_init is called once on construction."""

    def __init__(self, cfg: ConvConfig, device="cuda", stream=None):
        self.cfg = cfg
        conv_sizes(cfg)  # validates
        self.Cc = cfg.W - 1 + cfg.T_max
        self.ring = torch.empty((cfg.B, self.Cc, cfg.D), dtype=torch.float32, device=device)
        self.start = torch.empty(cfg.B, dtype=torch.int32, device=device)
        self.pend = torch.empty(cfg.B, dtype=torch.int32, device=device)
        self.arrive = torch.empty(cfg.B, dtype=torch.int32, device=device)
        self.err = torch.empty(4, dtype=torch.int32, device=device)
        self.struct = ConvState(*[t.data_ptr() for t in (self.ring, self.start, self.pend, self.arrive, self.err)])
        conv_init(cfg, self.struct, stream)


# ---- the prompt side: ragged tables, query/key norm, the delta rule over sequences ----

# These calls may be a few microseconds of GPU work, so the checks read each tensor attribute once.

def _device_and_stream(stream):
    """The current GPU and the stream a call goes to."""
    try:
        dev = torch.cuda.current_device()
    except RuntimeError as e:
        raise ValueError(f"tensors must be on the GPU: {e}") from e
    if stream is None:
        return dev, torch._C._cuda_getCurrentRawStream(dev)
    return dev, stream.cuda_stream if hasattr(stream, "cuda_stream") else stream


def _off_device(t, dev, what):
    if not t.is_cuda:
        return ValueError(f"{what} must be on the GPU")
    return ValueError(f"{what} is on {t.device}, the current device is cuda:{dev}")


def _dev(t, dev, dtype, shape, what):
    """Pointer of a contiguous tensor of GPU `dev` with this type and shape (None: any); None stays None."""
    if t is None:
        return None
    if t.get_device() != dev:
        raise _off_device(t, dev, what)
    if t.dtype is not dtype:
        raise TypeError(f"{what}: {dtype} tensor expected, got {t.dtype}")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{what}: shape {tuple(shape)} expected, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{what} must be contiguous")
    return t.data_ptr()


def _rows(t, dev, dtype, shape, stride, what):
    """Pointer of [tokens, heads, dim] rows whose heads lie together and whose tokens lie `stride` elements apart; None stays
    None, which the library refuses by name."""
    if t is None:
        return None
    if t.get_device() != dev:
        raise _off_device(t, dev, what)
    if t.dtype is not dtype:
        raise TypeError(f"{what}: {dtype} tensor expected, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{what}: shape {shape} expected, got {tuple(t.shape)}")
    s = t.stride()
    if s[2] != 1 or (s[1] != shape[2] and shape[1] > 1) or (s[0] != stride and shape[0] > 1):
        raise ValueError(f"{what}: strides ({stride}, {shape[2]}, 1) expected, got {s}")
    return t.data_ptr()


def _workspace(t, dev, need):
    if t is None:
        return None
    if t.get_device() != dev:
        raise _off_device(t, dev, "workspace")
    if t.numel() * t.element_size() < need or not t.is_contiguous():
        raise ValueError(f"workspace must be contiguous and hold {need} bytes")
    return t.data_ptr()


def _torch_dtype(value, where):
    if value not in TORCH_DTYPES:
        raise ReplaySSMError(EINVAL, where, f"dtype {value} unknown")
    return TORCH_DTYPES[value]


def make_ragged_config(n_seqs, max_tokens, block=DELTA_BLOCK) -> RaggedConfig:
    return RaggedConfig(int(n_seqs), int(block), int(max_tokens))


def ragged_sizes(cfg: RaggedConfig) -> int:
    n = _i64(0)
    _check(lib().replayssm_ragged_sizes(ctypes.byref(cfg), ctypes.byref(n)), "ragged_sizes")
    return int(n.value)


def ragged_maps(cfg, maps, lengths, history=None, stream=None):
    """replayssm_ragged_maps. Tables of a RaggedMaps have to be large enough for cfg's batches."""
    n = (cfg.n_seqs,)
    room = getattr(maps, "room", None)
    if room is not None:
        need = (cfg.n_seqs, cfg.max_tokens, cfg.max_tokens // max(cfg.block, 1) + cfg.n_seqs)
        for have, want, what in zip(room, need, ("cu_tokens and cu_blocks: requests", "token_seq: tokens", "block_seq: blocks")):
            if want > have:
                raise ValueError(f"{what}: the tables have room for {have}, the configuration needs {want}")
    dev, s = _device_and_stream(stream)
    if room is not None and maps.tensors[0].get_device() != dev:
        raise _off_device(maps.tensors[0], dev, "maps")
    _check(lib().replayssm_ragged_maps(ctypes.byref(cfg), ctypes.byref(maps),
                                       _dev(lengths, dev, torch.int32, n, "lengths"),
                                       _dev(history, dev, torch.int32, n, "history"), s), "ragged_maps")


class RaggedMaps:
    """Device memory (torch tensors) for one packed batch's tables, plus the C struct. Filled by ragged_maps."""

    def __init__(self, cfg: RaggedConfig, device="cuda"):
        self.cfg = cfg
        self.max_blocks = ragged_sizes(cfg)  # validates
        i32 = torch.int32
        self.cu_tokens = torch.zeros(cfg.n_seqs + 1, dtype=i32, device=device)
        self.cu_blocks = torch.zeros(cfg.n_seqs + 1, dtype=i32, device=device)
        self.token_seq = torch.full((cfg.max_tokens,), -1, dtype=i32, device=device)
        self.token_pos = torch.full((cfg.max_tokens,), -1, dtype=i32, device=device)
        self.block_seq = torch.full((self.max_blocks,), -1, dtype=i32, device=device)
        self.err = torch.zeros(4, dtype=i32, device=device)
        tensors = (self.cu_tokens, self.cu_blocks, self.token_seq, self.token_pos, self.block_seq, self.err)
        self.struct = Ragged(*[t.data_ptr() for t in tensors])
        self.struct.tensors = tensors  # the struct may outlive this object
        self.struct.room = (cfg.n_seqs, cfg.max_tokens, self.max_blocks)


def make_qk_norm_config(n_tokens, Hq, Hk, D, norm="l2", rot=0, interleaved=False, rep=1, eps=1e-6, q_scale=1.0,
                        dtype="bf16", out_dtype=None, q_stride=None, k_stride=None) -> QkNormConfig:
    """Strides default to contiguous rows, out_dtype to dtype."""
    out_dtype = dtype if out_dtype is None else out_dtype
    return QkNormConfig(int(n_tokens), int(Hq), int(Hk), int(D), NORMS.get(norm, norm), int(rot),
                        int(bool(interleaved)), int(rep), DTYPES.get(dtype, dtype), DTYPES.get(out_dtype, out_dtype),
                        float(eps), float(q_scale), int(Hq * D if q_stride is None else q_stride),
                        int(Hk * D if k_stride is None else k_stride))


def qk_norm_sizes(cfg: QkNormConfig) -> int:
    n = _i64(0)
    _check(lib().replayssm_qk_norm_sizes(ctypes.byref(cfg), ctypes.byref(n)), "qk_norm_sizes")
    return int(n.value)


def _qk_inputs(cfg, dev, q, k, wq, wk, positions, inv_freq):
    t, n, D, rot, f32 = _torch_dtype(cfg.dtype, "qk_norm"), cfg.n_tokens, cfg.D, cfg.rot, torch.float32
    try:
        return (_rows(q, dev, t, (n, cfg.Hq, D), cfg.q_stride, "q") if cfg.Hq else None,
                _rows(k, dev, t, (n, cfg.Hk, D), cfg.k_stride, "k") if cfg.Hk else None,
                _dev(wq, dev, f32, (D,), "wq"), _dev(wk, dev, f32, (D,), "wk"),
                _dev(positions, dev, torch.int32, (n,), "positions") if rot else None,
                _dev(inv_freq, dev, f32, (rot // 2,), "inv_freq") if rot else None)
    except (TypeError, ValueError):
        qk_norm_sizes(cfg)  # a configuration that the library refuses is named first
        raise


def qk_norm(cfg, q, k, wq, wk, positions, inv_freq, q_out, k_out, stream=None):
    dev, s = _device_and_stream(stream)
    o, n = _torch_dtype(cfg.out_dtype, "qk_norm"), cfg.n_tokens
    _check(lib().replayssm_qk_norm(
        ctypes.byref(cfg), *_qk_inputs(cfg, dev, q, k, wq, wk, positions, inv_freq),
        _dev(q_out, dev, o, (n, cfg.Hq * cfg.rep, cfg.D), "q_out") if cfg.Hq else None,
        _dev(k_out, dev, o, (n, cfg.Hk * cfg.rep, cfg.D), "k_out") if cfg.Hk else None, s), "qk_norm")


def qk_norm_backward(cfg, q, k, wq, wk, positions, inv_freq, dq_out, dk_out, dq, dk, dwq=None, dwk=None,
                     workspace=None, stream=None):
    dev, s = _device_and_stream(stream)
    need = qk_norm_sizes(cfg) if dwq is not None or dwk is not None else 0
    t, o, n, D = _torch_dtype(cfg.dtype, "qk_norm"), _torch_dtype(cfg.out_dtype, "qk_norm"), cfg.n_tokens, cfg.D
    _check(lib().replayssm_qk_norm_backward(
        ctypes.byref(cfg), *_qk_inputs(cfg, dev, q, k, wq, wk, positions, inv_freq),
        _dev(dq_out, dev, o, (n, cfg.Hq * cfg.rep, D), "dq_out") if cfg.Hq else None,
        _dev(dk_out, dev, o, (n, cfg.Hk * cfg.rep, D), "dk_out") if cfg.Hk else None,
        _dev(dq, dev, t, (n, cfg.Hq, D), "dq") if cfg.Hq else None,
        _dev(dk, dev, t, (n, cfg.Hk, D), "dk") if cfg.Hk else None,
        _dev(dwq, dev, torch.float32, (D,), "dwq"), _dev(dwk, dev, torch.float32, (D,), "dwk"),
        _workspace(workspace, dev, need), s), "qk_norm_backward")


def make_delta_config(n_seqs, n_tokens, H, Hk, dk, dv, dtype="bf16", scale=1.0, q_stride=None, k_stride=None,
                      v_stride=None) -> DeltaConfig:
    """Strides default to contiguous rows."""
    return DeltaConfig(int(n_seqs), int(H), int(Hk), int(dk), int(dv), DTYPES.get(dtype, dtype), int(n_tokens),
                       int(Hk * dk if q_stride is None else q_stride), int(Hk * dk if k_stride is None else k_stride),
                       int(H * dv if v_stride is None else v_stride), float(scale))


def delta_sizes(cfg: DeltaConfig):
    """(bytes of delta_prompt's workspace, bytes of delta_prompt_backward's)"""
    f, b = _i64(0), _i64(0)
    _check(lib().replayssm_delta_sizes(ctypes.byref(cfg), ctypes.byref(f), ctypes.byref(b)), "delta_sizes")
    return int(f.value), int(b.value)


def _delta_inputs(cfg, dev, t, q, k, v, g, beta):
    n, f32 = cfg.n_tokens, torch.float32
    return (_rows(q, dev, t, (n, cfg.Hk, cfg.dk), cfg.q_stride, "q"),
            _rows(k, dev, t, (n, cfg.Hk, cfg.dk), cfg.k_stride, "k"),
            _rows(v, dev, t, (n, cfg.H, cfg.dv), cfg.v_stride, "v"), _dev(g, dev, f32, (n, cfg.H), "g"),
            _dev(beta, dev, f32, (n, cfg.H), "beta"))


def _maps(cfg, maps):
    """The C arguments of a batch's configuration and tables; those of a RaggedMaps are checked against the batch. Where
    they have room for fewer tokens than the arrays hold, the call is told that room: no sequence goes further, and the
    kernels then read no table past its end, whatever is in it."""
    room = getattr(maps, "room", None)
    if room is not None:
        n_seqs, tokens, blocks = room
        if n_seqs != cfg.n_seqs:
            raise ValueError(f"cu_tokens: tables of {cfg.n_seqs} sequences expected, got {n_seqs}")
        if blocks < tokens // DELTA_BLOCK + n_seqs:
            raise ValueError(f"block_seq: tables of blocks of {DELTA_BLOCK} expected")
        if tokens < cfg.n_tokens:
            cfg = DeltaConfig.from_buffer_copy(cfg)
            cfg.n_tokens = tokens
    return ctypes.byref(cfg), ctypes.byref(maps)


def _maps_device(maps, dev):
    tensors = getattr(maps, "tensors", None)
    if tensors is not None and tensors[0].get_device() != dev:
        raise _off_device(tensors[0], dev, "maps")


def delta_step(cfg, cu_tokens, slots, n_slots, q, k, v, g, beta, S_in, S_out, out, err, stream=None):
    dev, s = _device_and_stream(stream)
    t, i32, n = _torch_dtype(cfg.dtype, "delta_step"), torch.int32, cfg.n_seqs
    pool = (n_slots, cfg.H, cfg.dv, cfg.dk)
    _check(lib().replayssm_delta_step(
        ctypes.byref(cfg), _dev(cu_tokens, dev, i32, (n + 1,), "cu_tokens"), _dev(slots, dev, i32, (n,), "slots"),
        int(n_slots), *_delta_inputs(cfg, dev, t, q, k, v, g, beta), _dev(S_in, dev, torch.float32, pool, "S_in"),
        _dev(S_out, dev, torch.float32, pool, "S_out"), _dev(out, dev, t, (cfg.n_tokens, cfg.H, cfg.dv), "out"),
        _dev(err, dev, i32, None, "err"), s), "delta_step")


def delta_prompt(cfg, maps, q, k, v, g, beta, S0, out, S_out, workspace, err, stream=None):
    config, tables = _maps(cfg, maps)
    dev, s = _device_and_stream(stream)
    _maps_device(maps, dev)
    need = delta_sizes(cfg)[0]
    t, f32 = _torch_dtype(cfg.dtype, "delta_prompt"), torch.float32
    states = (cfg.n_seqs, cfg.H, cfg.dv, cfg.dk)
    _check(lib().replayssm_delta_prompt(
        config, tables, *_delta_inputs(cfg, dev, t, q, k, v, g, beta),
        _dev(S0, dev, f32, states, "S0"), _dev(out, dev, t, (cfg.n_tokens, cfg.H, cfg.dv), "out"),
        _dev(S_out, dev, f32, states, "S_out"), _workspace(workspace, dev, need),
        _dev(err, dev, torch.int32, None, "err"), s), "delta_prompt")


def delta_prompt_backward(cfg, maps, q, k, v, g, beta, S0, dout, dS_out, dq, dk, dv, dg, dbeta, dS0, workspace, err,
                          stream=None):
    config, tables = _maps(cfg, maps)
    dev, s = _device_and_stream(stream)
    _maps_device(maps, dev)
    need = delta_sizes(cfg)[1]
    t, n, f32 = _torch_dtype(cfg.dtype, "delta_prompt_backward"), cfg.n_tokens, torch.float32
    states, keys, values = (cfg.n_seqs, cfg.H, cfg.dv, cfg.dk), (n, cfg.Hk, cfg.dk), (n, cfg.H, cfg.dv)
    _check(lib().replayssm_delta_prompt_backward(
        config, tables, *_delta_inputs(cfg, dev, t, q, k, v, g, beta),
        _dev(S0, dev, f32, states, "S0"), _dev(dout, dev, t, values, "dout"),
        _dev(dS_out, dev, f32, states, "dS_out"), _dev(dq, dev, t, keys, "dq"), _dev(dk, dev, t, keys, "dk"),
        _dev(dv, dev, t, values, "dv"), _dev(dg, dev, f32, (n, cfg.H), "dg"),
        _dev(dbeta, dev, f32, (n, cfg.H), "dbeta"), _dev(dS0, dev, f32, states, "dS0"),
        _workspace(workspace, dev, need), _dev(err, dev, torch.int32, None, "err"), s), "delta_prompt_backward")


# ---- a Mamba-2 layer on whole sequences: convolution, linear attention, gated norm ----

def make_conv_prompt_config(n_seqs, n_tokens, D, W=4, silu=True, dtype="bf16", x_stride=None) -> ConvPromptConfig:
    """x_stride defaults to contiguous rows."""
    return ConvPromptConfig(int(n_seqs), int(D), int(W), int(bool(silu)), DTYPES.get(dtype, dtype), int(n_tokens),
                            int(D if x_stride is None else x_stride))


def conv_prompt_sizes(cfg: ConvPromptConfig) -> int:
    n = _i64(0)
    _check(lib().replayssm_conv_prompt_sizes(ctypes.byref(cfg), ctypes.byref(n)), "conv_prompt_sizes")
    return int(n.value)


def _channel_rows(t, dev, dtype, shape, stride, what):
    """Pointer of [tokens, channels] rows whose tokens lie `stride` elements apart."""
    if t is None:
        return None
    if t.dim() != 2:
        raise ValueError(f"{what}: shape {shape} expected, got {tuple(t.shape)}")
    return _rows(t.unsqueeze(1), dev, dtype, (shape[0], 1, shape[1]), stride, what)


def _table_room(cfg, maps):
    """The room of a RaggedMaps in (tokens, blocks), checked against the batch; None for tables of the caller's own."""
    room = getattr(maps, "room", None)
    if room is None:
        return None
    if room[0] != cfg.n_seqs:
        raise ValueError(f"cu_tokens: tables of {cfg.n_seqs} sequences expected, got {room[0]}")
    return room[1:]


def _conv_maps(cfg, maps):
    """As _maps: tables with room for fewer tokens than the arrays hold tell the call so."""
    room = _table_room(cfg, maps)
    if room is not None and room[0] < cfg.n_tokens:
        cfg = ConvPromptConfig.from_buffer_copy(cfg)
        cfg.n_tokens = room[0]
    return ctypes.byref(cfg), ctypes.byref(maps)


def _conv_inputs(cfg, dev, x, w, bias, first):
    f32, D, W = torch.float32, cfg.D, cfg.W
    return (_channel_rows(x, dev, _torch_dtype(cfg.dtype, "conv_prompt"), (cfg.n_tokens, D), cfg.x_stride, "x"),
            _dev(w, dev, f32, (D, W), "w"), _dev(bias, dev, f32, (D,), "bias"),
            _dev(first, dev, f32, (cfg.n_seqs, W - 1, D), "first") if W > 1 else None)


def conv_prompt(cfg, maps, x, w, bias, first, y, last, err, stream=None):
    config, tables = _conv_maps(cfg, maps)
    dev, s = _device_and_stream(stream)
    _maps_device(maps, dev)
    conv_prompt_sizes(cfg)
    t, f32 = _torch_dtype(cfg.dtype, "conv_prompt"), torch.float32
    _check(lib().replayssm_conv_prompt(
        config, tables, *_conv_inputs(cfg, dev, x, w, bias, first), _dev(y, dev, t, (cfg.n_tokens, cfg.D), "y"),
        _dev(last, dev, f32, (cfg.n_seqs, cfg.W - 1, cfg.D), "last") if cfg.W > 1 else None,
        _dev(err, dev, torch.int32, None, "err"), s), "conv_prompt")


def conv_prompt_backward(cfg, maps, x, w, bias, first, dy, dlast, dx, dw, dbias, dfirst, workspace, err, stream=None):
    config, tables = _conv_maps(cfg, maps)
    dev, s = _device_and_stream(stream)
    _maps_device(maps, dev)
    need = conv_prompt_sizes(cfg) if dw is not None or dbias is not None else 0
    t, f32, D, W = _torch_dtype(cfg.dtype, "conv_prompt_backward"), torch.float32, cfg.D, cfg.W
    window = (cfg.n_seqs, W - 1, D)
    _check(lib().replayssm_conv_prompt_backward(
        config, tables, *_conv_inputs(cfg, dev, x, w, bias, first), _dev(dy, dev, t, (cfg.n_tokens, D), "dy"),
        _dev(dlast, dev, f32, window, "dlast") if W > 1 else None, _dev(dx, dev, t, (cfg.n_tokens, D), "dx"),
        _dev(dw, dev, f32, (D, W), "dw"), _dev(dbias, dev, f32, (D,), "dbias"),
        _dev(dfirst, dev, f32, window, "dfirst") if W > 1 else None, _workspace(workspace, dev, need),
        _dev(err, dev, torch.int32, None, "err"), s), "conv_prompt_backward")


def conv_restore(cfg, st, seqs, windows, stream=None):
    """Starts sequences seqs of a ConvLayer from the windows that conv_prompt left."""
    n = seqs.shape[0]
    dev, s = _device_and_stream(stream)
    _check(lib().replayssm_conv_restore(
        ctypes.byref(cfg), ctypes.byref(st), int(n), _dev(seqs, dev, torch.int32, (n,), "seqs") if n else None,
        _dev(windows, dev, torch.float32, (n, cfg.W - 1, cfg.D), "windows") if n and cfg.W > 1 else None, s), "conv_restore")


def make_linear_config(n_seqs, n_tokens, H, Hk, dk, dv, dtype="bf16", scale=1.0, q_stride=None, k_stride=None,
                       v_stride=None, segment=None) -> LinearConfig:
    """Strides default to contiguous rows, segment to replayssm_linear_segment's (which refuses bad sizes)."""
    cfg = LinearConfig(int(n_seqs), int(H), int(Hk), int(dk), int(dv), DTYPES.get(dtype, dtype), int(n_tokens),
                       int(Hk * dk if q_stride is None else q_stride), int(Hk * dk if k_stride is None else k_stride),
                       int(H * dv if v_stride is None else v_stride), float(scale), DELTA_BLOCK)
    if segment is not None:
        cfg.segment = int(segment)
    elif cfg.n_seqs <= RAGGED_SEQS:  # (only the step takes more)
        cfg.segment = linear_segment(cfg)
    return cfg


def linear_segment(cfg: LinearConfig) -> int:
    n = _i32(0)
    _check(lib().replayssm_linear_segment(ctypes.byref(cfg), ctypes.byref(n)), "linear_segment")
    return int(n.value)


def linear_sizes(cfg: LinearConfig):
    """(bytes of linear_prompt's workspace, bytes of linear_prompt_backward's)"""
    f, b = _i64(0), _i64(0)
    _check(lib().replayssm_linear_sizes(ctypes.byref(cfg), ctypes.byref(f), ctypes.byref(b)), "linear_sizes")
    return int(f.value), int(b.value)


def _linear_inputs(cfg, dev, t, q, k, v, g, beta, skip):
    n, f32 = cfg.n_tokens, torch.float32
    return (_rows(q, dev, t, (n, cfg.Hk, cfg.dk), cfg.q_stride, "q"),
            _rows(k, dev, t, (n, cfg.Hk, cfg.dk), cfg.k_stride, "k"),
            _rows(v, dev, t, (n, cfg.H, cfg.dv), cfg.v_stride, "v"), _dev(g, dev, f32, (n, cfg.H), "g"),
            _dev(beta, dev, f32, (n, cfg.H), "beta"), _dev(skip, dev, f32, (cfg.H,), "skip"))


def _linear_maps(cfg, maps):
    """As _maps, for tables whose blocks are the configuration's segments."""
    room = _table_room(cfg, maps)
    if room is not None:
        tokens, blocks = room
        if blocks != tokens // cfg.segment + cfg.n_seqs:
            raise ValueError(f"block_seq: tables of blocks of {cfg.segment} expected")
        if tokens < cfg.n_tokens:
            cfg = LinearConfig.from_buffer_copy(cfg)
            cfg.n_tokens = tokens
    return ctypes.byref(cfg), ctypes.byref(maps)


def linear_step(cfg, cu_tokens, slots, n_slots, q, k, v, g, beta, skip, S_in, S_out, out, err, stream=None):
    dev, s = _device_and_stream(stream)
    t, i32, n = _torch_dtype(cfg.dtype, "linear_step"), torch.int32, cfg.n_seqs
    pool = (n_slots, cfg.H, cfg.dv, cfg.dk)
    _check(lib().replayssm_linear_step(
        ctypes.byref(cfg), _dev(cu_tokens, dev, i32, (n + 1,), "cu_tokens"), _dev(slots, dev, i32, (n,), "slots"),
        int(n_slots), *_linear_inputs(cfg, dev, t, q, k, v, g, beta, skip), _dev(S_in, dev, torch.float32, pool, "S_in"),
        _dev(S_out, dev, torch.float32, pool, "S_out"), _dev(out, dev, t, (cfg.n_tokens, cfg.H, cfg.dv), "out"),
        _dev(err, dev, i32, None, "err"), s), "linear_step")


def linear_prompt(cfg, maps, q, k, v, g, beta, skip, S0, out, S_out, workspace, err, stream=None):
    dev, s = _device_and_stream(stream)
    need = linear_sizes(cfg)[0]
    config, tables = _linear_maps(cfg, maps)
    _maps_device(maps, dev)
    t, f32 = _torch_dtype(cfg.dtype, "linear_prompt"), torch.float32
    states = (cfg.n_seqs, cfg.H, cfg.dv, cfg.dk)
    _check(lib().replayssm_linear_prompt(
        config, tables, *_linear_inputs(cfg, dev, t, q, k, v, g, beta, skip), _dev(S0, dev, f32, states, "S0"),
        _dev(out, dev, t, (cfg.n_tokens, cfg.H, cfg.dv), "out"), _dev(S_out, dev, f32, states, "S_out"),
        _workspace(workspace, dev, need), _dev(err, dev, torch.int32, None, "err"), s), "linear_prompt")


def linear_prompt_backward(cfg, maps, q, k, v, g, beta, skip, S0, dout, dS_out, dq, dk, dv, dg, dbeta, dskip, dS0,
                           workspace, err, stream=None):
    dev, s = _device_and_stream(stream)
    need = linear_sizes(cfg)[1]
    config, tables = _linear_maps(cfg, maps)
    _maps_device(maps, dev)
    t, n, f32 = _torch_dtype(cfg.dtype, "linear_prompt_backward"), cfg.n_tokens, torch.float32
    states, keys, values = (cfg.n_seqs, cfg.H, cfg.dv, cfg.dk), (n, cfg.Hk, cfg.dk), (n, cfg.H, cfg.dv)
    _check(lib().replayssm_linear_prompt_backward(
        config, tables, *_linear_inputs(cfg, dev, t, q, k, v, g, beta, skip), _dev(S0, dev, f32, states, "S0"),
        _dev(dout, dev, t, values, "dout"), _dev(dS_out, dev, f32, states, "dS_out"), _dev(dq, dev, t, keys, "dq"),
        _dev(dk, dev, t, keys, "dk"), _dev(dv, dev, t, values, "dv"), _dev(dg, dev, f32, (n, cfg.H), "dg"),
        _dev(dbeta, dev, f32, (n, cfg.H), "dbeta"), _dev(dskip, dev, f32, (cfg.H,), "dskip"),
        _dev(dS0, dev, f32, states, "dS0"), _workspace(workspace, dev, need), _dev(err, dev, torch.int32, None, "err"),
        s), "linear_prompt_backward")


def make_gated_norm_config(n_tokens, groups, D, gate="before", shared=False, eps=1e-5, dtype="bf16", x_stride=None,
                           z_stride=None) -> GatedNormConfig:
    """gate: "before" or "after" the norm, or "none". Strides default to contiguous rows."""
    row = int(groups) * int(D)
    return GatedNormConfig(int(n_tokens), int(groups), int(D), GATES.get(gate, gate), int(bool(shared)),
                           DTYPES.get(dtype, dtype), float(eps), int(row if x_stride is None else x_stride),
                           int(row if z_stride is None else z_stride))


def gated_norm_sizes(cfg: GatedNormConfig) -> int:
    n = _i64(0)
    _check(lib().replayssm_gated_norm_sizes(ctypes.byref(cfg), ctypes.byref(n)), "gated_norm_sizes")
    return int(n.value)


def _norm_inputs(cfg, dev, x, z, w):
    t, shape = _torch_dtype(cfg.dtype, "gated_norm"), (cfg.n_tokens, cfg.groups, cfg.D)
    return (_rows(x, dev, t, shape, cfg.x_stride, "x"),
            _rows(z, dev, t, shape, cfg.z_stride, "z") if cfg.gate != GATE_NONE else None,
            _dev(w, dev, torch.float32, (cfg.D,) if cfg.shared else shape[1:], "w"))


def gated_norm(cfg, x, z, w, y, stream=None):
    dev, s = _device_and_stream(stream)
    gated_norm_sizes(cfg)
    t, shape = _torch_dtype(cfg.dtype, "gated_norm"), (cfg.n_tokens, cfg.groups, cfg.D)
    _check(lib().replayssm_gated_norm(ctypes.byref(cfg), *_norm_inputs(cfg, dev, x, z, w), _dev(y, dev, t, shape, "y"), s),
           "gated_norm")


def gated_norm_backward(cfg, x, z, w, dy, dx, dz, dw=None, workspace=None, stream=None):
    dev, s = _device_and_stream(stream)
    need = gated_norm_sizes(cfg)
    t, shape = _torch_dtype(cfg.dtype, "gated_norm"), (cfg.n_tokens, cfg.groups, cfg.D)
    _check(lib().replayssm_gated_norm_backward(
        ctypes.byref(cfg), *_norm_inputs(cfg, dev, x, z, w), _dev(dy, dev, t, shape, "dy"), _dev(dx, dev, t, shape, "dx"),
        _dev(dz, dev, t, shape, "dz") if cfg.gate != GATE_NONE else None,
        _dev(dw, dev, torch.float32, (cfg.D,) if cfg.shared else shape[1:], "dw"),
        _workspace(workspace, dev, need if dw is not None else 0), s), "gated_norm_backward")

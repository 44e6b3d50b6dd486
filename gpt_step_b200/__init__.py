"""Python binding of libgpt2step (the GPT-2 training step on one B200).

Argument marshalling only: every step of the path runs in the library's CUDA
kernels. torch is used for device memory (the arena, token buffers) and for
the current CUDA stream. Importing this package does not load the library;
the first call that needs it does, and raises if it is missing.
"""
from __future__ import annotations

import ctypes
import os
from dataclasses import dataclass

import numpy as np

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libgpt2step.so")

GPT2_PARAMS, GPT2_GRADS, GPT2_ADAM_M, GPT2_ADAM_V, GPT2_WEIGHTS_BF16 = 0, 1, 2, 3, 4
STATUS = {0: "GPT2_OK", 1: "GPT2_ERR_ARG", 2: "GPT2_ERR_CUDA", 3: "GPT2_ERR_TOKEN_RANGE",
          4: "GPT2_ERR_NONFINITE", 5: "GPT2_ERR_STATE", 6: "GPT2_ERR_TIMEOUT"}


class GPT2Error(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {STATUS.get(status, status)} ({_status_string(status)})")


class Config(ctypes.Structure):
    _fields_ = [("n_layer", ctypes.c_int32), ("n_head", ctypes.c_int32),
                ("n_embd", ctypes.c_int32), ("seq_len", ctypes.c_int32),
                ("vocab_real", ctypes.c_int32), ("vocab_padded", ctypes.c_int32),
                ("micro_batch", ctypes.c_int32), ("grad_accum", ctypes.c_int32),
                ("max_lr", ctypes.c_float), ("min_lr", ctypes.c_float),
                ("warmup_steps", ctypes.c_int32), ("total_steps", ctypes.c_int32),
                ("beta1", ctypes.c_float), ("beta2", ctypes.c_float), ("eps", ctypes.c_float),
                ("weight_decay", ctypes.c_float), ("grad_clip", ctypes.c_float)]

    @classmethod
    def make(cls, n_layer, n_head, n_embd, seq_len, vocab_real, vocab_padded=0, micro_batch=1,
             grad_accum=1, max_lr=6e-4, min_lr=0.0, warmup_steps=700, total_steps=18865,
             beta1=0.9, beta2=0.95, eps=1e-8, weight_decay=0.1, grad_clip=1.0, **_):
        return cls(n_layer, n_head, n_embd, seq_len, vocab_real, vocab_padded, micro_batch,
                   grad_accum, max_lr, min_lr, warmup_steps, total_steps, beta1, beta2, eps,
                   weight_decay, grad_clip)


_lib_handle = None
_c = ctypes
_P = ctypes.c_void_p
_I = ctypes.c_int
_I32 = ctypes.c_int32
_I64 = ctypes.c_int64
_F = ctypes.c_float
_FP = ctypes.POINTER(ctypes.c_float)
_SZ = ctypes.c_size_t

_SIGNATURES = {
    "gpt2_arena_bytes": (_SZ, [ctypes.POINTER(Config)]),
    "gpt2_num_params": (_I64, [ctypes.POINTER(Config), _I]),
    "gpt2_create": (_I, [ctypes.POINTER(Config), ctypes.c_uint64, _P, _SZ, _P, ctypes.POINTER(_P)]),
    "gpt2_destroy": (None, [_P]),
    "gpt2_fwd_bwd": (_I, [_P, _P, _P, _FP]),
    "gpt2_clip_adamw": (_I, [_P, _I32, _FP]),
    "gpt2_last_step_stats": (_I, [_P, _FP, _FP]),
    "gpt2_eval_loss": (_I, [_P, _P, _P, _I32, _FP]),
    "gpt2_train_step_host": (_I, [_P, _P, _P, _I32, _I32, _FP, _FP]),
    "gpt2_token_losses": (_I, [_P, _FP, _I64]),
    "gpt2_lr": (_F, [_P, _I32]),
    "gpt2_schedule_lr": (ctypes.c_double, [ctypes.POINTER(Config), _I32]),
    "gpt2_kernel_launches": (_I64, [_P]),
    "gpt2_profile_enable": (_I, [_P, _I]),
    "gpt2_profile_num_classes": (_I, []),
    "gpt2_profile_class_name": (ctypes.c_char_p, [_I]),
    "gpt2_profile_read": (_I, [_P, _I, ctypes.POINTER(ctypes.c_double), ctypes.POINTER(_I64),
                               ctypes.POINTER(ctypes.c_double)]),
    "gpt2_status_string": (ctypes.c_char_p, [_I]),
    "gpt2_num_tensors": (_I, [_P]),
    "gpt2_tensor_info": (_I, [_P, _I, ctypes.POINTER(ctypes.c_char_p), ctypes.POINTER(_I64),
                              ctypes.POINTER(_I)]),
    "gpt2_read": (_I, [_P, _I, _I, _FP]),
    "gpt2_write": (_I, [_P, _I, _I, _FP]),
    "gpt2_state_device_ptr": (_I, [_P, _I, ctypes.POINTER(ctypes.c_void_p), ctypes.POINTER(_I64)]),
    "gpt2_num_buckets": (_I, [_P]),
    "gpt2_bucket_range": (_I, [_P, _I, ctypes.POINTER(_I64), ctypes.POINTER(_I64)]),
    "gpt2_set_bucket_events": (_I, [_P, ctypes.POINTER(_P), _I]),
    "gpt2_grad_sumsq": (_I, [_P, ctypes.POINTER(_I64), _I, _P]),
    "gpt2_clip_adamw_ranges": (_I, [_P, _I32, ctypes.POINTER(_I64), _I, _P, _FP]),
    "gpt2op_linear_fwd": (_I, [_P, _P, _P, _P, _P, _I, _I, _I, _P, _P]),
    "gpt2op_linear_fwd_gelu": (_I, [_P, _P, _P, _P, _P, _I, _I, _I, _P, _P]),
    "gpt2op_linear_dgrad": (_I, [_P, _P, _P, _P, _I, _I, _I, _P, _P]),
    "gpt2op_linear_wgrad": (_I, [_P, _P, _P, _I, _I, _I, _I, _P, _P]),
    "gpt2op_linear_bwd": (_I, [_P, _P, _P, _P, _P, _P, _P, _I, _I, _I, ctypes.POINTER(_I), _P, _P]),
    "gpt2op_bias_grad_workspace": (_SZ, [_I, _I]),
    "gpt2op_bias_grad": (_I, [_P, _P, _I, _I, _P, _SZ, _P]),
    "gpt2op_layernorm_fwd": (_I, [_P, _P, _P, _P, _P, _P, _I, _I, _P]),
    "gpt2op_layernorm_bwd_workspace": (_SZ, [_I, _I]),
    "gpt2op_layernorm_bwd": (_I, [_P, _P, _P, _P, _P, _P, _P, _P, _P, _I, _I, _P, _SZ, _P]),
    "gpt2op_layernorm_bwd_noalloc_max_bytes": (_SZ, []),
    "gpt2op_layernorm_bwd_noalloc": (_I, [_P, _P, _P, _P, _P, _P, _P, _P, _P, _I, _I, _P]),
    "gpt2op_attention_fwd": (_I, [_P, _P, _P, _I, _I, _I, _I, _P, _P]),
    "gpt2op_attention_bwd_workspace": (_SZ, [_I, _I, _I, _I]),
    "gpt2op_attention_bwd": (_I, [_P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _P, _SZ, _P, _P]),
    "gpt2op_softmax_ce": (_I, [_P, _P, _P, _I, _I, _I, _F, _P, _P]),
    "gpt2op_softmax_ce_masked": (_I, [_P, _P, _P, _I, _I, _I, _I, _F, _P, _P]),
    "gpt2op_lm_head_loss": (_I, [_P, _P, _P, _P, _I, _I, _I, _I, _P, _SZ, _P, _P]),
    "gpt2op_lm_head_ce_workspace": (_SZ, [_I, _I]),
    "gpt2op_lm_head_ce": (_I, [_P, _P, _P, _P, _P, _I, _I, _I, _I, _F, _I, _P, _SZ, _P, _P]),
    "gpt2_token_logps": (_I, [_P, _P, _P, _I32, _I32, _P]),
    "gpt2_fwd_bwd_policy": (_I, [_P, _P, _P, _P, _P, _P, _P, _I32, _F, _F, _F, _F, _P, _FP]),
    "gpt2_fwd_bwd_preference": (_I, [_P, _P, _P, _P, _I32, _I, _I, _F, _F, _P, _FP]),
    "gpt2_muon_workspace": (_SZ, [ctypes.POINTER(Config)]),
    "gpt2_clip_muon": (_I, [_P, _I32, _F, _P, _SZ, _FP]),
    "gpt2op_token_logps": (_I, [_P, _P, _P, _I, _I, _I, _I, _P, _P]),
    "gpt2op_policy_loss": (_I, [_P, _P, _P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _F, _F, _F, _F, _P, _P]),
    "gpt2op_preference_loss_workspace": (_SZ, [_I, _I]),
    "gpt2op_preference_loss": (_I, [_P, _P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _I, _F, _F, _F, _P, _SZ,
                                    _P, _P]),
    "gpt2op_orthogonalize_workspace": (_SZ, [_I, _I, _I]),
    "gpt2op_orthogonalize": (_I, [_P, _I, _I64, _P, _I64, _I, _I, _I, _I, _P, _SZ, _P, _P]),
    "gpt2op_embedding_fwd": (_I, [_P, _P, _P, _P, _I, _I, _I, _I, _P, _P]),
    "gpt2op_embedding_bwd": (_I, [_P, _P, _P, _P, _I, _I, _I, _I, _P]),
    "gpt2op_wait_selftest": (_I, [_I64, _P, _P]),
}


def lib():
    """Load libgpt2step.so (raises if it has not been built)."""
    global _lib_handle
    if _lib_handle is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                               "`python -m gpt_step_b200.build` (there is no fallback path)")
        h = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in _SIGNATURES.items():
            f = getattr(h, name)
            f.restype = res
            f.argtypes = args
        _lib_handle = h
    return _lib_handle


def _status_string(st: int) -> str:
    try:
        return lib().gpt2_status_string(st).decode()
    except Exception:  # pragma: no cover
        return "?"


def check(st: int, what: str):
    if st != 0:
        raise GPT2Error(st, what)


def _ptr(t):
    """Device (or host numpy) pointer of a tensor/array, None for None."""
    if t is None:
        return None
    if isinstance(t, np.ndarray):
        return t.ctypes.data
    return t.data_ptr()


def _stream_handle(stream=None):
    import torch
    s = stream if stream is not None else torch.cuda.current_stream()
    return s.cuda_stream


def arena_bytes(cfg: Config) -> int:
    return lib().gpt2_arena_bytes(ctypes.byref(cfg))


def schedule_lr(cfg: Config, step: int) -> float:
    """The learning-rate schedule of `cfg` at `step` (host arithmetic in the library)."""
    return lib().gpt2_schedule_lr(ctypes.byref(cfg), step)


def muon_workspace(cfg: Config) -> int:
    """Bytes of workspace GPT2.clip_muon needs for `cfg`."""
    return lib().gpt2_muon_workspace(ctypes.byref(cfg))


def num_params(cfg: Config, padded: bool = False) -> int:
    return lib().gpt2_num_params(ctypes.byref(cfg), 1 if padded else 0)


PREFERENCE_KINDS = {"sigmoid": 0, "squared": 1}


def _kind(name: str) -> int:
    if name not in PREFERENCE_KINDS:
        raise ValueError(f"kind {name!r}: one of {sorted(PREFERENCE_KINDS)}")
    return PREFERENCE_KINDS[name]


def _rows_of(T: int, tokens) -> int:
    n = tokens.numel()
    if n == 0 or n % T:
        raise ValueError(f"tokens: {n} positions are not whole sequences of {T}")
    return n


_dtypes = None


def _types():
    """(bfloat16, float32, int32, uint8), once torch is needed."""
    global _dtypes
    if _dtypes is None:
        import torch
        _dtypes = (torch.bfloat16, torch.float32, torch.int32, torch.uint8)
    return _dtypes


def _device_of(t, name) -> int:
    dev = t.get_device()
    if dev < 0:
        raise ValueError(f"{name}: a device tensor is needed")
    return dev


def _need(t, name, dtype, numel, dev):
    """Check a contiguous tensor's type, element count (-1: any but none) and device; returns its pointer."""
    if t is None:
        raise ValueError(f"{name} is required")
    n = t.numel()
    if t.dtype is dtype and t.get_device() == dev and t.is_contiguous() and (n == numel or (numel < 0 and n)):
        return t.data_ptr()
    _device_of(t, name)
    if t.dtype is not dtype:
        raise ValueError(f"{name}: {t.dtype}, not {dtype}")
    if t.get_device() != dev:
        raise ValueError(f"{name}: on {t.device}, not cuda:{dev}")
    if not t.is_contiguous():
        raise ValueError(f"{name}: not contiguous")
    raise ValueError(f"{name}: {n} elements" + (f", not {numel}" if numel >= 0 else ""))


def _opt(t, name, dtype, numel, dev):
    return None if t is None else _need(t, name, dtype, numel, dev)


@dataclass
class TensorInfo:
    name: str
    shape: tuple


class GPT2:
    """One model: create(config, seed), fwd_bwd, clip_adamw, eval_loss, introspection."""

    def __init__(self, cfg: Config, seed: int, stream=None):
        import torch
        self.cfg = cfg
        self.torch = torch
        self.stream = stream if stream is not None else torch.cuda.current_stream()
        nbytes = arena_bytes(cfg)
        if nbytes == 0:
            raise GPT2Error(1, "gpt2_arena_bytes (unsupported configuration)")
        self.arena = torch.empty(nbytes + 1024, dtype=torch.uint8, device="cuda")
        base = self.arena.data_ptr()
        self._base = (base + 1023) // 1024 * 1024
        h = ctypes.c_void_p()
        check(lib().gpt2_create(ctypes.byref(cfg), ctypes.c_uint64(seed), ctypes.c_void_p(self._base),
                                nbytes, ctypes.c_void_p(self.stream.cuda_stream), ctypes.byref(h)),
              "gpt2_create")
        self.h = h
        self.T = cfg.seq_len
        self.B = cfg.micro_batch
        self._infos = None
        self.sharded = False     # set by the sharded data-parallel step: a rank's update is its shards' alone

    def close(self):
        if getattr(self, "h", None):
            lib().gpt2_destroy(self.h)
            self.h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    # -- the step --------------------------------------------------------------------------
    def fwd_bwd(self, tokens, targets, want_loss: bool = False):
        out = ctypes.c_float()
        check(lib().gpt2_fwd_bwd(self.h, _ptr(tokens), _ptr(targets),
                                 ctypes.byref(out) if want_loss else None), "gpt2_fwd_bwd")
        return out.value if want_loss else None

    def token_logps(self, tokens, targets, logps, ignore_index: int = -1):
        """logps (device fp32, tokens' shape) = the targets' log-probabilities, 0 where ignored."""
        _, f32, i32, _ = _types()
        n, dev = _rows_of(self.T, tokens), self.arena.get_device()
        check(lib().gpt2_token_logps(self.h, _need(tokens, "tokens", i32, n, dev), _need(targets, "targets", i32, n, dev),
                                     n // self.T, ignore_index, _need(logps, "logps", f32, n, dev)), "gpt2_token_logps")

    def fwd_bwd_policy(self, tokens, targets, old_logp, adv, ref_logp=None, weight=None, ignore_index: int = -1,
                       clip_low: float = 0.2, clip_high: float = 0.2, kl_coef: float = 0.0, scale: float = 1.0,
                       logps=None, want_loss: bool = False):
        """One micro-step on the clipped policy loss; per-position inputs are device fp32 [B, T]."""
        _, f32, i32, _ = _types()
        n, dev = self.B * self.T, self.arena.get_device()
        out = ctypes.c_float()
        check(lib().gpt2_fwd_bwd_policy(
            self.h, _need(tokens, "tokens", i32, n, dev), _need(targets, "targets", i32, n, dev),
            _need(old_logp, "old_logp", f32, n, dev), _opt(ref_logp, "ref_logp", f32, n, dev),
            _need(adv, "adv", f32, n, dev), _opt(weight, "weight", f32, n, dev), ignore_index, clip_low, clip_high,
            kl_coef, scale, _opt(logps, "logps", f32, n, dev), ctypes.byref(out) if want_loss else None),
            "gpt2_fwd_bwd_policy")
        return out.value if want_loss else None

    def fwd_bwd_preference(self, tokens, targets, ref_logp=None, ignore_index: int = -1, kind: str = "sigmoid",
                           average: bool = False, beta: float = 0.1, smoothing: float = 0.0, seq_logps=None,
                           want_loss: bool = False):
        """One micro-step on the paired preference loss: sequences 2p (chosen) and 2p + 1 (rejected)."""
        _, f32, i32, _ = _types()
        n, dev = self.B * self.T, self.arena.get_device()
        out = ctypes.c_float()
        check(lib().gpt2_fwd_bwd_preference(
            self.h, _need(tokens, "tokens", i32, n, dev), _need(targets, "targets", i32, n, dev),
            _opt(ref_logp, "ref_logp", f32, self.B, dev), ignore_index, _kind(kind), 1 if average else 0, beta,
            smoothing, _opt(seq_logps, "seq_logps", f32, self.B, dev), ctypes.byref(out) if want_loss else None),
            "gpt2_fwd_bwd_preference")
        return out.value if want_loss else None

    def clip_muon(self, step: int, workspace, momentum: float = 0.95, want_norm: bool = False):
        """The optimizer step with orthogonalised momentum for the blocks' 2-D weights;
        workspace: a device tensor of at least muon_workspace(cfg) bytes. On several ranks with
        DataParallel(mode="allreduce"): sync_grads(), then this; the sharded form cuts through matrices."""
        if self.sharded:
            raise ValueError("clip_muon: the model's update is sharded over ranks, which cuts through matrices "
                             "(DataParallel(mode=\"allreduce\") keeps them whole)")
        out = ctypes.c_float()
        ws = _need(workspace, "workspace", _types()[3], -1, self.arena.get_device())
        check(lib().gpt2_clip_muon(self.h, step, momentum, ws, workspace.numel(),
                                   ctypes.byref(out) if want_norm else None), "gpt2_clip_muon")
        return out.value if want_norm else None

    def clip_adamw(self, step: int, want_norm: bool = False):
        out = ctypes.c_float()
        check(lib().gpt2_clip_adamw(self.h, step, ctypes.byref(out) if want_norm else None),
              "gpt2_clip_adamw")
        return out.value if want_norm else None

    def last_step_stats(self):
        l, n = ctypes.c_float(), ctypes.c_float()
        check(lib().gpt2_last_step_stats(self.h, ctypes.byref(l), ctypes.byref(n)), "gpt2_last_step_stats")
        return l.value, n.value

    def eval_loss(self, tokens, targets) -> float:
        out = ctypes.c_float()
        check(lib().gpt2_eval_loss(self.h, _ptr(tokens), _ptr(targets), tokens.shape[0], ctypes.byref(out)),
              "gpt2_eval_loss")
        return out.value

    def train_step_host(self, tokens_host: np.ndarray, targets_host: np.ndarray, step: int):
        """tokens/targets: host int32 [n_micro, B, T] (pinned or pageable)."""
        l, n = ctypes.c_float(), ctypes.c_float()
        check(lib().gpt2_train_step_host(self.h, _ptr(tokens_host), _ptr(targets_host),
                                         tokens_host.shape[0], step, ctypes.byref(l), ctypes.byref(n)),
              "gpt2_train_step_host")
        return l.value, n.value

    def train_step_host_ptr(self, tok_ptr: int, tgt_ptr: int, n_micro: int, step: int):
        l, n = ctypes.c_float(), ctypes.c_float()
        check(lib().gpt2_train_step_host(self.h, tok_ptr, tgt_ptr, n_micro, step, ctypes.byref(l),
                                         ctypes.byref(n)), "gpt2_train_step_host")
        return l.value, n.value

    def token_losses(self) -> np.ndarray:
        out = np.empty(self.B * self.T, np.float32)
        check(lib().gpt2_token_losses(self.h, out.ctypes.data_as(_FP), out.size), "gpt2_token_losses")
        return out.reshape(self.B, self.T)

    def lr(self, step: int) -> float:
        return lib().gpt2_lr(self.h, step)

    def kernel_launches(self) -> int:
        return lib().gpt2_kernel_launches(self.h)

    def profile(self, on: bool):
        check(lib().gpt2_profile_enable(self.h, 1 if on else 0), "gpt2_profile_enable")

    def profile_read(self) -> dict:
        out = {}
        for c in range(lib().gpt2_profile_num_classes()):
            ms, n, work = ctypes.c_double(), ctypes.c_int64(), ctypes.c_double()
            check(lib().gpt2_profile_read(self.h, c, ctypes.byref(ms), ctypes.byref(n), ctypes.byref(work)),
                  "gpt2_profile_read")
            name = lib().gpt2_profile_class_name(c).decode()
            key = "flops" if name.startswith(("gemm", "attention")) else "bytes"
            out[name] = {"ms": ms.value, "launches": n.value, key: work.value}
        return out

    # -- introspection ---------------------------------------------------------------------
    def tensors(self):
        if self._infos is None:
            n = lib().gpt2_num_tensors(self.h)
            infos = []
            for i in range(n):
                name = ctypes.c_char_p()
                shape = (ctypes.c_int64 * 2)()
                nd = ctypes.c_int()
                check(lib().gpt2_tensor_info(self.h, i, ctypes.byref(name), shape, ctypes.byref(nd)),
                      "gpt2_tensor_info")
                infos.append(TensorInfo(name.value.decode(), tuple(shape[: nd.value])))
            self._infos = infos
        return self._infos

    def read(self, what: int, idx: int) -> np.ndarray:
        info = self.tensors()[idx]
        out = np.empty(info.shape, np.float32)
        check(lib().gpt2_read(self.h, what, idx, out.ctypes.data_as(_FP)), "gpt2_read")
        return out

    def write(self, what: int, idx: int, arr: np.ndarray):
        info = self.tensors()[idx]
        a = np.ascontiguousarray(arr, dtype=np.float32)
        if a.shape != info.shape:
            raise ValueError(f"{info.name}: shape {a.shape} != {info.shape}")
        check(lib().gpt2_write(self.h, what, idx, a.ctypes.data_as(_FP)), "gpt2_write")

    def state_tensor(self, what: int):
        """The flat state array `what` (fp32; bf16 for GPT2_WEIGHTS_BF16) as a torch view of the arena."""
        ptr, n = ctypes.c_void_p(), ctypes.c_int64()
        check(lib().gpt2_state_device_ptr(self.h, what, ctypes.byref(ptr), ctypes.byref(n)),
              "gpt2_state_device_ptr")
        off = ptr.value - self.arena.data_ptr()
        if what == GPT2_WEIGHTS_BF16:
            return self.arena[off: off + 2 * n.value].view(self.torch.bfloat16)
        return self.arena[off: off + 4 * n.value].view(self.torch.float32)

    # -- sharded optimizer step -------------------------------------------------------------
    def num_buckets(self) -> int:
        return lib().gpt2_num_buckets(self.h)

    def bucket_range(self, b: int):
        """(begin, end) elements of bucket b, or of the 1-D region for b = -1."""
        lo, hi = ctypes.c_int64(), ctypes.c_int64()
        check(lib().gpt2_bucket_range(self.h, b, ctypes.byref(lo), ctypes.byref(hi)), "gpt2_bucket_range")
        return lo.value, hi.value

    def set_bucket_events(self, events):
        """Register torch.cuda.Event objects (one per bucket); [] clears."""
        self._bucket_events = list(events)
        arr = (ctypes.c_void_p * max(1, len(events)))(*[e.cuda_event for e in events])
        check(lib().gpt2_set_bucket_events(self.h, arr, len(events)), "gpt2_set_bucket_events")

    @staticmethod
    def _ranges(ranges):
        flat = [int(v) for r in ranges for v in r]
        return (ctypes.c_int64 * len(flat))(*flat), len(ranges)

    def grad_sumsq(self, ranges, dev_out):
        """Enqueue: dev_out (a device float64 tensor of one element) = sum of g^2 over the ranges."""
        arr, n = self._ranges(ranges)
        check(lib().gpt2_grad_sumsq(self.h, arr, n, _ptr(dev_out)), "gpt2_grad_sumsq")

    def clip_adamw_ranges(self, step: int, ranges, dev_sumsq, want_norm: bool = False):
        arr, n = self._ranges(ranges)
        out = ctypes.c_float()
        check(lib().gpt2_clip_adamw_ranges(self.h, step, arr, n, _ptr(dev_sumsq),
                                           ctypes.byref(out) if want_norm else None), "gpt2_clip_adamw_ranges")
        return out.value if want_norm else None

    def read_all(self, what: int) -> dict:
        return {t.name: self.read(what, i) for i, t in enumerate(self.tensors())}

    def write_all(self, what: int, named: dict):
        for i, t in enumerate(self.tensors()):
            self.write(what, i, named[t.name])


# -- op-level calls (device tensors in, device tensors out) -----------------------------------

def _s(stream):
    return ctypes.c_void_p(_stream_handle(stream))


def linear_fwd(inp, w, bias, resid, out, err, stream=None):
    M, K = inp.shape
    N = w.shape[0]
    check(lib().gpt2op_linear_fwd(_ptr(inp), _ptr(w), _ptr(bias), _ptr(resid), _ptr(out), M, N, K,
                                  _ptr(err), _s(stream)), "gpt2op_linear_fwd")


def linear_fwd_gelu(inp, w, bias, pre_out, gelu_out, err, stream=None):
    M, K = inp.shape
    N = w.shape[0]
    check(lib().gpt2op_linear_fwd_gelu(_ptr(inp), _ptr(w), _ptr(bias), _ptr(pre_out), _ptr(gelu_out),
                                       M, N, K, _ptr(err), _s(stream)), "gpt2op_linear_fwd_gelu")


def linear_dgrad(dout, w, gelu_pre, din, err, stream=None):
    M, N = dout.shape
    K = w.shape[1]
    check(lib().gpt2op_linear_dgrad(_ptr(dout), _ptr(w), _ptr(gelu_pre), _ptr(din), M, N, K,
                                    _ptr(err), _s(stream)), "gpt2op_linear_dgrad")


def linear_wgrad(dout, inp, dw, err, splits=0, stream=None):
    M, N = dout.shape
    K = inp.shape[1]
    check(lib().gpt2op_linear_wgrad(_ptr(dout), _ptr(inp), _ptr(dw), M, N, K, splits, _ptr(err),
                                    _s(stream)), "gpt2op_linear_wgrad")


def linear_bwd(dout, w, inp, gelu_pre, din, dw, colsum, err, stream=None) -> int:
    """Grouped input + weight gradient of a linear layer; returns the dw reduction split."""
    M, N = dout.shape
    K = w.shape[1]
    sp = ctypes.c_int()
    check(lib().gpt2op_linear_bwd(_ptr(dout), _ptr(w), _ptr(inp), _ptr(gelu_pre), _ptr(din), _ptr(dw),
                                  _ptr(colsum), M, N, K, ctypes.byref(sp), _ptr(err), _s(stream)),
          "gpt2op_linear_bwd")
    return sp.value


def wait_selftest(limit_ns, err, stream=None) -> int:
    """Run the bounded-wait self-test; returns the raw status (6 = timed out as designed)."""
    return lib().gpt2op_wait_selftest(int(limit_ns), _ptr(err), _s(stream))


def bias_grad_workspace(M, N):
    return lib().gpt2op_bias_grad_workspace(M, N)


def bias_grad(dout, db, workspace, stream=None):
    M, N = dout.shape
    check(lib().gpt2op_bias_grad(_ptr(dout), _ptr(db), M, N, _ptr(workspace),
                                 0 if workspace is None else workspace.numel(), _s(stream)), "gpt2op_bias_grad")


def layernorm_fwd(x, w, b, y, mean, rstd, stream=None):
    rows, C = x.shape
    check(lib().gpt2op_layernorm_fwd(_ptr(x), _ptr(w), _ptr(b), _ptr(y), _ptr(mean), _ptr(rstd),
                                     rows, C, _s(stream)), "gpt2op_layernorm_fwd")


def layernorm_bwd_workspace(rows, C):
    return lib().gpt2op_layernorm_bwd_workspace(rows, C)


def layernorm_bwd(dy, x, mean, rstd, w, dresid, dx, dw, db, workspace, stream=None):
    rows, C = x.shape
    check(lib().gpt2op_layernorm_bwd(_ptr(dy), _ptr(x), _ptr(mean), _ptr(rstd), _ptr(w), _ptr(dresid),
                                     _ptr(dx), _ptr(dw), _ptr(db), rows, C, _ptr(workspace),
                                     0 if workspace is None else workspace.numel(), _s(stream)),
          "gpt2op_layernorm_bwd")


def layernorm_bwd_noalloc(dy, x, mean, rstd, w, dresid, dx, dw, db, stream=None):
    """LayerNorm backward with the library's own fixed scratch (no workspace argument)."""
    rows, C = x.shape
    check(lib().gpt2op_layernorm_bwd_noalloc(_ptr(dy), _ptr(x), _ptr(mean), _ptr(rstd), _ptr(w),
                                             _ptr(dresid), _ptr(dx), _ptr(dw), _ptr(db), rows, C,
                                             _s(stream)), "gpt2op_layernorm_bwd_noalloc")


def attention_fwd(qkv, out, lse, n_head, err, stream=None):
    B, T, C3 = qkv.shape
    hd = C3 // 3 // n_head
    check(lib().gpt2op_attention_fwd(_ptr(qkv), _ptr(out), _ptr(lse), B, T, n_head, hd, _ptr(err),
                                     _s(stream)), "gpt2op_attention_fwd")


def attention_bwd_workspace(B, T, H, hd):
    return lib().gpt2op_attention_bwd_workspace(B, T, H, hd)


def attention_bwd(qkv, out, dout, lse, dqkv, n_head, workspace, err, stream=None, dbias=None):
    """dbias (fp32 [3C]) or None: += the qkv bias gradient (column sums of dqkv)."""
    B, T, C3 = qkv.shape
    hd = C3 // 3 // n_head
    check(lib().gpt2op_attention_bwd(_ptr(qkv), _ptr(out), _ptr(dout), _ptr(lse), _ptr(dqkv), _ptr(dbias),
                                     B, T, n_head, hd, _ptr(workspace), workspace.numel(), _ptr(err),
                                     _s(stream)), "gpt2op_attention_bwd")


def softmax_ce(logits, targets, losses, V, dscale, err, stream=None):
    N, Vp = logits.shape
    check(lib().gpt2op_softmax_ce(_ptr(logits), _ptr(targets), _ptr(losses), N, V, Vp, dscale,
                                  _ptr(err), _s(stream)), "gpt2op_softmax_ce")


def softmax_ce_masked(logits, targets, losses, V, ignore_index, dscale, err, stream=None):
    """Softmax-CE where rows with target == ignore_index get loss 0 and zero gradient."""
    N, Vp = logits.shape
    check(lib().gpt2op_softmax_ce_masked(_ptr(logits), _ptr(targets), _ptr(losses), N, V, Vp, ignore_index,
                                         dscale, _ptr(err), _s(stream)), "gpt2op_softmax_ce_masked")


def lm_head_ce_workspace(N, Vp):
    return lib().gpt2op_lm_head_ce_workspace(N, Vp)


def lm_head_ce(h, wte, targets, logits, losses, V, dscale, write_grad, ws, err, stream=None):
    """Tied lm_head GEMM + softmax-CE: logits = h . wte^T, then losses (and dz in place)."""
    N, C = h.shape
    Vp = wte.shape[0]
    check(lib().gpt2op_lm_head_ce(_ptr(h), _ptr(wte), _ptr(targets), _ptr(logits), _ptr(losses), N, C, V, Vp,
                                  dscale, 1 if write_grad else 0, _ptr(ws),
                                  0 if ws is None else ws.numel() * ws.element_size(), _ptr(err), _s(stream)),
          "gpt2op_lm_head_ce")


def lm_head_loss(h, wte, targets, losses, V, ws, err, stream=None):
    """Per-row losses of the tied lm_head with the logits never stored."""
    N, C = h.shape
    Vp = wte.shape[0]
    check(lib().gpt2op_lm_head_loss(_ptr(h), _ptr(wte), _ptr(targets), _ptr(losses), N, C, V, Vp, _ptr(ws),
                                    0 if ws is None else ws.numel() * ws.element_size(), _ptr(err), _s(stream)),
          "gpt2op_lm_head_loss")


def embedding_fwd(tokens, wte, wpe, out, V, err, stream=None):
    B, T = tokens.shape
    C = wte.shape[1]
    check(lib().gpt2op_embedding_fwd(_ptr(tokens), _ptr(wte), _ptr(wpe), _ptr(out), B, T, C, V,
                                     _ptr(err), _s(stream)), "gpt2op_embedding_fwd")


def embedding_bwd(tokens, dx, dwte, dwpe, V, stream=None):
    B, T = tokens.shape
    C = dwte.shape[1]
    check(lib().gpt2op_embedding_bwd(_ptr(tokens), _ptr(dx), _ptr(dwte), _ptr(dwpe), B, T, C, V,
                                     _s(stream)), "gpt2op_embedding_bwd")


# The post-training operators check their tensors (the checks cost about as much as
# the launch, which is what a call on few rows takes) and run on the tensors' device.

_torch = _raw_stream = None


def _call(name, dev, stream, *args):
    """lib().<name>(*args, stream) with device `dev` current."""
    global _torch, _raw_stream
    if _torch is None:
        import torch
        # the handle of a device's current stream, without the Stream object around it (1.3 us of a call's 10)
        _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
            (lambda d: torch.cuda.current_stream(d).cuda_stream)
        _torch = torch
    if stream is None:
        handle = _raw_stream(dev)
    elif stream.device.index != dev:
        raise ValueError(f"stream on {stream.device}, tensors on cuda:{dev}")
    else:
        handle = stream.cuda_stream
    f = getattr(lib(), name)
    if _torch.cuda.current_device() == dev:
        st = f(*args, handle)
    else:
        with _torch.cuda.device(dev):
            st = f(*args, handle)
    if st:
        raise GPT2Error(st, name)


def _logits_shape(logits, V):
    if logits.dim() != 2:
        raise ValueError(f"logits: [rows, padded ids] are needed, not {tuple(logits.shape)}")
    N, Vp = logits.shape
    if not 0 < V <= Vp:
        raise ValueError(f"V = {V} real ids of {Vp} columns")
    return N, Vp


def token_logps(logits, targets, logps, V, err, ignore_index=-1, stream=None):
    """logps = each row's log-probability of its target over the V real ids (0 where ignored)."""
    b16, f32, i32, _ = _types()
    N, Vp = _logits_shape(logits, V)
    d = _device_of(logits, "logits")
    _call("gpt2op_token_logps", d, stream, _need(logits, "logits", b16, -1, d), _need(targets, "targets", i32, N, d),
          _need(logps, "logps", f32, N, d), N, V, Vp, ignore_index, _need(err, "err", i32, -1, d))


def policy_loss(logits, targets, old_logp, adv, dlogits, logps, losses, V, err, ref_logp=None, weight=None,
                ignore_index=-1, clip_low=0.2, clip_high=0.2, kl_coef=0.0, dscale=1.0, stream=None):
    """Clipped policy loss with a KL term and its gradient over the logits.

    dlogits: None (losses alone), the logits (in place) or a tensor of their shape;
    logps may be None; ref_logp is required with kl_coef > 0."""
    b16, f32, i32, _ = _types()
    N, Vp = _logits_shape(logits, V)
    d = _device_of(logits, "logits")
    _call("gpt2op_policy_loss", d, stream, _need(logits, "logits", b16, -1, d), _need(targets, "targets", i32, N, d),
          _need(old_logp, "old_logp", f32, N, d), _opt(ref_logp, "ref_logp", f32, N, d), _need(adv, "adv", f32, N, d),
          _opt(weight, "weight", f32, N, d), _opt(dlogits, "dlogits", b16, N * Vp, d), _opt(logps, "logps", f32, N, d),
          _need(losses, "losses", f32, N, d), N, V, Vp, ignore_index, clip_low, clip_high, kl_coef, dscale,
          _need(err, "err", i32, -1, d))


def preference_loss_workspace(N, P):
    return lib().gpt2op_preference_loss_workspace(N, P)


def preference_loss(logits, targets, seq_start, dlogits, logps, seq_logps, losses, V, workspace, err, ref_logp=None,
                    ignore_index=-1, kind="sigmoid", average=False, beta=0.1, smoothing=0.0, dscale=1.0, stream=None):
    """Paired preference loss and its gradient over the logits; seq_start int32 [2P + 1],
    sequence 2p chosen and 2p + 1 rejected. dlogits as in policy_loss; seq_logps may be None."""
    b16, f32, i32, u8 = _types()
    N, Vp = _logits_shape(logits, V)
    P = (seq_start.numel() - 1) // 2
    if P < 1 or seq_start.numel() != 2 * P + 1:
        raise ValueError(f"seq_start: {seq_start.numel()} bounds are not 2P + 1")
    d = _device_of(logits, "logits")
    _call("gpt2op_preference_loss", d, stream, _need(logits, "logits", b16, -1, d),
          _need(targets, "targets", i32, N, d), _need(seq_start, "seq_start", i32, -1, d),
          _opt(ref_logp, "ref_logp", f32, 2 * P, d), _opt(dlogits, "dlogits", b16, N * Vp, d),
          _need(logps, "logps", f32, N, d), _opt(seq_logps, "seq_logps", f32, 2 * P, d),
          _need(losses, "losses", f32, P, d), N, P, V, Vp, ignore_index, _kind(kind), 1 if average else 0, beta,
          smoothing, dscale, _need(workspace, "workspace", u8, -1, d), workspace.numel(), _need(err, "err", i32, -1, d))


def orthogonalize_workspace(batch, rows, cols):
    return lib().gpt2op_orthogonalize_workspace(batch, rows, cols)


def _matrices(name, t):
    """(batch, rows, cols, elements between matrices) of contiguous [rows, cols] matrices."""
    if t.dim() not in (2, 3):
        raise ValueError(f"{name}: [rows, cols] or [batch, rows, cols], not {tuple(t.shape)}")
    b, r, c = (1, *t.shape) if t.dim() == 2 else t.shape
    if t.stride(-1) != 1 and c > 1 or t.stride(-2) != c and r > 1:
        raise ValueError(f"{name}: the matrices are not contiguous")
    return b, r, c, t.stride(0) if t.dim() == 3 and b > 1 else r * c


def orthogonalize(x, out, workspace, err, steps=5, stream=None):
    """out = the Newton-Schulz orthogonalisation of x: [rows, cols] or [batch, rows, cols]
    (matrices may lie apart), x fp32 or bf16, out bf16."""
    b16, f32, i32, u8 = _types()
    b, r, c, xs = _matrices("x", x)
    ob, orows, oc, os_ = _matrices("out", out)
    if (ob, orows, oc) != (b, r, c):
        raise ValueError(f"out: {tuple(out.shape)}, x: {tuple(x.shape)}")
    if x.dtype is not f32 and x.dtype is not b16:
        raise ValueError(f"x: {x.dtype}, not float32 or bfloat16")
    if out.dtype is not b16:
        raise ValueError(f"out: {out.dtype}, not bfloat16")
    d = _device_of(x, "x")
    if out.get_device() != d:
        raise ValueError(f"out: on {out.device}, not cuda:{d}")
    _call("gpt2op_orthogonalize", d, stream, x.data_ptr(), 1 if x.dtype is f32 else 0, xs, out.data_ptr(), os_, b, r, c,
          steps, _need(workspace, "workspace", u8, -1, d), workspace.numel(), _need(err, "err", i32, -1, d))

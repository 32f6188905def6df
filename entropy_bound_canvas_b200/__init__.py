"""Python binding of the B200 entropy-bound canvas sampler (libebsampler.so).

Argument marshalling only: every step of the sampler runs in the CUDA
kernels behind the C ABI of ``include/eb_sampler.h``.  PyTorch supplies device
buffers and the current stream; nothing here computes on the data, and there
is no CPU fallback -- importing fails loudly when the library is missing.

    from entropy_bound_canvas_b200 import EBSampler
    s = EBSampler(B=1, L=256, V=262144, seed=1)
    canvas, committed, stop = s.new_canvas()
    H, amax = s.outputs()
    for step in range(48):
        s.step(logits[step], step, canvas, committed, H, amax, stop)
        if s.done(stop):
            break
"""
from __future__ import annotations

import ctypes as C
import dataclasses
import os
from typing import Any, NamedTuple

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libebsampler.so")

F32, BF16 = 0, 1
RULE_ENTROPY_BOUND, RULE_BLOCK_REFINEMENT, RULE_ENTROPY_BOUND_MI = 0, 1, 2
STOP_ACTIVE, STOP_ADAPTIVE, STOP_ALL_COMMITTED, STOP_LAST_STEP = 0, 1, 2, 3
STATUS_BAD_TOKEN, STATUS_NONFINITE, STATUS_TIMEOUT, STATUS_BAD_OFFSETS = 1, 2, 4, 8
GUMBEL_GROUP = 64

EB_OK = 0
ERRORS = {
    1: "EB_ERR_INVALID_ARG", 2: "EB_ERR_CUDA", 3: "EB_ERR_OUT_OF_MEMORY",
    4: "EB_ERR_STEP_ORDER", 5: "EB_ERR_UNSUPPORTED", 6: "EB_ERR_OVERFLOW",
    7: "EB_ERR_DEVICE_STATUS",
}


class EBError(RuntimeError):
    def __init__(self, code: int, what: str):
        self.code = code
        super().__init__(f"{what}: {ERRORS.get(code, code)} ({_lib().eb_strerror(code).decode()})")


class Config(C.Structure):
    """eb_config_t (same field order and types as include/eb_sampler.h)."""
    _fields_ = [
        ("B", C.c_int32), ("L", C.c_int32), ("V", C.c_int32), ("num_steps", C.c_int32),
        ("t_max", C.c_double), ("t_min", C.c_double),
        ("entropy_bound", C.c_double), ("stop_entropy", C.c_double),
        ("stability_steps", C.c_int32), ("rule", C.c_int32),
        ("threshold", C.c_double), ("quota", C.c_int32), ("greedy", C.c_int32),
        ("canvas_offset", C.c_int32), ("seed", C.c_uint64),
        ("editing_threshold", C.c_double), ("vocab_offset", C.c_int32), ("vocab_total", C.c_int32),
    ]


class ScoreInput(C.Structure):
    """eb_score_input_t."""
    _fields_ = [
        ("logits", C.c_void_p), ("dtype", C.c_int32), ("rows", C.c_int32), ("V", C.c_int32),
        ("ld", C.c_int64), ("tokens", C.c_void_p), ("temperatures", C.c_void_p),
        ("temperature", C.c_double),
    ]


class Policy(C.Structure):
    """eb_policy_t."""
    _fields_ = [
        ("old_logprobs", C.c_void_p), ("advantages", C.c_void_p), ("ref_logprobs", C.c_void_p),
        ("weights", C.c_void_p), ("clip_low", C.c_double), ("clip_high", C.c_double),
        ("kl_coef", C.c_double), ("entropy_coef", C.c_double), ("scale", C.c_double),
    ]


class Preference(C.Structure):
    """eb_preference_t."""
    _fields_ = [
        ("offsets", C.c_void_p), ("pairs", C.c_int32), ("ref_logprobs", C.c_void_p),
        ("beta", C.c_double), ("label_smoothing", C.c_double), ("margin", C.c_double),
        ("average", C.c_int32), ("scale", C.c_double),
    ]


class TokenScores(NamedTuple):
    logprobs: Any        # [rows] fp32
    entropies: Any       # [rows] fp32, or None


class PolicyLoss(NamedTuple):
    terms: Any           # [5] fp32: loss, policy term, KL, entropy, clipped share
    logprobs: Any        # [rows] fp32
    entropies: Any       # [rows] fp32
    d_logits: Any        # as the logits, or None


class PreferenceLoss(NamedTuple):
    loss: Any               # [1] fp32
    losses: Any             # [pairs] fp32
    sequence_logprobs: Any  # [2 pairs] fp32
    logprobs: Any           # [rows] fp32
    d_logits: Any           # as the logits, or None


_LIB = None


def _lib():
    global _LIB
    if _LIB is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(
                f"{LIB_PATH} is missing: build it with `python -m entropy_bound_canvas_b200.build` "
                "(nvcc, sm_100a). There is no CPU fallback.")
        L = C.CDLL(LIB_PATH)
        vp, i32, u32p = C.c_void_p, C.c_int, C.POINTER(C.c_uint32)
        L.eb_config_default.argtypes = [C.POINTER(Config), C.c_int32, C.c_int32, C.c_int32]
        L.eb_config_default.restype = None
        L.eb_sampler_init.argtypes = [C.POINTER(vp), C.POINTER(Config), i32]
        L.eb_sampler_init.restype = i32
        L.eb_sampler_init_canvas.argtypes = [vp, vp, vp, vp, vp]
        L.eb_sampler_init_canvas.restype = i32
        L.eb_sampler_step.argtypes = [vp, vp, i32, i32, vp, vp, vp, vp, vp, vp]
        L.eb_sampler_step.restype = i32
        L.eb_canvas_done.argtypes = [vp, vp, i32, C.POINTER(C.c_int), vp]
        L.eb_canvas_done.restype = i32
        L.eb_sampler_status.argtypes = [vp, u32p, i32, vp]
        L.eb_sampler_status.restype = i32
        L.eb_sampler_draws.argtypes = [vp, vp, vp, vp]
        L.eb_sampler_draws.restype = i32
        L.eb_sampler_set_state.argtypes = [vp, vp, vp, i32, vp]
        L.eb_sampler_set_state.restype = i32
        L.eb_sampler_step_slice.argtypes = [vp, vp, i32, i32, vp, vp, vp, vp]
        L.eb_sampler_step_slice.restype = i32
        L.eb_sampler_combine.argtypes = [vp, vp, i32, i32, vp, vp, vp, vp, vp, vp]
        L.eb_sampler_combine.restype = i32
        L.eb_slice_record_bytes.argtypes = []
        L.eb_slice_record_bytes.restype = C.c_size_t
        L.eb_sampler_set_split_event.argtypes = [vp, vp]
        L.eb_sampler_set_split_event.restype = i32
        L.eb_sampler_set_wait_limit.argtypes = [vp, C.c_uint64]
        L.eb_sampler_set_wait_limit.restype = i32
        L.eb_sampler_workspace_bytes.argtypes = [vp]
        L.eb_sampler_workspace_bytes.restype = C.c_size_t
        L.eb_sampler_destroy.argtypes = [vp]
        L.eb_sampler_destroy.restype = None
        L.eb_strerror.argtypes = [i32]
        L.eb_strerror.restype = C.c_char_p
        L.eb_version.argtypes = []
        L.eb_version.restype = i32
        L.eb_lmhead_logits.argtypes = [vp, vp, i32, i32, i32, vp, vp]
        L.eb_lmhead_logits.restype = i32
        L.eb_lmhead_reserve.argtypes = [vp, i32]
        L.eb_lmhead_reserve.restype = i32
        L.eb_lmhead_step.argtypes = [vp, vp, vp, i32, i32, vp, vp, vp, vp, vp, vp]
        L.eb_lmhead_step.restype = i32
        sip, i64, dbl = C.POINTER(ScoreInput), C.c_int64, C.c_double
        L.eb_scorer_init.argtypes = [C.POINTER(vp), C.c_int32, i32]
        L.eb_scorer_init.restype = i32
        L.eb_token_logprobs.argtypes = [vp, sip, vp, vp, vp]
        L.eb_token_logprobs.restype = i32
        L.eb_token_logprobs_backward.argtypes = [vp, sip, vp, vp, vp, i64, vp]
        L.eb_token_logprobs_backward.restype = i32
        L.eb_policy_loss.argtypes = [vp, sip, C.POINTER(Policy), vp, vp, vp, vp, i64, vp]
        L.eb_policy_loss.restype = i32
        L.eb_preference_loss.argtypes = [vp, sip, C.POINTER(Preference), vp, vp, vp, vp, vp, i64,
                                         vp]
        L.eb_preference_loss.restype = i32
        L.eb_lmhead_logprobs.argtypes = [vp, vp, vp, i32, i32, i32, vp, vp, dbl, vp, vp, vp]
        L.eb_lmhead_logprobs.restype = i32
        L.eb_scorer_status.argtypes = [vp, u32p, i32, vp]
        L.eb_scorer_status.restype = i32
        L.eb_scorer_set_wait_limit.argtypes = [vp, C.c_uint64]
        L.eb_scorer_set_wait_limit.restype = i32
        L.eb_scorer_workspace_bytes.argtypes = [vp]
        L.eb_scorer_workspace_bytes.restype = C.c_size_t
        L.eb_scorer_destroy.argtypes = [vp]
        L.eb_scorer_destroy.restype = None
        _LIB = L
    return _LIB


def library():
    """The loaded ctypes library (raises ImportError if it was not built)."""
    return _lib()


def default_config(B: int, L: int, V: int) -> Config:
    c = Config()
    _lib().eb_config_default(C.byref(c), B, L, V)
    return c


def make_config(B, L, V, **kw) -> Config:
    c = default_config(B, L, V)
    for k, v in kw.items():
        if not hasattr(c, k):
            raise TypeError(f"unknown config field {k!r}")
        setattr(c, k, v)
    return c


def _check(rc: int, what: str):
    if rc != EB_OK:
        raise EBError(rc, what)


def _torch():
    import torch
    return torch


def _cuda_device(device):
    """The CUDA device of this index: the current one where none is named."""
    torch = _torch()
    index = None if device is None else torch.device(device).index
    return torch.device("cuda", torch.cuda.current_device() if index is None else index)


def lmhead_logits(hidden, weight, out=None):
    """The LM head's logits hidden @ weight^T (bf16 [rows, d] and [V, d] on
    one device) formed by the fused LM-head kernel's tensor-core contraction,
    written as fp32 [rows, V]: the diagnostic form of eb_lmhead_step."""
    torch = _torch()
    for t, n in ((hidden, "hidden"), (weight, "weight")):
        if t.dtype != torch.bfloat16 or t.dim() != 2 or not t.is_contiguous():
            raise ValueError(f"{n} must be a contiguous 2-D bf16 tensor")
    rows, d = hidden.shape
    V = weight.shape[0]
    if weight.shape[1] != d:
        raise ValueError("hidden and weight disagree on the hidden size")
    if out is None:
        out = torch.empty((rows, V), dtype=torch.float32, device=hidden.device)
    stream = torch.cuda.current_stream(hidden.device).cuda_stream
    _check(_lib().eb_lmhead_logits(C.c_void_p(hidden.data_ptr()), C.c_void_p(weight.data_ptr()),
                                   int(rows), int(V), int(d), C.c_void_p(out.data_ptr()),
                                   C.c_void_p(stream)), "eb_lmhead_logits")
    return out


def shard_canvases(B: int, world: int, rank: int):
    """Contiguous split of B canvases over `world` ranks: (canvas_offset, count)."""
    base, extra = divmod(B, world)
    count = base + (1 if rank < extra else 0)
    offset = rank * base + min(rank, extra)
    return offset, count


class EBSampler:
    """One sampler handle on one CUDA device (see include/eb_sampler.h)."""

    def __init__(self, B: int, L: int, V: int, device=None, **config):
        torch = _torch()
        self.device = _cuda_device(device)
        self.cfg = make_config(B, L, V, **config)
        self.B, self.L, self.V = B, L, V
        h = C.c_void_p()
        _check(_lib().eb_sampler_init(C.byref(h), C.byref(self.cfg), self.device.index),
               "eb_sampler_init")
        self._h = h

    # -- helpers --------------------------------------------------------------
    def _stream(self):
        return C.c_void_p(_torch().cuda.current_stream(self.device).cuda_stream)

    def _ptr(self, t, dtype, shape, name):
        torch = _torch()
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{name} must be a torch tensor")
        if t.device != self.device:
            raise ValueError(f"{name} is on {t.device}, sampler is on {self.device}")
        if dtype is not None and t.dtype != dtype:
            raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
        if shape is not None and tuple(t.shape) != tuple(shape):
            raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
        return C.c_void_p(t.data_ptr())

    # -- buffers --------------------------------------------------------------
    def new_canvas(self):
        """Allocate (canvas, committed, stop_flags) and start fresh canvases."""
        torch = _torch()
        canvas = torch.empty((self.B, self.L), dtype=torch.int32, device=self.device)
        committed = torch.empty((self.B, self.L), dtype=torch.uint8, device=self.device)
        stop = torch.empty((self.B,), dtype=torch.uint8, device=self.device)
        self.init_canvas(canvas, committed, stop)
        return canvas, committed, stop

    def outputs(self):
        """Allocate (entropies, argmax) output buffers."""
        torch = _torch()
        return (torch.empty((self.B, self.L), dtype=torch.float32, device=self.device),
                torch.empty((self.B, self.L), dtype=torch.int32, device=self.device))

    # -- ABI calls ------------------------------------------------------------
    def init_canvas(self, canvas, committed, stop_flags):
        torch = _torch()
        _check(_lib().eb_sampler_init_canvas(
            self._h, self._ptr(canvas, torch.int32, (self.B, self.L), "canvas"),
            self._ptr(committed, torch.uint8, (self.B, self.L), "committed"),
            self._ptr(stop_flags, torch.uint8, (self.B,), "stop_flags"), self._stream()),
            "eb_sampler_init_canvas")

    def step(self, logits, step: int, canvas, committed, entropies, argmax, stop_flags):
        torch = _torch()
        if logits.dtype == torch.float32:
            dt = F32
        elif logits.dtype == torch.bfloat16:
            dt = BF16
        else:
            raise TypeError("logits must be float32 or bfloat16")
        if logits.device != self.device or tuple(logits.shape) != (self.B, self.L, self.V):
            raise ValueError(f"logits must be [{self.B}, {self.L}, {self.V}] on {self.device}")
        if not logits.is_contiguous():
            raise ValueError("logits must be contiguous")
        _check(_lib().eb_sampler_step(
            self._h, C.c_void_p(logits.data_ptr()), dt, int(step),
            self._ptr(canvas, torch.int32, (self.B, self.L), "canvas"),
            self._ptr(committed, torch.uint8, (self.B, self.L), "committed"),
            self._ptr(entropies, torch.float32, (self.B, self.L), "entropies"),
            self._ptr(argmax, torch.int32, (self.B, self.L), "argmax"),
            self._ptr(stop_flags, torch.uint8, (self.B,), "stop_flags"), self._stream()),
            "eb_sampler_step")

    # -- the sampler fused into the LM head --------------------------------------
    def lmhead_step(self, hidden, weight, step: int, canvas, committed, entropies, argmax,
                    stop_flags):
        """A step from the decoder's hidden states: hidden [B, L, d] (or
        [B*L, d]) and the LM head weight [V, d], both bf16; the logits are
        formed on the tensor cores and reduced on chip (never written)."""
        torch = _torch()
        for t, n in ((hidden, "hidden"), (weight, "weight")):
            if t.dtype != torch.bfloat16 or not t.is_contiguous() or t.device != self.device:
                raise ValueError(f"{n} must be a contiguous bf16 tensor on {self.device}")
        d = int(hidden.shape[-1])
        if hidden.numel() != self.B * self.L * d or tuple(weight.shape) != (self.V, d):
            raise ValueError(f"hidden must hold [{self.B}*{self.L}, d], weight [{self.V}, d]")
        if not getattr(self, "_lm_reserved", False):
            _check(_lib().eb_lmhead_reserve(self._h, d), "eb_lmhead_reserve")
            self._lm_reserved = True
        _check(_lib().eb_lmhead_step(
            self._h, C.c_void_p(hidden.data_ptr()), C.c_void_p(weight.data_ptr()), d, int(step),
            self._ptr(canvas, torch.int32, (self.B, self.L), "canvas"),
            self._ptr(committed, torch.uint8, (self.B, self.L), "committed"),
            self._ptr(entropies, torch.float32, (self.B, self.L), "entropies"),
            self._ptr(argmax, torch.int32, (self.B, self.L), "argmax"),
            self._ptr(stop_flags, torch.uint8, (self.B,), "stop_flags"), self._stream()),
            "eb_lmhead_step")

    # -- vocabulary-sharded logits ---------------------------------------------
    def slice_records(self):
        """A records buffer for one slice: [B, L, record bytes] uint8."""
        torch = _torch()
        n = int(_lib().eb_slice_record_bytes())
        return torch.empty((self.B, self.L, n), dtype=torch.uint8, device=self.device)

    def step_slice(self, logits, step: int, committed, stop_flags, records):
        """This device's vocabulary slice of a step: per-position records."""
        torch = _torch()
        dt = self._dtype(logits)
        n = int(_lib().eb_slice_record_bytes())
        _check(_lib().eb_sampler_step_slice(
            self._h, C.c_void_p(logits.data_ptr()), dt, int(step),
            self._ptr(committed, torch.uint8, (self.B, self.L), "committed"),
            self._ptr(stop_flags, torch.uint8, (self.B,), "stop_flags"),
            self._ptr(records, torch.uint8, (self.B, self.L, n), "records"), self._stream()),
            "eb_sampler_step_slice")

    def combine(self, all_records, step: int, canvas, committed, entropies, argmax, stop_flags):
        """Every slice's records ([n_slices, B, L, record bytes], slice order) ->
        the step's results and canvas decisions, as step() gives them."""
        torch = _torch()
        n = int(_lib().eb_slice_record_bytes())
        if all_records.dim() != 4 or tuple(all_records.shape[1:]) != (self.B, self.L, n):
            raise ValueError(f"records must be [n_slices, {self.B}, {self.L}, {n}]")
        _check(_lib().eb_sampler_combine(
            self._h, self._ptr(all_records, torch.uint8, None, "records"),
            int(all_records.shape[0]), int(step),
            self._ptr(canvas, torch.int32, (self.B, self.L), "canvas"),
            self._ptr(committed, torch.uint8, (self.B, self.L), "committed"),
            self._ptr(entropies, torch.float32, (self.B, self.L), "entropies"),
            self._ptr(argmax, torch.int32, (self.B, self.L), "argmax"),
            self._ptr(stop_flags, torch.uint8, (self.B,), "stop_flags"), self._stream()),
            "eb_sampler_combine")

    def step_split(self, logits, step: int, canvas, committed, entropies, argmax, stop_flags,
                   group=None):
        """A step over vocabulary-sharded logits: this rank's slice, one
        all-gather of the records over `group` (ranks ordered by slice), then
        the combine.  Without a process group the handle is the only slice."""
        torch = _torch()
        rec = self.slice_records()
        self.step_slice(logits, step, committed, stop_flags, rec)
        world = 1
        if group is not None or (torch.distributed.is_available()
                                 and torch.distributed.is_initialized()):
            world = torch.distributed.get_world_size(group)
        if world == 1:
            allr = rec.unsqueeze(0)
        else:
            allr = torch.empty((world,) + tuple(rec.shape), dtype=rec.dtype, device=rec.device)
            torch.distributed.all_gather_into_tensor(allr, rec, group=group)
        self.combine(allr, step, canvas, committed, entropies, argmax, stop_flags)

    def _dtype(self, logits):
        torch = _torch()
        if logits.dtype == torch.float32:
            dt = F32
        elif logits.dtype == torch.bfloat16:
            dt = BF16
        else:
            raise TypeError("logits must be float32 or bfloat16")
        if logits.device != self.device or tuple(logits.shape) != (self.B, self.L, self.V):
            raise ValueError(f"logits must be [{self.B}, {self.L}, {self.V}] on {self.device}")
        if not logits.is_contiguous():
            raise ValueError("logits must be contiguous")
        return dt

    def step_ptr(self, logits_ptr: int, dtype: int, step: int, canvas_ptr: int,
                 committed_ptr: int, entropies_ptr: int, argmax_ptr: int, stop_ptr: int,
                 stream_ptr: int = 0) -> int:
        """Raw pointer form of eb_sampler_step (returns the status code)."""
        return _lib().eb_sampler_step(self._h, C.c_void_p(logits_ptr), dtype, step,
                                      C.c_void_p(canvas_ptr), C.c_void_p(committed_ptr),
                                      C.c_void_p(entropies_ptr), C.c_void_p(argmax_ptr),
                                      C.c_void_p(stop_ptr), C.c_void_p(stream_ptr))

    def done(self, stop_flags, b: int = -1, check_status: bool = True) -> bool:
        torch = _torch()
        d = C.c_int(0)
        rc = _lib().eb_canvas_done(self._h, self._ptr(stop_flags, torch.uint8, (self.B,),
                                                      "stop_flags"), b, C.byref(d), self._stream())
        if rc != EB_OK and (check_status or rc != 7):
            raise EBError(rc, "eb_canvas_done")
        return bool(d.value)

    def status(self, clear: bool = False) -> int:
        s = C.c_uint32(0)
        _check(_lib().eb_sampler_status(self._h, C.byref(s), int(clear), self._stream()),
               "eb_sampler_status")
        return int(s.value)

    def draws(self):
        """(sample [B, L] int32, pmax [B, L] float32) of the last step."""
        torch = _torch()
        smp = torch.empty((self.B, self.L), dtype=torch.int32, device=self.device)
        pm = torch.empty((self.B, self.L), dtype=torch.float32, device=self.device)
        _check(_lib().eb_sampler_draws(self._h, C.c_void_p(smp.data_ptr()),
                                       C.c_void_p(pm.data_ptr()), self._stream()),
               "eb_sampler_draws")
        return smp, pm

    def set_state(self, prev_argmax, stable=None, next_step: int = 0):
        torch = _torch()
        sp = self._ptr(stable, torch.int32, (self.B,), "stable") if stable is not None else None
        _check(_lib().eb_sampler_set_state(
            self._h, self._ptr(prev_argmax, torch.int32, (self.B, self.L), "prev_argmax"),
            sp, next_step, self._stream()), "eb_sampler_set_state")

    def set_split_event(self, event=None):
        """Record `event` (a torch.cuda.Event, or None to stop) between the two
        kernels of every following step, for timing them apart."""
        ptr = None
        if event is not None:
            if not event.cuda_event:  # torch creates the CUDA event on first record
                event.record(_torch().cuda.current_stream(self.device))
            ptr = C.c_void_p(event.cuda_event)
        _check(_lib().eb_sampler_set_split_event(self._h, ptr), "eb_sampler_set_split_event")

    def set_wait_limit(self, limit_ns: int = 0):
        """Limit (ns) of the stream kernel's pipeline waits; 0 = the default
        2 s.  A diagnostic hook: a tiny limit makes a wait run out, which sets
        STATUS_TIMEOUT instead of hanging (see include/eb_sampler.h)."""
        _check(_lib().eb_sampler_set_wait_limit(self._h, int(limit_ns)),
               "eb_sampler_set_wait_limit")

    def workspace_bytes(self) -> int:
        return int(_lib().eb_sampler_workspace_bytes(self._h))

    def close(self):
        if getattr(self, "_h", None):
            _lib().eb_sampler_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        self.close()


class EBScorer:
    """Scores sampled tokens and learns from them, on one CUDA device: token
    log-probabilities and entropies with their gradient, the clipped policy
    loss and the preference loss with theirs (eb_scorer_t of
    include/eb_sampler.h, which gives the formulas).

    A row is one position.  Logits are [rows, V] with unit stride along V (a
    [B, L, V] tensor is taken as B*L rows), fp32 or bf16; tokens int32, a
    negative one ignores its row; temperature a number or an fp32 tensor of
    one per row.  Results are allocated here unless ``out`` gives the
    gradient's buffer, which may be the logits themselves.  Calls run on the
    device's current stream, never synchronise, and can be captured in a CUDA
    graph (keep the scorer as long as its graphs); one scorer per stream at a
    time.
    """

    def __init__(self, max_rows: int, device=None):
        torch = _torch()
        self.device = _cuda_device(device)
        self.max_rows = int(max_rows)
        h = C.c_void_p()
        _check(_lib().eb_scorer_init(C.byref(h), self.max_rows, self.device.index),
               "eb_scorer_init")
        self._h = h
        self._f32 = torch.empty((1,), dtype=torch.float32, device=self.device)
        self._shapes = {}
        self._i32, self._bf16, self._Tensor = torch.int32, torch.bfloat16, torch.Tensor
        self._like, self._dense = torch.empty_like, torch.contiguous_format
        # the stream's handle without a Stream object, where torch offers it
        raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
        self._raw_stream = raw or (lambda i: torch.cuda.current_stream(i).cuda_stream)

    # -- helpers --------------------------------------------------------------
    def _stream(self):
        return self._raw_stream(self.device.index)

    def _vector(self, t, n, dtype, name):
        """Address of a contiguous tensor of n values (None: a null pointer)."""
        if t is None:
            return None
        if not isinstance(t, self._Tensor):
            raise TypeError(f"{name} must be a torch tensor")
        if t.dtype is dtype and t.device == self.device and t.numel() == n and t.is_contiguous():
            return t.data_ptr()
        if t.device != self.device:
            raise ValueError(f"{name} is on {t.device}, scorer is on {self.device}")
        if t.dtype != dtype:
            raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
        raise ValueError(f"{name} must be contiguous and hold {n} values, got {tuple(t.shape)}")

    def _matrix(self, t, name):
        """(address, rows, V, elements between rows) of logits or a gradient."""
        if not isinstance(t, self._Tensor):
            raise TypeError(f"{name} must be a torch tensor")
        if t.dtype is not self._f32.dtype and t.dtype is not self._bf16:
            raise TypeError(f"{name} must be float32 or bfloat16")
        if t.device != self.device:
            raise ValueError(f"{name} is on {t.device}, scorer is on {self.device}")
        if t.dim() != 2:
            if t.dim() < 2:
                raise ValueError(f"{name} must be [rows, V]")
            try:
                t = t.view(-1, t.shape[-1])
            except RuntimeError:
                raise ValueError(f"{name}: the rows must lie at one stride") from None
        rows, V = t.shape
        ld, step = t.stride()
        if V > 1 and step != 1:
            raise ValueError(f"{name} must have unit stride along V")
        if rows <= 1:
            ld = V
        elif ld < V:
            raise ValueError(f"{name}: rows overlap")
        return t.data_ptr(), rows, V, ld

    def _input(self, logits, tokens, temperature):
        ptr, rows, V, ld = self._matrix(logits, "logits")
        dtype = F32 if logits.dtype is self._f32.dtype else BF16
        tok = self._vector(tokens, rows, self._i32, "tokens")
        if isinstance(temperature, self._Tensor):
            return ScoreInput(ptr, dtype, rows, V, ld, tok,
                              self._vector(temperature, rows, self._f32.dtype, "temperature"), 0.0)
        return ScoreInput(ptr, dtype, rows, V, ld, tok, None, temperature)

    def _gradient(self, logits, s, out):
        """(gradient tensor shaped as the logits, its address, its row stride)."""
        if out is None:
            out = self._like(logits, memory_format=self._dense)
            return out, out.data_ptr(), s.V
        if not isinstance(out, self._Tensor):
            raise TypeError("out must be a torch tensor")
        if out.shape != logits.shape or out.dtype != logits.dtype:
            raise ValueError("out must have the logits' shape and type")
        ptr, _, _, ldd = self._matrix(out, "out")
        return out, ptr, ldd

    def _new(self, n):
        """n fp32 values (empty_like of a kept shape without memory of its own:
        the cheapest of torch's allocations)."""
        shape = self._shapes.get(n)
        if shape is None:
            if len(self._shapes) >= 256:
                self._shapes.clear()
            shape = self._shapes[n] = self._f32.expand(n)
        return self._like(shape, memory_format=self._dense)

    # -- calls ------------------------------------------------------------------
    def token_logprobs(self, logits, tokens, temperature=1.0, entropies: bool = True):
        """Each row's log p[token] and (unless entropies=False) entropy."""
        s = self._input(logits, tokens, temperature)
        lp = self._new(s.rows)
        h = self._new(s.rows) if entropies else None
        _check(_lib().eb_token_logprobs(self._h, C.byref(s), lp.data_ptr(),
                                        h.data_ptr() if entropies else None, self._stream()),
               "eb_token_logprobs")
        return TokenScores(lp, h)

    def token_logprobs_backward(self, logits, tokens, d_logprobs, d_entropies=None,
                                temperature=1.0, out=None):
        """The gradient for the logits from those of token_logprobs' results."""
        s = self._input(logits, tokens, temperature)
        n, f32 = s.rows, self._f32.dtype
        out, ptr, ldd = self._gradient(logits, s, out)
        _check(_lib().eb_token_logprobs_backward(
            self._h, C.byref(s), self._vector(d_logprobs, n, f32, "d_logprobs"),
            self._vector(d_entropies, n, f32, "d_entropies"), ptr, ldd, self._stream()),
            "eb_token_logprobs_backward")
        return out

    def policy_loss(self, logits, tokens, old_logprobs, advantages, ref_logprobs=None,
                    weights=None, temperature=1.0, clip_low=0.2, clip_high=0.2, kl_coef=0.0,
                    entropy_coef=0.0, scale=1.0, grad: bool = True, out=None):
        """Clipped policy loss with a KL term and an entropy bonus, and its
        gradient for the logits (grad=False: the loss alone)."""
        s = self._input(logits, tokens, temperature)
        n, f32 = s.rows, self._f32.dtype
        p = Policy(self._vector(old_logprobs, n, f32, "old_logprobs"),
                   self._vector(advantages, n, f32, "advantages"),
                   self._vector(ref_logprobs, n, f32, "ref_logprobs"),
                   self._vector(weights, n, f32, "weights"), clip_low, clip_high, kl_coef,
                   entropy_coef, scale)
        d, ptr, ldd = self._gradient(logits, s, out) if grad else (None, None, 0)
        terms, lp, h = self._new(5), self._new(n), self._new(n)
        _check(_lib().eb_policy_loss(self._h, C.byref(s), C.byref(p), terms.data_ptr(),
                                     lp.data_ptr(), h.data_ptr(), ptr, ldd, self._stream()),
               "eb_policy_loss")
        return PolicyLoss(terms, lp, h, d)

    def preference_loss(self, logits, tokens, offsets, ref_logprobs=None, beta=0.1,
                        label_smoothing=0.0, margin=0.0, average: bool = False, temperature=1.0,
                        scale=1.0, grad: bool = True, out=None):
        """Preference loss over pairs of sequences and its gradient for the
        logits.  offsets [2 pairs + 1] int32 (device): sequence s is the rows
        offsets[s]..offsets[s+1], the chosen sequences first, then the
        rejected ones; ref_logprobs [2 pairs] a reference model's sums."""
        s = self._input(logits, tokens, temperature)
        n, f32 = s.rows, self._f32.dtype
        if not isinstance(offsets, self._Tensor) or offsets.dim() != 1 \
                or offsets.numel() % 2 != 1:
            raise ValueError("offsets must be a 1-D tensor of 2 * pairs + 1 values")
        pairs = offsets.numel() // 2
        p = Preference(self._vector(offsets, 2 * pairs + 1, self._i32, "offsets"), pairs,
                       self._vector(ref_logprobs, 2 * pairs, f32, "ref_logprobs"),
                       beta, label_smoothing, margin, int(average), scale)
        d, ptr, ldd = self._gradient(logits, s, out) if grad else (None, None, 0)
        loss, losses, seq, lp = (self._new(1), self._new(pairs), self._new(2 * pairs),
                                 self._new(n))
        _check(_lib().eb_preference_loss(self._h, C.byref(s), C.byref(p), loss.data_ptr(),
                                         losses.data_ptr(), seq.data_ptr(), lp.data_ptr(), ptr,
                                         ldd, self._stream()), "eb_preference_loss")
        return PreferenceLoss(loss, losses, seq, lp, d)

    def lmhead_logprobs(self, hidden, weight, tokens, temperature=1.0, entropies: bool = True):
        """token_logprobs on the logits hidden @ weight^T (bf16 [rows, d] or
        [B, L, d], and [V, d]) without forming them in memory."""
        for t, n in ((hidden, "hidden"), (weight, "weight")):
            if not isinstance(t, self._Tensor):
                raise TypeError(f"{n} must be a torch tensor")
            if t.dtype != self._bf16 or not t.is_contiguous() or t.device != self.device:
                raise ValueError(f"{n} must be a contiguous bf16 tensor on {self.device}")
        if hidden.dim() < 2 or weight.dim() != 2 or weight.shape[1] != hidden.shape[-1]:
            raise ValueError("hidden must be [rows, d] and weight [V, d]")
        V, d = weight.shape
        rows = hidden.numel() // d if d else 0
        lp = self._new(rows)
        h = self._new(rows) if entropies else None
        tensor = isinstance(temperature, self._Tensor)
        _check(_lib().eb_lmhead_logprobs(
            self._h, hidden.data_ptr(), weight.data_ptr(), rows, V, d,
            self._vector(tokens, rows, self._i32, "tokens"),
            self._vector(temperature, rows, self._f32.dtype, "temperature") if tensor else None,
            1.0 if tensor else float(temperature), lp.data_ptr(),
            h.data_ptr() if entropies else None, self._stream()), "eb_lmhead_logprobs")
        return TokenScores(lp, h)

    def status(self, clear: bool = False) -> int:
        s = C.c_uint32(0)
        _check(_lib().eb_scorer_status(self._h, C.byref(s), int(clear), self._stream()),
               "eb_scorer_status")
        return int(s.value)

    def set_wait_limit(self, limit_ns: int = 0):
        """Limit (ns) of the internal waits; 0 = the default 2 s (a diagnostic
        hook, see include/eb_sampler.h)."""
        _check(_lib().eb_scorer_set_wait_limit(self._h, int(limit_ns)),
               "eb_scorer_set_wait_limit")

    def workspace_bytes(self) -> int:
        return int(_lib().eb_scorer_workspace_bytes(self._h))

    def close(self):
        if getattr(self, "_h", None):
            _lib().eb_scorer_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        self.close()

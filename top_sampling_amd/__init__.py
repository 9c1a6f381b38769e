"""Python binding of ``libtopsampling.so`` (MI355X / gfx950).

Argument marshalling only: every step of the sampling path runs in the HIP
kernels behind the C ABI (``include/top_sampling.h``).  PyTorch supplies device
memory and the current stream.  Importing this package fails if the library is
not built (``python top_sampling_amd/build.py``); there is no fallback.

Calls mirror the C entry points:
  lmhead_logits_local            local vocabulary projection, bf16 -> fp32
  lmhead_logits_local_lora       the same, each row with its own low-rank
                                 adapter
  quantize_rows_e4m3             per-row FP8 (E4M3) quantization of bf16 rows
  lmhead_logits_local_e4m3       the same projection from FP8 codes and scales
  (de)quantize_groups_e2m1       4-bit (MX FP4) quantization of rows, a scale
                                 per group of 32, and the values it stands for
  lmhead_logits_local_e2m1       the projection of bf16 hidden states from a
                                 4-bit lm_head
  sampler_assemble_vocab_slices  stitch received vocabulary slices
  sampler_sample                 per-row temperature / top-k / top-p /
                                 logprobs / Gumbel-max sampling
  sampler_sample_slices          the same, reading the received vocabulary
                                 slices in place (no stitched buffer)
  sampler_sample_ex              slices plus flags (processed log-probabilities)
  sampler_workspace_bytes(_slices)  workspace size queries
  token_logprobs(_backward[_ex]) log-probability and entropy of given tokens,
                                 and the gradient of a function of them
  token_logprobs_topn            the same with the tokens' ranks and the rows'
                                 most likely alternatives
  token_logprobs_listed(_backward)  log-probabilities of several listed tokens
                                 a row, and the gradient of a function of them
  policy_loss                    clipped policy loss with a KL term
  preference_loss                loss of paired log ratios
``stream`` (None: the current one) is where a call's kernels run.  The scoring,
loss, adapter and 4-bit calls allocate outputs and workspaces for it; inputs have to be
ready there, and to live until the kernels have run (``record_stream`` where they
were allocated for another one).
``compute_logits_local`` returns the rank's own ``[rows, V_local]`` slice,
the local-logits hook of batch-sharded sampling (page "Qwen4Exp batch-sharded
sampling: inside vLLM PR #61018", section "Why three lines were the whole
job").
"""
from __future__ import annotations

import ctypes
import os
from dataclasses import dataclass

import numpy as np

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libtopsampling.so")

TS_OK, TS_EINVAL, TS_EUNSUPPORTED, TS_EWORKSPACE, TS_EHIP = 0, -1, -2, -3, -4
TS_ROW_OK, TS_ROW_BAD_PARAMS, TS_ROW_BAD_LOGITS = 0, 1, 2
TS_MAX_LOGPROBS = 1024
TS_MAX_SLICES = 64
TS_LOGPROBS_PROCESSED = 1
TS_PROBE_SMALL_OPERANDS, TS_PROBE_RANDOM_OPERANDS = 0, 1
TS_NOALLOC_SCRATCH_BYTES = 96 << 20
PARAMS_BYTES = 24
TS_F32, TS_BF16 = 0, 1
TS_PREFERENCE_MEAN = 1
TS_MAX_LORA_RANK = 256
TS_MAX_LISTED = 1024
TS_MAX_LORA_ROWS = 1 << 20

# (name, restype, argtypes) of every symbol the headers declare
# (include/top_sampling.h and the measurement aids of top_sampling_measure.h).
_VP, _I64, _I32, _SZ = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_size_t
_F64 = ctypes.c_double
SYMBOLS = {
    "lmhead_logits_local": (ctypes.c_int, [_VP, _I64, _I64, _I64, _VP, _I64, _I64, _VP, _I64, _VP]),
    "lmhead_lora_workspace_bytes": (_SZ, [_I64, _I64]),
    "lmhead_logits_local_lora": (ctypes.c_int, [_VP, _I64, _I64, _I64, _VP, _I64, _I64, _VP, _I64,
                                                _I64, _VP, _I64, _I64, _I64, _I64, _VP, _VP, _VP,
                                                _I64, _VP, _SZ, _VP]),
    "quantize_rows_e4m3": (ctypes.c_int, [_VP, _I64, _I64, _I64, _VP, _I64, _VP, _VP]),
    "lmhead_logits_local_e4m3": (ctypes.c_int, [_VP, _VP, _I64, _I64, _I64, _VP, _VP, _I64, _I64,
                                                _VP, _I64, _VP]),
    "quantize_groups_e2m1": (ctypes.c_int, [_VP, _I32, _I64, _I64, _I64, _VP, _I64, _VP, _I64,
                                            _VP]),
    "dequantize_groups_e2m1": (ctypes.c_int, [_VP, _I64, _I64, _I64, _VP, _I64, _VP, _I32, _I64,
                                              _VP]),
    "lmhead_logits_local_e2m1": (ctypes.c_int, [_VP, _I64, _I64, _I64, _VP, _VP, _I64, _I64, _I64,
                                                _VP, _I64, _VP]),
    "sampler_workspace_bytes": (_SZ, [_I64, _I64, _I32]),
    "sampler_sample": (ctypes.c_int, [_VP, _I64, _I64, _I64, _VP, _I64, _I32, _VP, _VP, _VP, _VP,
                                      _VP, _VP, _SZ, _VP]),
    "sampler_sample_noalloc": (ctypes.c_int, [_VP, _I64, _I64, _I64, _VP, _I64, _I32, _VP, _VP,
                                              _VP, _VP, _VP, _VP]),
    "sampler_workspace_bytes_slices": (_SZ, [_I64, _VP, _I32, _I32]),
    "sampler_sample_slices": (ctypes.c_int, [_VP, _VP, _VP, _I32, _I64, _VP, _I64, _I32, _VP, _VP,
                                             _VP, _VP, _VP, _VP, _SZ, _VP]),
    "sampler_sample_ex": (ctypes.c_int, [_VP, _VP, _VP, _I32, _I64, _VP, _I64, _I32, _I32, _VP,
                                         _VP, _VP, _VP, _VP, _VP, _SZ, _VP]),
    "sampler_assemble_vocab_slices": (ctypes.c_int, [_VP, _VP, _VP, _I32, _I64, _VP, _I64, _VP]),
    "sampler_assemble_and_sample": (ctypes.c_int, [_VP, _VP, _VP, _I32, _I64, _VP, _I64, _VP, _I64,
                                                   _I32, _I32, _VP, _VP, _VP, _VP, _VP, _VP, _SZ,
                                                   _VP]),
    "ts_mfma_clock_probe": (ctypes.c_int, [_VP, _I32, _I64, _I32, _VP]),
    "ts_gumbel_keys": (ctypes.c_int, [_VP, _VP, _VP, _VP, _VP, _VP, _I64, _VP, _VP, _VP]),
    "token_logprobs_workspace_bytes": (_SZ, [_I64, _I64]),
    "token_logprobs": (ctypes.c_int, [_VP, _I32, _I64, _I64, _I64, _VP, _F64, _VP, _VP, _VP, _VP,
                                      _VP, _SZ, _VP]),
    "token_logprobs_backward": (ctypes.c_int, [_VP, _I32, _I64, _I64, _I64, _VP, _F64, _VP, _VP,
                                               _VP, _VP, _VP, _I64, _VP]),
    "token_logprobs_backward_ex": (ctypes.c_int, [_VP, _I32, _I64, _I64, _I64, _VP, _F64, _VP, _VP,
                                                  _VP, _VP, _VP, _VP, _I64, _VP]),
    "token_logprobs_topn_workspace_bytes": (_SZ, [_I64, _I64]),
    "token_logprobs_topn": (ctypes.c_int, [_VP, _I32, _I64, _I64, _I64, _VP, _F64, _I32, _VP, _VP,
                                           _VP, _VP, _VP, _VP, _VP, _VP, _SZ, _VP]),
    "token_logprobs_listed_workspace_bytes": (_SZ, [_I64, _I64]),
    "token_logprobs_listed": (ctypes.c_int, [_VP, _I32, _I64, _I64, _I64, _VP, _I32, _F64, _VP,
                                             _VP, _VP, _VP, _VP, _SZ, _VP]),
    "token_logprobs_listed_backward": (ctypes.c_int, [_VP, _I32, _I64, _I64, _I64, _VP, _I32,
                                                      _F64, _VP, _VP, _VP, _VP, _VP, _VP, _I64,
                                                      _VP]),
    "policy_loss": (ctypes.c_int, [_VP, _I32, _I64, _I64, _I64, _VP, _VP, _VP, _VP, _VP, _VP, _VP,
                                   _VP, _VP, _VP, _VP, _VP, _VP, _I64, _VP, _SZ, _VP]),
    "preference_loss_workspace_bytes": (_SZ, [_I64, _I64, _I64]),
    "preference_loss": (ctypes.c_int, [_VP, _I32, _I64, _I64, _I64, _VP, _VP, _I64, _VP, _VP, _VP,
                                       _VP, _VP, _VP, _VP, _VP, _VP, _VP, _I64, _VP, _SZ, _VP]),
    "ts_status_string": (ctypes.c_char_p, [ctypes.c_int]),
    "ts_last_error": (ctypes.c_char_p, []),
}


def _load() -> ctypes.CDLL:
    # PyTorch ships its own HIP runtime.  Load it first so the library binds to
    # that same runtime: a second copy of the HIP/HSA runtime in the process
    # (the one under /opt/rocm) would own the device independently.
    import torch  # noqa: F401

    if not os.path.exists(LIB_PATH):
        raise ImportError(
            f"{LIB_PATH} is not built; run `python top_sampling_amd/build.py` (hipcc, gfx950)")
    lib = ctypes.CDLL(LIB_PATH)
    for name, (res, args) in SYMBOLS.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    return lib


lib = _load()
import torch  # noqa: E402  (_load has loaded it)


class TopSamplingError(RuntimeError):
    def __init__(self, code: int, msg: str):
        super().__init__(f"{lib.ts_status_string(code).decode()}: {msg}")
        self.code = code


class TopSamplingValueError(TopSamplingError, ValueError):
    pass


def _check(code: int) -> None:
    if code == TS_OK:
        return
    msg = lib.ts_last_error().decode()
    if code in (TS_EINVAL, TS_EUNSUPPORTED, TS_EWORKSPACE):
        raise TopSamplingValueError(code, msg)
    raise TopSamplingError(code, msg)


def _torch():
    import torch

    return torch


def _stream_ptr(stream) -> int:
    torch = _torch()
    if stream is None:
        stream = torch.cuda.current_stream()
    return int(stream.cuda_stream) if hasattr(stream, "cuda_stream") else int(stream)


def _ptr(t) -> int | None:
    return None if t is None else t.data_ptr()


# ---------------------------------------------------------------- projection
def lmhead_logits_local(hidden, lm_head, out=None, stream=None):
    """fp32 ``[rows, V_local]`` logits of bf16 ``hidden [rows, H]`` against the
    bf16 vocabulary slice ``lm_head [V_local, H]``.  ``out`` may be a column
    slice of a wider fp32 buffer (its row stride is the leading dimension)."""
    torch = _torch()
    rows, h = hidden.shape
    vocab, h2 = lm_head.shape
    if h != h2:
        raise ValueError(f"hidden size mismatch: {h} vs {h2}")
    if hidden.dtype != torch.bfloat16 or lm_head.dtype != torch.bfloat16:
        raise TypeError("hidden and lm_head must be bfloat16")
    if hidden.stride(1) != 1 or lm_head.stride(1) != 1:
        raise ValueError("hidden and lm_head must be K-contiguous")
    if out is None:
        out = torch.empty(rows, vocab, dtype=torch.float32, device=hidden.device)
    if out.shape != (rows, vocab) or out.dtype != torch.float32 or out.stride(1) != 1:
        raise ValueError("out must be fp32 [rows, V_local] with unit column stride")
    _check(lib.lmhead_logits_local(_ptr(hidden), rows, h, hidden.stride(0), _ptr(lm_head), vocab,
                                   lm_head.stride(0), _ptr(out), out.stride(0),
                                   _stream_ptr(stream)))
    return out


def compute_logits_local(hidden, lm_head, out=None, stream=None):
    """The rank's own vocabulary shard ``[rows, V_local]``: no gather, no
    full-vocabulary buffer anywhere."""
    return lmhead_logits_local(hidden, lm_head, out=out, stream=stream)


# ---------------------------------------------------------- FP8 projection
def quantize_rows_e4m3(x, out=None, scales=None, stream=None):
    """bf16 ``[rows, cols]`` -> (uint8 E4M3 codes ``[rows, cols]``, fp32 per-row
    scales ``[rows]``): scale = max|x| / 448, code = nearest E4M3 of x / scale."""
    torch = _torch()
    if x.dtype != torch.bfloat16 or x.dim() != 2 or x.stride(1) != 1:
        raise ValueError("x must be bf16 [rows, cols] with unit column stride")
    rows, cols = x.shape
    if out is None:
        out = torch.empty(rows, cols, dtype=torch.uint8, device=x.device)
    if scales is None:
        scales = torch.empty(rows, dtype=torch.float32, device=x.device)
    _check(lib.quantize_rows_e4m3(_ptr(x), rows, cols, x.stride(0), _ptr(out), out.stride(0),
                                  _ptr(scales), _stream_ptr(stream)))
    return out, scales


def lmhead_logits_local_e4m3(hidden, hidden_scales, lm_head, lm_head_scales, out=None,
                             stream=None):
    """fp32 ``[rows, V_local]`` = s_x[r] * s_w[v] * (codes_x @ codes_w^T) for
    uint8 E4M3 codes ``hidden [rows, H]``, ``lm_head [V_local, H]`` and fp32
    per-row scales: the rank's own vocabulary slice, no gather."""
    torch = _torch()
    rows, h = hidden.shape
    vocab, h2 = lm_head.shape
    if h != h2 or hidden.dtype != torch.uint8 or lm_head.dtype != torch.uint8:
        raise ValueError("hidden and lm_head must be uint8 codes with the same hidden size")
    if hidden.stride(1) != 1 or lm_head.stride(1) != 1:
        raise ValueError("codes must have unit column stride")
    if out is None:
        out = torch.empty(rows, vocab, dtype=torch.float32, device=hidden.device)
    _check(lib.lmhead_logits_local_e4m3(
        _ptr(hidden), _ptr(hidden_scales), rows, h, hidden.stride(0), _ptr(lm_head),
        _ptr(lm_head_scales), vocab, lm_head.stride(0), _ptr(out), out.stride(0),
        _stream_ptr(stream)))
    return out


# ------------------------------------------------------------------ assembly
def sampler_assemble_vocab_slices(slices, out=None, stream=None):
    """``out[:, off_s:off_s+cols_s] = slices[s]`` (bit-exact)."""
    torch = _torch()
    n, rows, ptrs, cols, lds = _slice_arrays(slices)
    total = sum(int(s.shape[1]) for s in slices)
    if out is None:
        out = torch.empty(rows, total, dtype=torch.float32, device=slices[0].device)
    if out.shape != (rows, total) or out.stride(1) != 1 or out.dtype != torch.float32:
        raise ValueError("out must be fp32 [rows, sum cols] with unit column stride")
    _check(lib.sampler_assemble_vocab_slices(ptrs, cols, lds, n, rows, _ptr(out), out.stride(0),
                                             _stream_ptr(stream)))
    return out


# ------------------------------------------------------------------- sampler
def sampler_workspace_bytes(rows: int, vocab: int, max_logprobs: int) -> int:
    return int(lib.sampler_workspace_bytes(rows, vocab, max_logprobs))


def params_to_device(params: np.ndarray, device):
    """Copy a record array of row parameters (24-byte records) to the device."""
    torch = _torch()
    raw = np.ascontiguousarray(params).view(np.uint8).reshape(-1)
    if raw.shape[0] != PARAMS_BYTES * params.shape[0]:
        raise ValueError("parameter records must be 24 bytes")
    return torch.from_numpy(raw.copy()).to(device)


@dataclass
class SampleOutput:
    token_ids: object       # int32 [rows]
    token_logprobs: object  # fp32 [rows]
    topn_ids: object        # int32 [rows, max_logprobs]
    topn_logprobs: object   # fp32 [rows, max_logprobs]
    row_status: object      # int32 [rows]


def allocate_sample_output(rows: int, max_logprobs: int, device) -> SampleOutput:
    torch = _torch()
    return SampleOutput(
        torch.empty(rows, dtype=torch.int32, device=device),
        torch.empty(rows, dtype=torch.float32, device=device),
        torch.empty(rows, max_logprobs, dtype=torch.int32, device=device),
        torch.empty(rows, max_logprobs, dtype=torch.float32, device=device),
        torch.empty(rows, dtype=torch.int32, device=device),
    )


def allocate_workspace(rows: int, vocab: int, max_logprobs: int, device):
    torch = _torch()
    n = max(256, sampler_workspace_bytes(rows, vocab, max_logprobs))
    return torch.empty(n, dtype=torch.uint8, device=device)


def sampler_sample(logits, params, row_offset: int = 0, max_logprobs: int = 0, out=None,
                   workspace=None, stream=None, processed: bool = False) -> SampleOutput:
    """Sample one token per row of fp32 ``logits [rows, V]`` (row stride = its
    leading dimension).  ``params`` is a device uint8 tensor of 24-byte
    ``ts_row_params`` records (see ``params_to_device``).  ``processed``
    returns log-probabilities of the sampled distribution (sampler_sample_ex
    with TS_LOGPROBS_PROCESSED) instead of the raw log_softmax."""
    if processed:
        return sampler_sample_slices([logits], params, row_offset, max_logprobs, out=out,
                                     workspace=workspace, stream=stream, processed=True)
    torch = _torch()
    rows, vocab = logits.shape
    if logits.dtype != torch.float32 or logits.stride(1) != 1:
        raise ValueError("logits must be fp32 with unit column stride")
    if params.dtype != torch.uint8 or params.numel() != PARAMS_BYTES * rows:
        raise ValueError("params must be rows x 24 bytes (uint8)")
    if out is None:
        out = allocate_sample_output(rows, max_logprobs, logits.device)
    if workspace is None:
        workspace = allocate_workspace(rows, vocab, max_logprobs, logits.device)
    _check(lib.sampler_sample(
        _ptr(logits), rows, vocab, logits.stride(0), _ptr(params), row_offset, max_logprobs,
        _ptr(out.token_ids), _ptr(out.token_logprobs),
        _ptr(out.topn_ids) if max_logprobs > 0 else None,
        _ptr(out.topn_logprobs) if max_logprobs > 0 else None,
        _ptr(out.row_status), _ptr(workspace), workspace.numel(), _stream_ptr(stream)))
    return out


def sampler_sample_noalloc(logits, params, row_offset: int = 0, max_logprobs: int = 0, out=None,
                           stream=None) -> SampleOutput:
    """``sampler_sample`` with the library's built-in scratch as the
    workspace (no workspace argument; nothing is allocated by the call
    itself, ``out`` aside when it is not given).  Calls that overlap on one
    GPU share the scratch and must be serialised."""
    torch = _torch()
    rows, vocab = logits.shape
    if logits.dtype != torch.float32 or logits.stride(1) != 1:
        raise ValueError("logits must be fp32 with unit column stride")
    if params.dtype != torch.uint8 or params.numel() != PARAMS_BYTES * rows:
        raise ValueError("params must be rows x 24 bytes (uint8)")
    if out is None:
        out = allocate_sample_output(rows, max_logprobs, logits.device)
    _check(lib.sampler_sample_noalloc(
        _ptr(logits), rows, vocab, logits.stride(0), _ptr(params), row_offset, max_logprobs,
        _ptr(out.token_ids), _ptr(out.token_logprobs),
        _ptr(out.topn_ids) if max_logprobs > 0 else None,
        _ptr(out.topn_logprobs) if max_logprobs > 0 else None,
        _ptr(out.row_status), _stream_ptr(stream)))
    return out


def _slice_arrays(slices):
    torch = _torch()
    n = len(slices)
    if n < 1 or n > TS_MAX_SLICES:
        raise ValueError(f"need 1..{TS_MAX_SLICES} slices")
    rows = slices[0].shape[0]
    for s in slices:
        if s.dtype != torch.float32 or s.dim() != 2 or s.shape[0] != rows or s.stride(1) != 1:
            raise ValueError("slices must be fp32 [rows, cols_s] with unit column stride")
    ptrs = (ctypes.c_void_p * n)(*[_ptr(s) for s in slices])
    cols = (ctypes.c_int64 * n)(*[int(s.shape[1]) for s in slices])
    lds = (ctypes.c_int64 * n)(*[max(int(s.stride(0)), int(s.shape[1])) for s in slices])
    return n, rows, ptrs, cols, lds


def sampler_workspace_bytes_slices(rows: int, slice_cols, max_logprobs: int) -> int:
    n = len(slice_cols)
    cols = (ctypes.c_int64 * max(n, 1))(*[int(c) for c in slice_cols])
    return int(lib.sampler_workspace_bytes_slices(rows, cols, n, max_logprobs))


def sampler_sample_slices(slices, params, row_offset: int = 0, max_logprobs: int = 0, out=None,
                          workspace=None, stream=None, processed: bool = False) -> SampleOutput:
    """``sampler_sample`` over the column-wise concatenation of ``slices``
    (fp32 ``[rows, cols_s]`` each), read in place.  Token ids are global
    columns of that concatenation."""
    torch = _torch()
    n, rows, ptrs, cols, lds = _slice_arrays(slices)
    if params.dtype != torch.uint8 or params.numel() != PARAMS_BYTES * rows:
        raise ValueError("params must be rows x 24 bytes (uint8)")
    device = slices[0].device
    if out is None:
        out = allocate_sample_output(rows, max_logprobs, device)
    if workspace is None:
        nb = max(256, sampler_workspace_bytes_slices(rows, list(cols), max_logprobs))
        workspace = torch.empty(nb, dtype=torch.uint8, device=device)
    head = (ptrs, cols, lds, n, rows, _ptr(params), row_offset, max_logprobs)
    call = (lambda *t: lib.sampler_sample_ex(*head, TS_LOGPROBS_PROCESSED, *t)) if processed \
        else (lambda *t: lib.sampler_sample_slices(*head, *t))
    _check(call(
        _ptr(out.token_ids), _ptr(out.token_logprobs),
        _ptr(out.topn_ids) if max_logprobs > 0 else None,
        _ptr(out.topn_logprobs) if max_logprobs > 0 else None,
        _ptr(out.row_status), _ptr(workspace), workspace.numel(), _stream_ptr(stream)))
    return out


def sampler_assemble_and_sample(slices, params, row_offset: int = 0, max_logprobs: int = 0,
                                assembled=None, out=None, workspace=None, stream=None,
                                processed: bool = False):
    """``sampler_assemble_vocab_slices`` into ``assembled`` and
    ``sampler_sample_slices`` of the same slices in one call, which reads the
    logits once.  Returns ``(assembled, SampleOutput)``."""
    torch = _torch()
    n, rows, ptrs, cols, lds = _slice_arrays(slices)
    total = sum(int(c) for c in cols)
    if params.dtype != torch.uint8 or params.numel() != PARAMS_BYTES * rows:
        raise ValueError("params must be rows x 24 bytes (uint8)")
    device = slices[0].device
    if assembled is None:
        assembled = torch.empty(rows, total, dtype=torch.float32, device=device)
    if assembled.shape != (rows, total) or assembled.stride(1) != 1 or \
            assembled.dtype != torch.float32:
        raise ValueError("assembled must be fp32 [rows, sum cols] with unit column stride")
    if out is None:
        out = allocate_sample_output(rows, max_logprobs, device)
    if workspace is None:
        nb = max(256, sampler_workspace_bytes_slices(rows, list(cols), max_logprobs))
        workspace = torch.empty(nb, dtype=torch.uint8, device=device)
    _check(lib.sampler_assemble_and_sample(
        ptrs, cols, lds, n, rows, _ptr(assembled), assembled.stride(0), _ptr(params), row_offset,
        max_logprobs, TS_LOGPROBS_PROCESSED if processed else 0,
        _ptr(out.token_ids), _ptr(out.token_logprobs),
        _ptr(out.topn_ids) if max_logprobs > 0 else None,
        _ptr(out.topn_logprobs) if max_logprobs > 0 else None,
        _ptr(out.row_status), _ptr(workspace), workspace.numel(), _stream_ptr(stream)))
    return assembled, out


# ------------------------------------------------------- scoring and losses
class _PolicyParams(ctypes.Structure):
    _fields_ = [("temperature", _F64), ("clip_low", _F64), ("clip_high", _F64),
                ("kl_coef", _F64)]


class _PreferenceParams(ctypes.Structure):
    _fields_ = [("temperature", _F64), ("beta", _F64), ("label_smoothing", _F64),
                ("margin", _F64), ("flags", _I32)]


@dataclass
class TokenLogprobs:
    logprobs: object    # fp32 [rows]
    entropies: object   # fp32 [rows], or None if not asked for
    row_stats: object   # fp32 [rows, 2], for token_logprobs_backward
    row_status: object  # int32 [rows]


@dataclass
class TokenLogprobsTopn:
    logprobs: object       # fp32 [rows], or None without tokens
    ranks: object          # int32 [rows], or None without tokens
    entropies: object      # fp32 [rows], or None if not asked for
    topn_ids: object       # int32 [rows, max_logprobs]
    topn_logprobs: object  # fp32 [rows, max_logprobs]
    row_stats: object      # fp32 [rows, 2], for the backward passes
    row_status: object     # int32 [rows]


@dataclass
class PolicyLoss:
    loss: object         # fp32 scalar
    logprobs: object     # fp32 [rows]
    ratios: object       # fp32 [rows]
    kl: object           # fp32 [rows]
    row_status: object   # int32 [rows]
    grad_logits: object  # the logits' type [rows, vocab], or None


@dataclass
class PreferenceLoss:
    loss: object         # fp32 scalar
    pair_losses: object  # fp32 [n_pairs]
    rewards: object      # fp32 [2 n_pairs]: chosen, then rejected
    logprobs: object     # fp32 [rows]
    row_status: object   # int32 [rows]
    grad_logits: object  # the logits' type [rows, vocab], or None


def _public_current_device():
    return torch.cuda.current_device()


def _public_current_stream(index):
    return torch.cuda.current_stream(index).cuda_stream


# torch's own short ways to the two, where it has them (1 us less a call).
_current_device = getattr(torch._C, "_cuda_getDevice", _public_current_device)
_current_stream = getattr(torch._C, "_cuda_getCurrentRawStream", _public_current_stream)


class _OnDevice:
    """Makes the device of a call's tensors and its stream current, so that
    outputs and workspaces are allocated for that stream.  Where they are
    already, which is the usual call, nothing is switched (switching takes
    longer than a small kernel)."""

    __slots__ = ("pointer", "_guard")

    def __init__(self, device, stream):
        index = device.index
        if index is None:
            raise ValueError("tensors must be on the GPU")
        self._guard = None
        if stream is None:
            if index != _current_device():
                self._guard = torch.cuda.device(device)
            self.pointer = _current_stream(index)
            return
        if not hasattr(stream, "cuda_stream"):
            stream = torch.cuda.ExternalStream(int(stream), device=device)
        elif stream.device != device:
            raise ValueError("the stream belongs to another device than the tensors")
        self.pointer = int(stream.cuda_stream)
        self._guard = torch.cuda.stream(stream)

    def __enter__(self):
        if self._guard is not None:
            self._guard.__enter__()
        return self.pointer

    def __exit__(self, *exc):
        if self._guard is not None:
            self._guard.__exit__(*exc)


_LOGITS_TYPES = {torch.float32: TS_F32, torch.bfloat16: TS_BF16}


def _check_vector(t, name, n, device, dtype=torch.float32):
    if t is None:
        return
    if t.dtype is not dtype or t.numel() != n or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of {n} values")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, the logits on {device}")


def _token_rows(logits, token_ids, each: int = 1):
    """Checks logits and token ids (`each` a row); returns (type code, leading
    dimension)."""
    kind = _LOGITS_TYPES.get(logits.dtype)
    shape = logits.shape
    if len(shape) != 2 or kind is None:
        raise ValueError("logits must be fp32 or bf16 [rows, vocab]")
    rows, vocab = shape
    ld, step = logits.stride()
    if vocab > 1 and step != 1:
        raise ValueError("logits must have unit column stride")
    if rows > 1 and ld < vocab:
        raise ValueError("logits rows overlap")
    _check_vector(token_ids, "token_ids", rows * each, logits.device, torch.int32)
    return kind, max(ld, vocab)


def _grad_rows(grad_logits, logits):
    if grad_logits.shape != logits.shape or grad_logits.dtype != logits.dtype or \
            grad_logits.device != logits.device:
        raise ValueError("grad_logits must have the shape, type and device of logits")
    (rows, vocab), stride = grad_logits.shape, grad_logits.stride()
    if vocab > 1 and stride[1] != 1:
        raise ValueError("grad_logits must have unit column stride")
    if rows > 1 and stride[0] < vocab:
        raise ValueError("grad_logits rows overlap")
    return max(stride[0], vocab)


def _gradient(grad_logits, wanted, logits):
    """The buffer of the logits' gradient (checked, or a new one if wanted)
    and its leading dimension."""
    if grad_logits is not None:
        return grad_logits, _grad_rows(grad_logits, logits)
    if not wanted:
        return None, 0
    rows, vocab = logits.shape
    return torch.empty(rows, vocab, dtype=logits.dtype, device=logits.device), vocab


def _workspace(workspace, need, device):
    if workspace is None:
        return torch.empty(max(256, need), dtype=torch.uint8, device=device)
    if workspace.dtype != torch.uint8 or not workspace.is_contiguous() or \
            workspace.device != device:
        raise ValueError("workspace must be a contiguous uint8 tensor on the logits' device")
    return workspace


def _outputs(sizes, device):
    """fp32 tensors of these sizes, and the first one's address.  One allocation
    holds them side by side, which takes less time than one each.  They are no
    views (this split makes none) and each has a version of its own, so that one
    can be changed in place while a graph holds another."""
    base = torch.empty(sum(sizes), dtype=torch.float32, device=device)
    return base.unsafe_split_with_sizes(sizes), base.data_ptr()


def token_logprobs_workspace_bytes(rows: int, vocab: int) -> int:
    return int(lib.token_logprobs_workspace_bytes(rows, vocab))


def preference_loss_workspace_bytes(rows: int, vocab: int, n_pairs: int) -> int:
    return int(lib.preference_loss_workspace_bytes(rows, vocab, n_pairs))


def token_logprobs(logits, token_ids, temperature: float = 1.0, entropies: bool = False,
                   workspace=None, stream=None) -> TokenLogprobs:
    """Log-probability of ``token_ids[r]`` (int32; negative: row left out)
    under ``softmax(logits[r] / temperature)``, fp32 or bf16 ``logits [rows,
    vocab]``, and with ``entropies`` that distribution's entropy.  The outputs
    share one allocation."""
    kind, ld = _token_rows(logits, token_ids)
    rows, vocab = logits.shape
    dev = logits.device
    with _OnDevice(dev, stream) as s:
        workspace = _workspace(workspace, token_logprobs_workspace_bytes(rows, vocab), dev)
        (stats, logprobs, status, h), at = _outputs(
            (2 * rows, rows, rows, rows if entropies else 0), dev)
        out = TokenLogprobs(logprobs, h if entropies else None, stats.view(rows, 2).data,
                            status.view(torch.int32).data)
        _check(lib.token_logprobs(
            logits.data_ptr(), kind, rows, vocab, ld, token_ids.data_ptr(), temperature,
            at + 8 * rows, at + 16 * rows if entropies else None, at, at + 12 * rows,
            workspace.data_ptr(), workspace.numel(), s))
    return out


def token_logprobs_backward(logits, token_ids, forward: TokenLogprobs, grad_logprobs,
                            grad_entropies=None, temperature: float = 1.0, grad_logits=None,
                            stream=None):
    """Gradient of the logits from ``grad_logprobs`` (fp32 ``[rows]``) and
    ``grad_entropies`` (or None), with the ``TokenLogprobs`` that
    ``token_logprobs`` gave for the same logits, tokens and temperature (calls
    ``token_logprobs_backward_ex`` with its log-probabilities where they are
    still as that call gave them).  ``grad_logits`` may be ``logits`` itself."""
    kind, ld = _token_rows(logits, token_ids)
    rows, vocab = logits.shape
    dev = logits.device
    _check_vector(grad_logprobs, "grad_logprobs", rows, dev)
    _check_vector(grad_entropies, "grad_entropies", rows, dev)
    _check_vector(forward.row_stats, "forward.row_stats", 2 * rows, dev)
    _check_vector(forward.entropies, "forward.entropies", rows, dev)
    logprobs = forward.logprobs
    if logprobs is not None and (logprobs.dtype is not torch.float32 or logprobs.device != dev or
                                 logprobs.numel() != rows or not logprobs.is_contiguous()):
        logprobs = None  # the caller has put something of its own there
    with _OnDevice(dev, stream) as s:
        grad_logits, ldg = _gradient(grad_logits, True, logits)
        _check(lib.token_logprobs_backward_ex(
            logits.data_ptr(), kind, rows, vocab, ld, token_ids.data_ptr(), temperature,
            _ptr(forward.row_stats), _ptr(logprobs), _ptr(grad_logprobs),
            _ptr(forward.entropies), _ptr(grad_entropies), grad_logits.data_ptr(), ldg, s))
    return grad_logits


def token_logprobs_topn_workspace_bytes(rows: int, vocab: int) -> int:
    return int(lib.token_logprobs_topn_workspace_bytes(rows, vocab))


def token_logprobs_listed_workspace_bytes(rows: int, vocab: int) -> int:
    return int(lib.token_logprobs_listed_workspace_bytes(rows, vocab))


def token_logprobs_topn(logits, token_ids, max_logprobs: int, temperature: float = 1.0,
                        entropies: bool = False, workspace=None,
                        stream=None) -> TokenLogprobsTopn:
    """``token_logprobs`` with each token's rank (from 1, in the order of logit
    descending and id ascending) and the row's first ``max_logprobs`` tokens of
    that order with their log-probabilities.  ``token_ids`` None asks for the
    alternatives alone, of every row.  The outputs share one allocation."""
    kind, ld = _token_rows(logits, token_ids)
    rows, vocab = logits.shape
    n, dev = int(max_logprobs), logits.device
    if n < 0 or n > TS_MAX_LOGPROBS:
        raise ValueError(f"max_logprobs {n} outside 0..{TS_MAX_LOGPROBS}")
    asked = token_ids is not None
    given = rows if asked else 0
    with _OnDevice(dev, stream) as s:
        workspace = _workspace(workspace, token_logprobs_topn_workspace_bytes(rows, vocab), dev)
        (stats, logprobs, ranks, status, ids, top, h), at = _outputs(
            (2 * rows, given, given, rows, rows * n, rows * n, rows if entropies else 0), dev)
        out = TokenLogprobsTopn(
            logprobs if asked else None, ranks.view(torch.int32).data if asked else None,
            h if entropies else None,
            ids.view(torch.int32).view(rows, n).data, top.view(rows, n).data,
            stats.view(rows, 2).data, status.view(torch.int32).data)
        after = at + 4 * (2 * rows + 2 * given)
        _check(lib.token_logprobs_topn(
            logits.data_ptr(), kind, rows, vocab, ld, _ptr(token_ids), temperature, n,
            at + 8 * rows if given else None, at + 4 * (2 * rows + given) if given else None,
            after + 4 * (rows + 2 * rows * n) if entropies else None, after + 4 * rows,
            after + 4 * (rows + rows * n), at, after, workspace.data_ptr(), workspace.numel(), s))
    return out


def token_logprobs_listed(logits, listed_ids, temperature: float = 1.0, entropies: bool = False,
                          workspace=None, stream=None) -> TokenLogprobs:
    """Log-probabilities of ``listed_ids [rows, n]`` (int32; negative: unused
    place, all of a row negative: row left out) under ``softmax(logits[r] /
    temperature)``: a ``TokenLogprobs`` whose ``logprobs`` are ``[rows, n]``.  The
    outputs share one allocation."""
    n = _listed(logits, listed_ids)
    kind, ld = _token_rows(logits, listed_ids, n)
    rows, vocab = logits.shape
    dev = logits.device
    with _OnDevice(dev, stream) as s:
        workspace = _workspace(workspace, token_logprobs_listed_workspace_bytes(rows, vocab), dev)
        (stats, logprobs, status, h), at = _outputs(
            (2 * rows, rows * n, rows, rows if entropies else 0), dev)
        out = TokenLogprobs(logprobs.view(rows, n).data, h if entropies else None,
                            stats.view(rows, 2).data, status.view(torch.int32).data)
        after = at + 4 * (2 * rows + rows * n)
        _check(lib.token_logprobs_listed(
            logits.data_ptr(), kind, rows, vocab, ld, listed_ids.data_ptr(), n, temperature,
            at + 8 * rows, after + 4 * rows if entropies else None, at, after,
            workspace.data_ptr(), workspace.numel(), s))
    return out


def _listed(logits, listed_ids):
    if listed_ids.dim() != 2 or logits.dim() != 2 or listed_ids.shape[0] != logits.shape[0]:
        raise ValueError("listed_ids must be [rows, n] and logits [rows, vocab]")
    n = listed_ids.shape[1]
    if n < 1 or n > TS_MAX_LISTED:
        raise ValueError(f"{n} listed tokens a row, outside 1..{TS_MAX_LISTED}")
    return n


def token_logprobs_listed_backward(logits, listed_ids, forward: TokenLogprobs, grad_logprobs,
                                   grad_entropies=None, temperature: float = 1.0,
                                   grad_logits=None, stream=None):
    """Gradient of the logits from ``grad_logprobs`` (fp32 ``[rows, n]``) and
    ``grad_entropies`` (fp32 ``[rows]`` or None), with the ``TokenLogprobs`` that
    ``token_logprobs_listed`` gave for the same logits, ids and temperature.  For the
    alternatives ``top`` of ``token_logprobs_topn`` (``listed_ids`` its ``topn_ids``)
    that is ``TokenLogprobs(top.topn_logprobs, top.entropies, top.row_stats,
    top.row_status)``; ``top`` itself is refused, as its ``logprobs`` are the given
    tokens'.  ``grad_logits`` may be ``logits`` itself."""
    if isinstance(forward, TokenLogprobsTopn):
        raise ValueError("the logprobs of a TokenLogprobsTopn are the given tokens': pass "
                         "TokenLogprobs(topn_logprobs, entropies, row_stats, row_status)")
    n = _listed(logits, listed_ids)
    kind, ld = _token_rows(logits, listed_ids, n)
    rows, vocab = logits.shape
    dev = logits.device
    if grad_logprobs is None or forward.logprobs is None or forward.row_stats is None:
        raise ValueError("grad_logprobs and the forward pass's outputs are needed")
    _check_vector(grad_logprobs, "grad_logprobs", rows * n, dev)
    _check_vector(grad_entropies, "grad_entropies", rows, dev)
    _check_vector(forward.row_stats, "forward.row_stats", 2 * rows, dev)
    _check_vector(forward.logprobs, "forward.logprobs", rows * n, dev)
    _check_vector(forward.entropies, "forward.entropies", rows, dev)
    with _OnDevice(dev, stream) as s:
        grad_logits, ldg = _gradient(grad_logits, True, logits)
        _check(lib.token_logprobs_listed_backward(
            logits.data_ptr(), kind, rows, vocab, ld, listed_ids.data_ptr(), n, temperature,
            _ptr(forward.row_stats), _ptr(forward.logprobs), _ptr(grad_logprobs),
            _ptr(forward.entropies), _ptr(grad_entropies), grad_logits.data_ptr(), ldg, s))
    return grad_logits


def policy_loss(logits, token_ids, old_logprobs, advantages, ref_logprobs=None, weights=None, *,
                clip_low: float = 0.2, clip_high: float = 0.2, kl_coef: float = 0.0,
                temperature: float = 1.0, backward: bool = False, grad_loss=None,
                grad_logits=None, workspace=None, stream=None) -> PolicyLoss:
    """Clipped policy loss with a KL term over rows of ``logits`` (see
    ``policy_loss`` in top_sampling.h for the formula).  ``weights`` (fp32
    ``[rows]``) holds the average wanted; None sums the rows.  With
    ``backward``, or a ``grad_logits`` buffer (``logits`` itself is allowed),
    the same call writes ``grad_loss`` (a device scalar, None for 1) times
    the gradient of the logits.  The outputs but ``grad_logits`` share one
    allocation: clone a loss that is kept for long."""
    kind, ld = _token_rows(logits, token_ids)
    rows, vocab = logits.shape
    dev = logits.device
    _check_vector(old_logprobs, "old_logprobs", rows, dev)
    _check_vector(advantages, "advantages", rows, dev)
    _check_vector(ref_logprobs, "ref_logprobs", rows, dev)
    _check_vector(weights, "weights", rows, dev)
    _check_vector(grad_loss, "grad_loss", 1, dev)
    with _OnDevice(dev, stream) as s:
        workspace = _workspace(workspace, token_logprobs_workspace_bytes(rows, vocab), dev)
        grad_logits, ldg = _gradient(grad_logits, backward, logits)
        (loss, logprobs, ratios, kl, status), at = _outputs((1, rows, rows, rows, rows), dev)
        out = PolicyLoss(loss.view(()).data, logprobs, ratios, kl,
                         status.view(torch.int32).data, grad_logits)
        params = _PolicyParams(temperature, clip_low, clip_high, kl_coef)
        _check(lib.policy_loss(
            logits.data_ptr(), kind, rows, vocab, ld, token_ids.data_ptr(),
            ctypes.addressof(params), _ptr(old_logprobs), _ptr(ref_logprobs), _ptr(advantages),
            _ptr(weights), _ptr(grad_loss), at, at + 4, at + 4 * (1 + rows),
            at + 4 * (1 + 2 * rows), at + 4 * (1 + 3 * rows), _ptr(grad_logits), ldg,
            workspace.data_ptr(), workspace.numel(), s))
    return out


def preference_loss(logits, token_ids, seq_offsets, ref_logprobs=None, pair_weights=None, *,
                    beta: float = 0.1, label_smoothing: float = 0.0, margin: float = 0.0,
                    mean: bool = False, temperature: float = 1.0, backward: bool = False,
                    grad_loss=None, grad_logits=None, workspace=None,
                    stream=None) -> PreferenceLoss:
    """Loss of paired log ratios (see ``preference_loss`` in top_sampling.h).
    ``seq_offsets`` (int32 ``[2 n_pairs + 1]``) bounds the sequences, chosen
    answers first, then the rejected ones in the same order.  ``mean`` divides
    each sequence's sum by its tokens.  ``backward``, ``grad_loss``,
    ``grad_logits`` and the outputs' memory as in ``policy_loss``."""
    kind, ld = _token_rows(logits, token_ids)
    rows, vocab = logits.shape
    dev = logits.device
    if seq_offsets.numel() % 2 != 1:
        raise ValueError("seq_offsets must hold 2 n_pairs + 1 values")
    n_pairs = seq_offsets.numel() // 2
    _check_vector(seq_offsets, "seq_offsets", 2 * n_pairs + 1, dev, torch.int32)
    _check_vector(ref_logprobs, "ref_logprobs", rows, dev)
    _check_vector(pair_weights, "pair_weights", n_pairs, dev)
    _check_vector(grad_loss, "grad_loss", 1, dev)
    with _OnDevice(dev, stream) as s:
        workspace = _workspace(workspace, preference_loss_workspace_bytes(rows, vocab, n_pairs),
                               dev)
        grad_logits, ldg = _gradient(grad_logits, backward, logits)
        (loss, pair_losses, rewards, logprobs, status), at = _outputs(
            (1, n_pairs, 2 * n_pairs, rows, rows), dev)
        out = PreferenceLoss(loss.view(()).data, pair_losses, rewards, logprobs,
                             status.view(torch.int32).data, grad_logits)
        params = _PreferenceParams(temperature, beta, label_smoothing, margin,
                                   TS_PREFERENCE_MEAN if mean else 0)
        _check(lib.preference_loss(
            logits.data_ptr(), kind, rows, vocab, ld, token_ids.data_ptr(),
            seq_offsets.data_ptr(), n_pairs, ctypes.addressof(params), _ptr(ref_logprobs),
            _ptr(pair_weights), _ptr(grad_loss), at, at + 4, at + 4 * (1 + n_pairs),
            at + 4 * (1 + 3 * n_pairs), at + 4 * (1 + 3 * n_pairs + rows), _ptr(grad_logits),
            ldg, workspace.data_ptr(), workspace.numel(), s))
    return out


# ------------------------------------------------------ projection with adapters
def lmhead_lora_workspace_bytes(rows: int, rank: int) -> int:
    return int(lib.lmhead_lora_workspace_bytes(rows, rank))


def lmhead_logits_local_lora(hidden, lm_head, lora_a, lora_b, adapter_ids, adapter_scales=None,
                             out=None, workspace=None, stream=None):
    """``lmhead_logits_local`` with a low-rank adapter per row: fp32 ``[rows,
    V_local]`` = hidden @ lm_head^T + scale (hidden @ A^T) @ B^T with the
    row's own ``A = lora_a[id]``, ``B = lora_b[id]`` (bf16 ``[n, rank, H]`` and
    ``[n, V_local, rank]``, inner stride 1) and ``adapter_scales[id]`` (fp32,
    None for 1); id -1 has no adapter."""
    shapes = hidden.shape, lm_head.shape, lora_a.shape, lora_b.shape
    if tuple(map(len, shapes)) != (2, 2, 3, 3):
        raise ValueError("hidden and lm_head must be 2-D, lora_a and lora_b 3-D")
    (rows, h), (vocab, h_w), (n, rank, h_a), shape_b = shapes
    if h_w != h or h_a != h or shape_b != (n, vocab, rank):
        raise ValueError("sizes do not fit: hidden [rows, H], lm_head [V, H], lora_a [n, rank, H], "
                         "lora_b [n, V, rank]")
    dev = hidden.device
    ld = []
    for t, name in ((hidden, "hidden"), (lm_head, "lm_head"), (lora_a, "lora_a"),
                    (lora_b, "lora_b")):
        if t.dtype != torch.bfloat16:
            raise TypeError(f"{name} must be bfloat16")
        stride, (count, width) = t.stride(), t.shape[-2:]
        if width > 1 and stride[-1] != 1:
            raise ValueError(f"{name} must have unit inner stride")
        if t.device != dev:
            raise ValueError(f"{name} is on {t.device}, hidden on {dev}")
        ld.append(stride[-2] if count > 1 else width)
    ld_hidden, ld_lm_head, ld_a, ld_b = ld
    stride_a, stride_b = (lora_a.stride(0), lora_b.stride(0)) if n > 1 else (0, 0)
    _check_vector(adapter_ids, "adapter_ids", rows, dev, torch.int32)
    _check_vector(adapter_scales, "adapter_scales", n, dev)
    with _OnDevice(dev, stream) as s:
        if out is None:
            out = torch.empty(rows, vocab, dtype=torch.float32, device=dev)
        if out.shape != (rows, vocab) or out.dtype != torch.float32 or out.device != dev or \
                (vocab > 1 and out.stride(1) != 1):
            raise ValueError("out must be fp32 [rows, V_local] with unit column stride")
        workspace = _workspace(workspace, lmhead_lora_workspace_bytes(rows, rank), dev)
        _check(lib.lmhead_logits_local_lora(
            hidden.data_ptr(), rows, h, ld_hidden, lm_head.data_ptr(), vocab, ld_lm_head,
            lora_a.data_ptr(), stride_a, ld_a, lora_b.data_ptr(), stride_b, ld_b, n, rank,
            _ptr(adapter_scales), _ptr(adapter_ids), out.data_ptr(),
            out.stride(0) if rows > 1 else vocab, workspace.data_ptr(), workspace.numel(), s))
    return out


# ------------------------------------------------------ 4-bit rows and projection
E2M1_GROUP = 32


def _group_rows(t, name, dtype, rows, width, device):
    """Checks a matrix of a 4-bit call; returns its leading dimension."""
    if t.dtype is not dtype or t.shape != (rows, width):
        raise ValueError(f"{name} must be {dtype} [{rows}, {width}]")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, not on {device}")
    ld, step = t.stride()
    if width > 1 and step != 1:
        raise ValueError(f"{name} must have unit column stride")
    if rows > 1 and ld < width:
        raise ValueError(f"{name} rows overlap")
    return max(ld, width) if rows > 1 else width


def _group_out(t, name, dtype, rows, width, device):
    """An output (checked, or a new one) and its leading dimension."""
    if t is None:
        return torch.empty(rows, width, dtype=dtype, device=device), width
    return t, _group_rows(t, name, dtype, rows, width, device)


def _values_type(dtype):
    kind = _LOGITS_TYPES.get(dtype)
    if kind is None:
        raise ValueError("values must be fp32 or bf16")
    return kind


def quantize_groups_e2m1(x, codes=None, scales=None, stream=None):
    """fp32 or bf16 ``x [rows, cols]`` (cols a multiple of 32) as OCP MX FP4:
    uint8 codes ``[rows, cols / 2]`` (two a byte, the even column's in the low
    half) and a scale byte for every 32 columns, ``[rows, cols / 32]`` (see
    ``quantize_groups_e2m1`` in top_sampling.h)."""
    if x.dim() != 2:
        raise ValueError("x must be [rows, cols]")
    kind, dev = _values_type(x.dtype), x.device
    rows, cols = x.shape
    if cols % E2M1_GROUP:
        raise ValueError(f"cols {cols} is no multiple of {E2M1_GROUP}")
    ld_x = _group_rows(x, "x", x.dtype, rows, cols, dev)
    with _OnDevice(dev, stream) as s:
        codes, ld_codes = _group_out(codes, "codes", torch.uint8, rows, cols // 2, dev)
        scales, ld_scales = _group_out(scales, "scales", torch.uint8, rows, cols // E2M1_GROUP,
                                       dev)
        _check(lib.quantize_groups_e2m1(x.data_ptr(), kind, rows, cols, ld_x, codes.data_ptr(),
                                        ld_codes, scales.data_ptr(), ld_scales, s))
    return codes, scales


def dequantize_groups_e2m1(codes, scales, dtype=torch.bfloat16, out=None, stream=None):
    """The values that 4-bit ``codes [rows, cols / 2]`` and their ``scales
    [rows, cols / 32]`` stand for, in ``dtype`` (fp32 or bf16, both exact)."""
    if codes.dim() != 2:
        raise ValueError("codes must be [rows, cols / 2]")
    dev = codes.device
    rows, cols = codes.shape[0], 2 * codes.shape[1]
    if cols % E2M1_GROUP:
        raise ValueError(f"cols {cols} is no multiple of {E2M1_GROUP}")
    ld_codes = _group_rows(codes, "codes", torch.uint8, rows, cols // 2, dev)
    ld_scales = _group_rows(scales, "scales", torch.uint8, rows, cols // E2M1_GROUP, dev)
    kind = _values_type(dtype if out is None else out.dtype)
    with _OnDevice(dev, stream) as s:
        out, ld_out = _group_out(out, "out", dtype if out is None else out.dtype, rows, cols, dev)
        _check(lib.dequantize_groups_e2m1(codes.data_ptr(), rows, cols, ld_codes,
                                          scales.data_ptr(), ld_scales, out.data_ptr(), kind,
                                          ld_out, s))
    return out


def lmhead_logits_local_e2m1(hidden, lm_head, lm_head_scales, out=None, stream=None):
    """``lmhead_logits_local`` with a 4-bit lm_head: fp32 ``[rows, V_local]`` of
    bf16 ``hidden [rows, H]`` against the codes ``lm_head [V_local, H / 2]`` and
    their ``lm_head_scales [V_local, H / 32]`` (uint8, from
    ``quantize_groups_e2m1``).  ``out`` may be columns of a wider buffer."""
    if hidden.dim() != 2 or lm_head.dim() != 2:
        raise ValueError("hidden and lm_head must be 2-D")
    dev = hidden.device
    rows, h = hidden.shape
    vocab = lm_head.shape[0]
    if h % E2M1_GROUP:
        raise ValueError(f"hidden size {h} is no multiple of {E2M1_GROUP}")
    ld_hidden = _group_rows(hidden, "hidden", torch.bfloat16, rows, h, dev)
    ld_lm_head = _group_rows(lm_head, "lm_head", torch.uint8, vocab, h // 2, dev)
    ld_scales = _group_rows(lm_head_scales, "lm_head_scales", torch.uint8, vocab,
                            h // E2M1_GROUP, dev)
    with _OnDevice(dev, stream) as s:
        out, ld_out = _group_out(out, "out", torch.float32, rows, vocab, dev)
        _check(lib.lmhead_logits_local_e2m1(
            hidden.data_ptr(), rows, h, ld_hidden, lm_head.data_ptr(), lm_head_scales.data_ptr(),
            vocab, ld_lm_head, ld_scales, out.data_ptr(), ld_out, s))
    return out


def mfma_clock_probe(workgroups: int, iters: int, device, stream=None, random: bool = False):
    """Launch the matrix-core clock probe (a measurement aid) and return the
    device tensor of per-workgroup ticks [workgroups, 4] (uint64 stored as
    int64): shader clock start / end, 100 MHz real time start / end.
    ``random`` selects random operand bits instead of a few small values."""
    torch = _torch()
    ticks = torch.zeros(workgroups, 4, dtype=torch.int64, device=device)
    mode = TS_PROBE_RANDOM_OPERANDS if random else TS_PROBE_SMALL_OPERANDS
    _check(lib.ts_mfma_clock_probe(_ptr(ticks), workgroups, iters, mode, _stream_ptr(stream)))
    return ticks


def gumbel_keys(logits, row_max, temperature, seeds, rows, ids, stream=None):
    """The sampler's own fp32 Gumbel-max keys and Philox noise words for listed
    tokens (a check aid): all arguments are 1-D device tensors of one length
    (fp32 logits / row_max / temperature, int64 seeds (uint64 bits) and rows,
    int32 ids).  Returns (keys fp32, words int32 holding the uint32 bits)."""
    torch = _torch()
    n = int(ids.numel())
    keys = torch.empty(n, dtype=torch.float32, device=ids.device)
    words = torch.empty(n, dtype=torch.int32, device=ids.device)
    _check(lib.ts_gumbel_keys(_ptr(logits), _ptr(row_max), _ptr(temperature), _ptr(seeds),
                              _ptr(rows), _ptr(ids), n, _ptr(keys), _ptr(words),
                              _stream_ptr(stream)))
    return keys, words

"""Python binding of libetg: the static embedding / tied lm_head service on MI355X.

Argument marshalling only.  Every step of the path runs in the HIP kernels of
``libetg.so`` (built in-tree by ``embedding_table_gather_amd/build.py``);
PyTorch supplies device memory and the current stream.  There is no CPU
fallback: if the library is missing, every call raises.

    t = Table(rows, BF16, vocab, hidden)          # rows: device tensor, borrowed
    x = t.embed_gather(ids)                       # ADR-0008 "POST /v1/embed"
    ids, scores = t.logits_topk(residual, k=10)   # ADR-0008 "POST /v1/logits"
    ids, scores, probs = t.logits_topk_probs(residual, k=10, temperature=1.0)
    logits = t.logits_raw(residual)               # raw logits mode, [B, vocab]
    rows = t.embed_gather_wire(ids, WIRE_I8)      # ADR-0009 wire rows (f16 or i8)
    ids, scores = t.logits_topk_wire(rows, WIRE_I8, k=10)
    ids, probs = t.sample(residual, uniform, temperature=0.8, top_p=0.95)   # next tokens
    q = t.quantize_i8()                           # int8 rows, a scale each: an I8Table
    logits = q.logits_raw(residual)               # int8 product, f32 [B, vocab]
    ids, probs = sample(logits, uniform, top_k=50, min_p=0.05)
    loss, lse = t.cross_entropy(residual, labels)              # training and evaluation
    dx, dt = t.cross_entropy_grad(residual, labels, lse, 1 / count)
    t.embed_gather_grad(dx0, ids, scale="sqrt_d", out=dt, accumulate=True)   # the tied table's gradient
"""
from __future__ import annotations

import ctypes
import os
import warnings

import torch

F32, BF16, Q8_0, F16 = 0, 1, 2, 3
WIRE_F32, WIRE_F16, WIRE_I8 = 0, 1, 2
PATH_AUTO, PATH_VALU, PATH_STREAM, PATH_GEMM, PATH_WIDE, PATH_Q8, PATH_ROW, PATH_RANK = 0, 1, 2, 3, 4, 5, 6, 7

# ETG_LIBRARY names another build of the same library (e.g. one whose host code
# carries sanitizers); by default the in-tree libetg.so
LIB_PATH = os.environ.get("ETG_LIBRARY") or os.path.join(os.path.dirname(os.path.abspath(__file__)), "libetg.so")

_STATUS = {
    0: "ETG_OK", -1: "ETG_EINVAL", -2: "ETG_EDTYPE", -3: "ETG_ESHAPE", -4: "ETG_EALIGN",
    -5: "ETG_ERANGE", -6: "ETG_EWORKSPACE", -8: "ETG_EHIP",
}

# Functions declared in include/etg.h, with their ctypes signatures.
_I32, _I64, _VP, _F = ctypes.c_int32, ctypes.c_int64, ctypes.c_void_p, ctypes.c_float
SIGNATURES = {
    "etg_version": (_I32, []),
    "etg_row_bytes": (_I64, [_I32, _I64]),
    "etg_sqrt_d": (_F, [_I64]),
    "etg_table_create": (_I32, [_VP, _I32, _I64, _I64, ctypes.POINTER(_VP)]),
    "etg_table_destroy": (_I32, [_VP]),
    "etg_embed_gather": (_I32, [_VP, _VP, _I64, _F, _VP, _VP, _VP]),
    "etg_logits_topk_workspace": (_I64, [_VP, _I64, _I32]),
    "etg_logits_topk_workspace_ex": (_I64, [_VP, _I64, _I32, _I32]),
    "etg_logits_topk": (_I32, [_VP, _VP, _I64, _I32, _VP, _VP, _VP, ctypes.c_size_t, _VP]),
    "etg_logits_topk_ex": (_I32, [_VP, _VP, _I64, _I32, _VP, _VP, _VP, ctypes.c_size_t, _I32, _VP]),
    "etg_logits_topk_profiled": (_I32, [_VP, _VP, _I64, _I32, _VP, _VP, _VP, ctypes.c_size_t, _I32, _VP, _VP,
                                        _VP]),
    "etg_logits_topk_probs": (_I32, [_VP, _VP, _I64, _I32, _F, _VP, _VP, _VP, _VP, ctypes.c_size_t, _I32, _VP]),
    "etg_logits_raw_workspace": (_I64, [_VP, _I64, _I32]),
    "etg_logits_raw": (_I32, [_VP, _VP, _I64, _VP, _VP, ctypes.c_size_t, _I32, _VP]),
    "etg_wire_row_bytes": (_I64, [_I32, _I64]),
    "etg_embed_gather_wire": (_I32, [_VP, _VP, _I64, _F, _I32, _VP, _VP, _VP]),
    "etg_logits_topk_wire": (_I32, [_VP, _VP, _I32, _I64, _I32, _VP, _VP, _VP, ctypes.c_size_t, _I32, _VP]),
    "etg_logits_topk_to_host": (_I32, [_VP, _VP, _I64, _I32, _VP, _VP, _VP, ctypes.c_size_t, _I32, _VP, _VP, _VP,
                                       _VP]),
    "etg_hbm_read_probe": (_I32, [_VP, _I64, _VP, _VP]),
    "etg_hbm_write_probe": (_I32, [_VP, _I64, ctypes.c_uint32, _VP]),
    "etg_logits_topk_noalloc": (_I32, [_VP, _VP, _I64, _I32, _VP, _VP, _VP]),
    "etg_step_cache_ids_capacity": (_I64, [_I64]),
    "etg_step_cache_workspace": (_I64, [_VP, _I64, _I32]),
    "etg_step_cache_create": (_I32, [_VP, _I64, _I64, _I32, _I32, _VP, _VP, _VP, _VP, _VP, _VP, ctypes.c_size_t, _VP,
                                     _VP, _VP, ctypes.POINTER(_VP)]),
    "etg_step_cache_destroy": (_I32, [_VP]),
    "etg_step_cache_stats": (_I32, [_VP, ctypes.POINTER(_I64), ctypes.POINTER(_I64)]),
    "etg_step_gather": (_I32, [_VP, _VP, _I64, _F, _VP]),
    "etg_step_logits": (_I32, [_VP, _I64, _VP, _VP]),
    "etg_quantize_i8": (_I32, [_VP, _I32, _I64, _I64, _I64, _VP, _I64, _VP, _I64, _VP]),
    "etg_matmul_i8_workspace": (_I64, [_I64, _I64, _I64]),
    "etg_matmul_i8": (_I32, [_VP, _I64, _VP, _I64, _VP, _I64, _VP, _I64, _I64, _I64, _I64, _VP, _I32, _I64, _VP,
                             ctypes.c_size_t, _VP]),
    "etg_logits_i8_workspace": (_I64, [_I64, _I64, _I64]),
    "etg_logits_i8": (_I32, [_VP, _I64, _VP, _I64, _I64, _I64, _VP, _I32, _I64, _I64, _VP, _I32, _I64, _VP,
                             ctypes.c_size_t, _VP]),
    "etg_sample_workspace": (_I64, [_I64, _I64]),
    "etg_sample": (_I32, [_VP, _I32, _I64, _I64, _I64, _VP, _VP, _VP, _VP, _VP, ctypes.c_size_t, _VP]),
    "etg_cross_entropy_workspace": (_I64, [_VP, _I64]),
    "etg_cross_entropy": (_I32, [_VP, _VP, _I64, _I64, _VP, _VP, _VP, _VP, ctypes.c_size_t, _VP]),
    "etg_cross_entropy_grad_workspace": (_I64, [_VP, _I64]),
    "etg_cross_entropy_grad": (_I32, [_VP, _VP, _I64, _I64, _VP, _VP, _F, _VP, _VP, _VP, _I64, _VP, _I32, _VP,
                                      ctypes.c_size_t, _VP]),
    "etg_embed_gather_grad_workspace": (_I64, [_VP, _I64]),
    "etg_embed_gather_grad": (_I32, [_VP, _VP, _I64, _VP, _I32, _I64, _F, _VP, _I32, _I32, _VP, ctypes.c_size_t, _VP]),
    "etg_last_error": (ctypes.c_char_p, []),
}

_lib = None


class EtgError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"{_STATUS.get(status, status)}: {message}")
        self.status = status


def lib() -> ctypes.CDLL:
    """Load libetg.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with embedding_table_gather_amd/build.py "
                               "(there is no fallback path)")
        L = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in SIGNATURES.items():
            fn = getattr(L, name)
            fn.restype = res
            fn.argtypes = args
        _lib = L
    return _lib


def _check(status: int) -> None:
    if status != 0:
        raise EtgError(status, lib().etg_last_error().decode())


def row_bytes(dtype: int, hidden: int) -> int:
    return int(lib().etg_row_bytes(int(dtype), int(hidden)))


def sqrt_d(hidden: int) -> float:
    return float(lib().etg_sqrt_d(int(hidden)))


def _stream_ptr(device: torch.device):
    return ctypes.c_void_p(torch.cuda.current_stream(device).cuda_stream)


def _ptr(t: torch.Tensor):
    return ctypes.c_void_p(t.data_ptr())


def _event_handle(ev, device: torch.device) -> int:
    """The hipEvent_t behind a torch event (created on first record), or a raw
    hipEvent_t handle passed as an int."""
    if isinstance(ev, int):
        return ev
    if ev.cuda_event == 0:
        ev.record(torch.cuda.current_stream(device))
    return ev.cuda_event


class Table:
    """A V x hidden table already in device memory (f32, bf16, f16 or Q8_0 rows).

    ``rows`` is any contiguous CUDA tensor holding exactly vocab * row_bytes bytes
    (e.g. uint16 [V, d] bf16 or f16 bits, float32 [V, d], uint8 [V, 34 d / 32]).  It is
    borrowed: the handle keeps a reference but never copies it.
    """

    def __init__(self, rows: torch.Tensor, dtype: int, vocab: int, hidden: int):
        if not rows.is_cuda:
            raise ValueError("table rows must be a device tensor")
        if not rows.is_contiguous():
            raise ValueError("table rows must be contiguous")
        rb = row_bytes(dtype, hidden)
        if rb < 0:
            raise ValueError(f"hidden {hidden} cannot be stored as dtype {dtype}")
        nbytes = rows.numel() * rows.element_size()
        if nbytes != vocab * rb:
            raise ValueError(f"rows hold {nbytes} bytes, expected {vocab} * {rb}")
        self.rows, self.dtype, self.vocab, self.hidden, self.row_bytes = rows, int(dtype), int(vocab), int(hidden), rb
        self.device = rows.device
        h = ctypes.c_void_p()
        _check(lib().etg_table_create(_ptr(rows), self.dtype, self.vocab, self.hidden, ctypes.byref(h)))
        self._h = h
        self._ws = {}

    def __del__(self):
        h = getattr(self, "_h", None)
        if h is not None and _lib is not None:
            _lib.etg_table_destroy(h)
            self._h = None

    @property
    def handle(self):
        return self._h

    # ------------------------------------------------------------------ gather
    def embed_gather(self, ids: torch.Tensor, scale=None, out: torch.Tensor | None = None,
                     bad_count: torch.Tensor | None = None, check: bool = True) -> torch.Tensor:
        """f32 [n, hidden] rows for int32 ids (ADR-0008 "POST /v1/embed").

        scale: None (no scale), "sqrt_d" (the f32 nearest sqrt(hidden)), or a number.
        check: count bad ids on the device, synchronize, and raise ValueError if
        any; with check=False nothing waits (bad rows are still zero-filled, and
        counted into ``bad_count`` if one is given).
        """
        if ids.dtype != torch.int32 or ids.device != self.device:
            raise ValueError("ids must be an int32 tensor on the table's device")
        ids = ids.contiguous().view(-1)
        n = ids.numel()
        sc = 1.0 if scale is None else (sqrt_d(self.hidden) if scale == "sqrt_d" else float(scale))
        if out is None:
            out = torch.empty((n, self.hidden), dtype=torch.float32, device=self.device)
        elif out.dtype != torch.float32 or not out.is_contiguous() or out.numel() != n * self.hidden:
            raise ValueError("out must be a contiguous float32 tensor of n * hidden values")
        if check and bad_count is None:
            bad_count = torch.zeros(1, dtype=torch.int32, device=self.device)
        bad_ptr = _ptr(bad_count) if bad_count is not None else None
        with torch.cuda.device(self.device):
            _check(lib().etg_embed_gather(self._h, _ptr(ids), n, sc, _ptr(out), bad_ptr,
                                          _stream_ptr(self.device)))
            if check:
                nbad = int(bad_count.item())
                if nbad:
                    raise ValueError(f"bad token id: {nbad} of {n} ids are not in [0, {self.vocab})")
        return out

    def embed_gather_wire(self, ids: torch.Tensor, wire: int, scale=None, out: torch.Tensor | None = None,
                          bad_count: torch.Tensor | None = None) -> torch.Tensor:
        """Rows encoded in a residual wire format: uint8 [n, wire_row_bytes(wire, hidden)]
        (ADR-0009: f16, or per-position [scale][zero point][int8 x hidden]).  No check
        of bad ids beyond counting them into ``bad_count`` if one is given."""
        if ids.dtype != torch.int32 or ids.device != self.device:
            raise ValueError("ids must be an int32 tensor on the table's device")
        ids = ids.contiguous().view(-1)
        n = ids.numel()
        rb = wire_row_bytes(wire, self.hidden)
        sc = 1.0 if scale is None else (sqrt_d(self.hidden) if scale == "sqrt_d" else float(scale))
        if out is None:
            out = torch.empty((n, rb), dtype=torch.uint8, device=self.device)
        elif out.numel() * out.element_size() != n * rb or not out.is_contiguous():
            raise ValueError("out must be a contiguous buffer of n * wire_row_bytes bytes")
        bad_ptr = _ptr(bad_count) if bad_count is not None else None
        with torch.cuda.device(self.device):
            _check(lib().etg_embed_gather_wire(self._h, _ptr(ids), n, sc, int(wire), _ptr(out), bad_ptr,
                                               _stream_ptr(self.device)))
        return out

    # ------------------------------------------------------------------ logits
    def workspace_bytes(self, batch: int, k: int, path: int = PATH_AUTO) -> int:
        n = int(lib().etg_logits_topk_workspace_ex(self._h, int(batch), int(k), int(path)))
        if n < 0:
            _check(n)
        return n

    def workspace(self, batch: int, k: int, path: int = PATH_AUTO) -> torch.Tensor:
        """A device workspace for this shape, cached per (shape, path, current stream).

        Calls on one stream run in order, so they can share a workspace; calls on
        different streams get different ones.  Threads that enqueue on the same
        stream concurrently must pass their own ``workspace``."""
        key = (int(batch), int(k), int(path), torch.cuda.current_stream(self.device).cuda_stream)
        ws = self._ws.get(key)
        if ws is None:
            ws = torch.empty(max(self.workspace_bytes(batch, k, path), 256), dtype=torch.uint8, device=self.device)
            self._ws[key] = ws
        return ws

    def logits_topk(self, residual: torch.Tensor, k: int, path: int = PATH_AUTO,
                    workspace: torch.Tensor | None = None, out_ids: torch.Tensor | None = None,
                    out_scores: torch.Tensor | None = None, events=None):
        """Top-k (ids int32 [B, k], logits f32 [B, k]) of residual @ table.T per row.

        events: optional (before, after) torch.cuda.Event pair, recorded around the
        kernel that streams the table (for timing that kernel alone).
        """
        if residual.dtype != torch.float32 or residual.device != self.device:
            raise ValueError("residual must be a float32 tensor on the table's device")
        R = residual.contiguous().view(-1, self.hidden)
        B = R.shape[0]
        if workspace is None:
            workspace = self.workspace(B, k, path)
        if out_ids is None:
            out_ids = torch.empty((B, k), dtype=torch.int32, device=self.device)
        if out_scores is None:
            out_scores = torch.empty((B, k), dtype=torch.float32, device=self.device)
        ev0 = ev1 = None
        if events is not None:
            ev0, ev1 = (ctypes.c_void_p(_event_handle(e, self.device)) for e in events)
        with torch.cuda.device(self.device):
            _check(lib().etg_logits_topk_profiled(self._h, _ptr(R), B, int(k), _ptr(out_ids), _ptr(out_scores),
                                                  _ptr(workspace), workspace.numel(), int(path), ev0, ev1,
                                                  _stream_ptr(self.device)))
        return out_ids, out_scores

    def logits_topk_noalloc(self, residual: torch.Tensor, k: int, out_ids: torch.Tensor,
                            out_scores: torch.Tensor):
        """logits_topk with the library's own device scratch as the workspace (for
        callers that cannot allocate): writes into the given int32 / float32 [B, k]
        device tensors and allocates nothing.  Calls that overlap on one GPU race."""
        R = self._residual(residual)
        B = R.shape[0]
        for o, dt in ((out_ids, torch.int32), (out_scores, torch.float32)):
            if o.dtype != dt or o.device != self.device or not o.is_contiguous() or o.numel() != B * k:
                raise ValueError("out_ids / out_scores must be contiguous int32 / float32 [B, k] device tensors")
        with torch.cuda.device(self.device):
            _check(lib().etg_logits_topk_noalloc(self._h, _ptr(R), B, int(k), _ptr(out_ids), _ptr(out_scores),
                                                 _stream_ptr(self.device)))
        return out_ids, out_scores

    def logits_topk_to_host(self, residual: torch.Tensor, k: int, path: int = PATH_AUTO,
                            workspace: torch.Tensor | None = None, host_out=None):
        """logits_topk whose answer is also copied, without a synchronisation, into
        page-locked host tensors (host_out: a reusable (int32, float32) pair of
        [B, k] pinned CPU tensors, else new ones).  Returns (host ids, host scores,
        event): the host tensors hold the answer once event.synchronize() (or a true
        event.query())."""
        R = self._residual(residual)
        B = R.shape[0]
        if workspace is None:
            workspace = self.workspace(B, k, path)
        ids = torch.empty((B, k), dtype=torch.int32, device=self.device)
        sc = torch.empty((B, k), dtype=torch.float32, device=self.device)
        if host_out is None:
            host_out = (torch.empty((B, k), dtype=torch.int32, pin_memory=True),
                        torch.empty((B, k), dtype=torch.float32, pin_memory=True))
        h_ids, h_sc = host_out
        if (h_ids.dtype != torch.int32 or h_sc.dtype != torch.float32 or h_ids.device.type != "cpu"
                or h_sc.device.type != "cpu" or h_ids.numel() < B * k or h_sc.numel() < B * k
                or not h_ids.is_contiguous() or not h_sc.is_contiguous()):
            raise ValueError("host_out must be contiguous CPU int32 / float32 tensors of at least B * k entries")
        ev = torch.cuda.Event()
        with torch.cuda.device(self.device):
            evh = ctypes.c_void_p(_event_handle(ev, self.device))
            _check(lib().etg_logits_topk_to_host(self._h, _ptr(R), B, int(k), _ptr(ids), _ptr(sc), _ptr(workspace),
                                                 workspace.numel(), int(path), _ptr(h_ids), _ptr(h_sc), evh,
                                                 _stream_ptr(self.device)))
        return h_ids, h_sc, ev

    def _residual(self, residual: torch.Tensor) -> torch.Tensor:
        if residual.dtype != torch.float32 or residual.device != self.device:
            raise ValueError("residual must be a float32 tensor on the table's device")
        return residual.contiguous().view(-1, self.hidden)

    def logits_topk_probs(self, residual: torch.Tensor, k: int, temperature: float = 1.0,
                          path: int = PATH_AUTO, workspace: torch.Tensor | None = None):
        """Top-k (ids int32 [B, k], logits f32 [B, k], probabilities f32 [B, k]); the
        probabilities are the softmax of logits / temperature over the whole vocabulary."""
        R = self._residual(residual)
        B = R.shape[0]
        if workspace is None:
            workspace = self.workspace(B, k, path)
        ids = torch.empty((B, k), dtype=torch.int32, device=self.device)
        scores = torch.empty((B, k), dtype=torch.float32, device=self.device)
        probs = torch.empty((B, k), dtype=torch.float32, device=self.device)
        with torch.cuda.device(self.device):
            _check(lib().etg_logits_topk_probs(self._h, _ptr(R), B, int(k), float(temperature), _ptr(ids),
                                               _ptr(scores), _ptr(probs), _ptr(workspace), workspace.numel(),
                                               int(path), _stream_ptr(self.device)))
        return ids, scores, probs

    def logits_topk_wire(self, residual: torch.Tensor, wire: int, k: int, path: int = PATH_AUTO,
                         workspace: torch.Tensor | None = None):
        """Top-k (ids, logits) of residual rows given in a wire format: a contiguous
        device buffer of batch * wire_row_bytes(wire, hidden) bytes."""
        rb = wire_row_bytes(wire, self.hidden)
        nbytes = residual.numel() * residual.element_size()
        if residual.device != self.device or not residual.is_contiguous() or nbytes % rb:
            raise ValueError("residual must be a contiguous device buffer of whole wire rows")
        B = nbytes // rb
        if workspace is None:
            workspace = self.workspace(B, k, path)
        ids = torch.empty((B, k), dtype=torch.int32, device=self.device)
        scores = torch.empty((B, k), dtype=torch.float32, device=self.device)
        with torch.cuda.device(self.device):
            _check(lib().etg_logits_topk_wire(self._h, _ptr(residual), int(wire), B, int(k), _ptr(ids), _ptr(scores),
                                              _ptr(workspace), workspace.numel(), int(path),
                                              _stream_ptr(self.device)))
        return ids, scores

    def logits_raw(self, residual: torch.Tensor, path: int = PATH_AUTO, out: torch.Tensor | None = None,
                   workspace: torch.Tensor | None = None) -> torch.Tensor:
        """Raw logits mode: f32 [B, vocab] = residual @ table.T."""
        R = self._residual(residual)
        B = R.shape[0]
        if workspace is None:
            n = int(lib().etg_logits_raw_workspace(self._h, B, int(path)))
            if n < 0:
                _check(n)
            workspace = torch.empty(max(n, 256), dtype=torch.uint8, device=self.device)
        if out is None:
            out = torch.empty((B, self.vocab), dtype=torch.float32, device=self.device)
        elif out.dtype != torch.float32 or out.device != self.device or out.shape != (B, self.vocab) \
                or not out.is_contiguous():
            raise ValueError("out must be a contiguous float32 [batch, vocab] tensor on the table's device")
        with torch.cuda.device(self.device):
            _check(lib().etg_logits_raw(self._h, _ptr(R), B, _ptr(out), _ptr(workspace), workspace.numel(),
                                        int(path), _stream_ptr(self.device)))
        return out

    def sample(self, residual: torch.Tensor, uniform: torch.Tensor, path: int = PATH_AUTO, **kw):
        """The next token of each residual row: ``sample`` of its raw logits (temperature,
        top_k, top_p, min_p, allowed as there)."""
        return sample(self.logits_raw(residual, path=path), uniform, **kw)

    def quantize_i8(self) -> "I8Table":
        """The table's rows as an int8 lm_head (f32, bf16 and f16 tables)."""
        if self.dtype not in _TORCH_FLOATS:
            raise ValueError("only f32, bf16 and f16 tables can be quantised to int8 rows")
        rows = self.rows.view(-1).view(torch.uint8).view(_TORCH_FLOATS[self.dtype]).view(self.vocab, self.hidden)
        return I8Table(*quantize_i8(rows))

    # ---------------------------------------------------------------- training
    def _float_type(self) -> torch.dtype:
        if self.dtype not in _TORCH_FLOATS:
            raise ValueError("a Q8_0 table has no gradients: the table must be f32, bf16 or f16")
        return _TORCH_FLOATS[self.dtype]

    def _train_rows(self, residual: torch.Tensor, labels: torch.Tensor):
        """(row stride, batch) of residual rows of the table's type with a label each, checked."""
        dtype = self._float_type()
        if residual.dtype != dtype:
            raise ValueError(f"residual must be a {dtype} tensor, the table's type")
        stride = _rows(residual, "residual", self.device)
        batch, hidden = residual.shape
        if hidden != self.hidden:
            raise ValueError(f"residual has {hidden} columns, the table {self.hidden}")
        if labels.dtype != torch.int32 or labels.device != self.device or labels.shape != (batch,) \
                or not labels.is_contiguous():
            raise ValueError(f"labels must be a contiguous int32 tensor of {batch} values on the table's device")
        return stride, batch

    def cross_entropy(self, residual: torch.Tensor, labels: torch.Tensor, out_loss: torch.Tensor | None = None,
                      out_lse: torch.Tensor | None = None, workspace: torch.Tensor | None = None):
        """(loss, lse) float32 [B] of residual rows [B, hidden] of the table's type against int32
        labels [B]: lse = ln sum_v exp(residual @ table.T), loss = lse - the label's logit, 0
        where the label is not in [0, vocab).  The logits are never in memory.

        Nothing is recorded for autograd: the caller's backward pass calls ``cross_entropy_grad``,
        in a torch.autograd.Function for instance (whose forward runs without gradients).  A
        residual that requires grad where they are recorded gets a warning.  The outputs must not
        overlap each other or the inputs."""
        if residual.requires_grad and torch.is_grad_enabled():
            warnings.warn("residual requires grad, but cross_entropy records nothing for autograd: its gradient is "
                          "what cross_entropy_grad gives", stacklevel=2)
        stride, batch = self._train_rows(residual, labels)
        dev = self.device
        loss = torch.empty(batch, dtype=torch.float32, device=dev) if out_loss is None \
            else _floats(out_loss, batch, "out_loss", dev)
        lse = torch.empty(batch, dtype=torch.float32, device=dev) if out_lse is None \
            else _floats(out_lse, batch, "out_lse", dev)
        L = lib()
        workspace, ws_ptr, ws_bytes = _workspace_for(L.etg_cross_entropy_workspace(self._h, batch), dev, workspace)
        _call(L.etg_cross_entropy, dev, self._h, residual.data_ptr(), stride, batch, labels.data_ptr(),
              loss.data_ptr(), lse.data_ptr(), ws_ptr, ws_bytes)
        return loss, lse

    def cross_entropy_grad(self, residual: torch.Tensor, labels: torch.Tensor, lse: torch.Tensor, grad_loss=1.0,
                           grad_lse: torch.Tensor | None = None, residual_grad: bool = True, table_grad: bool = True,
                           out_residual: torch.Tensor | None = None, out_table: torch.Tensor | None = None,
                           accumulate: bool = False, workspace: torch.Tensor | None = None):
        """Gradients of ``cross_entropy`` in the table's type: (residual's [B, hidden], table's
        [vocab, hidden]), None in the place of one that is not wanted.

        lse: as cross_entropy gave it.  grad_loss: the gradient of each loss, a number or a
        float32 tensor [B]; grad_lse: that of each lse, a float32 tensor [B] or None.
        accumulate: add the table's gradient to ``out_table``.  The logits are computed again,
        by pieces of the vocabulary.  The outputs must not overlap each other or the inputs (the
        table's rows among them).
        """
        stride, batch = self._train_rows(residual, labels)
        dev, dtype = self.device, residual.dtype
        _floats(lse, batch, "lse", dev)
        d_gl = None
        if isinstance(grad_loss, torch.Tensor):
            d_gl, grad_loss = _floats(grad_loss, batch, "grad_loss", dev).data_ptr(), 0.0
        d_gz = None if grad_lse is None else _floats(grad_lse, batch, "grad_lse", dev).data_ptr()
        dx_ptr, dx_stride = None, self.hidden
        if residual_grad:
            if out_residual is None:
                out_residual = torch.empty((batch, self.hidden), dtype=dtype, device=dev)
            elif out_residual.dtype != dtype or out_residual.shape != residual.shape:
                raise ValueError("out_residual must be a tensor of the residual's type and shape")
            dx_ptr, dx_stride = out_residual.data_ptr(), _rows(out_residual, "out_residual", dev)
        elif out_residual is not None:
            raise ValueError("out_residual is given, but residual_grad is not wanted")
        if table_grad:
            out_table = self._table_grad(out_table, (dtype,), dtype, accumulate)
        elif out_table is not None or accumulate:
            raise ValueError("out_table or accumulate is given, but table_grad is not wanted")
        L = lib()
        workspace, ws_ptr, ws_bytes = _workspace_for(L.etg_cross_entropy_grad_workspace(self._h, batch), dev, workspace)
        _call(L.etg_cross_entropy_grad, dev, self._h, residual.data_ptr(), stride, batch, labels.data_ptr(),
              lse.data_ptr(), grad_loss, d_gl, d_gz, dx_ptr, dx_stride,
              out_table.data_ptr() if table_grad else None, int(accumulate), ws_ptr, ws_bytes)
        return out_residual, out_table

    def _table_grad(self, out, types, dtype, accumulate) -> torch.Tensor:
        """The gradient [vocab, hidden] given as ``out``, checked, or a new one."""
        if out is None:
            if accumulate:
                raise ValueError("accumulate needs the tensor to add to")
            return torch.empty((self.vocab, self.hidden), dtype=dtype, device=self.device)
        if out.dtype not in types or out.device != self.device or out.shape != (self.vocab, self.hidden) \
                or not out.is_contiguous():
            raise ValueError(f"the table's gradient must be a contiguous {' or '.join(map(str, types))} tensor "
                             f"[{self.vocab}, {self.hidden}] on the table's device")
        return out

    def embed_gather_grad(self, grad: torch.Tensor, ids: torch.Tensor, scale=None, out: torch.Tensor | None = None,
                          out_dtype=None, accumulate: bool = False, workspace: torch.Tensor | None = None):
        """Gradient of ``embed_gather`` with respect to the table, [vocab, hidden] in the table's
        type (or float32: out_dtype or the type of ``out``): out[v] = scale * the sum of grad's
        rows [n, hidden] (float32, bfloat16 or float16) whose id is v, added to what ``out``
        holds with accumulate.  Bad ids add nothing.  Sums are in a fixed order, without
        atomics.  scale: as in embed_gather.  ``out`` must not overlap grad or ids (it is written
        while they are read); the table itself is not read."""
        dtype = self._float_type()
        if ids.dtype != torch.int32 or ids.device != self.device:
            raise ValueError("ids must be an int32 tensor on the table's device")
        ids = ids.contiguous().view(-1)
        n = ids.numel()
        gtype = _FLOATS.get(grad.dtype)
        if gtype is None:
            raise ValueError("grad must be a float32, bfloat16 or float16 tensor")
        stride = _rows(grad, "grad", self.device)
        if grad.shape != (n, self.hidden):
            raise ValueError(f"grad must have {n} rows of {self.hidden} values")
        sc = 1.0 if scale is None else (sqrt_d(self.hidden) if scale == "sqrt_d" else float(scale))
        want = dtype if out_dtype is None else _float_dtype(out_dtype)
        if want not in (dtype, torch.float32):
            raise ValueError(f"out_dtype must be {dtype} or float32")
        if out is not None and out_dtype is not None and out.dtype != want:
            raise ValueError(f"out is not a {want} tensor")
        types = (dtype,) if dtype == torch.float32 else (dtype, torch.float32)
        out = self._table_grad(out, types, want, accumulate)
        L = lib()
        workspace, ws_ptr, ws_bytes = _workspace_for(L.etg_embed_gather_grad_workspace(self._h, n), self.device,
                                                     workspace)
        _call(L.etg_embed_gather_grad, self.device, self._h, ids.data_ptr(), n, grad.data_ptr(), gtype, stride, sc,
              out.data_ptr(), _FLOATS[out.dtype], int(accumulate), ws_ptr, ws_bytes)
        return out


_FLOATS = {torch.float32: F32, torch.bfloat16: BF16, torch.float16: F16}
_TORCH_FLOATS = {F32: torch.float32, BF16: torch.bfloat16, F16: torch.float16}


def _float_dtype(dtype) -> torch.dtype:
    """A torch dtype from F32 / BF16 / F16 or the torch dtype itself."""
    if dtype not in _FLOATS:
        dtype = _TORCH_FLOATS.get(dtype)
        if dtype is None:
            raise ValueError("a dtype is float32, bfloat16 or float16 (F32, BF16 or F16)")
    return dtype


# the current stream's handle without a Stream object around it (0.1 us instead of 1.9)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) \
    or (lambda index: torch.cuda.current_stream(index).cuda_stream)


def _call(fn, device: torch.device, *args) -> None:
    """fn(*args, current stream of the device), with the device current; raises on an error."""
    stream = _raw_stream(device.index)
    if torch.cuda.current_device() == device.index:
        status = fn(*args, stream)
    else:
        with torch.cuda.device(device):
            status = fn(*args, stream)
    if status != 0:
        _check(status)


def _rows(t: torch.Tensor, what: str, device: torch.device | None = None) -> int:
    """The row stride of a 2-D device tensor whose rows are contiguous and do not overlap."""
    if t.dim() != 2 or not t.is_cuda or (device is not None and t.device != device):
        raise ValueError(f"{what} must be a 2-D tensor on the {'same' if device is not None else 'GPU'} device")
    n, cols = t.shape
    stride, inner = t.stride()
    if cols > 1 and inner != 1:
        raise ValueError(f"{what} must have contiguous rows")
    if n <= 1:
        return cols
    if stride < cols:
        raise ValueError(f"{what} rows overlap (stride {stride}, {cols} values)")
    return stride


def _scales(t: torch.Tensor, n: int, what: str, device: torch.device) -> int:
    """Checks a vector of n f32 scales; returns its stride in floats."""
    if t.dtype != torch.float32 or t.device != device or t.shape != (n,):
        raise ValueError(f"{what} must be a float32 tensor of {n} values on the operands' device")
    s = t.stride(0) if n > 1 else 1
    if s < 1:
        raise ValueError(f"{what} must have a positive stride")
    return s


def _floats(t: torch.Tensor, n: int, what: str, device: torch.device) -> torch.Tensor:
    """A contiguous vector of n f32 values, checked."""
    if t.dtype != torch.float32 or t.device != device or t.shape != (n,) or not t.is_contiguous():
        raise ValueError(f"{what} must be a contiguous float32 tensor of {n} values on the table's device")
    return t


def _workspace_for(need: int, device: torch.device, given: torch.Tensor | None = None):
    """(tensor, pointer, bytes) of a call's workspace: the given tensor checked (its size by
    the call itself), or a fresh one, as calls on other streams and captured graphs keep their
    own (the caching allocator makes that cheap); no tensor where none is needed."""
    if given is not None:
        if given.dtype != torch.uint8 or given.device != device or not given.is_contiguous():
            raise ValueError("workspace must be a contiguous uint8 tensor on the operands' device")
        return given, given.data_ptr(), given.numel()
    if need == 0:
        return None, None, 0
    if need < 0:
        _check(need)
    space = torch.empty(need, dtype=torch.uint8, device=device)
    return space, space.data_ptr(), need


def quantize_i8(x: torch.Tensor, codes: torch.Tensor | None = None, scale: torch.Tensor | None = None):
    """(int8 codes [rows, cols], f32 scales [rows]) of the rows of a float32, bfloat16 or
    float16 matrix: scale = max|x| / 127, codes = round(x / scale) (ADR-0009's i8 wire
    definition).  A row with a NaN or an infinity gets scale NaN.  ``codes`` and ``scale``
    may be given, with any row stride."""
    dtype = _FLOATS.get(x.dtype)
    if dtype is None:
        raise ValueError("x must be a float32, bfloat16 or float16 tensor")
    xs = _rows(x, "x")
    rows, cols = x.shape
    dev = x.device
    if codes is None:
        codes, qs = torch.empty((rows, cols), dtype=torch.int8, device=dev), cols
    elif codes.dtype != torch.int8 or codes.shape != x.shape:
        raise ValueError("codes must be an int8 tensor of x's shape")
    else:
        qs = _rows(codes, "codes", dev)
    if scale is None:
        scale, ss = torch.empty(rows, dtype=torch.float32, device=dev), 1
    else:
        ss = _scales(scale, rows, "scale", dev)
    _call(lib().etg_quantize_i8, dev, x.data_ptr(), dtype, rows, cols, xs, codes.data_ptr(), qs, scale.data_ptr(), ss)
    return codes, scale


def _out(out: torch.Tensor | None, out_dtype, m: int, n: int, device: torch.device):
    """(output [m, n], its row stride): the given one checked, or a new one."""
    if out is None:
        return torch.empty((m, n), dtype=_float_dtype(out_dtype), device=device), max(n, 1)
    if out.dtype not in _FLOATS or out.shape != (m, n):
        raise ValueError("out must be a float32, bfloat16 or float16 tensor of the result's shape")
    return out, max(_rows(out, "out", device), 1)


def matmul_i8(a: torch.Tensor, a_scale: torch.Tensor, w: torch.Tensor, w_scale: torch.Tensor,
              out_dtype=torch.float32, out: torch.Tensor | None = None,
              workspace: torch.Tensor | None = None) -> torch.Tensor:
    """out [m, n] = (a @ w.T) * a_scale[:, None] * w_scale[None, :] for int8 a [m, k] and
    w [n, k] (rows of any stride; k <= 65536): exact int32 sums, scaled in f32, rounded
    once to ``out_dtype`` (float32, bfloat16, float16, or F32 / BF16 / F16)."""
    if a.dtype != torch.int8 or w.dtype != torch.int8:
        raise ValueError("a and w must be int8 tensors")
    dev = a.device
    a_stride, w_stride = _rows(a, "a"), _rows(w, "w", dev)
    m, k = a.shape
    n = w.shape[0]
    if w.shape[1] != k:
        raise ValueError(f"a has {k} columns, w {w.shape[1]}")
    sa, sw = _scales(a_scale, m, "a_scale", dev), _scales(w_scale, n, "w_scale", dev)
    out, out_stride = _out(out, out_dtype, m, n, dev)
    L = lib()
    workspace, ws_ptr, ws_bytes = _workspace_for(L.etg_matmul_i8_workspace(m, n, k), dev, workspace)
    _call(L.etg_matmul_i8, dev, a.data_ptr(), a_stride, a_scale.data_ptr(), sa, w.data_ptr(), w_stride,
          w_scale.data_ptr(), sw, m, n, k, out.data_ptr(), _FLOATS[out.dtype], out_stride, ws_ptr, ws_bytes)
    return out


class _Sampling(ctypes.Structure):
    """etg_sampling of include/etg.h."""
    _fields_ = [("temperature", _F), ("top_k", _I32), ("top_p", _F), ("min_p", _F), ("d_temperature", _VP),
                ("d_top_k", _VP), ("d_top_p", _VP), ("d_min_p", _VP), ("d_allowed", _VP), ("allowed_stride", _I64)]


def _setting(v, off, dtype: torch.dtype, rows: int, device: torch.device, what: str):
    """(scalar, device pointer or None) of a sampling setting."""
    if not isinstance(v, torch.Tensor):
        return v, None
    if v.dtype != dtype or v.device != device or v.shape != (rows,) or not v.is_contiguous():
        raise ValueError(f"{what} must be a number or a contiguous {dtype} tensor of {rows} values on the logits' device")
    return off, v.data_ptr()


def sample(logits: torch.Tensor, uniform: torch.Tensor, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0,
           allowed: torch.Tensor | None = None, out_ids: torch.Tensor | None = None,
           out_probs: torch.Tensor | None = None, workspace: torch.Tensor | None = None):
    """One token per row of logits (float32, bfloat16 or float16 [B, vocab]): (ids int32
    [B], probabilities f32 [B] they were drawn with), from random numbers ``uniform`` (f32
    [B] in [0, 1)).

    temperature (0: greedy), top_k (0: off), top_p (1: off) and min_p (0: off) are numbers
    or device tensors with one value per row (float32; top_k int32).  ``allowed`` is a bit
    mask, int32 [ceil(vocab / 32)] or [B, ceil(vocab / 32)], bit v % 32 of word v / 32 set
    where token v is allowed.  NaN and -inf logits are never drawn.  A row with nothing to
    draw, or with a setting or random number out of range, has id -1 and probability 0.
    """
    dtype = _FLOATS.get(logits.dtype)
    if dtype is None:
        raise ValueError("logits must be a float32, bfloat16 or float16 tensor")
    stride = _rows(logits, "logits")
    rows, vocab = logits.shape
    dev = logits.device
    if uniform.dtype != torch.float32 or uniform.device != dev or uniform.shape != (rows,) \
            or not uniform.is_contiguous():
        raise ValueError(f"uniform must be a contiguous float32 tensor of {rows} values on the logits' device")
    T, d_T = _setting(temperature, 1.0, torch.float32, rows, dev, "temperature")
    k, d_k = _setting(top_k, 0, torch.int32, rows, dev, "top_k")
    p, d_p = _setting(top_p, 1.0, torch.float32, rows, dev, "top_p")
    mp, d_mp = _setting(min_p, 0.0, torch.float32, rows, dev, "min_p")
    d_allowed, a_stride = None, 0
    if allowed is not None:
        words = (vocab + 31) // 32
        if allowed.dtype != torch.int32 or allowed.device != dev or allowed.dim() not in (1, 2) \
                or allowed.shape[-1] != words or (words > 1 and allowed.stride(-1) != 1) \
                or (allowed.dim() == 2 and allowed.shape[0] != rows):
            raise ValueError(f"allowed must be an int32 [{words}] or [{rows}, {words}] tensor with contiguous rows on "
                             "the logits' device")
        d_allowed = allowed.data_ptr()
        if allowed.dim() == 2 and rows > 1:
            a_stride = allowed.stride(0)  # 0: an expanded row, one for all
    if out_ids is None:
        out_ids = torch.empty(rows, dtype=torch.int32, device=dev)
    elif out_ids.dtype != torch.int32 or out_ids.device != dev or out_ids.shape != (rows,) \
            or not out_ids.is_contiguous():
        raise ValueError(f"out_ids must be a contiguous int32 tensor of {rows} values on the logits' device")
    if out_probs is None:
        out_probs = torch.empty(rows, dtype=torch.float32, device=dev)
    elif out_probs.dtype != torch.float32 or out_probs.device != dev or out_probs.shape != (rows,) \
            or not out_probs.is_contiguous():
        raise ValueError(f"out_probs must be a contiguous float32 tensor of {rows} values on the logits' device")
    L = lib()
    workspace, ws_ptr, ws_bytes = _workspace_for(L.etg_sample_workspace(rows, vocab), dev, workspace)
    if d_k is None:  # the C type's range: past every vocabulary is off, a negative one stays negative
        k = 0 if k > 0x7fffffff else max(k, -0x80000000)
    how = _Sampling(T, k, p, mp, d_T, d_k, d_p, d_mp, d_allowed, a_stride)
    _call(L.etg_sample, dev, logits.data_ptr(), dtype, rows, vocab, stride, ctypes.addressof(how), uniform.data_ptr(),
          out_ids.data_ptr(), out_probs.data_ptr(), ws_ptr, ws_bytes)
    return out_ids, out_probs


class I8Table:
    """A V x hidden lm_head as int8 rows with one f32 scale each (half the bytes of a bf16
    one): logits come from an int8 product with residual rows quantised the same way.

    ``codes`` is an int8 [V, hidden] device tensor (rows of any stride), ``scale`` float32
    [V]: Table.quantize_i8() or quantize_i8(rows) make them.  Both are borrowed.
    """

    def __init__(self, codes: torch.Tensor, scale: torch.Tensor):
        if codes.dtype != torch.int8:
            raise ValueError("codes must be an int8 tensor")
        self._stride = _rows(codes, "codes")
        self.codes, self.scale = codes, scale
        self.vocab, self.hidden = codes.shape
        self.device = codes.device
        self._scale_stride = _scales(scale, self.vocab, "scale", self.device)

    def logits_raw(self, residual: torch.Tensor, out_dtype=torch.float32, out: torch.Tensor | None = None,
                   workspace: torch.Tensor | None = None) -> torch.Tensor:
        """Logits [B, vocab] of float32, bfloat16 or float16 residual rows [B, hidden],
        each row quantised to int8 first."""
        dtype, dev = _FLOATS.get(residual.dtype), self.device
        if dtype is None:
            raise ValueError("residual must be a float32, bfloat16 or float16 tensor")
        stride = _rows(residual, "residual", dev)
        B, hidden = residual.shape
        if hidden != self.hidden:
            raise ValueError(f"residual has {hidden} columns, the table {self.hidden}")
        out, out_stride = _out(out, out_dtype, B, self.vocab, dev)
        L = lib()
        workspace, ws_ptr, ws_bytes = _workspace_for(L.etg_logits_i8_workspace(B, self.vocab, hidden), dev, workspace)
        _call(L.etg_logits_i8, dev, self.codes.data_ptr(), self._stride, self.scale.data_ptr(), self._scale_stride,
              self.vocab, hidden, residual.data_ptr(), dtype, stride, B, out.data_ptr(), _FLOATS[out.dtype], out_stride,
              ws_ptr, ws_bytes)
        return out

    def logits_raw_wire(self, residual: torch.Tensor, out_dtype=torch.float32,
                        out: torch.Tensor | None = None) -> torch.Tensor:
        """Logits of residual rows in the WIRE_I8 format (a contiguous device buffer of
        whole wire rows), whose codes are multiplied as they are."""
        rb = wire_row_bytes(WIRE_I8, self.hidden)
        nbytes = residual.numel() * residual.element_size()
        if residual.device != self.device or not residual.is_contiguous() or nbytes % rb:
            raise ValueError("residual must be a contiguous device buffer of whole wire rows")
        if rb % 4 or residual.data_ptr() % 4:
            raise ValueError("wire rows must be 4-byte aligned (hidden a multiple of 4)")
        rows = residual.view(-1).view(torch.int8).view(-1, rb)
        return matmul_i8(rows[:, 8:], residual.view(-1).view(torch.float32).view(-1, rb // 4)[:, 0], self.codes,
                         self.scale, out_dtype=out_dtype, out=out)

    def sample(self, residual: torch.Tensor, uniform: torch.Tensor, **kw):
        """The next token of each residual row: ``sample`` of its logits (same settings)."""
        return sample(self.logits_raw(residual), uniform, **kw)


class StepCache:
    """Embed and logits calls for small repeated shapes from host ids to a host
    answer: the kernels read the ids from, and write the top-k answer to, mapped
    page-locked memory (no copy operations), the answer tracked by an event.  With
    use_graphs=True each configuration (token counts bucketed to multiples of 64 or
    256) is captured into a HIP graph on its second hit and replayed after; on this
    platform a graph launch measured slower than the two to four kernel launches it
    replaces, so calls run eagerly by default.

    Owns its buffers as tensors and lends them to the library:
      rows      device f32 [ids capacity, hidden]: the gathered rows
      residual  device f32 [max_batch, hidden]: write the residual rows here
      ids, scores  page-locked CPU [max_batch, k]: the answer after event.synchronize()
    """

    STEP_ID_SLOTS = 4  # ETG_STEP_ID_SLOTS

    def __init__(self, table: Table, max_ids: int, max_batch: int, k: int, use_graphs: bool = False):
        L = lib()
        self.table, self.k, self.max_ids, self.max_batch = table, int(k), int(max_ids), int(max_batch)
        dev = table.device
        cap = int(L.etg_step_cache_ids_capacity(int(max_ids)))
        if cap < 0:
            raise ValueError(f"max_ids {max_ids} out of range")
        ws = int(L.etg_step_cache_workspace(table.handle, int(max_batch), int(k)))
        if ws < 0:
            _check(ws)
        self.d_ids = torch.zeros(cap, dtype=torch.int32, device=dev)
        self.rows = torch.empty((cap, table.hidden), dtype=torch.float32, device=dev)
        self.residual = torch.zeros((int(max_batch), table.hidden), dtype=torch.float32, device=dev)
        self.d_topk_ids = torch.empty((int(max_batch), int(k)), dtype=torch.int32, device=dev)
        self.d_topk_scores = torch.empty((int(max_batch), int(k)), dtype=torch.float32, device=dev)
        self.workspace = torch.empty(max(ws, 256), dtype=torch.uint8, device=dev)
        self.h_ids = torch.zeros((self.STEP_ID_SLOTS, cap), dtype=torch.int32, pin_memory=True)
        self.ids = torch.zeros((int(max_batch), int(k)), dtype=torch.int32, pin_memory=True)
        self.scores = torch.zeros((int(max_batch), int(k)), dtype=torch.float32, pin_memory=True)
        h = ctypes.c_void_p()
        _check(L.etg_step_cache_create(table.handle, int(max_ids), int(max_batch), int(k), int(bool(use_graphs)),
                                       _ptr(self.d_ids),
                                       _ptr(self.rows), _ptr(self.residual), _ptr(self.d_topk_ids),
                                       _ptr(self.d_topk_scores), _ptr(self.workspace), self.workspace.numel(),
                                       _ptr(self.h_ids), _ptr(self.ids), _ptr(self.scores), ctypes.byref(h)))
        self._h = h

    def __del__(self):
        h = getattr(self, "_h", None)
        if h is not None and _lib is not None:
            _lib.etg_step_cache_destroy(h)
            self._h = None

    def gather(self, ids, scale=None) -> torch.Tensor:
        """Rows for host int32 ids (a CPU tensor or array of n ids): a view of the
        first n rows of ``rows``, filled in stream order."""
        import numpy as np
        a = np.ascontiguousarray(ids.numpy() if isinstance(ids, torch.Tensor) else ids, dtype=np.int32).reshape(-1)
        sc = 1.0 if scale is None else (sqrt_d(self.table.hidden) if scale == "sqrt_d" else float(scale))
        with torch.cuda.device(self.table.device):
            _check(lib().etg_step_gather(self._h, a.ctypes.data_as(ctypes.c_void_p), a.size, sc,
                                         _stream_ptr(self.table.device)))
        return self.rows[:a.size]

    def logits(self, batch: int, event=None):
        """Top-k of residual rows [0, batch) into the page-locked ``ids`` / ``scores``;
        returns the event recorded after the copy (wait on it before reading)."""
        ev = event if event is not None else torch.cuda.Event()
        with torch.cuda.device(self.table.device):
            evh = ctypes.c_void_p(_event_handle(ev, self.table.device))
            _check(lib().etg_step_logits(self._h, int(batch), evh, _stream_ptr(self.table.device)))
        return ev

    def stats(self):
        g, r = ctypes.c_int64(), ctypes.c_int64()
        _check(lib().etg_step_cache_stats(self._h, ctypes.byref(g), ctypes.byref(r)))
        return g.value, r.value


def hbm_read_probe(t: torch.Tensor, sink: torch.Tensor | None = None) -> None:
    """Enqueue a plain read stream of the bytes of a contiguous device tensor (a
    multiple of 16 bytes) on the current stream: the measured HBM read reference."""
    if not t.is_cuda or not t.is_contiguous():
        raise ValueError("a contiguous device tensor is required")
    if sink is None:
        sink = torch.empty(1, dtype=torch.int32, device=t.device)
    _check(lib().etg_hbm_read_probe(t.data_ptr(), t.numel() * t.element_size(), sink.data_ptr(),
                                    torch.cuda.current_stream(t.device).cuda_stream))


def hbm_write_probe(t: torch.Tensor, value: int = 0) -> None:
    """Enqueue a plain write stream over the bytes of a contiguous device tensor (a
    multiple of 16 bytes), every 32-bit word set to `value`, on the current stream:
    the measured HBM write reference."""
    if not t.is_cuda or not t.is_contiguous():
        raise ValueError("a contiguous device tensor is required")
    _check(lib().etg_hbm_write_probe(t.data_ptr(), t.numel() * t.element_size(), int(value) & 0xFFFFFFFF,
                                     torch.cuda.current_stream(t.device).cuda_stream))


def wire_row_bytes(wire: int, hidden: int) -> int:
    n = int(lib().etg_wire_row_bytes(int(wire), int(hidden)))
    if n < 0:
        raise ValueError(f"unknown wire format {wire} or hidden {hidden}")
    return n


def embed_gather(table: Table, ids: torch.Tensor, scale=None, **kw) -> torch.Tensor:
    return table.embed_gather(ids, scale=scale, **kw)


def logits_topk(table: Table, residual: torch.Tensor, k: int, **kw):
    return table.logits_topk(residual, k, **kw)

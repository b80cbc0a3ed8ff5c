"""Torch-facing wrapper of the C ABI: one handle per layer's state pool.

PyTorch supplies device memory and streams only; every step runs in
``libsq.so``. Tensors must be CUDA, contiguous, on the handle's device and
of the dtypes the C ABI states (fp32 activations, int32 slot ids, uint8 or
fp32 pool); anything else raises before a launch.
"""
from __future__ import annotations

import ctypes

import numpy as np
import torch

from . import _abi


def _stream(stream) -> int:
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


def _ptr(t: torch.Tensor | None, dtype=None, name="tensor", numel=None, dev=None) -> int | None:
    """Address of a contiguous CUDA tensor, on device `dev` where given (None passes)."""
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if dev is not None and t.get_device() != dev:
        raise ValueError(f"{name} must be a CUDA tensor on device {dev}, not on {t.device}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if numel is not None and t.numel() != numel:
        raise ValueError(f"{name} has {t.numel()} elements, expected {numel}")
    return t.data_ptr()


def _host_ptr(t: torch.Tensor | None, dtype, name, numel) -> int | None:
    if t is None:
        return None
    if t.is_cuda:
        raise ValueError(f"{name} must be a CPU tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if t.numel() != numel:
        raise ValueError(f"{name} has {t.numel()} elements, expected {numel}")
    return t.data_ptr()


DTYPES = {torch.float32: _abi.SQ_F32, torch.bfloat16: _abi.SQ_BF16, torch.float16: _abi.SQ_F16}


def _raw_stream(stream, dev: int) -> int:
    """Address of a stream, or of device `dev`'s current one."""
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(dev)
    return stream.cuda_stream if isinstance(stream, torch.cuda.Stream) else int(stream)


def row_ptr(t: torch.Tensor, dtype, name, rows, heads, d, dev: int):
    """(address, row stride in elements) of a [rows, heads, d] tensor whose
    rows may lie apart (a column slice of a wider matrix)."""
    shape, st = t.shape, t.stride()
    if (t.get_device() == dev and t.dtype is dtype and shape == (rows, heads, d) and st[2] == 1
            and (st[1] == d or heads == 1)):
        return t.data_ptr(), st[0] if rows > 1 else heads * d
    if not t.is_cuda or t.get_device() != dev:
        raise ValueError(f"{name} must be a CUDA tensor on device {dev}, not on {t.device}")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if tuple(shape) != (rows, heads, d):
        raise ValueError(f"{name} has shape {tuple(shape)}, expected {(rows, heads, d)}")
    if t.numel():
        raise ValueError(f"{name}: the heads of a row must be contiguous")
    return t.data_ptr(), heads * d


class StatePool:
    """A layer's recurrent-state pool handle (calibration tables on device).

    fmt: _abi.SQ_FMT_PACKED (quantized) or _abi.SQ_FMT_FP32 (unquantized).
    gate_kind: _abi.SQ_GATE_HEAD (GDN) or _abi.SQ_GATE_KEY_CHANNEL (KDA).
    unit_bits, pivot: [h_v] (GDN) or [h_v, d] (KDA); col_scale, row_impact [h_v, d].
    """

    def __init__(self, n_slots, h_v, h_k, d, gate_kind, fmt=_abi.SQ_FMT_PACKED, unit_bits=None, pivot=None,
                 col_scale=None, row_impact=None, stream=None):
        self.n_slots, self.h_v, self.h_k, self.d = int(n_slots), int(h_v), int(h_k), int(d)
        self.gate_kind, self.fmt = int(gate_kind), int(fmt)
        self.device = torch.device("cuda", torch.cuda.current_device())
        desc = _abi.StateDesc(self.n_slots, self.h_v, self.h_k, self.d, self.d, self.fmt, self.gate_kind)
        calib = None
        self._keep = []
        if fmt == _abi.SQ_FMT_PACKED:
            arrs = [np.ascontiguousarray(unit_bits, dtype=np.int8), np.ascontiguousarray(pivot, dtype=np.uint8),
                    np.ascontiguousarray(col_scale, dtype=np.float32),
                    np.ascontiguousarray(row_impact, dtype=np.float32)]
            self._keep = arrs
            calib = _abi.Calib(*[a.ctypes.data for a in arrs])
        self._h, self.pool_bytes = _abi.sq_state_alloc(desc, calib, _stream(stream))
        rep = _abi.sq_state_bytes(self._h)
        self.slot_bytes = rep["slot_bytes"]
        self.report = rep

    # ----------------------------------------------------------- helpers
    def close(self):
        if getattr(self, "_h", None) is not None and self._h.value:
            _abi.sq_state_free(self._h)
            self._h = None

    def __del__(self):  # pragma: no cover
        try:
            self.close()
        except Exception:
            pass

    def new_pool(self) -> torch.Tensor:
        if self.fmt == _abi.SQ_FMT_PACKED:
            return torch.zeros(self.pool_bytes, dtype=torch.uint8, device=self.device)
        return torch.zeros((self.n_slots, self.h_v, self.d, self.d), dtype=torch.float32, device=self.device)

    def _arg(self, t, dtype=None, name="tensor", numel=None):
        return _ptr(t, dtype, name, numel, self.device.index)

    def _check_pool(self, pool):
        if pool.numel() * pool.element_size() != self.pool_bytes:
            raise ValueError(f"pool has {pool.numel() * pool.element_size()} bytes, expected {self.pool_bytes}")
        return self._arg(pool, name="pool")

    def head_layout(self, head: int):
        return _abi.sq_head_layout(self._h, head)

    def launches(self) -> int:
        return _abi.sq_launch_count(self._h)

    # --------------------------------------------------------- the calls
    def quantize_state(self, pool, S, slot_ids=None, stream=None):
        B = S.shape[0]
        d, hv = self.d, self.h_v
        _abi.sq_quantize_state(self._h, self._check_pool(pool),
                               self._arg(S, torch.float32, "S", B * hv * d * d),
                               self._arg(slot_ids, torch.int32, "slot_ids", B), B, _stream(stream))

    def decode_step(self, pool, q, k, v, beta, g, o, slot_ids=None, stream=None):
        B = q.shape[0]
        d, hv, hk = self.d, self.h_v, self.h_k
        gn = B * hv * (d if self.gate_kind == _abi.SQ_GATE_KEY_CHANNEL else 1)
        _abi.sq_decode_step(self._h, self._check_pool(pool),
                            self._arg(q, torch.float32, "q", B * hk * d), self._arg(k, torch.float32, "k", B * hk * d),
                            self._arg(v, torch.float32, "v", B * hv * d), self._arg(beta, torch.float32, "beta", B * hv),
                            self._arg(g, torch.float32, "g", gn), self._arg(o, torch.float32, "o", B * hv * d),
                            self._arg(slot_ids, torch.int32, "slot_ids", B), B, _stream(stream))

    def window_buffer_bytes(self, W: int):
        """(bytes of one (slot, head) window record, bytes of the whole buffer)."""
        return _abi.sq_window_buffer_bytes(self._h, int(W))

    def new_window_buffer(self, W: int) -> torch.Tensor:
        """A zeroed window buffer (every count 0) for windows of W tokens."""
        return torch.zeros(self.window_buffer_bytes(W)[1], dtype=torch.uint8, device=self.device)

    def window_step(self, pool, wbuf, W, q, k, v, beta, g, o, slot_ids=None, stream=None):
        """One token of the per-window variant (sq_window_step): the packed
        state stays frozen while the window buffer collects the tokens'
        updates; it is requantized when W tokens are buffered."""
        B = q.shape[0]
        d, hv, hk = self.d, self.h_v, self.h_k
        gn = B * hv * (d if self.gate_kind == _abi.SQ_GATE_KEY_CHANNEL else 1)
        nb = self.window_buffer_bytes(W)[1]
        if wbuf.numel() * wbuf.element_size() != nb:
            raise ValueError(f"window buffer has {wbuf.numel() * wbuf.element_size()} bytes, expected {nb}")
        _abi.sq_window_step(self._h, self._check_pool(pool), self._arg(wbuf, name="wbuf"), int(W),
                            self._arg(q, torch.float32, "q", B * hk * d), self._arg(k, torch.float32, "k", B * hk * d),
                            self._arg(v, torch.float32, "v", B * hv * d), self._arg(beta, torch.float32, "beta", B * hv),
                            self._arg(g, torch.float32, "g", gn), self._arg(o, torch.float32, "o", B * hv * d),
                            self._arg(slot_ids, torch.int32, "slot_ids", B), B, _stream(stream))

    def decode_step_host(self, pool, q, k, v, beta, g, o, slot_ids=None, stream=None):
        """The decode step with q, k, v, beta, g, slot_ids and o as CPU tensors
        (page-locked for overlapped copies; o page-locked is written by the
        kernel directly). The pool stays on the GPU. Read o after the stream
        has passed the call."""
        B = q.shape[0]
        d, hv, hk = self.d, self.h_v, self.h_k
        gn = B * hv * (d if self.gate_kind == _abi.SQ_GATE_KEY_CHANNEL else 1)
        _abi.sq_decode_step_host(self._h, self._check_pool(pool),
                                 _host_ptr(q, torch.float32, "q", B * hk * d),
                                 _host_ptr(k, torch.float32, "k", B * hk * d),
                                 _host_ptr(v, torch.float32, "v", B * hv * d),
                                 _host_ptr(beta, torch.float32, "beta", B * hv),
                                 _host_ptr(g, torch.float32, "g", gn), _host_ptr(o, torch.float32, "o", B * hv * d),
                                 _host_ptr(slot_ids, torch.int32, "slot_ids", B), B, _stream(stream))

    def prefill(self, pool, q, k, v, beta, g, o, S0=None, S_out=None, lengths=None, slot_ids=None, stream=None):
        """Run the prompt (q, k [B, L, h_k, d]; v, o [B, L, h_v, d]; beta [B, L, h_v];
        g [B, L, h_v] or [B, L, h_v, d]) through the gated delta rule from S0
        (or zeros) and store the final state once in the requests' slots."""
        B, L = q.shape[0], q.shape[1]
        d, hv, hk = self.d, self.h_v, self.h_k
        gn = B * L * hv * (d if self.gate_kind == _abi.SQ_GATE_KEY_CHANNEL else 1)
        n = B * L
        _abi.sq_prefill(self._h, self._check_pool(pool), self._arg(S0, torch.float32, "S0", B * hv * d * d),
                        self._arg(q, torch.float32, "q", n * hk * d), self._arg(k, torch.float32, "k", n * hk * d),
                        self._arg(v, torch.float32, "v", n * hv * d), self._arg(beta, torch.float32, "beta", n * hv),
                        self._arg(g, torch.float32, "g", gn), self._arg(o, torch.float32, "o", n * hv * d),
                        self._arg(S_out, torch.float32, "S_out", B * hv * d * d),
                        self._arg(lengths, torch.int32, "lengths", B), self._arg(slot_ids, torch.int32, "slot_ids", B),
                        B, L, _stream(stream))

    def ragged_workspace_bytes(self, B: int, rows: int, max_len: int | None = None, dtype=torch.bfloat16) -> int:
        """Bytes of workspace prefill_ragged needs for a batch of these sizes."""
        return _abi.sq_ragged_workspace_bytes(self._h, DTYPES[dtype], int(B), int(rows),
                                              int(rows if max_len is None else max_len))

    def new_ragged_workspace(self, B: int, rows: int, max_len: int | None = None, dtype=torch.bfloat16) -> torch.Tensor:
        """A workspace for prefill_ragged; calls that may overlap need one each."""
        return torch.empty(self.ragged_workspace_bytes(B, rows, max_len, dtype), dtype=torch.uint8,
                           device=self.device)

    def prefill_ragged(self, pool, q, k, v, beta, g, o, tables, slot_ids=None, max_len=None, workspace=None,
                       stream=None):
        """The gated delta rule over a ragged batch (sq_prefill_ragged): q, k
        [rows, h_k, d], v, o [rows, h_v, d] (bf16, fp16 or fp32; q, k and v may
        be column slices of wider matrices), beta [rows, h_v], g [rows, h_v]
        or [rows, h_v, d], tables a ragged.BatchTables. A request with
        past > 0 goes on from its slot's state, another starts from zeros.
        max_len: the longest request's rows (by default all rows): a batch of
        short requests that does not give it allocates the workspace of long
        ones (ragged_workspace_bytes) and runs three kernels in place of one."""
        B, rows, d, hv, hk = tables.cu_seqlens.numel() - 1, q.shape[0], self.d, self.h_v, self.h_k
        if q.dtype not in DTYPES:
            raise ValueError(f"q must be one of {tuple(DTYPES)}, got {q.dtype}")
        if tables.cu_blocks.numel() != B + 1 or tables.block_req.numel() < rows // _abi.SQ_RAGGED_BLOCK + B:
            raise ValueError("cu_blocks or block_req is too short for the batch")
        gn = rows * hv * (d if self.gate_kind == _abi.SQ_GATE_KEY_CHANNEL else 1)
        max_len = rows if max_len is None else int(max_len)
        dev = self.device.index
        if dev != torch.cuda.current_device():
            with torch.cuda.device(dev):
                return self.prefill_ragged(pool, q, k, v, beta, g, o, tables, slot_ids, max_len, workspace, stream)
        if workspace is None:
            need = self.ragged_workspace_bytes(B, rows, max_len, q.dtype)
            if need:  # allocated on the stream that uses it
                on = (torch.cuda.current_stream() if stream is None else
                      torch.cuda.ExternalStream(_raw_stream(stream, dev), device=self.device))
                with torch.cuda.stream(on):
                    workspace = torch.empty(need, dtype=torch.uint8, device=self.device)
        i32 = torch.int32
        t = _abi.RaggedTables(self._arg(tables.cu_seqlens, i32, "cu_seqlens", B + 1),
                              self._arg(tables.cu_blocks, i32, "cu_blocks", B + 1),
                              self._arg(tables.block_req, i32, "block_req"), self._arg(tables.past, i32, "past", B))
        qp, qs = row_ptr(q, q.dtype, "q", rows, hk, d, dev)
        kp, ks = row_ptr(k, q.dtype, "k", rows, hk, d, dev)
        vp, vs = row_ptr(v, q.dtype, "v", rows, hv, d, dev)
        _abi.sq_prefill_ragged(self._h, self._check_pool(pool), qp, kp, vp, qs, ks, vs, DTYPES[q.dtype],
                               self._arg(beta, torch.float32, "beta", rows * hv), self._arg(g, torch.float32, "g", gn),
                               self._arg(o, q.dtype, "o", rows * hv * d), t, self._arg(slot_ids, i32, "slot_ids", B), B, rows,
                               max_len, self._arg(workspace, torch.uint8, "workspace"),
                               workspace.numel() if workspace is not None else 0, _raw_stream(stream, dev))

    def dequantize_state(self, pool, S_out, slot_ids=None, stream=None):
        B = S_out.shape[0]
        d, hv = self.d, self.h_v
        _abi.sq_dequantize_state(self._h, self._check_pool(pool),
                                 self._arg(S_out, torch.float32, "S_out", B * hv * d * d),
                                 self._arg(slot_ids, torch.int32, "slot_ids", B), B, _stream(stream))

    def get_status(self, clear=True, stream=None) -> int:
        return _abi.sq_get_status(self._h, _stream(stream), clear)

    def exact_count(self, clear=True, stream=None) -> int:
        """Columns whose S^T k the packed steps summed exactly since the last clear."""
        return _abi.sq_get_exact_count(self._h, _stream(stream), clear)

    def launch_plan(self) -> dict:
        return _abi.sq_launch_plan(self._h)

    def set_wait_limit(self, ns: int) -> None:
        _abi.sq_set_wait_limit(self._h, ns)

    def test_stall_stages(self, extra_bytes: int) -> None:
        """Testing only: make CTA 0's waits run out (see include/sq.h)."""
        _abi.sq_test_stall_stages(self._h, extra_bytes)

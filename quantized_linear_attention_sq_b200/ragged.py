"""Ragged batches: torch-facing wrappers of include/sq_ragged.h.

A serving loop packs its requests' rows one after the other. ``batch_tables``
(or ``BatchTables.build``) turns the lengths into offsets, blocks, positions
and pool slots; ``qk_norm`` prepares queries and keys; then
``StatePool.prefill_ragged`` runs the gated delta rule over every request's
rows, from and into its pool slot.
"""
from __future__ import annotations

from dataclasses import dataclass

import torch

from . import _abi
from .state import DTYPES, _raw_stream, row_ptr

BLOCK = _abi.SQ_RAGGED_BLOCK
I32, U8, F32 = torch.int32, torch.uint8, torch.float32


def _arg(t, dtype, name, numel, dev):
    """Address of a contiguous tensor on CUDA device `dev` (None passes)."""
    if t is None:
        return None
    # get_device() is -1 for a CPU tensor
    if t.get_device() == dev and t.dtype is dtype and t.is_contiguous() and (numel is None or t.numel() == numel):
        return t.data_ptr()
    if not t.is_cuda or t.get_device() != dev:
        raise ValueError(f"{name} must be a CUDA tensor on device {dev}, not on {t.device}")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    raise ValueError(f"{name} has {t.numel()} elements, expected {numel}")


def _device_of(t, name):
    dev = t.get_device()
    if dev < 0:
        raise ValueError(f"{name} must be a CUDA tensor")
    return dev


def batch_tables(lengths, past, cu_seqlens, cu_blocks, positions, block_req, slot_ids=None, slot_used=None,
                 slot_out=None, used_out=None, status=None, stream=None, max_rows=None) -> None:
    """Write the tables of a ragged batch (sq_batch_tables): lengths, past
    int32 [B] (past may be None), cu_seqlens, cu_blocks int32 [B + 1],
    positions int32 [max_rows], or None (max_rows is needed then),
    block_req int32 [max_rows // 64 + B] or more.
    slot_ids, slot_out int32 [B] and slot_used, used_out uint8 [n_slots]: all
    four or none; requests with slot_ids < 0 take free slots."""
    dev = _device_of(lengths, "lengths")
    if dev != torch.cuda.current_device():
        with torch.cuda.device(dev):
            return batch_tables(lengths, past, cu_seqlens, cu_blocks, positions, block_req, slot_ids, slot_used,
                                slot_out, used_out, status, stream, max_rows)
    if max_rows is None:
        if positions is None:
            raise ValueError("max_rows is needed where positions is None")
        max_rows = positions.numel()
    B, rows = lengths.numel(), int(max_rows)
    if block_req.numel() < rows // BLOCK + B:
        raise ValueError(f"block_req has {block_req.numel()} elements, {rows // BLOCK + B} are needed")
    if not (slot_ids is None) == (slot_used is None) == (slot_out is None) == (used_out is None):
        raise ValueError("slot_ids, slot_used, slot_out and used_out go together")
    n_slots = 0 if slot_used is None else slot_used.numel()
    _abi.sq_batch_tables(_arg(lengths, I32, "lengths", None, dev), _arg(past, I32, "past", B, dev), B, rows,
                         _arg(cu_seqlens, I32, "cu_seqlens", B + 1, dev), _arg(cu_blocks, I32, "cu_blocks", B + 1, dev),
                         _arg(positions, I32, "positions", rows, dev), _arg(block_req, I32, "block_req", None, dev),
                         _arg(slot_ids, I32, "slot_ids", B, dev), _arg(slot_used, U8, "slot_used", None, dev), n_slots,
                         _arg(slot_out, I32, "slot_out", B, dev), _arg(used_out, U8, "used_out", n_slots, dev),
                         _arg(status, I32, "status", 1, dev), _raw_stream(stream, dev))


@dataclass
class BatchTables:
    """The tables of one ragged batch, on the GPU."""
    cu_seqlens: torch.Tensor              # int32 [B + 1]
    cu_blocks: torch.Tensor               # int32 [B + 1]
    block_req: torch.Tensor               # int32 [max_rows // 64 + B]
    past: torch.Tensor | None = None      # int32 [B]
    positions: torch.Tensor | None = None  # int32 [max_rows]

    @classmethod
    def empty(cls, B: int, max_rows: int, device=None) -> "BatchTables":
        """Buffers for batches of B requests and up to max_rows rows."""
        z = lambda n: torch.zeros(n, dtype=torch.int32, device=device or torch.device("cuda"))  # noqa: E731
        return cls(z(B + 1), z(B + 1), z(max_rows // BLOCK + B), None, z(max_rows))

    def build(self, lengths, past=None, slot_ids=None, slot_used=None, status=None, stream=None,
              max_rows=None) -> "BatchTables":
        """Fill the tables from lengths (int32 [B]); requests with slot_ids < 0
        take free slots of the pool, in place in slot_ids and slot_used.
        max_rows: the batch's most rows, needed where there are no positions."""
        batch_tables(lengths, past, self.cu_seqlens, self.cu_blocks, self.positions, self.block_req,
                     slot_ids=slot_ids, slot_used=slot_used, slot_out=slot_ids, used_out=slot_used, status=status,
                     stream=stream, max_rows=max_rows)
        self.past = past
        return self

    @property
    def n_rows(self) -> torch.Tensor:
        """The batch's row count, on the GPU (int32 [1])."""
        return self.cu_seqlens[-1:]


def qk_norm(q, k, q_out, k_out, mode="l2", eps=1e-6, q_weight=None, k_weight=None, q_scale=1.0, positions=None,
            rot_dim=0, base=10000.0, interleaved=False, n_rows=None, stream=None) -> None:
    """Norm of q [rows, h_q, d] and k [rows, h_k, d] for each head ("l2" or
    "rms"), times weight (fp32 [d]) and, for q, q_scale; then the first
    rot_dim channels turned by positions (int32 [rows]); sq_qk_norm. q and k
    may be column slices of a wider matrix; q_out and k_out are contiguous, of
    any of the element types. n_rows (int32 [1], on the GPU): only the rows
    below it are computed."""
    if mode not in ("l2", "rms"):
        raise ValueError(f"mode must be 'l2' or 'rms', got {mode!r}")
    for t, name in ((q, "q"), (q_out, "q_out")):
        if t.dtype not in DTYPES:
            raise ValueError(f"{name} must be one of {tuple(DTYPES)}, got {t.dtype}")
    dev = _device_of(q, "q")
    if dev != torch.cuda.current_device():
        with torch.cuda.device(dev):
            return qk_norm(q, k, q_out, k_out, mode, eps, q_weight, k_weight, q_scale, positions, rot_dim, base,
                           interleaved, n_rows, stream)
    rows, hq, d = q.shape
    hk = k.shape[1]
    desc = _abi.NormDesc(_abi.SQ_NORM_L2 if mode == "l2" else _abi.SQ_NORM_RMS, eps, q_scale, rot_dim,
                         1 if interleaved else 0, base)
    tin, tout = q.dtype, q_out.dtype
    qp, qs = row_ptr(q, tin, "q", rows, hq, d, dev)
    kp, ks = row_ptr(k, tin, "k", rows, hk, d, dev)
    _abi.sq_qk_norm(desc, qp, kp, qs, ks, DTYPES[tin], _arg(q_weight, F32, "q_weight", d, dev),
                    _arg(k_weight, F32, "k_weight", d, dev), _arg(positions, I32, "positions", rows, dev),
                    _arg(q_out, tout, "q_out", rows * hq * d, dev), _arg(k_out, tout, "k_out", rows * hk * d, dev),
                    DTYPES[tout], rows, _arg(n_rows, I32, "n_rows", 1, dev), hq, hk, d, _raw_stream(stream, dev))

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
from .state import DTYPES, _ptr, _stream, row_ptr

BLOCK = _abi.SQ_RAGGED_BLOCK


def _same_device(*ts):
    ts = [t for t in ts if t is not None]
    for t in ts:
        if not t.is_cuda:
            raise ValueError("every tensor must be a CUDA tensor")
        if t.device != ts[0].device:
            raise ValueError(f"tensors on {ts[0].device} and {t.device}")
    return ts[0].device


def batch_tables(lengths, past, cu_seqlens, cu_blocks, positions, block_req, slot_ids=None, slot_used=None,
                 slot_out=None, used_out=None, status=None, stream=None) -> None:
    """Write the tables of a ragged batch (sq_batch_tables): lengths, past
    int32 [B] (past may be None), cu_seqlens, cu_blocks int32 [B + 1],
    positions int32 [max_rows], block_req int32 [max_rows // 64 + B] or more.
    slot_ids, slot_out int32 [B] and slot_used, used_out uint8 [n_slots]: all
    four or none; requests with slot_ids < 0 take free slots."""
    B, rows = lengths.numel(), positions.numel()
    i32 = torch.int32
    dev = _same_device(lengths, past, cu_seqlens, cu_blocks, positions, block_req, slot_ids, slot_used, slot_out,
                       used_out, status)
    if block_req.numel() < rows // BLOCK + B:
        raise ValueError(f"block_req has {block_req.numel()} elements, {rows // BLOCK + B} are needed")
    slots = [slot_ids, slot_used, slot_out, used_out]
    if any(t is None for t in slots) and not all(t is None for t in slots):
        raise ValueError("slot_ids, slot_used, slot_out and used_out go together")
    n_slots = 0 if slot_used is None else slot_used.numel()
    with torch.cuda.device(dev):
        _abi.sq_batch_tables(_ptr(lengths, i32, "lengths"), _ptr(past, i32, "past", B), B, rows,
                             _ptr(cu_seqlens, i32, "cu_seqlens", B + 1), _ptr(cu_blocks, i32, "cu_blocks", B + 1),
                             _ptr(positions, i32, "positions"), _ptr(block_req, i32, "block_req"),
                             _ptr(slot_ids, i32, "slot_ids", B), _ptr(slot_used, torch.uint8, "slot_used"), n_slots,
                             _ptr(slot_out, i32, "slot_out", B), _ptr(used_out, torch.uint8, "used_out", n_slots),
                             _ptr(status, i32, "status", 1), _stream(stream))


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

    def build(self, lengths, past=None, slot_ids=None, slot_used=None, status=None, stream=None) -> "BatchTables":
        """Fill the tables from lengths (int32 [B]); requests with slot_ids < 0
        take free slots of the pool, in place in slot_ids and slot_used."""
        batch_tables(lengths, past, self.cu_seqlens, self.cu_blocks, self.positions, self.block_req,
                     slot_ids=slot_ids, slot_used=slot_used, slot_out=slot_ids, used_out=slot_used, status=status,
                     stream=stream)
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
    dev = _same_device(q, k, q_out, k_out, q_weight, k_weight, positions, n_rows)
    rows, hq, d = q.shape
    hk = k.shape[1]
    desc = _abi.NormDesc(_abi.SQ_NORM_L2 if mode == "l2" else _abi.SQ_NORM_RMS, float(eps), float(q_scale),
                         int(rot_dim), int(bool(interleaved)), float(base))
    with torch.cuda.device(dev):
        qp, qs = row_ptr(q, q.dtype, "q", (rows, hq, d), dev)
        kp, ks = row_ptr(k, q.dtype, "k", (rows, hk, d), dev)
        f32, i32 = torch.float32, torch.int32
        _abi.sq_qk_norm(desc, qp, kp, qs, ks, DTYPES[q.dtype], _ptr(q_weight, f32, "q_weight", d),
                        _ptr(k_weight, f32, "k_weight", d), _ptr(positions, i32, "positions", rows),
                        _ptr(q_out, q_out.dtype, "q_out", rows * hq * d), _ptr(k_out, q_out.dtype, "k_out", rows * hk * d),
                        DTYPES[q_out.dtype], rows, _ptr(n_rows, i32, "n_rows", 1), hq, hk, d, _stream(stream))

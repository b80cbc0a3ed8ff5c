"""Refusals of the ragged-batch calls on the host, before any launch (no GPU
needed), and the plain definitions the GPU tests rest on."""
import ctypes

import numpy as np
import pytest
import torch

from quantized_linear_attention_sq_b200 import _abi, build
from tests import ragged_ref as ref


@pytest.fixture(scope="module")
def L():
    build.build()
    return _abi.lib()


A = 1 << 20  # an aligned address nothing reads: every call below is refused


def _tables(L, **kw):
    a = dict(lengths=A, past=None, B=4, rows=256, cu=A, cb=A, pos=A, req=A, slot=None, used=None, n_slots=0,
             slot_out=None, used_out=None, status=None)
    a.update(kw)
    return L.sq_batch_tables(*a.values(), None), L.sq_last_error().decode()


@pytest.mark.parametrize("kw,code,needle", [
    (dict(B=-1), _abi.SQ_ERR_INVALID_ARG, "B, max_rows"),
    (dict(rows=-1), _abi.SQ_ERR_INVALID_ARG, "B, max_rows"),
    (dict(n_slots=-2), _abi.SQ_ERR_INVALID_ARG, "n_slots"),
    (dict(B=_abi.SQ_RAGGED_MAX_REQUESTS + 1), _abi.SQ_ERR_UNSUPPORTED, "requests"),
    (dict(rows=(1 << 30) + 1), _abi.SQ_ERR_UNSUPPORTED, "max_rows"),
    (dict(n_slots=(1 << 30) + 1), _abi.SQ_ERR_UNSUPPORTED, "n_slots"),
    (dict(lengths=None), _abi.SQ_ERR_INVALID_ARG, "lengths is NULL"),
    (dict(lengths=A + 2), _abi.SQ_ERR_INVALID_ARG, "lengths is not"),
    (dict(cu=None), _abi.SQ_ERR_INVALID_ARG, "cu_seqlens"),
    (dict(cb=None), _abi.SQ_ERR_INVALID_ARG, "cu_blocks"),
    (dict(req=None), _abi.SQ_ERR_INVALID_ARG, "block_req"),
    (dict(pos=A + 1), _abi.SQ_ERR_INVALID_ARG, "positions"),
    (dict(slot=A), _abi.SQ_ERR_INVALID_ARG, "slot_out"),
    (dict(slot=A, slot_out=A, n_slots=4), _abi.SQ_ERR_INVALID_ARG, "used"),
    (dict(used=A, n_slots=4), _abi.SQ_ERR_INVALID_ARG, "slot_ids"),
])
def test_tables_refusals(L, kw, code, needle):
    rc, msg = _tables(L, **kw)
    assert rc == code and needle in msg


def _norm(L, desc=None, **kw):
    d = dict(mode=_abi.SQ_NORM_L2, eps=1e-6, q_scale=1.0, rot=0, inter=0, base=1e4)
    d.update(desc or {})
    a = dict(q=A, k=A, qs=512, ks=512, tin=_abi.SQ_BF16, qw=None, kw=None, pos=A, qo=2 * A, ko=2 * A,
             tout=_abi.SQ_BF16, rows=8, n_rows=None, hq=4, hk=4, d=128)
    a.update(kw)
    return L.sq_qk_norm(ctypes.byref(_abi.NormDesc(*d.values())), *a.values(), None), L.sq_last_error().decode()


@pytest.mark.parametrize("desc,kw,code,needle", [
    (dict(mode=2), {}, _abi.SQ_ERR_INVALID_ARG, "mode"),
    (dict(eps=-1.0), {}, _abi.SQ_ERR_INVALID_ARG, "eps"),
    (dict(eps=float("nan")), {}, _abi.SQ_ERR_INVALID_ARG, "eps"),
    (dict(q_scale=float("inf")), {}, _abi.SQ_ERR_INVALID_ARG, "q_scale"),
    (dict(rot=3), {}, _abi.SQ_ERR_INVALID_ARG, "rot_dim"),
    (dict(rot=130), {}, _abi.SQ_ERR_INVALID_ARG, "rot_dim"),
    (dict(rot=64, base=0.0), {}, _abi.SQ_ERR_INVALID_ARG, "base"),
    (dict(rot=64), dict(pos=None), _abi.SQ_ERR_INVALID_ARG, "positions"),
    ({}, dict(tin=3), _abi.SQ_ERR_INVALID_ARG, "element type"),
    ({}, dict(tout=-1), _abi.SQ_ERR_INVALID_ARG, "element type"),
    ({}, dict(d=96), _abi.SQ_ERR_UNSUPPORTED, "d must be"),
    ({}, dict(rows=-1), _abi.SQ_ERR_INVALID_ARG, "rows"),
    ({}, dict(rows=(1 << 30) + 1), _abi.SQ_ERR_UNSUPPORTED, "rows"),
    ({}, dict(q=None), _abi.SQ_ERR_INVALID_ARG, "q is NULL"),
    ({}, dict(q=A + 8), _abi.SQ_ERR_INVALID_ARG, "q is not 16-byte"),
    ({}, dict(qs=500), _abi.SQ_ERR_INVALID_ARG, "below"),
    ({}, dict(ks=516), _abi.SQ_ERR_INVALID_ARG, "multiple of 16"),
    ({}, dict(qo=A), _abi.SQ_ERR_INVALID_ARG, "overlaps"),
    ({}, dict(ko=A + 4), _abi.SQ_ERR_INVALID_ARG, "k_out"),
])
def test_norm_refusals(L, desc, kw, code, needle):
    rc, msg = _norm(L, desc, **kw)
    assert rc == code and needle in msg


def test_norm_without_rows_or_heads_is_a_no_op(L):
    assert _norm(L, rows=0)[0] == _abi.SQ_OK
    assert _norm(L, hq=0, hk=0)[0] == _abi.SQ_OK


def test_ragged_needs_a_handle(L):
    t = _abi.RaggedTables(A, A, A, None)
    rc = L.sq_prefill_ragged(None, A, A, A, A, 128, 128, 128, _abi.SQ_BF16, A, A, A, ctypes.byref(t), None, 1, 1, 1,
                             None, 0, None)
    assert rc == _abi.SQ_ERR_INVALID_ARG and "handle" in L.sq_last_error().decode()
    n = ctypes.c_uint64()
    assert L.sq_ragged_workspace_bytes(None, _abi.SQ_BF16, 1, 1, 1, ctypes.byref(n)) == _abi.SQ_ERR_INVALID_ARG


def test_python_wrappers_refuse_cpu_tensors():
    from quantized_linear_attention_sq_b200 import ragged
    i = lambda n: torch.zeros(n, dtype=torch.int32)  # noqa: E731
    with pytest.raises(ValueError, match="CUDA"):
        ragged.batch_tables(i(2), None, i(3), i(3), i(64), i(3))
    x = torch.zeros(4, 2, 128)
    with pytest.raises(ValueError, match="CUDA"):
        ragged.qk_norm(x, x, x, x)
    with pytest.raises(ValueError, match="mode"):
        ragged.qk_norm(x, x, x, x, mode="layer")
    with pytest.raises(ValueError, match="q must be"):
        ragged.qk_norm(x.double(), x, x, x)


# ------------------------------------------------- the plain definitions
def test_reference_tables_by_hand():
    t = ref.tables([3, 0, -2, 70, 1], [5, 1, 1, 0, 9], 80, [-1, 4, -1, -1, 0], [1, 0, 0, 1, 1, 0])
    assert t["cu_seqlens"] == [0, 3, 3, 3, 73, 74]
    assert t["cu_blocks"] == [0, 1, 1, 1, 3, 4]
    assert t["positions"][:5] == [5, 6, 7, 0, 1] and t["positions"][72:] == [69, 9]
    assert t["block_req"] == [0, 3, 3, 4]
    assert t["slot_out"] == [1, 4, 2, 5, 0] and t["used_out"] == [1, 1, 1, 1, 1, 1] and t["status"] == 0


def test_reference_tables_cut_and_short_of_slots():
    t = ref.tables([60, 60, 60], None, 100, [-1, -1, -1], [0, 1])
    assert t["cu_seqlens"] == [0, 60, 100, 100] and t["cu_blocks"] == [0, 1, 2, 2]
    assert t["slot_out"] == [0, -1, -1]
    assert t["status"] == _abi.SQ_STATUS_TRUNCATED | _abi.SQ_STATUS_NO_SLOT


@pytest.mark.parametrize("channel", [False, True])
def test_reference_recurrence_is_the_textbook_step(channel):
    from tests.helpers import random_inputs, textbook_step
    rng = np.random.default_rng(3)
    hv, hk, d, n = 4, 2, 8, 5
    S = rng.standard_normal((1, hv, d, d))
    steps = [random_inputs(rng, 1, hv, hk, d, int(channel)) for _ in range(n)]
    rows = [torch.from_numpy(np.concatenate([s[x] for s in steps])) for x in range(5)]
    o, S1 = ref.recurrence(*rows, torch.from_numpy(S[0]))
    for t, (q, k, v, beta, g) in enumerate(steps):
        S, ot = textbook_step(S, q, k, v, beta, g, hk)
        assert np.allclose(o[t].numpy(), ot[0], rtol=1e-12, atol=1e-14)
    assert np.allclose(S1.numpy(), S[0], rtol=1e-12, atol=1e-14)


def test_reference_norm_turns_pairs():
    x = torch.tensor([[[3.0, 4.0, 0.0, 0.0]]], dtype=torch.float64)
    y = ref.norm(x, "l2", 0.0, None, 1.0, torch.tensor([1]), 2, 10.0, True)
    c, s = np.cos(1.0), np.sin(1.0)
    assert np.allclose(y[0, 0].numpy(), [0.6 * c - 0.8 * s, 0.8 * c + 0.6 * s, 0, 0])
    y = ref.norm(x, "rms", 0.0, None, 2.0, torch.tensor([1]), 4, 1.0, False)
    assert np.allclose(y[0, 0].numpy(), np.array([3 * c, 4 * c, 3 * s, 4 * s]) * 2 / 2.5)

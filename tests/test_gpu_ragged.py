"""GPU tests of the ragged-batch operators against their 64-bit definitions.

Tolerances (relative L2 per request and head, derived, not fitted):
- A row of the gated delta rule sums D terms through a chain of at most
  D / 8 + 8 + 3 <= 27 fp32 roundings and applies 4 more; roundings to nearest
  have no bias, so a row's relative error is about sqrt(31) 2^-24 < 8 2^-24,
  and the update is a contraction (gates <= 1, unit keys, beta <= 1): errors
  of earlier rows do not grow and add as independent ones,
  8 2^-24 sqrt(1 + n) after n rows.
- The stored outputs add half a step of their type, finfo.eps / 2.
- A norm sums d squares (<= 8 + 4 roundings, halved by the root), and
  multiplies 5 more times; the rotation adds 3: |error| <= 16 2^-24 of the
  head's largest value, plus half a step of the output type.
"""
import math

import pytest
import torch

from quantized_linear_attention_sq_b200 import _abi
from tests import ragged_ref as ref

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    from quantized_linear_attention_sq_b200 import build
    build.build()
    torch.cuda.init()


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


# ------------------------------------------------------------------ tables
def _check_tables(lengths, past, rows, slot_ids=None, used=None, in_place=False):
    from quantized_linear_attention_sq_b200.ragged import batch_tables
    B = len(lengths)
    mark = -77
    full = lambda n: torch.full((n,), mark, dtype=torch.int32, device="cuda")  # noqa: E731
    cu, cb, pos, req = full(B + 1), full(B + 1), full(rows), full(rows // 64 + B)
    status = i32([0])
    want = ref.tables(lengths, past, rows, slot_ids, used)
    kw = {}
    if slot_ids is not None:
        s, u = i32(slot_ids), torch.tensor(used, dtype=torch.uint8, device="cuda")
        so, uo = (s, u) if in_place else (full(B), torch.full((len(used),), 9, dtype=torch.uint8, device="cuda"))
        kw = dict(slot_ids=s, slot_used=u, slot_out=so, used_out=uo)
    batch_tables(i32(lengths), None if past is None else i32(past), cu, cb, pos, req, status=status, **kw)
    assert cu.tolist() == want["cu_seqlens"] and cb.tolist() == want["cu_blocks"]
    n, m = len(want["positions"]), len(want["block_req"])
    assert pos.tolist() == want["positions"] + [mark] * (rows - n)
    assert req.tolist() == want["block_req"] + [mark] * (rows // 64 + B - m)
    if slot_ids is not None:
        assert so.tolist() == want["slot_out"] and uo.tolist() == want["used_out"]
    assert status.item() == want["status"]


@pytest.mark.parametrize("lengths,past,rows", [
    ([1], None, 1), ([0], [3], 0), ([5], [7], 64), ([64, 63, 65, 0, 128, -4], [0, 1, 2, 3, 4, 5], 400),
    ([300, 300], [0, 9], 400), ([0, 0, 0], None, 10), ([2 ** 31 - 1, 2 ** 31 - 1], [1, 1], 3000),
])
def test_tables_small(lengths, past, rows):
    _check_tables(lengths, past, rows)


@pytest.mark.parametrize("B,hi", [(1023, 3), (1024, 1), (1025, 70), (2500, 9), (3000, 150)])
def test_tables_many_requests(B, hi):
    gen = torch.Generator().manual_seed(B)
    lengths = torch.randint(0, hi + 1, (B,), generator=gen).tolist()
    past = torch.randint(0, 5000, (B,), generator=gen).tolist()
    _check_tables(lengths, past, sum(lengths) + 11)


@pytest.mark.parametrize("B,n_slots,in_place", [(1, 1, True), (5, 3, False), (40, 4097, False), (700, 9001, True),
                                                (3000, 2000, False)])
def test_slots(B, n_slots, in_place):
    gen = torch.Generator().manual_seed(n_slots)
    used = (torch.rand(n_slots, generator=gen) < 0.7).int().tolist()
    taken = [s for s, u in enumerate(used) if u]
    slots = [taken[b % len(taken)] if taken and b % 3 else -1 for b in range(B)]
    _check_tables([1] * B, None, B, slots, used, in_place)


def test_tables_most_requests():
    """The largest batch: offsets by prefix sums on the host."""
    from quantized_linear_attention_sq_b200.ragged import BatchTables
    B = _abi.SQ_RAGGED_MAX_REQUESTS
    gen = torch.Generator().manual_seed(1)
    n = torch.randint(0, 200, (B,), generator=gen)
    rows = int(n.sum())
    used = torch.zeros(B, dtype=torch.uint8, device="cuda")
    slots = torch.full((B,), -1, dtype=torch.int32, device="cuda")
    t = BatchTables.empty(B, rows).build(n.int().cuda(), slot_ids=slots, slot_used=used)
    cu = torch.cat([torch.zeros(1, dtype=torch.int64), n.cumsum(0)])
    req = torch.repeat_interleave(torch.arange(B), n)
    assert torch.equal(t.cu_seqlens.cpu().long(), cu) and t.n_rows.item() == rows
    assert torch.equal(t.positions.cpu().long(), torch.arange(rows) - cu[req])
    assert torch.equal(slots.cpu().long(), torch.arange(B)) and bool(used.all())
    with pytest.raises(_abi.SQError):
        BatchTables.empty(B + 1, 64).build(torch.ones(B + 1, dtype=torch.int32, device="cuda"))


def test_tables_of_an_empty_batch():
    from quantized_linear_attention_sq_b200.ragged import BatchTables
    t = BatchTables.empty(0, 64)
    t.cu_seqlens.fill_(5)
    t.cu_blocks.fill_(5)
    t.build(i32([]))
    assert t.cu_seqlens.tolist() == [0] and t.cu_blocks.tolist() == [0]


# ------------------------------------------------------------------- norms
def _check_norm(rows, hq, hk, d, mode, rot, inter, tin, tout, weight=False, far=0, pad=0, eps=1e-6, n=None):
    from quantized_linear_attention_sq_b200.ragged import qk_norm
    gen = torch.Generator(device="cuda").manual_seed(rows + d + rot)
    x = (torch.randn((rows, (hq + hk) * d + pad), device="cuda", generator=gen) * 3).to(tin)
    q, k = x[:, :hq * d].unflatten(1, (hq, d)), x[:, hq * d:(hq + hk) * d].unflatten(1, (hk, d))
    wq, wk = (1 + 0.2 * torch.randn((2, d), device="cuda", generator=gen)).unbind(0) if weight else (None, None)
    pos = (far + torch.arange(rows, device="cuda")).int() if rot else None
    qo = torch.full((rows, hq, d), 7.0, dtype=tout, device="cuda")
    ko = torch.full((rows, hk, d), 7.0, dtype=tout, device="cuda")
    qk_norm(q, k, qo, ko, mode=mode, eps=eps, q_weight=wq, k_weight=wk, q_scale=d ** -0.5, positions=pos, rot_dim=rot,
            base=10000.0, interleaved=inter, n_rows=None if n is None else i32([n]))
    for y, src, w, scale in ((qo, q, wq, d ** -0.5), (ko, k, wk, 1.0)):
        if not src.numel():
            continue
        live = rows if n is None else n
        want = ref.norm(src[:live], mode, eps, w, scale, pos[:live] if rot else None, rot, 10000.0, inter)
        top = want.abs().amax(-1, keepdim=True)
        # fp16 steps below its normal range are 2^-24 apart
        tol = 16 * U * top + torch.finfo(tout).eps / 2 * want.abs() + (U if tout == torch.float16 else 0)
        assert ((y[:live].double() - want).abs() <= tol).all()
        assert (y[live:] == 7.0).all()


B16, F16, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.mark.parametrize("tin", [B16, F16, F32])
@pytest.mark.parametrize("tout", [B16, F16, F32])
@pytest.mark.parametrize("d,rot,inter", [(32, 32, False), (64, 0, False), (128, 64, True), (128, 64, False)])
def test_norm_types(tin, tout, d, rot, inter):
    _check_norm(33, 4, 2, d, "rms", rot, inter, tin, tout, weight=True, far=1000, pad=64)


@pytest.mark.parametrize("rot", [2, 6, 12, 16, 30, 48, 64])
@pytest.mark.parametrize("inter", [False, True])
def test_norm_rotary_widths(rot, inter):
    _check_norm(9, 3, 1, 64, "l2", rot, inter, F32, F32, far=17)


@pytest.mark.parametrize("rows,hq,hk,d", [(1, 1, 1, 32), (1, 5, 0, 128), (2, 0, 3, 64), (7, 3, 1, 128), (591, 2, 2, 32),
                                          (2400, 16, 16, 128), (5003, 12, 4, 64)])
def test_norm_shapes(rows, hq, hk, d):
    _check_norm(rows, hq, hk, d, "l2", d // 2, False, B16, F32)


def test_norm_far_positions():
    _check_norm(65, 2, 2, 128, "l2", 128, True, F32, F32, far=2 ** 31 - 70)


def test_norm_rows_behind_the_last():
    for n in (0, 1, 20, 33):
        _check_norm(33, 2, 2, 64, "l2", 64, False, B16, B16, n=n)


def test_norm_zero_rows_and_nan():
    from quantized_linear_attention_sq_b200.ragged import qk_norm
    x = torch.randn(3, 2, 64, device="cuda")
    x[0] = 0
    x[1, 0, 3] = float("nan")
    y, z = torch.empty_like(x), torch.empty_like(x)
    qk_norm(x, x.clone(), y, z)
    assert (y[0] == 0).all() and y[1, 0].isnan().all()
    assert y[1, 1].isfinite().all() and y[2].isfinite().all() and torch.equal(z[2], y[2])


# --------------------------------------------------------- gated delta rule
class Batch:
    """A ragged batch with garbage rows behind its last request and guard slots."""

    def __init__(self, lengths, hv=4, hk=2, d=128, channel=False, dtype=B16, packed=False, past=None, extra=5, seed=0,
                 slots=None, gates=None, pad=0, max_len=None):
        from quantized_linear_attention_sq_b200.ragged import BatchTables
        from quantized_linear_attention_sq_b200.state import StatePool
        gen = torch.Generator(device="cuda").manual_seed(seed + sum(lengths) + d)
        rnd = lambda *s: torch.randn(s, device="cuda", generator=gen)  # noqa: E731
        B = len(lengths)
        self.lengths, self.B, self.rows = lengths, B, sum(lengths) + extra
        self.past = [(b % 3) * 7 for b in range(B)] if past is None else past
        self.n_slots = B + 3
        self.slots = [(b * 5 + 2) % self.n_slots for b in range(B)] if slots is None else slots
        if slots is None and len(set(self.slots)) < B:
            self.slots = list(range(B))
        unit = lambda x: x / x.square().sum(-1, keepdim=True).sqrt()  # noqa: E731
        x = torch.zeros((self.rows, (2 * hk + hv) * d + pad), device="cuda", dtype=dtype)
        x[:, :hk * d] = unit(rnd(self.rows, hk, d) + 0.5 * rnd(1, hk, d)).flatten(1)
        x[:, hk * d:2 * hk * d] = unit(rnd(self.rows, hk, d) + 0.5 * rnd(1, hk, d)).flatten(1)
        x[:, 2 * hk * d:(2 * hk + hv) * d] = rnd(self.rows, hv * d)
        x[sum(lengths):] = float("nan")   # rows of no request are never read into a result
        self.q = x[:, :hk * d].unflatten(1, (hk, d))
        self.k = x[:, hk * d:2 * hk * d].unflatten(1, (hk, d))
        self.v = x[:, 2 * hk * d:(2 * hk + hv) * d].unflatten(1, (hv, d))
        self.beta = torch.sigmoid(rnd(self.rows, hv))
        hl = 2.0 ** (8 * torch.rand((hv, d) if channel else (hv,), device="cuda", generator=gen))
        self.g = torch.exp2(-torch.exp(0.3 * rnd(self.rows, *hl.shape)) / hl)
        if gates is not None:
            gates(self.g)
        self.o = torch.full((self.rows, hv, d), 3.0, device="cuda", dtype=dtype)
        kind = _abi.SQ_GATE_KEY_CHANNEL if channel else _abi.SQ_GATE_HEAD
        self.fp = StatePool(self.n_slots, hv, hk, d, kind, _abi.SQ_FMT_FP32)
        self.S0 = 0.2 * rnd(self.n_slots, hv, d, d)
        self.h, self.pool = self.fp, self.S0.clone()
        if packed:
            import numpy as np
            from tests.helpers import random_calib
            cal = random_calib(np.random.default_rng(seed + d), hv, d, int(channel))
            self.h = StatePool(self.n_slots, hv, hk, d, kind, _abi.SQ_FMT_PACKED, *cal)
            self.pool = self.h.new_pool()
            self.h.quantize_state(self.pool, self.S0)
            self.h.dequantize_state(self.pool, self.S0)
            self.packed0 = self.pool.clone()
            assert self.h.get_status() in (0, _abi.SQ_STATUS_SATURATED)
        self.tables = BatchTables.empty(B, self.rows).build(i32(lengths), i32(self.past))
        self.slot_ids = i32(self.slots)
        self.max_len = max_len

    def run(self, **kw):
        a = dict(slot_ids=self.slot_ids, max_len=self.max_len)
        a.update(kw)
        self.h.prefill_ragged(self.pool, self.q, self.k, self.v, self.beta, self.g, self.o, self.tables, **a)
        torch.cuda.synchronize()
        return self

    def expected(self):
        """[(o, S)] of every request in fp64."""
        out, at = [], 0
        for b, n in enumerate(self.lengths):
            r = slice(at, at + n)
            s = self.slots[b]
            S = self.S0[s] if self.past[b] > 0 and 0 <= s < self.n_slots else torch.zeros_like(self.S0[0])
            out.append(ref.recurrence(self.q[r], self.k[r], self.v[r], self.beta[r], self.g[r], S))
            at += n
        return out

    def close(self):
        self.fp.close()
        self.h.close()


def rel(a, b):
    """Largest relative L2 error over the leading head axis."""
    a, b = a.double().flatten(1), b.double().flatten(1)
    return ((a - b).norm(dim=1) / b.norm(dim=1).clamp(min=1e-30)).max().item()


def check_rows(bt, skip=()):
    at = 0
    for b, (o, S) in enumerate(bt.expected()):
        n = bt.lengths[b]
        tol = 8 * U * math.sqrt(1 + n)
        if b not in skip:
            if n:
                got = bt.o[at:at + n]
                # o = S^T q may cancel: its fp32 part is held to the size of |S| |q| <= 4 |o| rms
                assert rel(got.transpose(0, 1), o.transpose(0, 1)) <= torch.finfo(bt.o.dtype).eps / 2 + 4 * tol, (b, n)
            if n or bt.past[b] <= 0:
                state = bt.pool[bt.slots[b]]
                if S.abs().max() == 0:
                    assert (state == 0).all()
                else:
                    assert rel(state, S) <= tol, (b, n)
        at += n
    assert (bt.o[at:] == 3.0).all()


LENGTHS = [1, 0, 2, 17, 63, 64, 65, 0, 130, 5]


@pytest.mark.parametrize("d", [32, 64, 128])
@pytest.mark.parametrize("channel", [False, True])
@pytest.mark.parametrize("dtype", [B16, F16, F32])
def test_ragged_rows(d, channel, dtype):
    bt = Batch(LENGTHS, d=d, channel=channel, dtype=dtype, pad=64)
    try:
        check_rows(bt.run())
        # slots of no request, and of requests without rows that go on
        free = [s for s in range(bt.n_slots) if s not in bt.slots]
        free += [bt.slots[b] for b, n in enumerate(LENGTHS) if n == 0 and bt.past[b] > 0]
        assert torch.equal(bt.pool[free], bt.S0[free])
        assert bt.h.get_status() == 0
    finally:
        bt.close()


@pytest.mark.parametrize("hv,hk", [(1, 1), (3, 1), (8, 2), (32, 16)])
def test_ragged_heads(hv, hk):
    bt = Batch([70, 1, 128, 3], hv=hv, hk=hk)
    try:
        check_rows(bt.run())
    finally:
        bt.close()


@pytest.mark.parametrize("d,channel", [(32, False), (64, True), (128, False), (128, True)])
def test_ragged_packed_is_the_fp32_run_quantized(d, channel):
    """A packed pool takes the state an fp32 pool takes, quantized by sq_quantize_state, bit for bit."""
    lengths = [1, 0, 4, 90, 200, 0]
    a = Batch(lengths, d=d, channel=channel, packed=True)
    try:
        a.run()
        S = a.S0.clone()
        o = torch.full_like(a.o, 3.0)
        a.fp.prefill_ragged(S, a.q, a.k, a.v, a.beta, a.g, o, a.tables, slot_ids=a.slot_ids)
        assert torch.equal(o, a.o)
        want = a.packed0.clone()
        ran = [b for b in range(a.B) if a.lengths[b] or a.past[b] <= 0]
        a.h.quantize_state(want, S[[a.slots[b] for b in ran]].contiguous(), i32([a.slots[b] for b in ran]))
        torch.cuda.synchronize()
        assert torch.equal(want, a.pool)
    finally:
        a.close()


def test_ragged_more_requests_than_are_ranked():
    """Requests past the count up to which the longest start first, most of them short."""
    lengths = [(b * 7) % 5 for b in range(300)]
    lengths[3], lengths[150], lengths[299] = 90, 130, 64
    bt = Batch(lengths, hv=2, hk=1)
    try:
        check_rows(bt.run())
    finally:
        bt.close()


@pytest.mark.parametrize("n", [255, 256])
def test_ragged_ranked_requests(n):
    lengths = [10 + (b * 37) % 23 for b in range(n)]
    bt = Batch(lengths, hv=1, hk=1)
    try:
        check_rows(bt.run())
    finally:
        bt.close()


def test_ragged_longer_than_max_len():
    """max_len chooses the kernels; a request that passes it is still right."""
    for max_len in (1, 9, 10, 40):
        bt = Batch([1, 77, 0, 200, 9], max_len=max_len)
        try:
            check_rows(bt.run())
        finally:
            bt.close()


@pytest.mark.parametrize("packed", [False, True])
def test_ragged_on_another_stream(packed):
    """A call on a side stream, with the workspace that the call allocates."""
    bt = Batch([100, 3, 64, 1], packed=packed)
    try:
        torch.cuda.synchronize()
        side = torch.cuda.Stream()
        bt.run(stream=side)
        first = bt.o.clone(), bt.pool.clone()
        bt.pool.copy_(bt.packed0 if packed else bt.S0)
        torch.cuda.synchronize()
        bt.run(stream=side.cuda_stream)
        assert torch.equal(first[0], bt.o) and torch.equal(first[1], bt.pool)
        if not packed:
            check_rows(bt)
    finally:
        bt.close()


def test_ragged_nan_gate_and_beta():
    for name in ("g", "beta"):
        bt = Batch([100, 40, 3], past=[0, 0, 0])
        try:
            getattr(bt, name)[90, 1] = float("nan")   # request 0, row 90, head 1
            bt.run()
            check_rows(bt, skip=(0,))
            want, S = bt.expected()[0]
            assert rel(bt.o[:64].transpose(0, 1), want[:64].transpose(0, 1)) <= 2.0 ** -8 + 32 * U * 10
            others = [0, 2, 3]
            assert rel(bt.pool[bt.slots[0]][others], S[others]) <= 8 * U * math.sqrt(101)
            assert bt.pool[bt.slots[0]][1].isnan().any()
            assert bt.h.get_status() & _abi.SQ_STATUS_NAN
        finally:
            bt.close()


def test_ragged_guard_bytes_around_every_output():
    """o and the pool lie between guard regions that no call touches."""
    pad = 1024
    for packed, lengths in ((False, [130, 1, 65]), (True, [70, 0, 9, 129])):
        bt = Batch(lengths, packed=packed, extra=0)
        try:
            o = torch.full((bt.o.numel() + 2 * pad,), 5.0, device="cuda", dtype=bt.o.dtype)
            pool = torch.full((bt.pool.numel() + 2 * pad,), 5, device="cuda", dtype=bt.pool.dtype)
            pool[pad:-pad] = bt.pool.flatten()
            bt.h.prefill_ragged(pool[pad:-pad], bt.q, bt.k, bt.v, bt.beta, bt.g, o[pad:-pad], bt.tables,
                                slot_ids=bt.slot_ids)
            torch.cuda.synchronize()
            for x in (o, pool):
                assert (x[:pad] == 5).all() and (x[-pad:] == 5).all()
            bt.run()
            assert torch.equal(o[pad:-pad].view_as(bt.o), bt.o)
            assert torch.equal(pool[pad:-pad].view_as(bt.pool), bt.pool)
        finally:
            bt.close()


def test_ragged_gates_at_and_past_their_bounds():
    def gates(g):
        g[3::7] = 0.0
        g[5::11] = 1.0
        g[6::13] = 1.5
        g[8::17] = -0.25
        g[9::19] = 1e-30
    for channel in (False, True):
        bt = Batch([200, 65, 3], channel=channel, gates=gates)
        try:
            check_rows(bt.run())
        finally:
            bt.close()


def test_ragged_bad_slots():
    bt = Batch([3, 100, 70], slots=[-1, 1, 99])
    try:
        bt.run()
        check_rows(bt, skip=(0, 2))
        assert (bt.o[:3] == 0).all() and (bt.o[103:173] == 0).all()
        keep = [0, 2, 3, 4, 5]
        assert torch.equal(bt.pool[keep], bt.S0[keep])
        assert bt.h.get_status() == _abi.SQ_STATUS_BAD_SLOT
    finally:
        bt.close()


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_ragged_bad_values_stay_in_their_request(bad):
    bt = Batch([100, 3, 100, 64], past=[0, 0, 0, 5])
    try:
        bt.v[170, 1, 5] = bad    # request 2, row 67
        bt.run()
        check_rows(bt, skip=(2,))
        want, S = bt.expected()[2]
        early = bt.o[103:103 + 64].transpose(0, 1)
        assert rel(early, want[:64].transpose(0, 1)) <= 2.0 ** -8 + 32 * U * 9
        assert not bt.o[170:203, 1, 5].isfinite().any()
        assert bt.h.get_status() & _abi.SQ_STATUS_NAN
    finally:
        bt.close()


def test_ragged_refusals():
    bt = Batch([4, 70])
    try:
        a = dict(slot_ids=bt.slot_ids)
        call = lambda **kw: bt.h.prefill_ragged(*[kw.get(x, y) for x, y in (  # noqa: E731
            ("pool", bt.pool), ("q", bt.q), ("k", bt.k), ("v", bt.v), ("beta", bt.beta), ("g", bt.g), ("o", bt.o),
            ("tables", bt.tables))], **{**a, **kw.get("more", {})})
        with pytest.raises(ValueError, match="q must be"):
            call(q=bt.q.double())
        with pytest.raises(ValueError, match="k must be"):
            call(k=bt.k.float())
        with pytest.raises(ValueError, match="v has shape"):
            call(v=bt.v[:-1])
        with pytest.raises(ValueError, match="contiguous"):
            call(q=bt.q.flip(2).transpose(1, 2).contiguous().transpose(1, 2))
        with pytest.raises(ValueError, match="beta has"):
            call(beta=bt.beta[1:])
        with pytest.raises(ValueError, match="slot_ids has"):
            call(more=dict(slot_ids=bt.slot_ids[:1]))
        with pytest.raises(ValueError, match="pool has"):
            call(pool=bt.pool[1:])
        wide = torch.zeros((bt.rows, 2 * 128 + 4), dtype=B16, device="cuda")
        with pytest.raises(_abi.SQError, match="multiple of 16"):
            call(q=wide[:, :256].unflatten(1, (2, 128)))
        with pytest.raises(_abi.SQError, match="aligned"):
            call(q=torch.zeros(bt.rows * 256 + 4, dtype=B16, device="cuda")[4:].view(bt.rows, 2, 128))
        need = bt.h.ragged_workspace_bytes(2, bt.rows)
        if need:
            with pytest.raises(_abi.SQError, match="workspace has"):
                call(more=dict(workspace=torch.empty(need - 16, dtype=torch.uint8, device="cuda")))
        assert (bt.o == 3.0).all() and torch.equal(bt.pool, bt.S0)
    finally:
        bt.close()


def test_ragged_empty_batch_and_no_rows():
    bt = Batch([0, 0], past=[0, 4], extra=0)
    try:
        bt.run()
        assert (bt.pool[bt.slots[0]] == 0).all() and torch.equal(bt.pool[bt.slots[1]], bt.S0[bt.slots[1]])
        from quantized_linear_attention_sq_b200.ragged import BatchTables
        e = BatchTables.empty(0, 0).build(i32([]), i32([]))
        bt.h.prefill_ragged(bt.pool, bt.q, bt.k, bt.v, bt.beta, bt.g, bt.o, e)
        torch.cuda.synchronize()
    finally:
        bt.close()


def test_ragged_in_a_graph_and_beside_another_stream():
    """A captured call replays on new inputs, and two calls with workspaces of
    their own may run at once."""
    lengths = [300, 1, 64, 129]
    a, b, c = (Batch(lengths, hv=8, hk=4, seed=s) for s in (1, 2, 3))
    try:
        ws = [x.h.new_ragged_workspace(x.B, x.rows) for x in (a, b)]
        a.run(workspace=ws[0])
        first = a.o.clone(), a.pool.clone()
        check_rows(a)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            a.h.prefill_ragged(a.pool, a.q, a.k, a.v, a.beta, a.g, a.o, a.tables, slot_ids=a.slot_ids, workspace=ws[0])
        for src in (c, None):   # other inputs, then the first ones again
            if src is None:
                torch.manual_seed(0)
                src = Batch(lengths, hv=8, hk=4, seed=1)
            for x in ("q", "k", "v", "beta", "g"):
                getattr(a, x).copy_(getattr(src, x))
            a.S0.copy_(src.S0)
            a.pool.copy_(src.S0)
            side = torch.cuda.Stream()
            side.wait_stream(torch.cuda.current_stream())
            b.pool.copy_(b.S0)
            with torch.cuda.stream(side):
                b.h.prefill_ragged(b.pool, b.q, b.k, b.v, b.beta, b.g, b.o, b.tables, slot_ids=b.slot_ids,
                                   workspace=ws[1])
            graph.replay()
            torch.cuda.synchronize()
            check_rows(a)
            check_rows(b)
        assert torch.equal(first[0], a.o) and torch.equal(first[1], a.pool)
    finally:
        for x in (a, b, c):
            x.close()


def test_serving_loop_together():
    """Lengths to tables and slots, norms at the positions, prompts and continued
    prompts into the pool, then decode steps on the same slots, against fp64."""
    from quantized_linear_attention_sq_b200.ragged import BatchTables, qk_norm
    from quantized_linear_attention_sq_b200.state import StatePool
    gen = torch.Generator(device="cuda").manual_seed(5)
    rnd = lambda *s: torch.randn(s, device="cuda", generator=gen)  # noqa: E731
    hv, hk, d, B, n_slots = 4, 2, 128, 5, 9
    sp = StatePool(n_slots, hv, hk, d, _abi.SQ_GATE_HEAD, _abi.SQ_FMT_FP32)
    try:
        pool = rnd(n_slots, hv, d, d)
        used = torch.tensor([1, 0, 0, 1, 0, 0, 0, 0, 1], dtype=torch.uint8, device="cuda")
        slots = torch.full((B,), -1, dtype=torch.int32, device="cuda")
        past, S = i32([0] * B), [torch.zeros(hv, d, d, device="cuda", dtype=torch.float64) for _ in range(B)]
        for lengths in ([70, 3, 129, 64, 0], [1, 200, 0, 5, 66]):
            rows = sum(lengths) + 30
            t = BatchTables.empty(B, rows).build(i32(lengths), past, slot_ids=slots, slot_used=used)
            assert slots.tolist() == [1, 2, 4, 5, 6] and used.tolist() == [1, 1, 1, 1, 1, 1, 1, 0, 1]
            x = rnd(rows, (2 * hk + hv) * d).to(B16)
            q, k = (x[:, i * hk * d:(i + 1) * hk * d].unflatten(1, (hk, d)) for i in (0, 1))
            v = x[:, 2 * hk * d:].unflatten(1, (hv, d))
            qn, kn = torch.zeros(rows, hk, d, dtype=B16, device="cuda"), torch.zeros(rows, hk, d, dtype=B16, device="cuda")
            qk_norm(q, k, qn, kn, positions=t.positions, rot_dim=64, n_rows=t.n_rows)
            beta, g = torch.sigmoid(rnd(rows, hv)), torch.exp2(-torch.rand(rows, hv, device="cuda", generator=gen) / 30)
            o = torch.zeros(rows, hv, d, dtype=B16, device="cuda")
            sp.prefill_ragged(pool, qn, kn, v, beta, g, o, t, slot_ids=slots)
            cu = t.cu_seqlens.tolist()
            for b in range(B):
                r = slice(cu[b], cu[b + 1])
                want, S[b] = ref.recurrence(qn[r], kn[r], v[r], beta[r], g[r], S[b])
                if lengths[b]:
                    assert rel(o[r].transpose(0, 1), want.transpose(0, 1)) <= 2.0 ** -8 + 32 * U * math.sqrt(300)
            past = (past + i32(lengths)).contiguous()
        for step in range(2):
            q, k = (rnd(B, hk, d).to(B16) for _ in range(2))
            qf, kf = torch.empty(B, hk, d, device="cuda"), torch.empty(B, hk, d, device="cuda")
            qk_norm(q, k, qf, kf, positions=past, rot_dim=64)
            v, beta = rnd(B, hv, d), torch.sigmoid(rnd(B, hv))
            g, o = torch.full((B, hv), 0.97, device="cuda"), torch.empty(B, hv, d, device="cuda")
            sp.decode_step(pool, qf, kf, v, beta, g, o, slot_ids=slots)
            for b in range(B):
                want, S[b] = ref.recurrence(*(y[b:b + 1] for y in (qf, kf, v, beta, g)), S[b])
                assert rel(o[b], want[0]) <= 32 * U * math.sqrt(300)
            past = past + 1
        for b in range(B):
            assert rel(pool[slots[b].item()], S[b]) <= 8 * U * math.sqrt(300)
        assert sp.get_status() == 0
    finally:
        sp.close()

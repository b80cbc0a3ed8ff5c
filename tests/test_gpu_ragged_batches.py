"""GPU tests of ragged batches: calls that the documentation allows beside
those of test_gpu_ragged.py."""
import math

import pytest
import torch

from quantized_linear_attention_sq_b200 import _abi
from tests.test_gpu_ragged import U, Batch, check_rows, i32, rel

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    from quantized_linear_attention_sq_b200 import build
    build.build()
    torch.cuda.init()


@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("B", [2, 5, 37, 256])
def test_a_request_is_the_same_alone_and_in_a_batch(B, packed):
    """A batch of several requests sorts them by length in shared memory before
    its first tile arrives there; one request does not. Both give the same
    bits, call after call (fresh and resumed states)."""
    from quantized_linear_attention_sq_b200.ragged import BatchTables
    lengths = [10 + (b * 53) % 90 for b in range(B)]
    bt = Batch(lengths, hv=2, hk=1, packed=packed, past=[b % 2 for b in range(B)], extra=0)
    try:
        start = bt.pool.clone()
        alone, o, at = start.clone(), torch.full_like(bt.o, 3.0), 0
        for b, n in enumerate(lengths):
            r = slice(at, at + n)
            t = BatchTables.empty(1, n).build(i32([n]), i32([bt.past[b]]))
            bt.h.prefill_ragged(alone, bt.q[r], bt.k[r], bt.v[r], bt.beta[r], bt.g[r], o[r], t,
                                slot_ids=i32([bt.slots[b]]))
            at += n
        for _ in range(5):
            bt.pool.copy_(start)
            bt.o.fill_(3.0)
            bt.run()
            assert torch.equal(bt.o, o) and torch.equal(bt.pool, alone)
        assert not bt.h.get_status() & ~_abi.SQ_STATUS_SATURATED
    finally:
        bt.close()


@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("lengths", [[1, 2, 5, 1], [200, 20, 3, 64], [1] * 400])
def test_a_wait_that_runs_out_leaves_whole_states(lengths, packed):
    """The first wait of (request 0, head 0) expects 16 bytes more than are
    loaded, under a limit of 2 ms: every copy lands, the wait runs out. That
    state keeps its bytes and its o is not written; whatever else was left
    out is whole too, and the next call is right again."""
    hv, B = 4, len(lengths)
    bt = Batch(lengths, hv=hv, hk=2, packed=packed, past=[3] * B)
    try:
        start = bt.pool.clone()
        bt.run()
        assert not bt.h.get_status() & ~_abi.SQ_STATUS_SATURATED
        o, pool = bt.o.clone(), bt.pool.clone()
        bt.pool.copy_(start)
        bt.o.fill_(3.0)
        bt.h.set_wait_limit(2_000_000)
        bt.h.test_stall_stages(16)
        bt.run()
        assert bt.h.get_status() & _abi.SQ_STATUS_TIMEOUT

        def records(p):
            if not packed:
                return p
            at = [bt.h.head_layout(h) for h in range(hv)]
            per_slot = p.view(bt.n_slots, -1)
            return [[per_slot[s, off:off + nb] for off, nb in at] for s in range(bt.n_slots)]

        got, old, new = records(bt.pool), records(start), records(pool)
        left, first = 0, 0
        for b, n in enumerate(lengths):
            s = bt.slots[b]
            for h in range(hv):
                rows, want = bt.o[first:first + n, h], o[first:first + n, h]
                if torch.equal(got[s][h], old[s][h]):
                    left += 1
                    assert (rows == 3.0).all()
                else:
                    assert torch.equal(got[s][h], new[s][h]) and torch.equal(rows, want)
            first += n
        assert torch.equal(got[bt.slots[0]][0], old[bt.slots[0]][0])
        # the tiles of one CTA: (0, 0) and, row by row, every further one of its walk
        assert 1 <= left <= 1 + B * hv // 128
        if B * hv <= 128:
            assert left == 1
        free = [s for s in range(bt.n_slots) if s not in bt.slots]
        for s in free:
            assert all(torch.equal(x, y) for x, y in zip(got[s], old[s]))

        bt.h.test_stall_stages(0)
        bt.h.set_wait_limit(2_000_000_000)
        bt.pool.copy_(start)
        bt.o.fill_(3.0)
        bt.run()
        assert torch.equal(bt.o, o) and torch.equal(bt.pool, pool)
        assert not bt.h.get_status() & ~_abi.SQ_STATUS_SATURATED
    finally:
        bt.close()


def test_workspace_of_too_many_requests_is_refused():
    from quantized_linear_attention_sq_b200.state import StatePool
    sp = StatePool(1, 4, 2, 128, _abi.SQ_GATE_HEAD, _abi.SQ_FMT_FP32)
    try:
        most = _abi.SQ_RAGGED_MAX_REQUESTS
        one = sp.ragged_workspace_bytes(1, 10)
        assert one > 0 and sp.ragged_workspace_bytes(most, 2 ** 30) == (2 ** 24 + most) * one
        for B in (most + 1, 2 ** 31 - 1):
            with pytest.raises(_abi.SQError, match="requests"):
                sp.ragged_workspace_bytes(B, 2 ** 30)
    finally:
        sp.close()


@pytest.mark.parametrize("first", [2 ** 31 - 1, 2 ** 31 - 2, -1, -2 ** 31, 1000])
def test_first_blocks_outside_the_workspace_are_skipped(first):
    """A table entry that no call of sq_batch_tables writes: the request gets
    o = 0, a status bit and no state, the others are right."""
    bt = Batch([70, 200, 3, 64], past=[1, 0, 1, 1])
    try:
        bt.tables.cu_blocks[1] = first
        bt.run()
        check_rows(bt, skip=(1,))
        assert (bt.o[70:270] == 0).all()
        s = bt.slots[1]
        assert torch.equal(bt.pool[s], bt.S0[s])
        assert bt.h.get_status() == _abi.SQ_STATUS_BAD_SLOT
    finally:
        bt.close()


@pytest.mark.parametrize("gate", [0.0, -1.0, 1e-40])
@pytest.mark.parametrize("row", [0, 20, 63, 64])
def test_a_gate_of_zero_forgets_the_largest_state(row, gate):
    """Nothing of a state of 1e30 is left behind a gate of zero (or, at 1e-40,
    1e-10 of it beside values of 1): not 2^-126 of it."""
    def gates(g):
        g[row] = gate
    bt = Batch([100], past=[1], gates=gates, extra=0)
    try:
        if gate <= 0.0:
            bt.v.mul_(1e-8)
        bt.S0.mul_(1e30)
        bt.pool.copy_(bt.S0)
        bt.run()
        (o, S), = bt.expected()
        tol = 8 * U * math.sqrt(101)
        assert rel(bt.pool[bt.slots[0]], S) <= tol
        for r in (slice(0, row), slice(row, 100)):
            if r.stop > r.start:
                assert rel(bt.o[r].transpose(0, 1), o[r].transpose(0, 1)) <= 2.0 ** -8 + 4 * tol
        assert bt.h.get_status() == 0
    finally:
        bt.close()


def test_tables_without_positions():
    """The positions may be left out, as in the C call."""
    from quantized_linear_attention_sq_b200.ragged import BatchTables, batch_tables
    lengths, past = i32([5, 0, 130, 64, 9]), i32([1, 2, 3, 4, 5])
    want = BatchTables.empty(5, 200).build(lengths, past)
    t = BatchTables.empty(5, 200)
    t.positions = None
    t.build(lengths, past, max_rows=200)
    for x in ("cu_seqlens", "cu_blocks", "block_req"):
        assert torch.equal(getattr(t, x), getattr(want, x))
    assert t.cu_seqlens.tolist() == [0, 5, 5, 135, 199, 200] and t.positions is None
    with pytest.raises(ValueError, match="max_rows"):
        t.build(lengths, past)
    with pytest.raises(ValueError, match="block_req"):
        t.build(lengths, past, max_rows=264)
    with pytest.raises(ValueError, match="positions"):
        batch_tables(lengths, past, want.cu_seqlens, want.cu_blocks, want.positions, want.block_req, max_rows=199)
    # and a batch runs on such tables
    bt = Batch([70, 1, 20])
    try:
        bt.tables.positions = None
        bt.tables.build(i32(bt.lengths), i32(bt.past), max_rows=bt.rows)
        check_rows(bt.run())
    finally:
        bt.close()


def test_a_replay_beside_a_call_on_another_stream():
    """A captured call replays while another handle's call runs on a side
    stream, each with a workspace of its own; everything either reads is
    ordered before both."""
    lengths = [300, 1, 64, 129]
    a, b = (Batch(lengths, hv=8, hk=4, seed=s) for s in (4, 5))
    try:
        ws = [x.h.new_ragged_workspace(x.B, x.rows) for x in (a, b)]
        first = []
        for x, w in zip((a, b), ws):
            x.run(workspace=w)
            check_rows(x)
            first.append((x.o.clone(), x.pool.clone()))
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            a.h.prefill_ragged(a.pool, a.q, a.k, a.v, a.beta, a.g, a.o, a.tables, slot_ids=a.slot_ids, workspace=ws[0])
        side = torch.cuda.Stream()
        for _ in range(20):
            for x in (a, b):
                x.pool.copy_(x.S0)
                x.o.fill_(3.0)
            side.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(side):
                b.h.prefill_ragged(b.pool, b.q, b.k, b.v, b.beta, b.g, b.o, b.tables, slot_ids=b.slot_ids,
                                   workspace=ws[1])
            graph.replay()
            torch.cuda.current_stream().wait_stream(side)
            for x, (o, pool) in zip((a, b), first):
                assert torch.equal(x.o, o) and torch.equal(x.pool, pool)
        assert a.h.get_status() == 0 and b.h.get_status() == 0
    finally:
        a.close()
        b.close()

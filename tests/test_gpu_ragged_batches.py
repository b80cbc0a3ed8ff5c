"""GPU tests of ragged batches: calls that the documentation allows beside
those of test_gpu_ragged.py."""
import pytest
import torch

from quantized_linear_attention_sq_b200 import _abi
from tests.test_gpu_ragged import Batch, check_rows, i32

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

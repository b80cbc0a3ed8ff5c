"""GPU: o where a large old value is overwritten by a small one and read back.

With |k| = 1, q = k, beta = 1 and gates of 1 the row's output is v itself, the
difference of S^T q and (k . q)(v - S^T k): whatever S^T q and the update lose
on the way to o, o shows in full. The inputs lie on grids that make every sum
exact in fp32, whatever its order:
- S = N 2^-17 with 2^17 <= |N| < 2^18; k has four entries of +-1/2, so S^T k is
  a multiple of 2^-18 below 4 and the update u = v - S^T k, v = j 2^-17, as well;
- S + k u is a multiple of 2^-19 below 4, and the next S^T k sums multiples of
  2^-20 below 8: 23 bits;
- beta is 0 in the other rows and 1 in the writing ones, so the products q . k,
  k . k and every inverse over them hold only -1, 0 and 1.
So o has to be the 64-bit result rounded once to bf16, and the state the
64-bit state: no tolerance.
"""
import pytest
import torch

from quantized_linear_attention_sq_b200 import _abi
from tests import ragged_ref as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    from quantized_linear_attention_sq_b200 import build
    build.build()
    torch.cuda.init()


@pytest.mark.parametrize("in_blocks", [False, True])
@pytest.mark.parametrize("n,writes", [(10, [4]), (40, [0, 17, 18]), (64, [0, 33, 63]), (200, [5, 70, 130, 199])])
def test_an_overwritten_value_reads_back_exactly(n, writes, in_blocks):
    from quantized_linear_attention_sq_b200.ragged import BatchTables
    from quantized_linear_attention_sq_b200.state import StatePool
    gen = torch.Generator().manual_seed(n)
    hv, hk, d = 2, 1, 128
    sign = lambda *s: 2.0 * torch.randint(0, 2, s, generator=gen) - 1  # noqa: E731
    S0 = sign(1, hv, d, d) * torch.randint(2 ** 17, 2 ** 18, (1, hv, d, d), generator=gen) * 2.0 ** -17
    key = torch.zeros(d)
    key[torch.randperm(d, generator=gen)[:4]] = 0.5 * sign(4)
    k = key.expand(n, hk, d).contiguous()
    v = sign(n, hv, d) * torch.randint(1, 128, (n, hv, d), generator=gen) * 2.0 ** -17
    beta = torch.zeros(n, hv)
    beta[writes] = 1.0
    g = torch.ones(n, hv)
    want_o, want_S = ref.recurrence(k, k, v, beta, g, S0[0])
    last = torch.zeros_like(want_o)
    for t in range(n):
        last[t] = v[t] if beta[t, 0] else last[t - 1]
    assert torch.equal(want_o[writes[0]:], last[writes[0]:])   # what was written last, exactly

    sp = StatePool(1, hv, hk, d, _abi.SQ_GATE_HEAD, _abi.SQ_FMT_FP32)
    try:
        pool = S0.float().cuda()
        kb, vb = k.bfloat16().cuda(), v.bfloat16().cuda()
        assert torch.equal(vb.cpu().double(), v.double()) and torch.equal(pool.cpu().double(), S0.double())
        i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
        t = BatchTables.empty(1, n).build(i32([n]), i32([1]))
        o = torch.zeros((n, hv, d), dtype=torch.bfloat16, device="cuda")
        sp.prefill_ragged(pool, kb, kb.clone(), vb, beta.cuda(), g.cuda(), o, t, max_len=n if in_blocks else 1)
        torch.cuda.synchronize()
        assert torch.equal(o.cpu(), want_o.bfloat16())
        assert torch.equal(pool[0].cpu().double(), want_S)
        assert sp.get_status() == 0
    finally:
        sp.close()

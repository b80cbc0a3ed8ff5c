"""StatePool refuses tensors of another GPU than its handle's, whichever
argument they are (no GPU needed: the tensors are stand-ins, and the calls
behind the checks are replaced)."""
import types

import pytest
import torch

from quantized_linear_attention_sq_b200 import _abi, state

N_SLOTS, HV, HK, D, B, ROWS = 3, 4, 2, 32, 2, 5
I32, F32, U8 = torch.int32, torch.float32, torch.uint8


class On:
    """What the checks ask of a contiguous CUDA tensor."""
    is_cuda = True

    def __init__(self, dtype, *shape, dev=0):
        self.dtype, self.shape, self.dev = dtype, torch.Size(shape), dev
        self.device = torch.device("cuda", dev)

    def get_device(self):
        return self.dev

    def numel(self):
        return self.shape.numel()

    def element_size(self):
        return self.dtype.itemsize

    def stride(self):
        return torch.empty(self.shape, device="meta").stride()

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return 1 << 20


def calls():
    f = lambda *s: On(F32, *s)  # noqa: E731
    step = dict(q=f(B, HK, D), k=f(B, HK, D), v=f(B, HV, D), beta=f(B, HV), g=f(B, HV), o=f(B, HV, D))
    rows = dict(q=f(ROWS, HK, D), k=f(ROWS, HK, D), v=f(ROWS, HV, D), beta=f(ROWS, HV), g=f(ROWS, HV), o=f(ROWS, HV, D))
    prompt = {x: On(F32, t.shape[0], 7, *t.shape[1:]) for x, t in step.items()}
    pool, slots, S = f(N_SLOTS, HV, D, D), On(I32, B), f(B, HV, D, D)
    tables = dict(cu_seqlens=On(I32, B + 1), cu_blocks=On(I32, B + 1), block_req=On(I32, B), past=On(I32, B))
    return {
        "quantize_state": dict(pool=pool, S=S, slot_ids=slots),
        "dequantize_state": dict(pool=pool, S_out=S, slot_ids=slots),
        "decode_step": dict(pool=pool, slot_ids=slots, **step),
        "window_step": dict(pool=pool, wbuf=On(U8, 64), W=4, slot_ids=slots, **step),
        "prefill": dict(pool=pool, S0=S, S_out=S, lengths=On(I32, B), slot_ids=slots, **prompt),
        "prefill_ragged": dict(pool=pool, slot_ids=slots, workspace=On(U8, 64), **rows, **tables),
    }


def run(call, args):
    args = dict(args)
    if call == "prefill_ragged":
        args["tables"] = types.SimpleNamespace(**{x: args.pop(x) for x in ("cu_seqlens", "cu_blocks", "block_req", "past")})
    sp = object.__new__(state.StatePool)
    sp.n_slots, sp.h_v, sp.h_k, sp.d = N_SLOTS, HV, HK, D
    sp.gate_kind, sp.fmt = _abi.SQ_GATE_HEAD, _abi.SQ_FMT_FP32
    sp.device, sp._h, sp.pool_bytes = torch.device("cuda", 0), None, 4 * N_SLOTS * HV * D * D
    getattr(sp, call)(stream=0, **args)


CASES = [(call, name) for call, args in calls().items() for name, t in args.items() if isinstance(t, On)]


@pytest.fixture
def launched(monkeypatch):
    seen = []
    for name in ("sq_quantize_state", "sq_dequantize_state", "sq_decode_step", "sq_window_step", "sq_prefill",
                 "sq_prefill_ragged"):
        monkeypatch.setattr(_abi, name, lambda *a, name=name: seen.append(name))
    monkeypatch.setattr(_abi, "sq_window_buffer_bytes", lambda *a: (16, 64))
    monkeypatch.setattr(_abi, "sq_ragged_workspace_bytes", lambda *a: 64)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    return seen


@pytest.mark.parametrize("call", calls())
def test_tensors_of_the_pool_s_device_are_taken(call, launched):
    run(call, calls()[call])
    assert launched == ["sq_" + call]


@pytest.mark.parametrize("call,name", CASES)
def test_a_tensor_of_another_device_is_refused(call, name, launched):
    args = calls()[call]
    args[name] = On(args[name].dtype, *args[name].shape, dev=1)
    with pytest.raises(ValueError, match=f"{name} must be a CUDA tensor on device 0, not on cuda:1"):
        run(call, args)
    assert not launched

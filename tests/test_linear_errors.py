"""What a failed launch leaves behind: nothing that the next call could take for its own."""
import ctypes

import pytest
import torch

from test_linear_attention import draw

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("shape", [(4, 40, 40, 140, 64, 64, 4),  # equal shares
                                   (1, 1, 1, 2000, 64, 64, 1),   # segments
                                   (1, 1, 1, 140, 64, 64, 1)], ids=str)
def test_a_refused_launch_is_not_reported_again(shape):
    """While a stream of the blocking kind is captured, work on the legacy default stream is
    refused by the runtime: prefill says so, and a decode on another stream does not."""
    from gated_delta_rule_recurrent_b200 import binding

    L, P = binding.lib(), binding._ptr
    x = draw(*shape, seed=27, device="cuda")
    y = draw(1, 1, 1, 2, 64, 64, 1, seed=28, lengths=[2], device="cuda")
    B, Hq, Hv, T, Dk, Dv, pool = shape
    d, d_y = binding.Dims(B, T, Hq, Hv, Dk, Dv, pool), binding.Dims(1, 2, 1, 1, 64, 64, 1)
    names = ("query", "key", "value", "log_decay", "state_pool", "lengths", "indices")
    out, out_y = torch.zeros_like(x["value"]), torch.zeros_like(y["value"])
    need = ctypes.c_int64(0)
    assert L.gdr_linear_attention_prefill_workspace(ctypes.byref(d), ctypes.byref(need)) == 0
    work = torch.empty(max(need.value, 16), dtype=torch.uint8, device="cuda")
    before = x["state_pool"].clone()
    other = torch.cuda.Stream()

    def prefill(stream):
        return L.gdr_linear_attention_prefill(ctypes.byref(d), *(P(x[n]) for n in names),
                                              x["scale"], P(out), P(work), need.value, stream)

    def decode():
        return L.gdr_linear_attention_decode(ctypes.byref(d_y), *(P(y[n]) for n in names), None,
                                             y["scale"], P(out_y), other.cuda_stream)

    assert decode() == 0
    torch.cuda.synchronize()
    cu, stream, graph = ctypes.CDLL("libcuda.so.1"), ctypes.c_void_p(), ctypes.c_void_p()
    assert cu.cuStreamCreate(ctypes.byref(stream), 0) == 0  # 0: synchronises with the legacy one
    assert cu.cuStreamBeginCapture_v2(stream, 0) == 0
    try:
        refused = prefill(None)
        after = decode()
    finally:
        cu.cuStreamEndCapture(stream, ctypes.byref(graph))  # the capture was invalidated
        if graph.value:
            cu.cuGraphDestroy(graph)
        cu.cuStreamDestroy_v2(stream)
    torch.cuda.synchronize()
    assert refused == 5 and "launch" in L.gdr_last_error().decode()
    assert after == 0
    assert torch.equal(x["state_pool"].view(torch.int16), before.view(torch.int16))
    assert prefill(torch.cuda.current_stream().cuda_stream) == 0 and decode() == 0
    torch.cuda.synchronize()
    assert binding.device_error() == 0

"""CPU test of what a trace is told that calls the library itself: a trace would hold only the empty outputs."""

import pytest
import torch

q = pytest.importorskip("block_wise_bit_adam8bit_amd")


@pytest.mark.parametrize("call", [
    q.qopt_fp8_quantize, q.qopt_fp4_quantize, q.qopt_orthogonalize, lambda x: q.qopt_layer_norm_forward(x)[0],
    lambda x: q.qopt_muon32bit_step([], lr=1.0, momentum=0.5, weight_decay=0.0)])
def test_the_refusal_names_what_can_be_traced(call):
    with pytest.raises(RuntimeError, match="fp8_linear, fp4_linear and layer_norm"):
        torch.jit.trace(call, torch.ones(4, 8), check_trace=False)

"""A stack of experts and the payload of one layer are not taken for each other: the C struct of both
is the same, so a call for one layer would compute with the first expert alone."""
import pytest
import torch

import w4_gemm_amd as W

N, K, E = 8, 256, 3


def _payloads():
    one = W.W8Payload(torch.zeros((N, K), dtype=torch.int8), torch.ones(N, dtype=torch.float16), None, None)
    return one, W.stack_payloads_w8([one] * E)


X, DY = torch.zeros((4, K), dtype=torch.bfloat16), torch.zeros((4, N), dtype=torch.bfloat16)
OFFSETS = torch.tensor([0, 1, 2, 4], dtype=torch.int32)


@pytest.mark.parametrize("call", [
    lambda p: W.linear_fwd_w8a8(X, p), lambda p: W.linear_dgrad_w8(DY, p),
    lambda p: W.linear_fwd_w8(X, p), lambda p: W.reconstruct_bf16_w8(p),
    lambda p: W.fwd_w8a8_workspace_bytes(4, p), lambda p: W.dgrad_w8_workspace_bytes(4, p),
    lambda p: W.fwd_w8_workspace_bytes(4, p),
], ids=["fwd_w8a8", "dgrad_w8", "fwd_w8", "reconstruct_w8", "fwd_w8a8_ws", "dgrad_w8_ws", "fwd_w8_ws"])
def test_calls_for_one_layer_refuse_a_stack(call):
    with pytest.raises(TypeError, match="one layer"):
        call(_payloads()[1])


@pytest.mark.parametrize("call", [
    lambda p: W.grouped_fwd_w8a8(X, OFFSETS, p), lambda p: W.grouped_dgrad_w8(DY, OFFSETS, p),
    lambda p: W.grouped_fwd_w8a8_workspace_bytes(4, p), lambda p: W.grouped_dgrad_w8_workspace_bytes(4, p),
], ids=["fwd_w8a8", "dgrad_w8", "fwd_w8a8_ws", "dgrad_w8_ws"])
def test_grouped_calls_refuse_one_layer(call):
    with pytest.raises(TypeError, match="GroupedW8Payload"):
        call(_payloads()[0])


def test_grouped_calls_refuse_missing_offsets():
    for call, a in ((W.grouped_fwd_w8a8, X), (W.grouped_dgrad_w8, DY)):
        with pytest.raises(TypeError, match="offsets"):
            call(a, None, _payloads()[1])

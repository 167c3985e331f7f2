"""The even form of gate and up in the C ABI and the Python wrappers, on the host (no GPU needed)."""
import re

import pytest
import torch

import rank_orthonormalized_optimizer_amd as dion
from rank_orthonormalized_optimizer_amd import _lib, block
from tests.test_block_abi import HEADER, ffn, ffn_grad


def test_the_flag_is_the_headers():
    assert re.search(rf"#define DION_KEEP_EVEN {_lib.KEEP_EVEN}\b", open(HEADER).read())


@pytest.mark.parametrize("call", [ffn, ffn_grad])
def test_flag_goes_with_an_activation_and_bf16(call):
    for act in (_lib.SILU, _lib.GELU):
        assert call(act=act | _lib.KEEP_EVEN, nbytes=1) == _lib.ERR_WORKSPACE   # taken, up to the next check
        assert call(act=act | _lib.KEEP_EVEN, dt=0, xt=0, nbytes=1) == _lib.ERR_OPTION
        assert call(act=act | 2 * _lib.KEEP_EVEN, nbytes=1) == _lib.ERR_OPTION
    assert call(act=2 | _lib.KEEP_EVEN, nbytes=1) == _lib.ERR_OPTION


def test_what_holds_gate_and_up():
    f32, bf16 = torch.zeros(3, 8), torch.zeros(3, 8, dtype=torch.bfloat16)
    even = torch.zeros(3, 8, dtype=torch.int16)
    cpu = torch.device("cpu")
    with pytest.raises(ValueError, match="both or neither"):
        block._kept(even, None, torch.bfloat16, cpu, even.shape)
    assert block._kept(None, None, torch.bfloat16, cpu, even.shape) == 0
    assert block._kept(even, even, torch.bfloat16, cpu, even.shape) == _lib.KEEP_EVEN
    assert block._kept(bf16, bf16, torch.bfloat16, cpu, even.shape) == 0
    assert block._kept(f32, f32, torch.float32, cpu, even.shape) == 0


@pytest.mark.gpu
def test_types_of_gate_and_up_refused(cuda):
    x, W = torch.zeros(3, 64, device=cuda), torch.zeros(8, 64, device=cuda)
    even, half = torch.zeros(3, 8, device=cuda, dtype=torch.int16), torch.zeros(3, 8, device=cuda, dtype=torch.bfloat16)
    down = W.t().contiguous()
    with pytest.raises(TypeError):
        dion.gated_ffn_(x, W, W, down, gate=even, up=even)   # fp32 weights keep fp32
    b = [t.bfloat16() for t in (x, W, W, down)]
    for gate, up in ((even, half), (half, even), (torch.zeros(3, 8, device=cuda), torch.zeros(3, 8, device=cuda))):
        with pytest.raises(TypeError):
            dion.gated_ffn_(*b, gate=gate, up=up)
        with pytest.raises(TypeError):
            dion.gated_ffn_grad_(*b, b[0], gate, up, dX=torch.empty_like(b[0]))

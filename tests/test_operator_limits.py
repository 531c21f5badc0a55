"""Sizes at the ends of their types.  No GPU: the host-side checks run before any CUDA call."""
import pytest

import mxfp4_expert_ffn_moe_b200 as moe
from mxfp4_expert_ffn_moe_b200 import build as moe_build

P = 0x1000                                     # an address that is never used
INVALID = -1
BF16, F32 = 0, 2


@pytest.fixture(scope="module")
def lib():
    moe_build.build()
    return moe.load_library()


@pytest.mark.parametrize("T,k", [(2 ** 61, 8), (2 ** 62, 4), (2 ** 63 - 1, 2), (2 ** 31, 1), (2 ** 28, 8),
                                 ((2 ** 31 - 1) // 3 + 1, 3)])
def test_a_number_of_pairs_past_32_or_64_bits_is_refused(lib, T, k):
    # T * k of the first three is 0 or negative in 64 bits
    assert lib.moe_dispatch_rows(P, BF16, 64, T, 64, k, P, P, 16, P, BF16, 64, None) == INVALID
    assert lib.moe_dispatch_rows_backward(P, F32, 64, T, 64, k, 16, P, P, P, 64, P, F32, 64, P, None) == INVALID
    assert lib.moe_combine_rows(P, F32, 64, T, 64, k, 16, P, P, P, BF16, 64, None) == INVALID
    assert lib.moe_combine_rows_backward(P, BF16, 64, T, 64, k, P, P, P, 64, 16, P, BF16, 64, P, None) == INVALID
    assert lib.moe_route_backward(P, P, P, T, 16, k, P, None) == INVALID
    assert lib.moe_permute(P, T, k, 16, 32, P, P, P, P, None, None) == INVALID
    assert lib.moe_gather_pairs(P, T, 64, k, P, P, P, P, 16, P, P, P, None) == INVALID
    assert lib.moe_mxfp4_workspace_size(T, 128, 128, 16, k) == 0
    assert lib.moe_token_tile_rows(T, 128, 128, 16, k, 0) == INVALID


def test_flags_of_the_calls_that_write_expert_rows(lib):
    for flags in (1, 2, 4, 16, 9):
        assert lib.moe_dispatch_rows_ex(P, BF16, 64, 8, 64, 2, P, P, 16, P, BF16, 64, flags, None) == INVALID
        assert lib.moe_combine_rows_backward_ex(P, BF16, 64, 8, 64, 2, P, P, P, 64, 16, P, BF16, 64, P, flags, None) == INVALID
    # the other checks come before any CUDA call with a good flag too
    assert lib.moe_dispatch_rows_ex(None, BF16, 64, 8, 64, 2, P, P, 16, P, BF16, 64, moe.MOE_FLAG_ZERO_SKIPPED, None) == INVALID
    assert lib.moe_combine_rows_backward_ex(P, BF16, 64, 8, 64, 2, P, P, P, 64, 16, P, BF16, 63, P, moe.MOE_FLAG_ZERO_SKIPPED, None) == INVALID


def test_the_types_that_rows_may_have():
    # the mapping and the refusal that every call's rows go through
    torch = pytest.importorskip("torch")
    moe._dtype_code(torch.float32, "t")                       # imports torch into the binding
    call = object.__new__(moe._Call)
    call.device, call.side = -1, None
    for dtype, code in ((torch.bfloat16, 0), (torch.float16, 1), (torch.float32, 2)):
        assert call.rows(torch.zeros((3, 4), dtype=dtype), "x", 3, 4)[1:] == (code, 4)
    for dtype in (torch.float64, torch.int32, torch.uint8):
        with pytest.raises(ValueError, match="x: expected bfloat16, float16 or float32"):
            call.rows(torch.zeros((3, 4), dtype=dtype), "x", 3, 4)
    with pytest.raises(ValueError, match="tensor of torch.float16"):
        call.rows(torch.zeros((3, 4)), "x", 3, 4, torch.float16)


def test_a_stream_of_another_device_is_refused(monkeypatch):
    torch = pytest.importorskip("torch")
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda device: 0, raising=False)

    class Tensor:
        device = "cuda:0"

        @staticmethod
        def get_device():
            return 0

    class Stream:
        def __init__(self, device_index, cuda_stream):
            self.device_index, self.cuda_stream = device_index, cuda_stream

    for handle in (0, 7):                                   # every device's default stream has the handle 0
        with pytest.raises(ValueError, match="stream of cuda:0"):
            moe._Call(Tensor, Stream(1, handle))
    assert moe._Call(Tensor, Stream(0, 0)).side is None
    assert moe._Call(Tensor, Stream(0, 7)).stream == 7

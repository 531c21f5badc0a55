"""Waits that give up: the row and matvec kernels end, flag it, touch nothing outside their
outputs, and the next call is right.  The bounds-checked build makes the waits give up at
once, so nothing here takes long or stays on the GPU."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def checked(moe_gpu):
    from mxfp4_expert_ffn_moe_b200 import build as moe_build
    moe_build.build(checked=True)
    moe_gpu.use_checked_library(True)
    yield moe_gpu
    moe_gpu.use_checked_library(False)


def _guarded(shape, dtype):
    import torch
    n = int(np.prod(shape))
    buf = torch.full((n + 512,), 3.0, dtype=dtype, device="cuda")
    return buf, buf[256:256 + n].view(shape)


def _calls(moe):
    import torch
    g = torch.Generator().manual_seed(1)
    T, k, H = 700, 4, 2880
    x = torch.randn((T, H), generator=g).to("cuda", torch.bfloat16)
    y = torch.randn((T * k, H), generator=g).to("cuda", torch.bfloat16)
    xo, yo = x[:, :1001].contiguous(), y[:, :1001].contiguous()          # rows off 16-byte words
    w = torch.rand((T, k), generator=g).cuda()
    pair_rows = torch.randperm(T * k, generator=g).to(torch.int32).cuda()
    blocks = torch.randint(0, 256, (8, 768, 1440), dtype=torch.uint8, generator=g).cuda()
    e8m0 = torch.randint(118, 127, (8, 768, 90), dtype=torch.uint8, generator=g).cuda()
    e4m3 = torch.randint(8, 56, (8, 768, 180), dtype=torch.uint8, generator=g).cuda()
    ids = torch.randint(0, 8, (48,), dtype=torch.int32, generator=g).cuda()
    xm = x[:12]
    return {
        "dispatch, copies": ((T * k, H), x.dtype, lambda o: moe.moe_dispatch_rows(x, pair_rows, k, rows=o)),
        "dispatch, weighted": ((T * k, H), x.dtype, lambda o: moe.moe_dispatch_rows(x, pair_rows, k, weights=w, rows=o)),
        "dispatch, odd": ((T * k, 1001), x.dtype, lambda o: moe.moe_dispatch_rows(xo, pair_rows, k, weights=w, rows=o)),
        "combine": ((T, H), x.dtype, lambda o: moe.moe_combine_rows(y, pair_rows, T, k, weights=w, out=o)),
        "combine, odd": ((T, 1001), x.dtype, lambda o: moe.moe_combine_rows(yo, pair_rows, T, k, weights=w, out=o)),
        "combine backward": ((T * k, H), x.dtype,
                             lambda o: moe.moe_combine_rows_backward(x, pair_rows, k, weights=w, y_rows=y, drows=o)),
        "mxfp4": ((48, 768), torch.float32, lambda o: moe.mxfp4_matvec(xm, blocks, e8m0, row_ids=ids, rows_per_x=4, out=o)),
        "nvfp4": ((48, 768), torch.float32, lambda o: moe.nvfp4_matvec(xm, blocks, e4m3, row_ids=ids, rows_per_x=4, out=o)),
    }


@pytest.mark.parametrize("name", ["dispatch, copies", "dispatch, weighted", "dispatch, odd", "combine", "combine, odd",
                                  "combine backward", "mxfp4", "nvfp4"])
def test_a_wait_that_gives_up_ends_the_call(checked, name):
    import torch
    moe = checked
    lib = moe.load_library()
    shape, dtype, call = _calls(moe)[name]
    want = torch.empty(shape, dtype=dtype, device="cuda")
    call(want)
    torch.cuda.synchronize()
    assert moe.moe_get_device_error() == 0
    buf, out = _guarded(shape, dtype)
    assert lib.moe_checked_give_up_waits(1) == 0
    try:
        torch.empty(1 << 28, dtype=torch.uint8, device="cuda").fill_(1)      # inputs out of L2: waits are not over yet
        call(out)
        torch.cuda.synchronize()
    finally:
        assert lib.moe_checked_give_up_waits(0) == 0
    assert moe.moe_get_device_error() & moe.MOE_DEVERR_TIMEOUT
    n = int(np.prod(shape))
    assert bool((buf[:256] == 3).all()) and bool((buf[256 + n:] == 3).all())
    for _ in range(2):
        call(out)
        torch.cuda.synchronize()
        assert moe.moe_get_device_error() == 0
        assert torch.equal(out, want)

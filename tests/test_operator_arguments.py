"""Refusals of the dispatch, combine, route-gradient and matvec calls.  No GPU: the host-side
checks run before any CUDA call, and the binding's own before the library."""
import ctypes

import pytest

import mxfp4_expert_ffn_moe_b200 as moe
from mxfp4_expert_ffn_moe_b200 import build as moe_build

P = 0x1000                                     # an address that is never used
INVALID, UNSUPPORTED = -1, -2
BF16, F16, F32 = 0, 1, 2


@pytest.fixture(scope="module")
def lib():
    moe_build.build()
    return moe.load_library()


def _refused(fn, names, good, changes, status):
    args = dict(zip(names.split(), good))
    for k, v in changes.items():
        assert k in args, k
        args[k] = v
    assert fn(*args.values()) == status, changes


DISPATCH = "x x_dtype x_stride T H k pair_rows weights R rows rows_dtype rows_stride stream"
DISPATCH_GOOD = [P, BF16, 64, 8, 64, 2, P, P, 16, P, BF16, 64, None]


@pytest.mark.parametrize("changes,status", [
    (dict(x=None), INVALID), (dict(rows=None), INVALID), (dict(T=0), INVALID), (dict(H=0), INVALID), (dict(k=0), INVALID),
    (dict(k=9), INVALID), (dict(R=0), INVALID), (dict(T=2 ** 30), INVALID), (dict(R=2 ** 31), INVALID), (dict(H=2 ** 31), INVALID),
    (dict(x_stride=-1), INVALID), (dict(rows_stride=63), INVALID), (dict(x=P + 1), INVALID), (dict(rows=P + 1), INVALID),
    (dict(pair_rows=P + 2), INVALID), (dict(weights=P + 2), INVALID), (dict(x_dtype=3), INVALID), (dict(rows_dtype=-1), INVALID),
    (dict(pair_rows=None, R=15), INVALID), (dict(rows_dtype=F16), UNSUPPORTED), (dict(x_dtype=F32), UNSUPPORTED)])
def test_dispatch_refusals(lib, changes, status):
    _refused(lib.moe_dispatch_rows, DISPATCH, DISPATCH_GOOD, changes, status)


DISPATCH_BWD = "drows rows_dtype rows_stride T H k R pair_rows weights x x_stride dx x_dtype dx_stride dweights stream"
DISPATCH_BWD_GOOD = [P, F32, 64, 8, 64, 2, 16, P, P, P, 64, P, F32, 64, P, None]


@pytest.mark.parametrize("changes,status", [
    (dict(drows=None), INVALID), (dict(dx=None), INVALID), (dict(x=None), INVALID), (dict(dweights=None), INVALID),
    (dict(dx_stride=0), INVALID), (dict(x_stride=-64), INVALID), (dict(rows_stride=-1), INVALID), (dict(x=P + 2), INVALID),
    (dict(dweights=P + 1), INVALID), (dict(T=-1), INVALID), (dict(pair_rows=None, R=1), INVALID),
    (dict(rows_dtype=BF16), UNSUPPORTED)])
def test_dispatch_backward_refusals(lib, changes, status):
    _refused(lib.moe_dispatch_rows_backward, DISPATCH_BWD, DISPATCH_BWD_GOOD, changes, status)


COMBINE = "rows rows_dtype rows_stride T H k R pair_rows weights out out_dtype out_stride stream"
COMBINE_GOOD = [P, F32, 64, 8, 64, 2, 16, P, P, P, BF16, 64, None]


@pytest.mark.parametrize("changes,status", [
    (dict(rows=None), INVALID), (dict(out=None), INVALID), (dict(out_stride=32), INVALID), (dict(k=9), INVALID),
    (dict(rows=P + 2), INVALID), (dict(out_dtype=7), INVALID), (dict(rows_dtype=BF16, out_dtype=F32), UNSUPPORTED)])
def test_combine_refusals(lib, changes, status):
    _refused(lib.moe_combine_rows, COMBINE, COMBINE_GOOD, changes, status)


COMBINE_BWD = "dout out_dtype dout_stride T H k pair_rows weights rows rows_stride R drows rows_dtype drows_stride dweights stream"
COMBINE_BWD_GOOD = [P, BF16, 64, 8, 64, 2, P, P, P, 64, 16, P, BF16, 64, P, None]


@pytest.mark.parametrize("changes,status", [
    (dict(dout=None), INVALID), (dict(drows=None), INVALID), (dict(rows=None), INVALID), (dict(dweights=None), INVALID),
    (dict(drows_stride=1), INVALID), (dict(dout_stride=-1), INVALID), (dict(rows_stride=-1), INVALID),
    (dict(rows=P + 1), INVALID), (dict(rows_dtype=F16), UNSUPPORTED)])
def test_combine_backward_refusals(lib, changes, status):
    _refused(lib.moe_combine_rows_backward, COMBINE_BWD, COMBINE_BWD_GOOD, changes, status)


ROUTE_BWD = "dweights ids weights T E k dlogits stream"


@pytest.mark.parametrize("changes,status", [
    (dict(dweights=None), INVALID), (dict(ids=None), INVALID), (dict(weights=None), INVALID), (dict(dlogits=None), INVALID),
    (dict(T=0), INVALID), (dict(E=0), INVALID), (dict(k=0), INVALID), (dict(k=9), INVALID), (dict(E=3), INVALID),
    (dict(T=2 ** 30), INVALID), (dict(dlogits=P + 2), INVALID), (dict(ids=P + 1), INVALID), (dict(E=257), UNSUPPORTED)])
def test_route_backward_refusals(lib, changes, status):
    _refused(lib.moe_route_backward, ROUTE_BWD, [P, P, P, 8, 16, 4, P, None], changes, status)


MATVEC = "x x_dtype x_stride rows_per_x R N K E row_ids blocks scales bias flags alpha limit out out_dtype stream"
MATVEC_GOOD = [P, BF16, 64, 1, 4, 32, 64, 8, P, P, P, P, 0, 1.702, 7.0, P, BF16, None]
MATVEC_CHANGES = [
    (dict(x=None), INVALID), (dict(blocks=None), INVALID), (dict(scales=None), INVALID), (dict(out=None), INVALID),
    (dict(R=0), INVALID), (dict(N=0), INVALID), (dict(K=0), INVALID), (dict(K=48), INVALID), (dict(E=0), INVALID),
    (dict(rows_per_x=0), INVALID), (dict(row_ids=None), INVALID), (dict(flags=1), INVALID), (dict(flags=4), INVALID),
    (dict(flags=2, N=33), INVALID), (dict(x=P + 8), INVALID), (dict(blocks=P + 8), INVALID), (dict(scales=P + 4), INVALID),
    (dict(x_stride=68), INVALID), (dict(x_stride=-64), INVALID), (dict(bias=P + 2), INVALID), (dict(row_ids=P + 1), INVALID),
    (dict(out=P + 1), INVALID), (dict(x_dtype=5), INVALID), (dict(out_dtype=9), INVALID),
    (dict(R=1025), UNSUPPORTED), (dict(E=257), UNSUPPORTED), (dict(N=2 ** 24 + 1), UNSUPPORTED), (dict(K=2 ** 15 + 32), UNSUPPORTED), (dict(N=2 ** 24, E=128), UNSUPPORTED),
    (dict(x_dtype=F32), UNSUPPORTED), (dict(out_dtype=F16), UNSUPPORTED)]


@pytest.mark.parametrize("changes,status", MATVEC_CHANGES)
def test_matvec_refusals(lib, changes, status):
    _refused(lib.mxfp4_matvec, MATVEC, MATVEC_GOOD, changes, status)
    nv = MATVEC.replace("scales bias", "scales scale2 bias")
    good = MATVEC_GOOD[:11] + [P] + MATVEC_GOOD[11:]
    _refused(lib.nvfp4_matvec, nv, good, changes, status)


def test_nvfp4_matvec_scale2_alignment(lib):
    good = MATVEC_GOOD[:11] + [P + 2] + MATVEC_GOOD[11:]
    assert lib.nvfp4_matvec(*good) == INVALID


def test_the_binding_refuses_tensors_off_the_current_device():
    torch = pytest.importorskip("torch")
    x = torch.zeros((4, 32), dtype=torch.bfloat16)
    calls = [lambda: moe.moe_dispatch_rows(x, None, 1), lambda: moe.moe_combine_rows(x, None, 4, 1),
             lambda: moe.moe_dispatch_rows_backward(x, None, 4, 1), lambda: moe.moe_combine_rows_backward(x, None, 1),
             lambda: moe.moe_route_backward(x.float(), x.int(), x.float(), 32),
             lambda: moe.mxfp4_matvec(x, x.to(torch.uint8), x.to(torch.uint8)),
             lambda: moe.nvfp4_matvec(x, x.to(torch.uint8), x.to(torch.uint8))]
    for call in calls:
        with pytest.raises(ValueError):
            call()


def test_dtype_codes_match_the_header():
    torch = pytest.importorskip("torch")
    assert [moe._dtype_code(d, "t") for d in (torch.bfloat16, torch.float16, torch.float32)] == [BF16, F16, F32]
    with pytest.raises(ValueError):
        moe._dtype_code(torch.float64, "t")
    assert ctypes.sizeof(ctypes.c_int) == 4

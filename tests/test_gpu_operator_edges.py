"""The ends of the row and matvec calls' tensors, sizes and buffers on the GPU."""
import numpy as np
import pytest

from tests.test_gpu_matvec import _bank, _dev, _want, _weights
from tests.test_gpu_pair_rows import E24, _case, _close, _dt, _pairs64, _randn

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("tok,row", [("bfloat16", "bfloat16"), ("float32", "float32")])
def test_the_ends_of_a_tensor_take_turns_with_its_other_rows(moe_gpu, tok, row):
    # off 16-byte words the granules at a tensor's two ends come by plain loads, all others by copies, through
    # the same stages in turn: the first and the last row between others, the same bits as aligned rows
    import torch
    moe = moe_gpu
    T, k, H, R = 6000, 3, 37, 50
    g = torch.Generator().manual_seed(40)
    pair_rows = torch.randint(0, R, (T, k), generator=g)
    pair_rows[torch.rand((T, k), generator=g) < 0.3] = R - 1
    pair_rows[torch.rand((T, k), generator=g) < 0.3] = 0
    pair_rows = pair_rows.reshape(-1).to(torch.int32).cuda()
    x, y = _randn((T, H), tok, g), _randn((R, H), row, g)
    words = torch.zeros((R, 40), dtype=y.dtype, device="cuda")
    words[:, :H] = y
    want = moe.moe_combine_rows(words, pair_rows, T, k)[:, :H]
    for off in (0, 1, 5):
        at = torch.empty(R * H + 8, dtype=y.dtype, device="cuda")[off:off + R * H].view(R, H)
        at.copy_(y)
        assert torch.equal(moe.moe_combine_rows(at, pair_rows, T, k), want)
        dx, _ = moe.moe_dispatch_rows_backward(at, pair_rows, T, k, x=x)
        assert torch.equal(dx, want)


def test_the_bank_s_last_scales_take_turns_with_others(moe_gpu):
    # E * N * K/32 is no multiple of 16: the bank's last scale bytes come by plain loads, and with several
    # tiles of x of the last expert other items' copies follow into the same buffer
    import torch
    moe = moe_gpu
    rng = np.random.default_rng(50)
    E, N, K, R = 2, 331, 96, 200
    blocks, scales = _bank(rng, E, N, K, "mxfp4", exact=True)
    x = rng.integers(-3, 4, (R, K)).astype(np.float64)
    ids = np.where(rng.random(R) < 0.1, 0, 1).astype(np.int32)
    got = moe.mxfp4_matvec(_dev(x, torch.bfloat16), _dev(blocks), _dev(scales), row_ids=_dev(ids), out_dtype=torch.float32)
    want, _, _ = _want(x, _weights(blocks, scales, "mxfp4"), ids, 1, None, None, False)
    np.testing.assert_array_equal(got.double().cpu().numpy(), want)


def test_two_host_threads_at_once(moe_gpu):
    # one instantiation, a small and a large shared-memory size, from two threads on their own streams
    import threading

    import torch
    moe = moe_gpu
    g = torch.Generator().manual_seed(60)
    T, k = 40, 7
    cases, errors = [], []
    for H in (8, 2880):
        y, w = _randn((T * k, H), "float16", g), torch.rand((T, k), generator=g).cuda()
        cases.append((y, w, (y.double().view(T, k, H) * w.double()[:, :, None]).sum(1)))
    torch.cuda.synchronize()

    def work(case):
        y, w, want = case
        stream = torch.cuda.Stream()
        try:
            for _ in range(50):
                out = moe.moe_combine_rows(y, None, T, k, weights=w, stream=stream)
            stream.synchronize()
            # k fused steps of 2^-24 on sums below 2^6, and one rounding to fp16
            assert bool(((out.double() - want).abs() <= 2.0 ** -11 * want.abs() + k * 2.0 ** -18).all())
        except Exception as e:                                       # noqa: BLE001
            errors.append(e)

    threads = [threading.Thread(target=work, args=(c,)) for c in cases for _ in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors
    assert moe.moe_get_device_error() == 0


def _dot_steps(H, k, tok, row):
    """Roundings of a dot: a thread's terms, then 5 shuffle steps and the sums of 4 warps.  A row is cut into
    segments of at most 32 KB of a token's operands, equal but for the last, of 8 elements and a multiple; 128
    threads take chunks of 8 elements (1 where rows are off 16-byte words)."""
    import torch
    size = {d: torch.finfo(_dt(d)).bits // 8 for d in (tok, row)}
    segs = -(-H * (size[tok] + k * size[row]) // 32768)
    seg = -(-(-(-H // segs)) // 8) * 8
    ve = 8 if H % 8 == 0 else 1
    return sum(-(-min(seg, H - at) // (128 * ve)) * ve for at in range(0, H, seg)) + 5 + 4


@pytest.mark.parametrize("tok,row", [("bfloat16", "bfloat16"), ("float32", "float32"), ("float16", "float32")])
@pytest.mark.parametrize("T,k,H", [(40, 4, 2880), (9, 8, 8200), (9, 7, 8201), (30, 3, 64), (30, 2, 127), (3, 1, 40000)])
def test_dots_within_their_roundings(moe_gpu, T, k, H, tok, row):
    moe = moe_gpu
    pair_rows, w, R, g = _case(T, k, 9, H, 0.1, seed=H)
    x, y = _randn((T, H), tok, g), _randn((R, H), row, g)
    prods = _pairs64(y, pair_rows, T, k) * x.double()[:, None, :]
    steps = _dot_steps(H, k, tok, row)
    _, dw = moe.moe_dispatch_rows_backward(y, pair_rows, T, k, weights=w, x=x)
    _close(dw, prods.sum(2), prods.abs().sum(2), steps, "dispatch backward")
    _, dw = moe.moe_combine_rows_backward(x, pair_rows, k, weights=w, y_rows=y)
    _close(dw, prods.sum(2), prods.abs().sum(2), steps, "combine backward")


@pytest.mark.parametrize("H,off", [(2880, 0), (2881, 1)])
def test_rows_past_two_to_the_31_elements(moe_gpu, H, off):
    import torch
    moe = moe_gpu
    T, k, R = 12, 3, 2 ** 31 // 2880 + 1000
    g = torch.Generator().manual_seed(H)
    far = torch.cat((torch.tensor([0, 1, R - 1, R - 2, 2 ** 31 // H, 2 ** 31 // H + 1, 2 ** 30 // H]),
                     2000 + torch.randperm(R // 2 - 4000, generator=g)[:T * k - 7]))
    assert far.unique().numel() == T * k and R * H > 2 ** 31
    pair_rows = far[torch.randperm(T * k, generator=g)].to(torch.int32).cuda()
    w = torch.rand((T, k), generator=g).cuda()
    x, y = _randn((T, H), "bfloat16", g), _randn((T * k, H), "bfloat16", g)
    big = torch.empty(R * H + 8, dtype=torch.bfloat16, device="cuda")[off:off + R * H].view(R, H)
    big[pair_rows.long()] = y
    assert torch.equal(moe.moe_combine_rows(big, pair_rows, T, k, weights=w), moe.moe_combine_rows(y, None, T, k, weights=w))
    dx, dw = moe.moe_dispatch_rows_backward(big, pair_rows, T, k, weights=w, x=x)
    assert torch.equal(dx, moe.moe_combine_rows(y, None, T, k, weights=w))
    prods = y.double().view(T, k, H) * x.double()[:, None, :]
    _close(dw, prods.sum(2), prods.abs().sum(2), _dot_steps(H, k, "bfloat16", "bfloat16"), "dweights")
    drows, dw2 = moe.moe_combine_rows_backward(x, pair_rows, k, weights=w, y_rows=big)
    want = moe.moe_dispatch_rows(x, None, k, weights=w)
    assert torch.equal(drows[pair_rows.long()], want)
    _close(dw2, prods.sum(2), prods.abs().sum(2), _dot_steps(H, k, "bfloat16", "bfloat16"), "dweights")
    drows[pair_rows.long()] = 0
    assert int(torch.count_nonzero(drows.view(-1))) == 0                # every other row of the fresh buffer
    moe.moe_dispatch_rows(x, pair_rows, k, rows=big)
    assert torch.equal(big[pair_rows.long()], x.repeat_interleave(k, dim=0))
    assert moe.moe_get_device_error() == 0


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("R,E,N,K,swiglu", [(1, 1, 2880, 2880, False), (24, 5, 62, 288, True), (70, 3, 331, 96, False),
                                            (9, 1, 40, 20000, True)])
def test_matvec_in_the_bounds_checked_build(moe_gpu, R, E, N, K, swiglu, fmt):
    import torch

    from mxfp4_expert_ffn_moe_b200 import build as moe_build
    moe_build.build(checked=True)
    moe = moe_gpu
    rng = np.random.default_rng(R + N)
    if swiglu:
        N += N % 2
    blocks, scales = (_dev(a) for a in _bank(rng, E, N, K, fmt, exact=True))
    x = _dev(rng.standard_normal((R, K)), torch.bfloat16)
    ids = _dev(rng.integers(0, E, R).astype(np.int32)) if E > 1 else None
    call = moe.mxfp4_matvec if fmt == "mxfp4" else moe.nvfp4_matvec
    results = []
    for checked in (False, True):
        moe.use_checked_library(checked)
        try:
            moe.moe_get_device_error()
            results.append(call(x, blocks, scales, row_ids=ids, swiglu=swiglu))
            assert moe.moe_get_device_error() == 0
        finally:
            moe.use_checked_library(False)
    assert torch.equal(*results)

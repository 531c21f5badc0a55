"""The ends of the row and matvec calls' tensors, sizes and buffers on the GPU."""
import numpy as np
import pytest

from tests.test_gpu_matvec import _bank, _dev, _want, _weights
from tests.test_gpu_pair_rows import _randn

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

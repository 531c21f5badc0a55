"""mxfp4_matvec and nvfp4_matvec on the GPU against their definition in 64 bits.

Exact inputs first: small integers and scales that make every partial sum a multiple of a
power of two below 2^24 of them, so fp32 sums are exact in any order and fp32 outputs must
equal the definition.  Random inputs: a sum of K products with at most one rounding or
truncation per term is off by (K + 64) 2^-23 sum|w x|, the result by half a step of its
type; the SwiGLU adds its slope (below 1.2 (limit + 1) in each operand for alpha 1.702)
times the operands' error and 32 roundings (expf is good to 2 ulp, times alpha * limit).
"""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

VALUE = np.array([0, .5, 1, 1.5, 2, 3, 4, 6, 0, -.5, -1, -1.5, -2, -3, -4, -6])
ALPHA, LIMIT = 1.702, 7.0


def _e4m3(b):
    b = b.astype(np.int64)
    e, m, s = (b >> 3) & 15, b & 7, b >> 7
    v = np.where(e == 0, m * 2.0 ** -9, (8 + m) * 2.0 ** (e - 10.0))
    return np.where((e == 15) & (m == 7), np.nan, np.where(s == 1, -v, v))


def _weights(blocks, scales, fmt):
    codes = np.stack((blocks & 15, blocks >> 4), axis=-1).reshape(*blocks.shape[:-1], -1)
    sc = np.where(scales == 255, np.nan, 2.0 ** (scales.astype(np.float64) - 127)) if fmt == "mxfp4" else _e4m3(scales)
    return VALUE[codes] * np.repeat(sc, 32 if fmt == "mxfp4" else 16, axis=-1)


def _bank(rng, E, N, K, fmt, exact=False):
    blocks = rng.integers(0, 256, (E, N, K // 2), dtype=np.uint8)
    if fmt == "mxfp4":
        scales = rng.integers(126, 129, (E, N, K // 32), dtype=np.uint8) if exact else \
            rng.integers(110, 140, (E, N, K // 32), dtype=np.uint8)
    elif exact:
        scales = rng.choice(np.array([0x30, 0x34, 0x38, 0x3C, 0x40, 0xB8], np.uint8), (E, N, K // 16))  # .5 .75 1 1.5 2 -1
    else:
        scales = rng.integers(0, 0x7F, (E, N, K // 16), dtype=np.uint8) | (rng.integers(0, 2, (E, N, K // 16), dtype=np.uint8) << 7)
    return blocks, scales


def _dev(a, dtype=None):
    import torch
    return None if a is None else torch.from_numpy(np.ascontiguousarray(a)).to("cuda", dtype)


def _call(moe, fmt, x, blocks, scales, scale2=None, **kw):
    if fmt == "mxfp4":
        return moe.mxfp4_matvec(x, blocks, scales, **kw)
    return moe.nvfp4_matvec(x, blocks, scales, scale2, **kw)


def _want(x64, W, ids, rows_per_x, scale2, bias, swiglu):
    """(y or its SwiGLU, sum of |w x| per output, y) in 64 bits"""
    R = ids.size
    xr = x64[np.arange(R) // rows_per_x]
    y = np.einsum("rnk,rk->rn", W[ids], xr) if R * W[0].size < 2e7 else np.stack([W[e] @ v for e, v in zip(ids, xr)])
    mag = np.einsum("rnk,rk->rn", np.abs(W[ids]), np.abs(xr)) if R * W[0].size < 2e7 else \
        np.stack([np.abs(W[e]) @ np.abs(v) for e, v in zip(ids, xr)])
    if scale2 is not None:
        s = scale2.astype(np.float64)[ids]
        s = np.tile(s, (1, W.shape[1] // 2)) if swiglu else s[:, None]
        y, mag = y * s, mag * np.abs(s)
    if bias is not None:
        y = y + bias.astype(np.float64)[ids]
        mag = mag + np.abs(bias.astype(np.float64)[ids])
    if not swiglu:
        return y, mag, y
    g, u = np.minimum(y[:, ::2], LIMIT), np.clip(y[:, 1::2], -LIMIT, LIMIT)
    with np.errstate(over="ignore"):
        return (u + 1) * g / (1 + np.exp(-ALPHA * g)), mag, y


SHAPES = [
    # T, k, E, N, K, ids
    (1, 1, 1, 1, 32, False),            # one output
    (1, 1, 1, 2880, 2880, False),
    (1, 4, 32, 90, 96, True),
    (3, 1, 1, 34, 64, False),           # several rows, one matrix
    (8, 1, 1, 130, 160, False),
    (9, 1, 1, 48, 352, False),          # one row past a tile of eight
    (33, 1, 1, 20, 416, False),         # past four tiles
    (70, 1, 1, 66, 128, False),
    (16, 4, 5, 62, 288, True),          # several rows per expert
    (64, 4, 128, 32, 1024, True),
    (5, 3, 200, 18, 8192, True),        # long K, many experts
    (1, 1, 1, 6, 20000, False),
    (5, 1, 1, 70, 32768, False),        # the longest rows: fewer rows of x at a time
    (8, 1, 1, 8190, 512, False),        # items of 64 weight rows, one partial stage
    (16, 4, 4, 1500, 2912, True),       # items of 128, up to two tiles of x per expert, a ragged last stage
    (16, 4, 16, 1500, 640, True),
]


@pytest.mark.parametrize("swiglu", [False, True], ids=["linear", "swiglu"])
@pytest.mark.parametrize("fmt,xdt", [("mxfp4", "bfloat16"), ("mxfp4", "float16"), ("nvfp4", "bfloat16"), ("nvfp4", "float16")])
@pytest.mark.parametrize("T,k,E,N,K,has_ids", SHAPES)
def test_exact_inputs_and_random_inputs(moe_gpu, T, k, E, N, K, has_ids, fmt, xdt, swiglu):
    import torch
    moe = moe_gpu
    if swiglu and N % 2:
        N += 1
    rng = np.random.default_rng(T * 1000 + N + K)
    R = T * k
    ids = (np.stack([rng.permutation(E)[:k] for _ in range(T)]).reshape(-1) if has_ids else np.zeros(R, np.int64)).astype(np.int32)
    row_ids = _dev(ids) if has_ids else None
    dt = getattr(torch, xdt)
    moe.moe_get_device_error()
    # exact: |x| <= 4, |w| <= 12, steps of 1/8: K * 48 * 8 < 2^24 for K <= 43690
    blocks, scales = _bank(rng, E, N, K, fmt, exact=True)
    x = rng.integers(-4, 5, (T, K)).astype(np.float64)
    bias = rng.integers(-8, 9, (E, N)).astype(np.float32)
    kw = dict(bias=_dev(bias), row_ids=row_ids, rows_per_x=k)
    W = _weights(blocks, scales, fmt)
    want, _, _ = _want(x, W, ids, k, None, bias, False)
    got = _call(moe, fmt, _dev(x, dt), _dev(blocks), _dev(scales), out_dtype=torch.float32, **kw)
    np.testing.assert_array_equal(got.cpu().numpy().astype(np.float64), want)
    same = _call(moe, fmt, _dev(x, dt), _dev(blocks), _dev(scales), **kw)
    assert torch.equal(same, got.to(dt)) and same.dtype == dt
    # random
    blocks, scales = _bank(rng, E, N, K, fmt)
    xt = torch.from_numpy(rng.standard_normal((T, K))).to(dt)
    bias = rng.standard_normal((E, N)).astype(np.float32)
    scale2 = (0.5 + rng.random((E, 2) if swiglu else E)).astype(np.float32) / 64 if fmt == "nvfp4" else None
    kw = dict(bias=_dev(bias), row_ids=row_ids, rows_per_x=k, swiglu=swiglu)
    want, mag, y = _want(xt.double().numpy(), _weights(blocks, scales, fmt), ids, k, scale2, bias, swiglu)
    acc = (K + 64) * 2.0 ** -23 * mag
    if swiglu:
        acc = 1.2 * (LIMIT + 1) * (acc[:, ::2] + acc[:, 1::2]) + 32 * 2.0 ** -24 * (np.abs(want) + LIMIT)
    for odt in (torch.float32, dt):
        got = _call(moe, fmt, xt.cuda(), _dev(blocks), _dev(scales), _dev(scale2), out_dtype=odt, **kw)
        assert got.shape == want.shape
        tol = 1.01 * (torch.finfo(odt).eps / 2 * np.abs(want) + acc) + (2.0 ** -25 if odt == torch.float16 else 0)
        g = got.double().cpu().numpy()
        if odt == torch.float16:                        # results past its range are infinite
            top = np.abs(want) > 65504
            assert np.isinf(g[np.abs(want) > 65520 + acc]).all()
            g, want_, tol = np.where(top, 0, g), np.where(top, 0, want), np.where(top, 1, tol)
            g = np.where(np.isinf(g) & (np.abs(want_) + acc >= 65504), want_, g)
        else:
            want_ = want
        bad = ~(np.abs(g - want_) <= tol)
        assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[0], g[bad][:2], want_[bad][:2])
    assert moe.moe_get_device_error() == 0


@pytest.mark.parametrize("xdt", ["bfloat16", "float16"])
def test_every_code_scale_and_magnitude(moe_gpu, xdt):
    # one element at a time: out[r, n] = W[n, r] x exactly, over all codes and E8M0 scales 0..254
    # (products below 2^-149 or past the fp32 range excepted), with x tiny, one and large
    import torch
    moe = moe_gpu
    K, N = 256, 256
    codes = (np.arange(N)[:, None] + np.arange(K)[None, :]) % 16
    blocks = (codes[:, ::2] | (codes[:, 1::2] << 4)).astype(np.uint8)
    scales = np.minimum(np.arange(N)[:, None] + np.arange(K // 32)[None, :] * 3, 254).astype(np.uint8)
    W = _weights(blocks[None], scales[None], "mxfp4")[0]
    for value in (2.0 ** -14, 1.0, 1.0 + 2.0 ** -7, 2.0 ** 15):
        x = torch.zeros((K, K), dtype=getattr(torch, xdt))
        x.fill_diagonal_(value)
        got = moe.mxfp4_matvec(x.cuda(), _dev(blocks), _dev(scales), out_dtype=torch.float32).double().cpu().numpy()
        want = W.T * float(x[0, 0])
        ok = (np.abs(want) < 2.0 ** 126) & ((np.abs(want) >= 2.0 ** -110) | (want == 0))
        np.testing.assert_array_equal(got[ok], want[ok])
    assert moe.moe_get_device_error() == 0


def test_every_e4m3_scale(moe_gpu):
    import torch
    moe = moe_gpu
    K, N = 64, 256
    codes = (np.arange(N)[:, None] * 5 + np.arange(K)[None, :]) % 16
    blocks = (codes[:, ::2] | (codes[:, 1::2] << 4)).astype(np.uint8)
    scales = np.repeat(np.arange(N, dtype=np.uint8)[:, None], K // 16, axis=1)
    scales[(scales & 0x7F) == 0x7F] = 0x38
    W = _weights(blocks[None], scales[None], "nvfp4")[0]
    for dt in (torch.bfloat16, torch.float16):
        x = torch.eye(K, dtype=dt) * 1.5
        got = moe.nvfp4_matvec(x.cuda(), _dev(blocks), _dev(scales), out_dtype=torch.float32).double().cpu().numpy()
        np.testing.assert_array_equal(got, W.T * 1.5)
    assert moe.moe_get_device_error() == 0


def test_wide_ranging_x_keeps_its_small_values(moe_gpu):
    # a row of x whose values span 2^28 below its largest, each alone under a weight: nothing of it is lost
    import torch
    moe = moe_gpu
    K, N = 64, 64
    codes = np.where(np.eye(N, K, dtype=np.int64) == 1, 2, 0)              # W = identity (code 2 is 1.0)
    blocks = (codes[:, ::2] | (codes[:, 1::2] << 4)).astype(np.uint8)
    scales = np.full((N, K // 32), 127, np.uint8)
    for top in (2.0 ** 100, 1.0, 2.0 ** -90):
        x = torch.tensor([[top * (1 + 2.0 ** -7) * 2.0 ** -(i % 29) for i in range(K)]], dtype=torch.bfloat16)
        got = moe.mxfp4_matvec(x.cuda(), _dev(blocks), _dev(scales), out_dtype=torch.float32)
        np.testing.assert_array_equal(got.double().cpu().numpy(), x.double().numpy())
    assert moe.moe_get_device_error() == 0


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
def test_infinities_and_nan_in_x(moe_gpu, fmt):
    # they reach their own rows only; an infinity under a positive weight is infinite
    import torch
    moe = moe_gpu
    K, N = 96, 40
    blocks = np.full((N, K // 2), 0x22, np.uint8)                            # W = 1
    scales = np.full((N, K // 32), 127, np.uint8) if fmt == "mxfp4" else np.full((N, K // 16), 0x38, np.uint8)
    x = torch.ones((4, K), dtype=torch.bfloat16)
    x[1, 17] = float("inf")
    x[2, 50] = float("nan")
    got = _call(moe, fmt, x.cuda(), _dev(blocks), _dev(scales), out_dtype=torch.float32).cpu()
    assert bool((got[0] == K).all()) and bool((got[3] == K).all())
    assert bool(torch.isposinf(got[1]).all()) and bool(torch.isnan(got[2]).all())
    # zero weights: a row of zeros gives zero, all-zero x too
    zero = _call(moe, fmt, torch.zeros((1, K), dtype=torch.bfloat16).cuda(), _dev(blocks), _dev(scales))
    assert bool((zero == 0).all())
    assert moe.moe_get_device_error() == 0


@pytest.mark.parametrize("odt", ["bfloat16", "float32"])
def test_infinities_and_nan_through_the_activation(moe_gpu, odt):
    # NaN stays NaN in the gate and in the up output (an invalid scale among the causes); an infinite
    # gate or up output is clamped like any large one
    import torch
    moe = moe_gpu
    K, N = 64, 8
    blocks = np.zeros((N, K // 2), np.uint8)
    blocks[:, 0] = 0x02                                                     # W[n, 0] = 1, the rest 0
    blocks[0, :] = 0x00
    blocks[2:4, 16] = 0x02                                                  # outputs 2, 3 also read x[32]
    blocks[5, 16] = 0x02                                                    # output 5 (an up) does
    blocks[6, 16] = 0x02                                                    # output 6 (a gate) does
    scales = np.full((N, K // 32), 127, np.uint8)
    x = torch.zeros((4, K), dtype=torch.bfloat16)
    x[:, 0] = 1.0
    x[1, 32], x[2, 32], x[3, 0] = float("inf"), 1.0, 0.0
    gu = x.double().numpy()[:, [0]].repeat(N, axis=1)
    gu[:, 0] = 0
    bad = scales.copy()
    bad[6, 1] = 255
    got = moe.mxfp4_matvec(x.cuda(), _dev(blocks), _dev(scales), swiglu=True, out_dtype=getattr(torch, odt)).double().cpu().numpy()
    y = gu.copy()
    for n in (2, 3, 5, 6):
        y[:, n] += x.double().numpy()[:, 32]
    # every output reads 0 * x[32] too: row 1's infinity makes those NaN
    y[1, [0, 1, 4, 7]] = np.nan
    with np.errstate(invalid="ignore"):
        g = np.where(y[:, ::2] > LIMIT, LIMIT, y[:, ::2])
        u = np.where(y[:, 1::2] > LIMIT, LIMIT, y[:, 1::2])
        want = (u + 1) * g / (1 + np.exp(-ALPHA * g))
    np.testing.assert_array_equal(np.isnan(got), np.isnan(want))
    ok = ~np.isnan(want)
    # products and sums here are exact: 32 roundings of the activation, one of the result
    u_ = torch.finfo(getattr(torch, odt)).eps / 2
    assert (np.abs(got[ok] - want[ok]) <= (u_ + 32 * 2.0 ** -24) * np.abs(want[ok])).all()
    assert np.isnan(want).any() and np.isfinite(want[1]).any()
    moe.moe_get_device_error()
    got = moe.mxfp4_matvec(x.cuda(), _dev(blocks), _dev(bad), swiglu=True, out_dtype=getattr(torch, odt)).cpu()
    assert moe.moe_get_device_error() == moe.MOE_DEVERR_BAD_SCALE
    assert bool(torch.isnan(got[:, 3]).all()) and bool(torch.isfinite(got[0, :3]).all())


@pytest.mark.parametrize("fmt,bad", [("mxfp4", 255), ("nvfp4", 0x7F), ("nvfp4", 0xFF)])
def test_an_invalid_scale_is_nan_and_flagged(moe_gpu, fmt, bad):
    import torch
    moe = moe_gpu
    rng = np.random.default_rng(1)
    E, N, K = 3, 40, 96
    blocks, scales = _bank(rng, E, N, K, fmt, exact=True)
    scales[1, 7, 1] = bad
    x = torch.ones((2, K), dtype=torch.bfloat16, device="cuda")
    ids = torch.tensor([1, 2], dtype=torch.int32, device="cuda")
    moe.moe_get_device_error()
    got = _call(moe, fmt, x, _dev(blocks), _dev(scales), row_ids=ids, out_dtype=torch.float32).cpu()
    assert moe.moe_get_device_error() == moe.MOE_DEVERR_BAD_SCALE
    nan = torch.isnan(got)
    assert bool(nan[0, 7]) and int(nan.sum()) == 1
    # an expert that no row names is not read
    _call(moe, fmt, x, _dev(blocks), _dev(scales), row_ids=torch.tensor([0, 2], dtype=torch.int32, device="cuda"))
    assert moe.moe_get_device_error() == 0


def test_rows_of_bad_experts_stay_unwritten(moe_gpu):
    import torch
    moe = moe_gpu
    rng = np.random.default_rng(2)
    E, N, K = 4, 48, 64
    blocks, scales = _bank(rng, E, N, K, "mxfp4", exact=True)
    x = torch.from_numpy(rng.integers(-3, 4, (6, K))).to("cuda", torch.bfloat16)
    ids = torch.tensor([3, -1, 0, 4, 3, 2 ** 30], dtype=torch.int32, device="cuda")
    out = torch.full((6, N), 77.0, device="cuda")
    moe.moe_get_device_error()
    moe.mxfp4_matvec(x, _dev(blocks), _dev(scales), row_ids=ids, out=out)
    assert moe.moe_get_device_error() == moe.MOE_DEVERR_BAD_EXPERT_ID
    W = _weights(blocks, scales, "mxfp4")
    for r, e in enumerate(ids.tolist()):
        want = W[e] @ x[r].double().cpu().numpy() if 0 <= e < E else np.full(N, 77.0)
        np.testing.assert_array_equal(out[r].double().cpu().numpy(), want)


def test_strided_x_and_odd_matrix_starts(moe_gpu):
    # x rows inside wider rows; N * K/32 odd, so an expert's scales start at any byte
    import torch
    moe = moe_gpu
    rng = np.random.default_rng(3)
    for fmt in ("mxfp4", "nvfp4"):
        E, N, K = 7, 37, 96
        blocks, scales = _bank(rng, E, N, K, fmt, exact=True)
        wide = torch.from_numpy(rng.integers(-3, 4, (11, K + 40))).to("cuda", torch.bfloat16)
        x = wide[:, 16:16 + K]
        ids = torch.from_numpy(rng.integers(0, E, 11).astype(np.int32)).cuda()
        got = _call(moe, fmt, x, _dev(blocks), _dev(scales), row_ids=ids, out_dtype=torch.float32)
        W = _weights(blocks, scales, fmt)
        want = np.stack([W[e] @ v for e, v in zip(ids.tolist(), x.double().cpu().numpy())])
        np.testing.assert_array_equal(got.double().cpu().numpy(), want)


@pytest.mark.parametrize("R,E", [(1024, 3), (1024, 256), (700, 1)])
def test_many_rows(moe_gpu, R, E):
    import torch
    moe = moe_gpu
    rng = np.random.default_rng(R + E)
    N, K = 40, 64
    blocks, scales = _bank(rng, E, N, K, "mxfp4", exact=True)
    x = rng.integers(-3, 4, (R, K)).astype(np.float64)
    ids = rng.integers(0, E, R).astype(np.int32)
    got = moe.mxfp4_matvec(_dev(x, torch.bfloat16), _dev(blocks), _dev(scales), row_ids=_dev(ids), out_dtype=torch.float32)
    want, _, _ = _want(x, _weights(blocks, scales, "mxfp4"), ids, 1, None, None, False)
    np.testing.assert_array_equal(got.double().cpu().numpy(), want)


def test_same_bits_again_on_a_stream_and_in_a_graph(moe_gpu):
    import torch
    moe = moe_gpu
    rng = np.random.default_rng(4)
    E, N, K, T, k = 16, 192, 2880, 6, 4
    blocks, scales = (_dev(a) for a in _bank(rng, E, N, K, "mxfp4"))
    x = torch.from_numpy(rng.standard_normal((T, K))).to("cuda", torch.bfloat16)
    ids = torch.from_numpy(np.stack([rng.permutation(E)[:k] for _ in range(T)]).astype(np.int32)).cuda()
    run = lambda stream=None: moe.mxfp4_matvec(x, blocks, scales, row_ids=ids, rows_per_x=k, swiglu=True, stream=stream)  # noqa: E731
    want = run()
    assert torch.equal(run(), want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    two = [run(side), run()]                               # two calls at once
    torch.cuda.synchronize()
    assert torch.equal(two[0], want) and torch.equal(two[1], want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = run()
    ids.copy_(ids.flip(0).clone())
    x.copy_(x.flip(0).clone())
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(got.view(T, k, -1).flip(0).reshape(got.shape), want)


# ---- a decode step ---------------------------------------------------------------------
@pytest.mark.parametrize("name", ["tiny_woo", "20b_decode_T1", "20b_decode_T8", "nvfp4_20b_decode_T8"])
def test_a_decode_step_against_the_oracle(moe_gpu, oracle_mod, name):
    """route -> gate_up product with SwiGLU -> down product -> weighted sum, in pair order without a sort,
    within the layer's tolerance of the oracle."""
    import torch

    from mxfp4_expert_ffn_moe_b200.workloads import workload
    from tests._metrics import MAX_ABS_OVER_RMS_TOL, REL_L2_TOL, max_abs_over_rms, rel_l2
    from tests.gpu_util import bf16_tensor_to_f64, layer_to_device, nvfp4_layer_to_device, oracle_forward, oracle_nvfp4_forward
    moe = moe_gpu
    layer = workload(name)
    nv = layer.fmt == "nvfp4"
    dev = nvfp4_layer_to_device(layer) if nv else layer_to_device(layer)
    k = layer.k
    ids, w = moe.moe_route(dev["logits"], k)
    up = dict(bias=dev["gu_bias"], row_ids=ids, rows_per_x=k, swiglu=True, alpha=layer.alpha, limit=layer.limit)
    down = dict(bias=dev["d_bias"], row_ids=ids, out_dtype=torch.float32)
    if nv:
        act = moe.nvfp4_matvec(dev["x"], dev["gu_blocks"], dev["gu_scales"], dev["gu_scale2"], **up)
        y = moe.nvfp4_matvec(act, dev["d_blocks"], dev["d_scales"], dev["d_scale2"], **down)
    else:
        act = moe.mxfp4_matvec(dev["x"], dev["gu_blocks"], dev["gu_scales"], **up)
        y = moe.mxfp4_matvec(act, dev["d_blocks"], dev["d_scales"], **down)
    out = moe.moe_combine_rows(y, None, layer.T, k, weights=w, dtype=torch.bfloat16)
    assert moe.moe_get_device_error() == 0
    ids_o, w_o = oracle_mod.route(layer.logits, k)
    want = (oracle_nvfp4_forward if nv else oracle_forward)(oracle_mod, layer, ids_o, w_o)
    got = bf16_tensor_to_f64(out)
    assert rel_l2(got, want) <= REL_L2_TOL and max_abs_over_rms(got, want) <= MAX_ABS_OVER_RMS_TOL

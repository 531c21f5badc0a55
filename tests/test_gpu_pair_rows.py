"""moe_dispatch_rows, moe_combine_rows, their gradients and moe_route_backward on the GPU
against their definitions in 64 bits.

Tolerances, with u the half step of the result's type (bf16 2^-8, fp16 2^-11, fp32 2^-24)
and e = 2^-24 of an fp32 operation: a spread is one product and one rounding, (u + e)|v|;
a sum of k products is k fused steps and one rounding, u|v| + k e sum|s y|; a dot adds at
most ceil(H/32) terms in a thread, 5 shuffle steps and 8 warps, (ceil(H/32) + 13) e
sum|a y|.  fp16 results below the normal range round by at most 2^-25.  Second-order terms are below
the factor 1.01.
"""
import math

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

E24 = 2.0 ** -24
TYPES = [("bfloat16", "bfloat16"), ("float16", "float16"), ("float32", "float32"), ("bfloat16", "float32"),
         ("float16", "float32")]


def _dt(name):
    import torch
    return getattr(torch, name)


def _close(got, want, mag, steps, what):
    """|got - want| <= 1.01 (u |want| + steps e mag) (+ the fp16 subnormal half step)"""
    import torch
    u = torch.finfo(got.dtype).eps / 2
    tol = 1.01 * (u * want.abs() + steps * E24 * mag) + (2.0 ** -25 if got.dtype == torch.float16 else 2.0 ** -140)
    bad = (got.double() - want).abs() > tol
    assert not bool(bad.any()), f"{what}: {int(bad.sum())} of {bad.numel()} off, first at {bad.nonzero()[0].tolist()}"
    assert bool(torch.isfinite(got).all()), what


def _case(T, k, E, H, drop, seed, extra_rows=0):
    """A permutation as moe_permute makes it, with a share of pairs dropped: pair_rows, weights, R."""
    import torch
    g = torch.Generator().manual_seed(seed)
    ids = torch.rand((T, E), generator=g).argsort(dim=1)[:, :k].reshape(-1)
    kept = torch.rand(T * k, generator=g) >= drop
    if drop and T > 2:
        kept[k:2 * k] = False                                    # a token that is dropped altogether
        kept[0] = True
    key = torch.where(kept, ids, E)
    order = torch.argsort(key, stable=True)
    rows = torch.empty(T * k, dtype=torch.int64)
    rows[order] = torch.arange(T * k)
    pair_rows = torch.where(kept, rows, torch.tensor(-1)).to(torch.int32)
    weights = torch.softmax(torch.randn((T, k), generator=g), dim=1)
    return pair_rows.cuda(), weights.cuda(), int(kept.sum()) + extra_rows, g


def _randn(shape, dtype, g):
    import torch
    return torch.randn(shape, generator=g).to(_dt(dtype)).cuda()


def _spread64(a, pair_rows, w, R, k):
    """(rows [R, H], written [R]) in 64 bits"""
    import torch
    T, H = a.shape
    rows = torch.zeros((R, H), dtype=torch.float64, device="cuda")
    written = torch.zeros(R, dtype=torch.bool, device="cuda")
    ok = pair_rows >= 0
    p = ok.nonzero()[:, 0]
    rows[pair_rows[p].long()] = a.double()[p // k] * w.double().reshape(-1)[p, None]
    written[pair_rows[p].long()] = True
    return rows, written


def _pairs64(rows, pair_rows, T, k):
    import torch
    out = torch.zeros((T * k, rows.shape[1]), dtype=torch.float64, device="cuda")
    p = (pair_rows >= 0).nonzero()[:, 0]
    out[p] = rows.double()[pair_rows[p].long()]
    return out.view(T, k, -1)


SHAPES = [
    # T, k, E, H, drop
    (1, 1, 1, 1, 0.0),              # one element
    (1, 4, 32, 2880, 0.0),          # one token of the gpt-oss-20b layer
    (3, 2, 5, 7, 0.3),              # odd width, an empty token
    (37, 3, 7, 1001, 0.2),          # odd width over several chunks
    (64, 8, 256, 66, 0.1),          # most slots, width a multiple of 2 only
    (300, 4, 32, 2880, 0.05),
    (19, 5, 9, 40, 0.5),            # more slots than 4, few chunks
    (5000, 2, 4, 64, 0.0),          # a warp per token
    (6, 7, 8, 8200, 0.0),           # long rows, in segments
    (7, 8, 8, 8201, 0.2),           # the same off 16-byte words
    (700, 8, 16, 24, 0.1),
]


@pytest.mark.parametrize("weighted", [True, False], ids=["weighted", "plain"])
@pytest.mark.parametrize("tok,row", TYPES)
@pytest.mark.parametrize("T,k,E,H,drop", SHAPES)
def test_against_64_bits(moe_gpu, T, k, E, H, drop, tok, row, weighted):
    import torch
    moe = moe_gpu
    pair_rows, w, R, g = _case(T, k, E, H, drop, seed=T + H, extra_rows=2)
    ones = torch.ones_like(w)
    ww, w64 = (w, w) if weighted else (None, ones)
    x, y = _randn((T, H), tok, g), _randn((R, H), row, g)
    # spread
    rows = torch.full((R, H), 7.0, dtype=_dt(row), device="cuda")
    got = moe.moe_dispatch_rows(x, pair_rows, k, weights=ww, rows=rows)
    want, written = _spread64(x, pair_rows, w64, R, k)
    assert got is rows and int(written.sum()) == R - 2
    _close(got[written], want[written], want[written].abs(), 1, "dispatch")
    assert bool((got[~written] == 7.0).all())                    # rows no pair names stay
    # sum
    parts = _pairs64(y, pair_rows, T, k) * w64.double()[:, :, None]
    out = moe.moe_combine_rows(y, pair_rows, T, k, weights=ww, dtype=_dt(tok))
    assert out.dtype == _dt(tok)
    _close(out, parts.sum(1), parts.abs().sum(1), k, "combine")
    # gradients: of the dispatch (drows = y) and of the combine (dout = x), with the dots
    steps = math.ceil(H / 32) + 13
    prods = _pairs64(y, pair_rows, T, k) * x.double()[:, None, :]
    dx, dw = moe.moe_dispatch_rows_backward(y, pair_rows, T, k, weights=ww, x=x)
    _close(dx, parts.sum(1), parts.abs().sum(1), k, "dispatch backward: dx")
    _close(dw, prods.sum(2), prods.abs().sum(2), steps, "dispatch backward: dweights")
    drows = torch.full((R, H), -3.0, dtype=_dt(row), device="cuda")
    drows, dw2 = moe.moe_combine_rows_backward(x, pair_rows, k, weights=ww, y_rows=y, drows=drows)
    _close(drows[written], want[written], want[written].abs(), 1, "combine backward: drows")
    assert bool((drows[~written] == -3.0).all())
    _close(dw2, prods.sum(2), prods.abs().sum(2), steps, "combine backward: dweights")
    # without the dots: the same bits
    assert torch.equal(moe.moe_dispatch_rows_backward(y, pair_rows, T, k, weights=ww, dtype=_dt(tok)), dx)
    drows3 = torch.full((R, H), -3.0, dtype=_dt(row), device="cuda")
    assert torch.equal(moe.moe_combine_rows_backward(x, pair_rows, k, weights=ww, drows=drows3), drows)
    assert moe.moe_get_device_error() == 0


def test_dropped_pairs_read_nothing(moe_gpu):
    # NaN and infinity behind dropped pairs (their weights, and rows no pair names) reach nothing
    import torch
    moe = moe_gpu
    T, k, H = 40, 4, 96
    pair_rows, w, R, g = _case(T, k, 16, H, 0.4, seed=3, extra_rows=5)
    x, y = _randn((T, H), "bfloat16", g), _randn((R, H), "bfloat16", g)
    y[R - 5:] = float("nan")
    dropped = (pair_rows < 0).view(T, k)
    bad = w.clone()
    bad[dropped] = float("nan")
    bad2 = w.clone()
    bad2[dropped] = float("inf")
    for a, b in ((bad, bad2), (bad2, w)):
        assert torch.equal(moe.moe_combine_rows(y, pair_rows, T, k, weights=a), moe.moe_combine_rows(y, pair_rows, T, k, weights=b))
    dx, dw = moe.moe_dispatch_rows_backward(y, pair_rows, T, k, weights=bad, x=x)
    assert bool(torch.isfinite(dx).all()) and bool((dx[1] == 0).all()) and bool((dw[dropped] == 0).all())
    rows = torch.full((R, H), 5.0, dtype=torch.bfloat16, device="cuda")
    rows, dw = moe.moe_combine_rows_backward(x, pair_rows, k, weights=bad, y_rows=y, drows=rows)
    assert bool(torch.isfinite(rows).all()) and bool((rows[R - 5:] == 5.0).all()) and bool((dw[dropped] == 0).all())
    # any negative entry drops a pair
    neg = torch.where(pair_rows < 0, torch.tensor(-2 ** 31, dtype=torch.int32, device="cuda"), pair_rows)
    assert torch.equal(moe.moe_combine_rows(y, neg, T, k, weights=w), moe.moe_combine_rows(y, pair_rows, T, k, weights=w))
    # NaN and infinity in rows that are used come through
    y[int(pair_rows[0])] = float("nan")
    assert bool(torch.isnan(moe.moe_combine_rows(y, pair_rows, T, k, weights=w)[0]).all())
    assert moe.moe_get_device_error() == 0


def test_a_row_past_the_buffer_is_dropped_and_flagged(moe_gpu):
    # the host and the kernel check the entry: nothing outside the buffers is touched
    import torch
    moe = moe_gpu
    T, k, H = 10, 2, 64
    g = torch.Generator().manual_seed(1)
    pair_rows = torch.arange(T * k, dtype=torch.int32, device="cuda")
    good = pair_rows.clone()
    good[5] = -1
    x, y = _randn((T, H), "bfloat16", g), _randn((T * k, H), "bfloat16", g)
    for value in (T * k, 2 ** 31 - 1):
        pair_rows[5] = value
        moe.moe_get_device_error()
        out = moe.moe_combine_rows(y, pair_rows, T, k)
        assert moe.moe_get_device_error() == moe.MOE_DEVERR_OUT_OF_BOUNDS
        assert torch.equal(out, moe.moe_combine_rows(y, good, T, k))
        rows = torch.zeros_like(y)
        moe.moe_dispatch_rows(x, pair_rows, k, rows=rows)
        assert moe.moe_get_device_error() == moe.MOE_DEVERR_OUT_OF_BOUNDS
        assert bool((rows[5] == 0).all()) and torch.equal(rows[6], x[3])


def test_the_same_row_twice_is_summed_twice(moe_gpu):
    import torch
    moe = moe_gpu
    g = torch.Generator().manual_seed(4)
    y = _randn((3, 32), "float32", g)
    pair_rows = torch.tensor([2, 2, 0, 1], dtype=torch.int32, device="cuda")
    out = moe.moe_combine_rows(y, pair_rows, 2, 2)
    assert torch.equal(out, torch.stack((y[2] + y[2], y[0] + y[1])))


@pytest.mark.parametrize("tok,row", [("bfloat16", "bfloat16"), ("float32", "float32"), ("float16", "float32")])
@pytest.mark.parametrize("off,pad", [(0, 8), (1, 3), (2, 2), (8, 56), (3, 0)])
def test_strided_and_unaligned_rows(moe_gpu, tok, row, off, pad):
    # rows inside wider rows, at any element offset: the same bits as contiguous ones
    import torch
    moe = moe_gpu
    T, k, H = 23, 3, 64
    pair_rows, w, R, g = _case(T, k, 8, H, 0.1, seed=off + pad)

    def wide(t):
        buf = torch.full((t.shape[0], off + H + pad), 9.0, dtype=t.dtype, device="cuda")
        view = buf[:, off:off + H]
        view.copy_(t)
        return buf, view

    x, y = _randn((T, H), tok, g), _randn((R, H), row, g)
    _, xs = wide(x)
    _, ys = wide(y)
    buf, rows = wide(torch.zeros_like(y))
    moe.moe_dispatch_rows(xs, pair_rows, k, weights=w, rows=rows)
    assert torch.equal(rows, moe.moe_dispatch_rows(x, pair_rows, k, weights=w, n_rows=R, dtype=_dt(row)))
    assert bool((buf[:, :off] == 9).all()) and bool((buf[:, off + H:] == 9).all())
    buf, out = wide(torch.zeros_like(x))
    moe.moe_combine_rows(ys, pair_rows, T, k, weights=w, out=out)
    assert torch.equal(out, moe.moe_combine_rows(y, pair_rows, T, k, weights=w, dtype=_dt(tok)))
    assert bool((buf[:, :off] == 9).all()) and bool((buf[:, off + H:] == 9).all())
    # the order of a dot's terms goes by the chunk width, so dots are compared to their bound
    _, dx = wide(torch.zeros_like(x))
    _, dw = moe.moe_dispatch_rows_backward(ys, pair_rows, T, k, weights=w, x=xs, dx=dx)
    prods = _pairs64(y, pair_rows, T, k) * x.double()[:, None, :]
    _close(dw, prods.sum(2), prods.abs().sum(2), math.ceil(H / 32) + 13, "dweights")
    assert torch.equal(dx, moe.moe_dispatch_rows_backward(y, pair_rows, T, k, weights=w, dtype=_dt(tok)))


def test_repeated_rows_and_no_permutation(moe_gpu):
    # a gradient that is one row for all tokens (stride 0), and rows in pair order (pair_rows None)
    import torch
    moe = moe_gpu
    T, k, H = 33, 4, 128
    g = torch.Generator().manual_seed(5)
    w = torch.rand((T, k), generator=g).cuda()
    y = _randn((T * k, H), "bfloat16", g)
    one = _randn((1, H), "bfloat16", g)
    drows, dw = moe.moe_combine_rows_backward(one.expand(T, H), None, k, weights=w, y_rows=y)
    want, dw_want = moe.moe_combine_rows_backward(one.expand(T, H).contiguous(), None, k, weights=w, y_rows=y)
    assert torch.equal(drows, want) and torch.equal(dw, dw_want)
    identity = torch.arange(T * k, dtype=torch.int32, device="cuda")
    assert torch.equal(moe.moe_combine_rows(y, None, T, k, weights=w), moe.moe_combine_rows(y, identity, T, k, weights=w))
    x = _randn((T, H), "bfloat16", g)
    assert torch.equal(moe.moe_dispatch_rows(x, None, k), x.repeat_interleave(k, dim=0))


def test_it_follows_the_layer_s_own_gather_and_combine(moe_gpu):
    # the inference calls of the same permutation: equal bits
    import torch
    moe = moe_gpu
    T, k, E, H = 257, 4, 32, 2880
    g = torch.Generator().manual_seed(6)
    logits = torch.randn((T, E), generator=g).cuda()
    ids, w = moe.moe_route(logits, k)
    perm = moe.moe_permute(ids, E, 32)
    x = _randn((T, H), "bfloat16", g)
    rows, _, row_w = moe.moe_gather_pairs(x, ids, w, perm, E)
    assert torch.equal(moe.moe_dispatch_rows(x, perm["pair_rows"], k), rows)
    y = _randn((T * k, H), "float32", g)
    scaled = (y.double() * row_w.double()[:, None]).float()
    assert torch.equal(moe.moe_combine_rows(scaled, perm["pair_rows"], T, k, dtype=torch.bfloat16),
                       moe.moe_combine_pairs(scaled, perm["pair_rows"], T, k))


def test_the_same_call_gives_the_same_bits_on_any_stream_and_in_a_graph(moe_gpu):
    import torch
    moe = moe_gpu
    T, k, H = 500, 4, 720
    pair_rows, w, R, g = _case(T, k, 16, H, 0.1, seed=8)
    x, y = _randn((T, H), "bfloat16", g), _randn((R, H), "bfloat16", g)
    ids = torch.rand((T, 16), generator=g).argsort(dim=1)[:, :k].to(torch.int32).contiguous().cuda()

    def step(stream=None):
        rows, dw = moe.moe_combine_rows_backward(x, pair_rows, k, weights=w, y_rows=y, stream=stream)
        dx, dw2 = moe.moe_dispatch_rows_backward(rows, pair_rows, T, k, weights=w, x=x, stream=stream)
        return rows, dw, dx, dw2, moe.moe_route_backward(dw2, ids, w, 16, stream=stream)

    want = step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = [step(side) for _ in range(3)][-1]
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = step()
    keep = x.clone()
    x.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert bool((captured[0] == 0).all()) and bool((captured[3] == 0).all())
    x.copy_(keep)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(captured, want))


def test_the_bounds_checked_build_gives_the_same(moe_gpu):
    import torch
    from mxfp4_expert_ffn_moe_b200 import build as moe_build
    moe_build.build(checked=True)
    moe = moe_gpu
    T, k, H = 90, 3, 250
    pair_rows, w, R, g = _case(T, k, 8, H, 0.1, seed=21)
    x, y = _randn((T, H), "float16", g), _randn((R, H), "float16", g)
    results = []
    for checked in (False, True):
        moe.use_checked_library(checked)
        try:
            moe.moe_get_device_error()
            rows = moe.moe_dispatch_rows(x, pair_rows, k, weights=w, n_rows=R)
            results.append((rows, moe.moe_combine_rows(y, pair_rows, T, k, weights=w),
                            *moe.moe_combine_rows_backward(x, pair_rows, k, weights=w, y_rows=y),
                            *moe.moe_dispatch_rows_backward(y, pair_rows, T, k, weights=w, x=x)))
            assert moe.moe_get_device_error() == 0
        finally:
            moe.use_checked_library(False)
    assert all(torch.equal(a, b) for a, b in zip(*results))


# ---- the router's gradient -----------------------------------------------------------
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 4, 2), (37, 7, 7), (300, 32, 4), (65, 200, 8), (5, 255, 8),
                                   (513, 256, 8), (4096, 32, 4), (2, 3, 1)])
def test_route_backward_against_64_bits(moe_gpu, T, E, k):
    import torch
    moe = moe_gpu
    g = torch.Generator().manual_seed(T + E)
    logits = torch.randn((T, E), generator=g).cuda()
    ids, w = moe.moe_route(logits, k)
    dw = torch.randn((T, k), generator=g).cuda()
    got = moe.moe_route_backward(dw, ids, w, E, dlogits=torch.full((T, E), 9.0, device="cuda"))
    w64, d64 = w.double(), dw.double()
    s = (w64 * d64).sum(1, keepdim=True)
    want = torch.zeros((T, E), dtype=torch.float64, device="cuda").scatter_(1, ids.long(), w64 * (d64 - s))
    # the inner sum: k fused steps; the difference and the product: one rounding each
    mag = torch.zeros_like(want).scatter_(1, ids.long(), w64 * (d64.abs() + (w64 * d64).abs().sum(1, keepdim=True)))
    _close(got, want, mag, k + 2, "dlogits")
    chosen = torch.zeros((T, E), dtype=torch.bool, device="cuda").scatter_(1, ids.long(), True)
    assert bool((got[~chosen] == 0).all())
    assert moe.moe_get_device_error() == 0


def test_route_backward_into_an_unaligned_gradient(moe_gpu):
    import torch
    moe = moe_gpu
    T, E, k = 301, 32, 4
    g = torch.Generator().manual_seed(9)
    ids, w = moe.moe_route(torch.randn((T, E), generator=g).cuda(), k)
    dw = torch.randn((T, k), generator=g).cuda()
    want = moe.moe_route_backward(dw, ids, w, E)
    for off in (1, 2, 3):
        buf = torch.full((T * E + 8,), 5.0, device="cuda")
        got = moe.moe_route_backward(dw, ids, w, E, dlogits=buf[off:off + T * E].view(T, E))
        assert torch.equal(got, want)
        assert bool((buf[:off] == 5).all()) and bool((buf[off + T * E:] == 5).all())


def test_route_backward_against_differences(moe_gpu):
    # d<dw, w(logits)>/dlogits by central differences of the softmax over the chosen, in 64 bits.  With
    # step h = 2^-13 the truncation is h^2/6 |w'''| |dw| <= 2^-26/6 * 6 * sum|dw| (the third derivative of a
    # softmax entry is below 6) and the rounding 2^-52 / h = 2^-39: under 2^-25 sum|dw| together.
    import torch
    moe = moe_gpu
    T, E, k, h = 12, 16, 4, 2.0 ** -13
    g = torch.Generator().manual_seed(2)
    logits = torch.randn((T, E), generator=g)
    ids, w = moe.moe_route(logits.cuda(), k)
    dw = torch.randn((T, k), generator=g)
    got = moe.moe_route_backward(dw.cuda(), ids, w, E).cpu().double()
    ids = ids.cpu().long()
    base = logits.double()

    def loss(at):
        return (torch.softmax(at.gather(1, ids), dim=1) * dw.double()).sum(1)

    bound = (dw.abs().sum(1) * (2.0 ** -25 + 8 * E24)).double()      # the kernel's own steps, and w's rounding
    for e in range(E):
        step = torch.zeros(E, dtype=torch.float64)
        step[e] = h
        diff = (loss(base + step) - loss(base - step)) / (2 * h)
        assert bool(((got[:, e] - diff).abs() <= bound).all()), e


def test_route_backward_empty_bad_and_repeated_slots(moe_gpu):
    import torch
    moe = moe_gpu
    ids = torch.tensor([[2, -1, -1], [1, 1, 0], [3, 9, 0], [-1, -1, -1]], dtype=torch.int32, device="cuda")
    w = torch.tensor([[1.0, float("nan"), 0.0], [0.25, 0.25, 0.5], [0.5, float("inf"), 0.5], [0.0, 0.0, 0.0]], device="cuda")
    dw = torch.tensor([[3.0, float("nan"), 1.0], [1.0, 3.0, 2.0], [1.0, 1.0, 3.0], [1.0, 1.0, 1.0]], device="cuda")
    moe.moe_get_device_error()
    got = moe.moe_route_backward(dw, ids, w, 4).cpu().numpy()
    assert moe.moe_get_device_error() == moe.MOE_DEVERR_BAD_EXPERT_ID         # the 9
    want = np.array([[0, 0, 0, 0], [0, 0, 0, 0], [0.5, 0, 0, -0.5], [0, 0, 0, 0]], np.float32)
    want[1] = [0.5 * (2 - 2), 0.25 * (1 - 2) + 0.25 * (3 - 2), 0, 0]
    np.testing.assert_array_equal(got, want)


def test_combine_gradients_against_differences(moe_gpu):
    # The combine is linear in the rows and in the weights: L = <G, combine(rows, w)> changes by exactly h
    # times the gradient.  Differences of the kernel's own fp32 outputs, at single entries.
    import torch
    moe = moe_gpu
    T, k, H = 9, 3, 50
    pair_rows, w, R, g = _case(T, k, 6, H, 0.2, seed=12)
    y, G = _randn((R, H), "float32", g), _randn((T, H), "float32", g)
    drows = torch.zeros_like(y)
    drows, dw = moe.moe_combine_rows_backward(G, pair_rows, k, weights=w, y_rows=y, drows=drows)

    def loss(rows, weights):
        return float((moe.moe_combine_rows(rows, pair_rows, T, k, weights=weights).double() * G.double()).sum())

    # each output moves by at most (k + 1) roundings of its magnitude, on both sides; h = 1
    mag = float((_pairs64(y, pair_rows, T, k).abs() * w.double()[:, :, None]).sum(1).mul(G.abs().double()).sum())
    slack = 2 * (k + 1) * E24 * (mag + float(G.abs().sum()) * (float(y.abs().max()) + 1))
    for p in range(0, T * k, 4):
        step = torch.zeros_like(w)
        step.view(-1)[p] = 0.5
        diff = loss(y, w + step) - loss(y, w - step)
        assert abs(diff - float(dw.view(-1)[p])) <= slack
    for r in range(0, R, 5):
        step = torch.zeros_like(y)
        step[r, r % H] = 0.5
        diff = loss(y + step, w) - loss(y - step, w)
        assert abs(diff - float(drows[r, r % H])) <= slack


# ---- a training step ------------------------------------------------------------------
@pytest.mark.parametrize("T,E,k,H,I", [(50, 8, 2, 64, 32), (33, 5, 4, 40, 24)])
def test_a_training_step_against_autograd_in_64_bits(moe_gpu, T, E, k, H, I):
    """route -> permute -> dispatch -> experts -> combine and back, fp32, against torch's
    autograd of the same layer in 64 bits.  The experts (tanh between two products) run in
    64 bits on both sides, so only the library's calls round: a handful of fp32 roundings
    per value, 2^-24 each, amplified by the experts' products; 64 of them, on the scale of
    each result's largest entry, cover the chain."""
    import torch
    moe = moe_gpu
    g = torch.Generator().manual_seed(T)
    x = torch.randn((T, H), generator=g).cuda()
    wr = (torch.randn((E, H), generator=g) / H ** 0.5).cuda()
    w1 = (torch.randn((E, H, I), generator=g) / H ** 0.5).cuda().double()
    w2 = (torch.randn((E, I, H), generator=g) / I ** 0.5).cuda().double()
    dout = torch.randn((T, H), generator=g).cuda()

    # reference: autograd in 64 bits through the same choice of experts
    x64, wr64 = x.double().requires_grad_(), wr.double().requires_grad_()
    logits64 = x64 @ wr64.T
    logits = logits64.detach().float()
    ids, w = moe.moe_route(logits, k)
    chosen = torch.softmax(logits64.gather(1, ids.long()), dim=1)
    h = torch.tanh(torch.einsum("th,tkhi->tki", x64, w1[ids.long()]))
    y = torch.einsum("tki,tkih->tkh", h, w2[ids.long()])
    out64 = (y * chosen[:, :, None]).sum(1)
    (out64 * dout.double()).sum().backward()

    # the library's calls around the same experts
    perm = moe.moe_permute(ids, E, 32)
    pr = perm["pair_rows"]
    rows = moe.moe_dispatch_rows(x, pr, k)
    row_e = torch.repeat_interleave(torch.arange(E, device="cuda"), perm["counts"].long())
    hr = torch.tanh(torch.einsum("rh,rhi->ri", rows.double(), w1[row_e]))
    y_rows = torch.einsum("ri,rih->rh", hr, w2[row_e]).float()
    out = moe.moe_combine_rows(y_rows, pr, T, k, weights=w)
    dy, dw = moe.moe_combine_rows_backward(dout, pr, k, weights=w, y_rows=y_rows)
    dh = torch.einsum("rh,rih->ri", dy.double(), w2[row_e]) * (1 - hr * hr)
    drows = torch.einsum("ri,rhi->rh", dh, w1[row_e]).float()
    dx = moe.moe_dispatch_rows_backward(drows, pr, T, k)
    dlogits = moe.moe_route_backward(dw, ids, w, E)
    dx_all = dx.double() + dlogits.double() @ wr.double()
    for got, want, what in ((out, out64.detach(), "out"), (dx_all, x64.grad, "dx"),
                            (dlogits.double().T @ x.double(), wr64.grad, "dw_router")):
        off = float((got.double() - want).abs().max())
        assert off <= 64 * E24 * float(want.abs().max()), (what, off)
    assert moe.moe_get_device_error() == 0

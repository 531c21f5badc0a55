"""Rows that no pair names, in the calls that write expert rows: zeros where the binding
allocates them or is asked to, left as they were in a given buffer otherwise."""
import pytest

from tests.test_gpu_pair_rows import _case, _dt, _randn

pytestmark = pytest.mark.gpu


def _stale(shape, dtype):
    """Memory of this size, holding NaN, goes back to the allocator."""
    import torch
    t = torch.full(shape, float("nan"), dtype=dtype, device="cuda")
    torch.cuda.synchronize()
    del t


CASES = [
    # T, k, E, H, drop, extra rows
    (1, 1, 1, 8, 0.0, 5),                # one pair, rows past it
    (3, 2, 5, 7, 0.3, 0),
    (300, 4, 32, 2880, 0.05, 0),
    (300, 4, 32, 2880, 0.0, 40),
    (700, 8, 16, 24, 0.5, 0),
    (5000, 8, 16, 40, 0.02, 0),          # narrow rows: several tokens a block
    (5000, 8, 16, 41, 0.7, 3),
    (2, 8, 8, 64, 0.0, 9000),            # a buffer far longer than its pairs
    (40, 3, 8, 8200, 0.4, 0),            # rows in segments
    (9000, 8, 8, 32, 0.0005, 0),         # many pairs of short rows, few dropped
    (9000, 4, 8, 400, 0.01, 50),         # many pairs of longer rows
    (60000, 8, 8, 24, 0.3, 7),           # many more
]


def _scattered(pair_rows, R, n_rows, seed):
    """The same pairs on rows anywhere in a buffer of n_rows: holes between them."""
    import torch
    g = torch.Generator().manual_seed(seed)
    place = torch.randperm(n_rows, generator=g)[:R].to(torch.int32).cuda()
    return torch.where(pair_rows < 0, pair_rows, place[pair_rows.clamp(min=0).long()])


@pytest.mark.parametrize("tok,row", [("bfloat16", "bfloat16"), ("float32", "float32"), ("float16", "float32")])
@pytest.mark.parametrize("scattered", [False, True], ids=["compact", "scattered"])
@pytest.mark.parametrize("T,k,E,H,drop,extra", CASES)
def test_rows_that_no_pair_names(moe_gpu, T, k, E, H, drop, extra, scattered, tok, row):
    import torch
    moe = moe_gpu
    pair_rows, w, R, g = _case(T, k, E, H, drop, seed=T + H)
    n = T * k + extra
    if scattered:
        pair_rows = _scattered(pair_rows, R, n, seed=H)
    x, y = _randn((T, H), tok, g), _randn((n, H), row, g)
    named = torch.zeros(n, dtype=torch.bool, device="cuda")
    named[pair_rows[pair_rows >= 0].long()] = True
    n_rows = n if extra else None
    calls = {
        "plain": (lambda **kw: moe.moe_dispatch_rows(x, pair_rows, k, n_rows=n_rows, dtype=_dt(row), **kw), "rows"),
        "weighted": (lambda **kw: moe.moe_dispatch_rows(x, pair_rows, k, weights=w, n_rows=n_rows, dtype=_dt(row), **kw), "rows"),
        "gradient": (lambda **kw: moe.moe_combine_rows_backward(x, pair_rows, k, weights=w, n_rows=n_rows, dtype=_dt(row), **kw), "drows"),
        "with dots": (lambda **kw: moe.moe_combine_rows_backward(x, pair_rows, k, weights=w, y_rows=y, **kw)[0], "drows"),
    }
    for what, (call, name) in calls.items():
        buf = torch.full((n, H), 7.0, dtype=_dt(row), device="cuda")
        kept = call(**{name: buf}).clone()
        assert bool((kept[~named] == 7).all()), what                 # a given buffer
        want = torch.where(named[:, None], kept, torch.zeros_like(kept))
        _stale((n, H), _dt(row))
        assert torch.equal(call(), want), what                        # an allocated one
        assert torch.equal(call(**{name: torch.full_like(buf, float("nan"))}, zero_skipped=True), want), what
        left = call(zero_skipped=False)
        assert torch.equal(left[named], want[named]), what
    assert moe.moe_get_device_error() == 0


@pytest.mark.parametrize("off,pad", [(0, 8), (1, 2), (3, 0)])
@pytest.mark.parametrize("extra", [0, 30])
def test_only_the_rows_themselves_become_zeros(moe_gpu, off, pad, extra):
    # rows inside wider rows: what lies between them stays
    import torch
    moe = moe_gpu
    T, k, H = 50, 4, 96
    pair_rows, w, R, g = _case(T, k, 8, H, 0.3, seed=off)
    n = T * k + extra
    pair_rows = _scattered(pair_rows, R, n, seed=1)
    x = _randn((T, H), "bfloat16", g)
    want = moe.moe_dispatch_rows(x, pair_rows, k, weights=w, n_rows=n)
    for ww in (w, None):
        buf = torch.full((n, off + H + pad), 9.0, dtype=torch.bfloat16, device="cuda")
        rows = buf[:, off:off + H]
        moe.moe_dispatch_rows(x, pair_rows, k, weights=ww, rows=rows, zero_skipped=True)
        if ww is not None:
            assert torch.equal(rows, want)
        assert bool((buf[:, :off] == 9).all()) and bool((buf[:, off + H:] == 9).all())


def test_no_permutation_and_rows_past_the_pairs(moe_gpu):
    import torch
    moe = moe_gpu
    g = torch.Generator().manual_seed(3)
    for T, k, H, n in ((5, 2, 64, 10), (5, 2, 64, 17), (5, 2, 33, 4000), (1, 1, 2880, 5000)):
        x = _randn((T, H), "bfloat16", g)
        _stale((n, H), torch.bfloat16)
        rows = moe.moe_dispatch_rows(x, None, k, n_rows=n)
        assert torch.equal(rows[:T * k], x.repeat_interleave(k, dim=0)) and bool((rows[T * k:] == 0).all())


def test_an_entry_past_the_buffer_leaves_its_row_zero(moe_gpu):
    import torch
    moe = moe_gpu
    g = torch.Generator().manual_seed(4)
    T, k, H = 30, 2, 64
    x = _randn((T, H), "bfloat16", g)
    pair_rows = torch.arange(T * k, dtype=torch.int32, device="cuda")
    pair_rows[7] = T * k
    moe.moe_get_device_error()
    _stale((T * k, H), torch.bfloat16)
    rows = moe.moe_dispatch_rows(x, pair_rows, k)
    assert moe.moe_get_device_error() == moe.MOE_DEVERR_OUT_OF_BOUNDS
    want = x.repeat_interleave(k, dim=0)
    want[7] = 0
    assert torch.equal(rows, want)


@pytest.mark.parametrize("T,k", [(901, 3), (15000, 3)], ids=["beside", "behind"])        # past 32768 pairs: a launch of their own
def test_pair_rows_at_any_address_on_a_stream_and_in_a_graph(moe_gpu, T, k):
    import torch
    moe = moe_gpu
    H = 48
    pair_rows, w, R, g = _case(T, k, 8, H, 0.1, seed=9)
    x = _randn((T, H), "float32", g)
    want = moe.moe_dispatch_rows(x, pair_rows, k, weights=w)
    side = torch.cuda.Stream()
    for off in (1, 2, 3):
        at = torch.empty(T * k + 4, dtype=torch.int32, device="cuda")[off:off + T * k]
        at.copy_(pair_rows)
        side.wait_stream(torch.cuda.current_stream())
        got = moe.moe_dispatch_rows(x, at, k, weights=w, stream=side)
        torch.cuda.synchronize()
        assert torch.equal(got, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = moe.moe_dispatch_rows(x, pair_rows, k, weights=w)
    for _ in range(2):
        got.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(got, want)
    # another routing in the same graph: other rows are left out
    pair_rows.copy_(torch.where(pair_rows >= 0, R - 1 - pair_rows, pair_rows).flip(0))
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(got, moe.moe_dispatch_rows(x, pair_rows, k, weights=w))

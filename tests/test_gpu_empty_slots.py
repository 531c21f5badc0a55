"""Empty slots of the routing (id -1, weight 0) through the calls that follow it on the GPU."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu


def _stale(shape, dtype):
    """Memory of this size, holding NaN, goes back to the allocator."""
    import torch
    t = torch.full(shape, float("nan"), dtype=dtype, device="cuda")
    torch.cuda.synchronize()
    del t


@pytest.mark.parametrize("own_buffers", [False, True], ids=["allocated", "given"])
@pytest.mark.parametrize("name", ["tiny_woo", "20b_decode_T8", "nvfp4_20b_decode_T8"])
def test_a_decode_step_with_empty_slots_follows_the_layer(moe_gpu, name, own_buffers):
    """route -> gate_up -> down -> weighted sum, with tokens of too few non-NaN logits, against the layer over the
    same ids, which drops those slots: both are within the layer's tolerance of the definition, so within twice
    that of each other."""
    import torch

    from mxfp4_expert_ffn_moe_b200.workloads import workload
    from tests._metrics import MAX_ABS_OVER_RMS_TOL, REL_L2_TOL, max_abs_over_rms, rel_l2
    from tests.gpu_util import layer_to_device, nvfp4_layer_to_device
    moe = moe_gpu
    layer = workload(name)
    nv = layer.fmt == "nvfp4"
    dev = nvfp4_layer_to_device(layer) if nv else layer_to_device(layer)
    T, k, E = layer.T, layer.k, layer.E
    logits = dev["logits"].clone()
    logits[0, 1:] = float("nan")                         # one expert left
    logits[T // 2] = float("nan")                        # none
    moe.moe_get_device_error()
    ids, w = moe.moe_route(logits, k)
    assert int((ids < 0).sum()) >= 2 * k - 1 and bool((w[ids < 0] == 0).all())
    up = dict(bias=dev["gu_bias"], row_ids=ids, rows_per_x=k, swiglu=True, alpha=layer.alpha, limit=layer.limit)
    down = dict(bias=dev["d_bias"], row_ids=ids, out_dtype=torch.float32)
    act_shape, y_shape = (T * k, dev["d_blocks"].shape[2] * 2), (T * k, dev["d_blocks"].shape[1])
    if own_buffers:
        up.update(out=torch.full(act_shape, float("nan"), dtype=torch.bfloat16, device="cuda"), zero_skipped=True)
        down.update(out=torch.full(y_shape, float("nan"), device="cuda"), zero_skipped=True)
    else:
        _stale(act_shape, torch.bfloat16)
        _stale(y_shape, torch.float32)
    if nv:
        act = moe.nvfp4_matvec(dev["x"], dev["gu_blocks"], dev["gu_scales"], dev["gu_scale2"], **up)
        y = moe.nvfp4_matvec(act, dev["d_blocks"], dev["d_scales"], dev["d_scale2"], **down)
        want = moe.moe_nvfp4_forward_ex(dev["x"], ids, w, dev["gu_blocks"], dev["gu_scales"], dev["gu_scale2"], dev["gu_bias"],
                                        dev["d_blocks"], dev["d_scales"], dev["d_scale2"], dev["d_bias"],
                                        alpha=layer.alpha, limit=layer.limit)
    else:
        act = moe.mxfp4_matvec(dev["x"], dev["gu_blocks"], dev["gu_scales"], **up)
        y = moe.mxfp4_matvec(act, dev["d_blocks"], dev["d_scales"], **down)
        want = moe.moe_mxfp4_forward_ex(dev["x"], ids, w, dev["gu_blocks"], dev["gu_scales"], dev["gu_bias"],
                                        dev["d_blocks"], dev["d_scales"], dev["d_bias"], alpha=layer.alpha, limit=layer.limit)
    out = moe.moe_combine_rows(y, None, T, k, weights=w, dtype=torch.bfloat16)
    assert moe.moe_get_device_error() == moe.MOE_DEVERR_BAD_LOGIT | moe.MOE_DEVERR_BAD_EXPERT_ID
    empty = (ids < 0).view(-1)
    assert bool((act[empty] == 0).all()) and bool((y[empty] == 0).all())
    got, ref = out.double().cpu().numpy(), want.double().cpu().numpy()
    assert np.isfinite(got).all() and (got[T // 2] == 0).all() and (ref[T // 2] == 0).all()
    assert rel_l2(got, ref) <= 2 * REL_L2_TOL and max_abs_over_rms(got, ref) <= 2 * MAX_ABS_OVER_RMS_TOL


@pytest.mark.parametrize("odt", ["bfloat16", "float32"])
@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("R,N,swiglu", [(6, 48, False), (6, 50, True), (1000, 34, False), (3, 20000, False)])
def test_skipped_rows_become_zeros_and_the_others_stay_the_same(moe_gpu, R, N, swiglu, fmt, odt):
    import torch
    moe = moe_gpu
    g = torch.Generator().manual_seed(R + N)
    E, K = 4, 64
    blocks = torch.randint(0, 256, (E, N, K // 2), dtype=torch.uint8, generator=g).cuda()
    lo, hi, per = (118, 127, 32) if fmt == "mxfp4" else (8, 56, 16)
    scales = torch.randint(lo, hi, (E, N, K // per), dtype=torch.uint8, generator=g).cuda()
    x = torch.randn((R, K), generator=g).to("cuda", torch.bfloat16)
    call = moe.mxfp4_matvec if fmt == "mxfp4" else moe.nvfp4_matvec
    kw = dict(swiglu=swiglu, out_dtype=getattr(torch, odt))
    ids = torch.randint(-1, E + 2, (R,), dtype=torch.int32, generator=g)
    ids[:3] = torch.tensor([-1, E, -2 ** 31], dtype=torch.int32)
    good = ids.clamp(0, E - 1).cuda()
    ids = ids.cuda()
    skipped = (ids < 0) | (ids >= E)
    moe.moe_get_device_error()
    full = call(x, blocks, scales, row_ids=good, **kw)
    assert moe.moe_get_device_error() == 0
    _stale(full.shape, full.dtype)
    got = call(x, blocks, scales, row_ids=ids, **kw)
    assert moe.moe_get_device_error() == moe.MOE_DEVERR_BAD_EXPERT_ID
    assert bool((got[skipped] == 0).all()) and torch.equal(got[~skipped], full[~skipped])
    out = torch.full_like(full, 7.0)
    call(x, blocks, scales, row_ids=ids, out=out, **kw)
    assert bool((out[skipped] == 7).all()) and torch.equal(out[~skipped], full[~skipped])
    call(x, blocks, scales, row_ids=ids, out=out, zero_skipped=True, **kw)
    assert torch.equal(out, got)
    # every row skipped
    none = call(x, blocks, scales, row_ids=torch.full_like(ids, -1), **kw)
    assert bool((none == 0).all())
    # no ids: nothing is skipped
    one = call(x, blocks[0], scales[0], zero_skipped=True, **kw)
    assert torch.equal(one, call(x, blocks[:1], scales[:1], row_ids=torch.zeros_like(ids), **kw))
    moe.moe_get_device_error()

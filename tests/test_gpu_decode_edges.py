"""tv_decode_attention at its edges: the caller's workspace and what lies behind it, values
that are not finite, the same work repeated.  Bounds as in cache_cases.decode_bounds."""
import numpy as np
import pytest
import torch

import tree_speculative_decoding_07_b200 as tv
from cache_cases import Cache, as_type, decode_reference, to_gpu

pytestmark = pytest.mark.gpu


def _inputs(c, hq, q=None):
    q = as_type(c.rng.standard_normal((len(c.lens), hq, c.d)), c.dtype) if q is None else q
    return q, (to_gpu(q, c.dtype), to_gpu(c.k, c.dtype), to_gpu(c.v, c.dtype), to_gpu(c.table), to_gpu(c.lens))


def _within(got, ref, tol, what):
    got = got.float().cpu().numpy().astype(np.float64)
    assert np.array_equal(np.isneginf(got), np.isneginf(ref)), what
    fine = np.isfinite(ref)
    assert np.isfinite(got[fine]).all(), what
    assert (np.abs(got[fine] - ref[fine]) <= tol[fine]).all(), what


MANY = [0, 5, 40, 16] * 140 + [700]  # 561 sequences: their tile counts go through the workspace


# lengths, KV heads, query heads per KV head, head_dim, type, weights, whether clusters share a head
@pytest.mark.parametrize("lens,hkv,g,d,dtype,weights,clusters", [
    ([6000, 44], 2, 4, 64, "bf16", False, False),
    ([6000, 44], 2, 4, 64, "bf16", True, False),
    ([5000, 0, 300], 1, 3, 128, "f16", True, False),
    ([5000, 0, 300], 1, 11, 64, "bf16", True, False),
    ([4000, 90], 1, 40, 128, "bf16", True, False),
    ([300, 44], 1, 40, 64, "f32", True, False),
    ([3000, 1], 1, 11, 256, "f32", True, False),
    ([3000, 1], 2, 3, 96, "f32", False, False),
    (MANY, 1, 2, 64, "bf16", False, False),
    (MANY, 1, 3, 64, "f16", True, False),
    ([300, 44], 2, 4, 64, "bf16", True, True),
    ([300, 44, 0], 1, 11, 128, "f16", True, True),
    ([100, 7] * 4, 2, 3, 64, "f32", True, True),
])
def test_a_dirty_workspace_and_what_lies_behind_it(lens, hkv, g, d, dtype, weights, clusters):
    c = Cache(len(lens) + g, lens, hkv, d, dtype)
    q, args = _inputs(c, hkv * g)
    w = c.rng.random((len(lens), hkv, c.width * c.block)).astype(np.float32) if weights else None
    ref, tol = decode_reference(c, q, w)
    desc = tv.cache_desc(args[1], args[2], args[3], hkv * g)
    plan = tv.tv_decode_attention_plan(desc, weights)
    size = plan.workspace_bytes
    assert size > 0 and (plan.cluster_ctas > 0) == clusters
    tail = 1 << 16
    ws = torch.full((size + tail,), 0xff, dtype=torch.uint8, device="cuda")  # NaN, -1
    out, lse = torch.full_like(args[0], float("nan")), torch.full((len(lens), hkv * g), float("nan"), device="cuda")
    for _ in range(2):  # the second time on what the first left
        dw = None if w is None else to_gpu(w)
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        tv.decode_attention(*args, attn_weights=dw, out=out, lse=lse, workspace=ws[:size], dev_status=status)
        torch.cuda.synchronize()
        assert int(status.item()) == 0
        _within(out, ref[0], tol[0], "out")
        _within(lse, ref[1], tol[1], "lse")
        if weights:
            _within(dw, ref[2], tol[2], "weights")
    assert (ws[size:] == 0xff).all()
    assert not (ws[:size] == 0xff).all()
    with pytest.raises(tv.TreeVerifyError):
        tv.decode_attention(*args, attn_weights=dw, out=out, lse=lse, workspace=ws[:size - 256])


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("lens", [[40], [6000]])
@pytest.mark.parametrize("value", [np.inf, -np.inf, np.nan])
def test_values_that_are_not_finite(dtype, lens, value):
    """One element of one value row: that element of the head's outputs is not finite (in fp32 as the
    definition gives it), everything else stays as it was."""
    c = Cache(31, lens, 2, 64, dtype)
    q, _ = _inputs(c, 4, as_type(0.5 * c.rng.standard_normal((1, 4, 64)), dtype))  # no weight underflows
    w = np.zeros((1, 2, c.width * 16), np.float32)
    ref, tol = decode_reference(c, q, w)
    for t in (0, lens[0] // 2, lens[0] - 1):
        at = (c.table[0, t // 16], t % 16, 1, 7)
        keep, c.v[at] = c.v[at], value
        _, args = _inputs(c, 4, q)
        dw = to_gpu(w)
        out, lse = tv.decode_attention(*args, attn_weights=dw)
        c.v[at] = keep
        hit = out[0, 2:, 7].float().cpu().numpy()  # the two query heads of KV head 1
        assert not np.isfinite(hit).any()
        if dtype == "f32" and not np.isnan(value):
            assert (hit == value).all()
        if np.isnan(value):
            assert np.isnan(hit).all()
        out[0, 2:, 7] = to_gpu(ref[0][0, 2:, 7]).to(out.dtype)
        _within(out, ref[0], tol[0], "out")
        _within(lse, ref[1], tol[1], "lse")
        _within(dw, ref[2], tol[2], "weights")


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("lens", [[40, 21], [6000, 21]])
def test_an_infinite_score_makes_its_row_nan(dtype, lens):
    c = Cache(32, lens, 1, 64, dtype)
    q = as_type(c.rng.standard_normal((2, 2, 64)), dtype)
    q[0, :, 0] = 1
    c.k[c.table[0, 1], 3, 0, 0] = np.inf
    w = np.zeros((2, 1, c.width * 16), np.float32)
    _, args = _inputs(c, 2, q)
    dw = to_gpu(w)
    out, lse = tv.decode_attention(*args, attn_weights=dw)
    assert torch.isnan(out[0]).all() and torch.isnan(lse[0]).all() and torch.isnan(dw[0, 0, :lens[0]]).all()
    assert torch.isfinite(out[1]).all() and torch.isfinite(lse[1]).all() and torch.isfinite(dw[1]).all()

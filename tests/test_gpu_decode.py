"""tv_decode_attention against the 64-bit reference (bounds derived in cache_cases.decode_bounds)."""
import numpy as np
import pytest
import torch

import tree_speculative_decoding_07_b200 as tv
from cache_cases import TYPES, Cache, as_type, decode_reference, to_gpu

pytestmark = pytest.mark.gpu


def _queries(c, hq, scale=1.0):
    return as_type(scale * c.rng.standard_normal((len(c.lens), hq, c.d)), c.dtype)


def _within(got, ref, tol, what):
    got = got.float().cpu().numpy().astype(np.float64)
    assert np.array_equal(np.isnan(got), np.isnan(ref)), what
    assert np.array_equal(np.isneginf(got), np.isneginf(ref)), what
    fine = np.isfinite(ref)
    over = np.abs(got[fine] - ref[fine]) - tol[fine]
    assert over.size == 0 or over.max() <= 0, f"{what}: {over.max():.3g} past the bound"


def _run(c, q, weights=None, **kw):
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    w = None if weights is None else to_gpu(weights)
    out, lse = tv.decode_attention(to_gpu(q, c.dtype), to_gpu(c.k, c.dtype), to_gpu(c.v, c.dtype), to_gpu(c.table),
                                   to_gpu(c.lens), attn_weights=w, dev_status=status, **kw)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    return out, lse, w


def _check(c, hq, weights=True, scale=None, q=None, **kw):
    q = _queries(c, hq) if q is None else q
    w = None
    if weights:  # earlier sums, in rows a little wider than the table needs
        w = c.rng.random((len(c.lens), c.hkv, c.width * c.block + 5)).astype(np.float32)
    ref, tol = decode_reference(c, q, w, scale)
    if scale is not None:
        kw["softmax_scale"] = scale
    out, lse, got_w = _run(c, q, w, **kw)
    _within(out, ref[0], tol[0], "out")
    _within(lse, ref[1], tol[1], "lse")
    if weights:
        _within(got_w, ref[2], tol[2], "weights")
        for i, n in enumerate(c.lens):  # behind a sequence's tokens nothing is touched
            np.testing.assert_array_equal(got_w[i, :, n:].cpu().numpy(), w[i, :, n:])


SHORT = [0, 1, 15, 16, 17, 100, 0, 33]


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("d", [64, 96, 128, 256])
@pytest.mark.parametrize("hkv,g", [(2, 1), (1, 3), (2, 4), (1, 7), (2, 8), (1, 11), (1, 12), (2, 16), (1, 40)])
def test_types_heads_and_short_lengths(dtype, d, hkv, g):
    _check(Cache(d + g, SHORT, hkv, d, dtype), hkv * g)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("block", [1, 4, 16, 20, 32, 48, 100])
def test_block_sizes(dtype, block):
    # pages that end inside a tile, tiles that end inside a page
    _check(Cache(block, [1, 19, 20, 21, 333, 64], 2, 128, dtype, block=block), 8)


@pytest.mark.parametrize("dtype,g", [("bf16", 4), ("f16", 16), ("f32", 5)])
@pytest.mark.parametrize("lens,hkv", [([5000], 1), ([3000, 1, 0, 777, 2048], 2), ([1, 9000], 1), ([20000], 2)])
def test_heads_shared_by_many_ctas(dtype, g, lens, hkv):
    _check(Cache(len(lens), lens, hkv, 128, dtype), hkv * g)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d,g", [(128, 4), (256, 11), (64, 40), (96, 3)])
@pytest.mark.parametrize("lens,hkv", [([600, 3], 1), ([640], 8), ([500] * 20, 4), ([2000] * 4, 8), ([1100], 2),
                                      ([90, 2000, 17, 0, 2000], 4)])
def test_both_ways_of_sharing_the_work(dtype, d, g, lens, hkv):
    # short or many units by clusters, others by equal stretches; on either side of the borders
    _check(Cache(d, lens, hkv, d, dtype), hkv * g)


@pytest.mark.parametrize("weights", [False, True])
def test_large_ragged_batch(weights):
    rng = np.random.default_rng(3)
    _check(Cache(3, rng.integers(0, 70, 700), 1, 64, "bf16"), 2, weights)
    _check(Cache(4, rng.integers(0, 700, 130), 2, 64, "f16"), 6, weights)


@pytest.mark.parametrize("B", [511, 512, 513, 6000])
@pytest.mark.parametrize("weights", [False, True])
def test_batches_of_many_sequences(B, weights):
    """Sequences that share a pool of blocks (reading needs no blocks of one's own), most of them short, a few
    long: the equal stretches cover many sequences each.  The reference runs in float64 on the GPU."""
    rng = np.random.default_rng(B)
    hkv, g, d, pool, width = 2, 2, 64, 90, 45
    lens = rng.integers(0, 40, B)
    lens[rng.integers(0, B, B // 20)] = rng.integers(500, width * 16 + 1, B // 20)
    lens = lens.astype(np.int32)
    k, v = (torch.from_numpy(rng.standard_normal((pool, 16, hkv, d)).astype(np.float32)).cuda().bfloat16() for _ in range(2))
    q = torch.from_numpy(rng.standard_normal((B, hkv * g, d)).astype(np.float32)).cuda().bfloat16()
    table, dl = to_gpu(rng.integers(0, pool, (B, width)).astype(np.int32)), to_gpu(lens)
    w = torch.rand(B, hkv, width * 16, device="cuda") if weights else None
    w0 = w.clone() if weights else None
    out, lse = tv.decode_attention(q, k, v, table, dl, attn_weights=w)
    for b0 in range(0, B, 500):
        sel = slice(b0, min(B, b0 + 500))
        kk = k[table[sel].long()].flatten(1, 2).permute(0, 2, 3, 1).double()  # [b][hkv][d][t]
        vv = v[table[sel].long()].flatten(1, 2).permute(0, 2, 1, 3).double()
        qq = q[sel].double().reshape(-1, hkv, g, d)
        s = (qq @ kk) / 8
        size = (qq.abs() @ kk.abs()).amax(-1) / 8
        seen = torch.arange(width * 16, device="cuda") < dl[sel, None]
        s = s.masked_fill(~seen[:, None, None], -torch.inf)
        p = torch.nan_to_num(torch.softmax(s, -1))  # empty rows: zeros
        ref, ref_lse = (p @ vv).reshape(-1, hkv * g, d), torch.logsumexp(s, -1).reshape(-1, hkv * g)
        ds = (d + 8) * 2 ** -23 * size
        rel = (2 * ds + 2 ** -21 + 2 ** -16 + 2 * (width + 64) * 2 ** -23)  # as decode_bounds
        tol = (rel[..., None] * (p @ vv.abs())).reshape(ref.shape) + 2 ** -8 * ref.abs() * 1.01
        assert ((out[sel].double() - ref).abs() <= tol).all()
        fine = dl[sel] > 0
        assert ((lse[sel] - ref_lse).abs()[fine] <= (ds.reshape(ref_lse.shape) + 2 ** -20 + 2 ** -22 * ref_lse.abs())[fine]).all()
        assert torch.isneginf(lse[sel][~fine]).all()
        if weights:
            add = p.sum(2)
            want_w = w0[sel].double() + add
            assert ((w[sel] - want_w).abs() <= (rel[..., None] * p).sum(2) + 2 ** -23 * want_w * (add > 0)).all()


def test_every_sequence_empty():
    c = Cache(5, [0, 0, 0], 2, 64, "bf16", width=2)
    out, lse, w = _run(c, _queries(c, 4), np.ones((3, 2, 32), np.float32))
    assert (out == 0).all() and torch.isneginf(lse).all() and (w == 1).all()


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("scale", [1.0, 0.01])
def test_softmax_scale(dtype, scale):
    _check(Cache(6, [600, 40], 2, 64, dtype), 8, scale=scale)


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("order", ["rising", "falling"])
def test_scores_that_rise_or_fall_far(dtype, order):
    """The scores climb (or drop) by hundreds along the sequence: the reference moves many times."""
    c = Cache(7, [900, 90], 1, 64, dtype)
    for i, n in enumerate(c.lens):
        t = np.arange(n) if order == "rising" else np.arange(n)[::-1]
        c.k[c.table[i][np.arange(n) // 16], np.arange(n) % 16, 0, 0] = as_type(t / 4.0, dtype)
    q = _queries(c, 4)
    q[:, :, 0] = 8.0
    _check(c, 4, q=q)


def test_many_small_weights_beside_a_large_one():
    """fp16: 20,000 tokens whose weights are 2^-15 of the first one's keep their share."""
    c = Cache(8, [20000], 1, 64, "f16")
    t = np.arange(20000)
    at = (c.table[0][t // 16], t % 16, 0)
    c.k[at] = 0
    c.k[at[0][0], 0, 0, 0] = 1.0
    c.v[at] = as_type(1 + 0.01 * c.rng.standard_normal((20000, 64)), "f16")
    q = np.zeros((1, 2, 64), np.float32)
    q[0, :, 0] = as_type(np.array([15 * np.log(2) * 8, 14.5 * np.log(2) * 8]), "f16")
    _check(c, 2, q=q)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_infinite_scores(dtype):
    c = Cache(9, [50, 50, 50], 1, 64, dtype)
    q = _queries(c, 2)
    q[:2] = 0
    q[:2, :, 0] = 1
    at = lambda i: (c.table[i][np.arange(50) // 16], np.arange(50) % 16, 0, 0)  # noqa: E731
    c.k[at(0)] = -np.inf                    # every score is -inf: as an empty row
    k1 = c.k[at(1)].copy()
    k1[::2] = -np.inf                       # every second token has no weight
    c.k[at(1)] = k1
    k2 = c.k[at(2)].copy()
    k2[7] = np.nan                          # one NaN: the row is NaN
    c.k[at(2)] = k2
    w0 = np.ones((3, 1, c.width * 16), np.float32)
    out, lse, w = _run(c, q, w0)
    assert (out[0] == 0).all() and torch.isneginf(lse[0]).all() and (w[0] == 1).all()
    c1 = Cache(9, [50], 1, 64, dtype)
    c1.k, c1.v, c1.table, c1.lens = c.k, c.v, c.table[1:2], c.lens[1:2]
    ref = np.zeros((1, 2, 64))
    lref = np.zeros((1, 2))
    for h in range(2):
        s = c1.rows(c1.k, 0, 0)[:, 0] / 8
        p = np.exp(s - s.max())
        ref[0, h] = (p / p.sum()) @ c1.rows(c1.v, 0, 0)
        lref[0, h] = s.max() + np.log(p.sum())
    tol = 2 ** -7 if dtype == "bf16" else 1e-5
    np.testing.assert_allclose(out[1:2].float().cpu().numpy(), ref, rtol=tol, atol=tol / 8)
    np.testing.assert_allclose(lse[1:2].cpu().numpy(), lref, rtol=1e-5)
    assert (w[1, 0, 0:50:2] == 1).all() and (w[1, 0, 1:50:2] > 1).all()
    assert torch.isnan(out[2]).all() and torch.isnan(lse[2]).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("lens", [[40, 35, 20], [40, 6000, 20]])
@pytest.mark.parametrize("entry", [-1, 10 ** 6])
def test_bad_block_ids_touch_their_sequence_only(dtype, lens, entry):
    c = Cache(10, lens, 2, 64, dtype)
    q = _queries(c, 4)
    w0 = np.ones((3, 2, c.width * 16), np.float32)
    ref, tol = decode_reference(c, q, w0)
    c.table[1, (lens[1] - 1) // 16] = entry
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    w = to_gpu(w0)
    out, lse = tv.decode_attention(to_gpu(q, dtype), to_gpu(c.k, dtype), to_gpu(c.v, dtype), to_gpu(c.table),
                                   to_gpu(c.lens), attn_weights=w, dev_status=status)
    assert int(status.item()) == tv.TV_ERR_BLOCK_TABLE
    assert torch.isnan(out[1]).all() and torch.isnan(lse[1]).all() and (w[1] == 1).all()
    for i in (0, 2):
        _within(out[i], ref[0][i], tol[0][i], "out")
        _within(w[i], ref[2][i], tol[2][i], "weights")
    # an entry that no token needs is not looked at
    c = Cache(11, [20, 30], 2, 64, dtype, width=4)
    c.table[:, 2:] = entry
    _check(c, 4)


def test_lengths_out_of_range():
    c = Cache(12, [20, 30, 10], 2, 64, "bf16", width=3)
    q = _queries(c, 4)
    w0 = np.ones((3, 2, 48), np.float32)
    ref, tol = decode_reference(c, q, w0)
    for lens, kw in (([20, -1, 10], {}), ([20, 49, 10], {}), ([20, 31, 10], dict(max_kv_len=30))):
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        w = to_gpu(w0)
        out, lse = tv.decode_attention(to_gpu(q, "bf16"), to_gpu(c.k, "bf16"), to_gpu(c.v, "bf16"), to_gpu(c.table),
                                       to_gpu(np.array(lens, np.int32)), attn_weights=w, dev_status=status, **kw)
        assert int(status.item()) == tv.TV_ERR_INVALID_ARG
        assert torch.isnan(out[1]).all() and torch.isnan(lse[1]).all() and (w[1] == 1).all()
        for i in (0, 2):
            _within(out[i], ref[0][i], tol[0][i], "out")


def _plain(c, hq, weights=True):
    q = _queries(c, hq)
    w = np.zeros((len(c.lens), c.hkv, c.width * c.block), np.float32) if weights else None
    ref, tol = decode_reference(c, q, w)
    return q, w, ref, tol


@pytest.mark.parametrize("layout", ["heads first", "k and v side by side", "wide rows"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_cache_strides(dtype, layout):
    c = Cache(13, [100, 37], 2, 64, dtype)
    q, w, ref, tol = _plain(c, 8)
    k, v = to_gpu(c.k, dtype), to_gpu(c.v, dtype)
    if layout == "heads first":
        k, v = (x.transpose(1, 2).contiguous().transpose(1, 2) for x in (k, v))
    elif layout == "k and v side by side":
        both = torch.stack([k, v], dim=1)  # [blocks][2][slots][heads][dim]
        k, v = both[:, 0], both[:, 1]
    else:
        wide = torch.full((2, *k.shape[:3], 96), float("nan"), dtype=k.dtype, device="cuda")
        wide[0, ..., :64], wide[1, ..., :64] = k, v
        k, v = wide[0, ..., :64], wide[1, ..., :64]
    assert not k.is_contiguous()
    fused = torch.randn(2, 12, 64, device="cuda").to(k.dtype)  # a projection's q, k, v side by side
    fused[:, :8] = to_gpu(q, dtype)
    dw = to_gpu(w)
    out, lse = tv.decode_attention(fused[:, :8], k, v, to_gpu(c.table), to_gpu(c.lens), attn_weights=dw)
    _within(out, ref[0], tol[0], "out")
    _within(dw, ref[2], tol[2], "weights")


def test_offsets_past_32_bits():
    """Blocks more than 2^32 bytes into a cache of 5.4 GB."""
    nb, bs, hkv, d = 41000, 64, 8, 128
    k = torch.empty(nb, bs, hkv, d, dtype=torch.bfloat16, device="cuda")
    v = torch.empty_like(k)
    c = Cache(14, [150, 64], hkv, d, "bf16", block=bs)
    ids = np.array([[40999, 3, 40000], [39999, 1, 2]], np.int32)
    for i in range(2):
        for j in range(3):
            k[int(ids[i, j])] = to_gpu(c.k[c.table[i, j]], "bf16")
            v[int(ids[i, j])] = to_gpu(c.v[c.table[i, j]], "bf16")
    q, w, ref, tol = _plain(c, 16)
    dw = to_gpu(w)
    out, lse = tv.decode_attention(to_gpu(q, "bf16"), k, v, to_gpu(ids), to_gpu(c.lens), attn_weights=dw)
    _within(out, ref[0], tol[0], "out")
    _within(dw, ref[2], tol[2], "weights")


def test_one_token_of_a_tree_is_a_new_token():
    c = Cache(15, [500, 33], 2, 128, "bf16")
    q = _queries(c, 8)
    args = [to_gpu(x, "bf16") for x in (c.k, c.v)]
    out, _ = tv.decode_attention(to_gpu(q, "bf16"), *args, to_gpu(c.table), to_gpu(c.lens))
    tree = tv.tree_attention(to_gpu(q, "bf16")[:, None], *args, to_gpu(c.table), to_gpu(c.lens - 1), None)
    ref, tol = decode_reference(c, q)
    _within(out, ref[0], tol[0], "out")
    # the tree kernel also rounds its weights to bf16 (half a step, 2^-8 of each) and its splits' results
    # (2^-8 of those): each at most 2^-8 of the weights times |v|
    size, _ = tv.decode_attention(to_gpu(q, "bf16"), args[0], args[1].abs(), to_gpu(c.table), to_gpu(c.lens))
    size = size.float().cpu().numpy() * (1 + 2 ** -8)
    assert (np.abs(tree[:, 0].float().cpu().numpy() - ref[0]) <= tol[0] + 2 * 2 ** -8 * size).all()


def test_same_bits_every_time_and_on_any_stream():
    c = Cache(16, [3000, 20, 900], 2, 128, "bf16")
    q, w, ref, tol = _plain(c, 16)
    args = (to_gpu(q, "bf16"), to_gpu(c.k, "bf16"), to_gpu(c.v, "bf16"), to_gpu(c.table), to_gpu(c.lens))
    first = [to_gpu(w)]
    first += tv.decode_attention(*args, attn_weights=first[0])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for stream in (None, side, side.cuda_stream):
        dw = to_gpu(w)
        torch.cuda.synchronize()
        got = tv.decode_attention(*args, attn_weights=dw, stream=stream)
        torch.cuda.synchronize()
        for a, b in zip(first, (dw, *got)):
            assert torch.equal(a, b)
    # two calls at once, each with its own workspace
    dws = [to_gpu(w), to_gpu(w)]
    torch.cuda.synchronize()
    outs = [tv.decode_attention(*args, attn_weights=dws[i], stream=s) for i, s in enumerate((side, None))]
    torch.cuda.synchronize()
    for dw, got in zip(dws, outs):
        for a, b in zip(first, (dw, *got)):
            assert torch.equal(a, b)


def test_captured_and_replayed():
    c = Cache(17, [700, 20], 2, 64, "f16")
    q, w, ref, tol = _plain(c, 8)
    dq, dk, dv, dt, dl = to_gpu(q, "f16"), to_gpu(c.k, "f16"), to_gpu(c.v, "f16"), to_gpu(c.table), to_gpu(c.lens)
    dw = to_gpu(w)
    tv.decode_attention(dq, dk, dv, dt, dl, attn_weights=dw.clone())  # first use outside
    graphs, results = [], []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            results.append(tv.decode_attention(dq, dk, dv, dt, dl, attn_weights=dw))
        graphs.append(g)
    assert (dw == 0).all()
    graphs[0].replay()
    torch.cuda.synchronize()
    _within(results[0][0], ref[0], tol[0], "out")
    _within(dw, ref[2], tol[2], "weights")
    # the length is read at replay: one token fewer
    dl -= 1
    dw.zero_()
    for g in graphs + graphs:
        g.replay()
    torch.cuda.synchronize()
    c.lens = c.lens - 1
    ref, tol = decode_reference(c, q, w)
    for out, lse in results:
        _within(out, ref[0], tol[0], "out")
        _within(lse, ref[1], tol[1], "lse")
    _within(dw, 4 * ref[2], 4 * tol[2] + 2 ** -22 * np.abs(ref[2]), "weights")


def test_given_outputs_and_workspace():
    c = Cache(18, [300, 44], 2, 64, "bf16")
    q, _, ref, tol = _plain(c, 8, weights=False)
    args = (to_gpu(q, "bf16"), to_gpu(c.k, "bf16"), to_gpu(c.v, "bf16"), to_gpu(c.table), to_gpu(c.lens))
    desc = tv.cache_desc(args[1], args[2], args[3], 8)
    size = tv.tv_decode_attention_workspace_size(desc)
    ws = torch.full((size + 256,), 0xff, dtype=torch.uint8, device="cuda")
    out, lse = torch.empty_like(args[0]), torch.empty(2, 8, device="cuda")
    got = tv.decode_attention(*args, out=out, lse=lse, workspace=ws[:size])
    assert got[0] is out and got[1] is lse
    _within(out, ref[0], tol[0], "out")
    assert (ws[size:] == 0xff).all()
    out2 = torch.empty_like(out)  # without lse
    assert tv.tv_decode_attention(desc, *args, out2, None, None, ws, size) == tv.TV_OK
    torch.cuda.synchronize()
    assert torch.equal(out, out2)


def test_wrapper_refusals():
    c = Cache(19, [30, 20], 2, 64, "bf16")
    q, k, v = (to_gpu(x, "bf16") for x in (_queries(c, 8), c.k, c.v))
    table, lens = to_gpu(c.table), to_gpu(c.lens)
    w = torch.zeros(2, 2, c.width * 16, device="cuda")
    bad = [
        (dict(q=q.half()), TypeError), (dict(q=q[:1]), ValueError), (dict(q=q[:, :7]), Exception),
        (dict(q=q[:, :, :32]), ValueError), (dict(q=q.transpose(0, 1)), ValueError), (dict(q=q.cpu()), ValueError),
        (dict(k=k[:, :8]), TypeError), (dict(v=v.cpu()), ValueError), (dict(table=table.long()), TypeError),
        (dict(lens=lens.long()), TypeError), (dict(lens=lens[:1]), ValueError), (dict(lens=None), Exception),
        (dict(attn_weights=w.half()), TypeError), (dict(attn_weights=w[:, :1]), ValueError),
        (dict(attn_weights=w[:, :, :17].contiguous()), tv.TreeVerifyError), (dict(attn_weights=w[:, :, ::2]), ValueError),
        (dict(out=q), tv.TreeVerifyError), (dict(out=q.float()), TypeError),
        (dict(workspace=torch.zeros(256, dtype=torch.uint8, device="cuda"), attn_weights=w), tv.TreeVerifyError),
        (dict(max_kv_len=10 ** 6), tv.TreeVerifyError), (dict(softmax_scale=-1.0), tv.TreeVerifyError),
    ]
    for kw, error in bad:
        a = dict(q=q, k=k, v=v, table=table, lens=lens)
        a.update({x: kw[x] for x in kw if x in a})
        rest = {x: kw[x] for x in kw if x not in a}
        with pytest.raises(error):
            tv.decode_attention(a["q"], a["k"], a["v"], a["table"], a["lens"], **rest)
    torch.cuda.synchronize()

"""tv_evict_cache against the reference: positions, rows and sums bit for bit."""
import numpy as np
import pytest
import torch

import tree_speculative_decoding_07_b200 as tv
from cache_cases import Cache, evict_reference, to_gpu

pytestmark = pytest.mark.gpu


def _sums(c, kind="mixed", extra=0):
    shape = (len(c.lens), c.hkv, c.width * c.block + extra)
    if kind == "equal":
        w = np.full(shape, 0.25, np.float32)
    elif kind == "few values":  # ties everywhere, both zeros among them
        w = c.rng.choice(np.array([0.0, -0.0, 1.0, 2.0, 1e-30, 3.0], np.float32), shape)
    elif kind == "odd":  # infinities, NaN, negative, subnormal
        w = c.rng.standard_normal(shape).astype(np.float32)
        pick = c.rng.random(shape)
        w[pick < 0.1] = np.nan
        w[(pick > 0.1) & (pick < 0.15)] = np.inf
        w[(pick > 0.15) & (pick < 0.2)] = -np.inf
        w[(pick > 0.2) & (pick < 0.3)] *= np.float32(1e-42)
    else:
        w = np.exp(2 * c.rng.standard_normal(shape)).astype(np.float32)
        w[c.rng.random(shape) < 0.1] = 0
    return w


def _host(t):
    return t.float().cpu().numpy()


def _check(c, budget, sink=0, recent=0, kind="mixed", copy=False, out="other", extra=0, **kw):
    w = _sums(c, kind, extra)
    dst = None
    if copy:  # blocks of its own for every sequence
        width = -(-budget // c.block)
        more = len(c.lens) * min(width, c.width)
        first = c.k.shape[0]
        pad = np.full((more, *c.k.shape[1:]), np.nan, np.float32)
        c.k, c.v = np.concatenate([c.k, pad]), np.concatenate([c.v, pad])
        dst = np.full_like(c.table, -7)  # entries that are not needed are not looked at
        dst[:, :min(width, c.width)] = first + c.rng.permutation(more).reshape(len(c.lens), -1)
    ref = evict_reference(c, w, budget, sink, recent, dst)
    k, v, dw = to_gpu(c.k, c.dtype), to_gpu(c.v, c.dtype), to_gpu(w)
    wo = dict(other=torch.from_numpy(w.copy()).cuda(), same=dw, none=None)[out]
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    new, kept = tv.evict_cache(k, v, to_gpu(c.table), to_gpu(c.lens), dw, budget, sink, recent,
                               dst_block_table=None if dst is None else to_gpu(dst), weights_out=wo,
                               dev_status=status, **kw)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    np.testing.assert_array_equal(new.cpu().numpy(), ref[4])
    np.testing.assert_array_equal(kept.cpu().numpy(), ref[3])
    if wo is not None:
        np.testing.assert_array_equal(_host(wo), ref[2])
    if out != "same":
        np.testing.assert_array_equal(_host(dw), w)
    # rows behind the kept ones may hold anything in place; everything else is as it was
    for got, want in ((k, ref[0]), (v, ref[1])):
        got = _host(got)
        for i, n in enumerate(ref[4]):
            t = np.arange(n)
            tab = c.table if dst is None else dst
            np.testing.assert_array_equal(got[tab[i][t // c.block], t % c.block], want[tab[i][t // c.block], t % c.block])
        np.testing.assert_array_equal(got, want)


LENS = [0, 1, 30, 64, 65, 200, 333, 100]


@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("f16", 64), ("f32", 256), ("bf16", 16), ("f32", 48), ("bf16", 96)])
@pytest.mark.parametrize("copy", [False, True])
@pytest.mark.parametrize("budget,sink,recent", [(64, 4, 16), (64, 0, 0), (64, 32, 32), (1, 0, 0), (1, 1, 0), (99, 0, 50)])
def test_types_budgets_and_lengths(dtype, d, copy, budget, sink, recent):
    _check(Cache(budget, LENS, 2, d, dtype), budget, sink, recent, copy=copy)


@pytest.mark.parametrize("kind", ["equal", "few values", "odd"])
@pytest.mark.parametrize("out", ["other", "same", "none"])
def test_ties_and_odd_values(kind, out):
    _check(Cache(1, [300, 77, 2000], 2, 64, "bf16"), 70, 3, 10, kind=kind, out=out)


@pytest.mark.parametrize("block", [1, 5, 16, 40])
@pytest.mark.parametrize("copy", [False, True])
def test_block_sizes(block, copy):
    _check(Cache(2, [90, 41, 200], 2, 64, "bf16", block=block), 41, 2, 5, copy=copy)


@pytest.mark.parametrize("lens,hkv,budget", [([9000], 2, 3000), ([9000, 100, 5001], 1, 700), ([40000], 1, 39999),
                                              ([70000], 1, 1000)])
@pytest.mark.parametrize("copy", [False, True])
def test_long_caches(lens, hkv, budget, copy):
    _check(Cache(3, lens, hkv, 64, "bf16"), budget, 5, 64, copy=copy, out="same")


@pytest.mark.parametrize("n", [393217, 786432])
def test_the_longest_caches(n):
    """Clusters of 16: past eight CTAs' shared memory, and the largest length that is taken."""
    assert n <= tv.TV_EVICT_MAX_LEN
    _check(Cache(12, [n], 1, 16, "bf16", spare=0), 3001, 5, 64, kind="few values", out="same")


@pytest.mark.parametrize("copy", [False, True])
def test_batches_of_many_sequences(copy):
    rng = np.random.default_rng(5)
    _check(Cache(13, rng.integers(0, 60, 900), 2, 16, "bf16", block=8), 25, 2, 5, copy=copy, out="same")


def test_two_calls_at_once():
    """Two caches on two streams, again and again: nothing is shared between calls."""
    cs = [Cache(14 + i, [3000, 40, 700], 2, 64, "bf16") for i in range(2)]
    ws = [_sums(c, "few values") for c in cs]
    refs = [evict_reference(c, w, 300, 3, 20) for c, w in zip(cs, ws)]
    streams = [torch.cuda.Stream() for _ in cs]
    start = [(to_gpu(c.k, "bf16"), to_gpu(c.v, "bf16"), to_gpu(c.table), to_gpu(c.lens), to_gpu(w)) for c, w in zip(cs, ws)]
    for _ in range(5):
        work = [(k.clone(), v.clone()) for k, v, *_ in start]
        torch.cuda.synchronize()
        res = [tv.evict_cache(*work[i], *start[i][2:], 300, 3, 20, stream=streams[i]) for i in range(2)]
        torch.cuda.synchronize()
        for i in range(2):
            np.testing.assert_array_equal(res[i][1].cpu().numpy(), refs[i][3])
            np.testing.assert_array_equal(_host(work[i][0]), refs[i][0])
            np.testing.assert_array_equal(_host(work[i][1]), refs[i][1])


@pytest.mark.parametrize("kind", ["equal", "few values", "mixed"])
def test_ties_across_the_slices_of_a_cluster(kind):
    _check(Cache(4, [17000], 1, 16, "bf16"), 8500, 3, 100, kind=kind, out="same")


def test_a_budget_past_every_length():
    _check(Cache(5, [10, 64, 0], 2, 64, "bf16"), 1000, 10, 20)
    _check(Cache(5, [10, 64, 0], 2, 64, "bf16"), 1000, 10, 20, copy=True)


def test_rows_of_sums_that_are_not_16_byte_aligned():
    _check(Cache(6, [500, 300], 3, 64, "bf16"), 100, 3, 9, extra=3)


@pytest.mark.parametrize("layout", ["heads first", "k and v side by side"])
def test_cache_strides(layout):
    c = Cache(7, [100, 60], 2, 64, "bf16")
    w = _sums(c)
    ref = evict_reference(c, w, 40, 2, 8)
    k, v = to_gpu(c.k, "bf16"), to_gpu(c.v, "bf16")
    if layout == "heads first":
        k, v = (x.transpose(1, 2).contiguous().transpose(1, 2) for x in (k, v))
    else:
        both = torch.stack([k, v], dim=1)
        k, v = both[:, 0], both[:, 1]
    new, kept = tv.evict_cache(k, v, to_gpu(c.table), to_gpu(c.lens), to_gpu(w), 40, 2, 8)
    np.testing.assert_array_equal(kept.cpu().numpy(), ref[3])
    np.testing.assert_array_equal(_host(k), ref[0])
    np.testing.assert_array_equal(_host(v), ref[1])


def test_copies_leave_shared_source_blocks_alone():
    """Two sequences share a prefix's blocks; each keeps its own choice in blocks of its own."""
    c = Cache(8, [80, 80], 2, 64, "bf16")
    c.table[1, :3] = c.table[0, :3]
    _check(c, 30, 2, 5, copy=True)


@pytest.mark.parametrize("lens", [[100, 90, 50], [100, 9000, 50]])
def test_bad_tables_and_lengths_leave_the_sequence_as_it_was(lens):
    for what in ("block", "dst", "negative", "long"):
        c = Cache(9, lens, 2, 64, "bf16")
        w = _sums(c)
        dst, given = None, c.lens.copy()
        if what == "dst":
            first = c.k.shape[0]
            pad = np.zeros((9, *c.k.shape[1:]), np.float32)
            c.k, c.v = np.concatenate([c.k, pad]), np.concatenate([c.v, pad])
            dst = np.full_like(c.table, first)
            dst[:, :3] = first + np.arange(9).reshape(3, 3)
        good = evict_reference(c, w, 40, 2, 8, dst)
        k0, v0 = c.k.copy(), c.v.copy()
        table = c.table.copy()
        if what == "block":
            table[1, 3] = c.k.shape[0]
        elif what == "dst":
            dst[1, 2] = -1
        else:
            given[1] = -5 if what == "negative" else c.width * 16 + 1
        k, v, dw = to_gpu(c.k, "bf16"), to_gpu(c.v, "bf16"), to_gpu(w)
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        new, kept = tv.evict_cache(k, v, to_gpu(table), to_gpu(given), dw, 40, 2, 8,
                                   dst_block_table=None if dst is None else to_gpu(dst), weights_out=dw,
                                   dev_status=status)
        torch.cuda.synchronize()
        assert int(status.item()) == (tv.TV_ERR_BLOCK_TABLE if what in ("block", "dst") else tv.TV_ERR_INVALID_ARG)
        assert new.cpu().tolist() == [40, int(given[1]), 40] and (kept[1] == -1).all()
        np.testing.assert_array_equal(_host(dw)[1], w[1])
        np.testing.assert_array_equal(kept.cpu().numpy()[[0, 2]], good[3][[0, 2]])
        np.testing.assert_array_equal(_host(dw)[[0, 2]], good[2][[0, 2]])
        # the flagged sequence's blocks are untouched, the others' rows moved
        own = np.unique(c.table[1])
        np.testing.assert_array_equal(_host(k)[own], k0[own])
        np.testing.assert_array_equal(_host(v)[own], v0[own])
        t = np.arange(40)
        for i in (0, 2):
            tab = c.table if dst is None else dst
            np.testing.assert_array_equal(_host(k)[tab[i][t // 16], t % 16], good[0][tab[i][t // 16], t % 16])


def test_streams_capture_and_repetition():
    c = Cache(10, [500, 2500], 2, 64, "bf16")
    w = _sums(c, "few values")
    ref = evict_reference(c, w, 200, 3, 20)
    table, lens, dw = to_gpu(c.table), to_gpu(c.lens), to_gpu(w)
    side = torch.cuda.Stream()
    for stream in (None, side, side.cuda_stream):
        k, v = to_gpu(c.k, "bf16"), to_gpu(c.v, "bf16")
        torch.cuda.synchronize()
        new, kept = tv.evict_cache(k, v, table, lens, dw, 200, 3, 20, stream=stream)
        torch.cuda.synchronize()
        np.testing.assert_array_equal(kept.cpu().numpy(), ref[3])
        np.testing.assert_array_equal(_host(k), ref[0])
    k0, v0 = to_gpu(c.k, "bf16"), to_gpu(c.v, "bf16")
    k, v = k0.clone(), v0.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        new, kept = tv.evict_cache(k, v, table, lens, dw, 200, 3, 20)
    for _ in range(3):
        k.copy_(k0)
        v.copy_(v0)
        kept.fill_(5)
        g.replay()
        torch.cuda.synchronize()
        np.testing.assert_array_equal(kept.cpu().numpy(), ref[3])
        np.testing.assert_array_equal(_host(k), ref[0])
        np.testing.assert_array_equal(_host(v), ref[1])


def test_wrapper_refusals():
    c = Cache(11, [30, 20], 2, 64, "bf16")
    k, v, table, lens = to_gpu(c.k, "bf16"), to_gpu(c.v, "bf16"), to_gpu(c.table), to_gpu(c.lens)
    w = torch.zeros(2, 2, c.width * 16, device="cuda")
    bad = [
        (dict(budget=0), tv.TreeVerifyError), (dict(budget=8, sink=5, recent=4), tv.TreeVerifyError),
        (dict(weights=w.half()), TypeError), (dict(weights=w[:1]), ValueError), (dict(weights=None), Exception),
        (dict(weights=w[:, :, :20].contiguous()), tv.TreeVerifyError), (dict(weights_out=w[:, :, :20]), ValueError),
        (dict(dst_block_table=table[:, :1].contiguous()), ValueError), (dict(dst_block_table=table), tv.TreeVerifyError),
        (dict(new_kv_lens=lens), tv.TreeVerifyError), (dict(kept=table), ValueError), (dict(lens=lens.long()), TypeError),
    ]
    for kw, error in bad:
        a = dict(lens=lens, weights=w, budget=8)
        a.update({x: kw[x] for x in kw if x in a})
        rest = {x: kw[x] for x in kw if x not in a}
        with pytest.raises(error):
            tv.evict_cache(k, v, table, a["lens"], a["weights"], a["budget"], **rest)
    torch.cuda.synchronize()

"""tv_rotary_write against the 64-bit reference.

Tolerance: the turn's fraction is rounded once to fp32 (at most 2^-25 of half a
turn's unit, under 2^-23 of a radian), sincospi is good to 2 ulp (2^-22), so a
coefficient is off by less than 2^-21 and a result by 2^-21 (|x| + |y|), with the
two fp32 products and their sum 2^-20 (|x| + |y|); then one rounding to the
storage type, half a step."""
import numpy as np
import pytest
import torch

import tree_speculative_decoding_07_b200 as tv
from cache_cases import HALF_STEP, TYPES, as_type, depth_of, rotary_reference, to_gpu

pytestmark = pytest.mark.gpu


class Step:
    """One step's rows, cache and 64-bit results."""

    def __init__(self, seed, b, n, hq, hkv, d, dtype, rot=None, block=16, prefix=None, counts=None, tree=False,
                 axes=1, interleaved=False, positions=False, base=None, theta=1e4):
        rng = np.random.default_rng(seed)
        self.rng, self.b, self.n, self.hq, self.hkv, self.d, self.dtype, self.block = rng, b, n, hq, hkv, d, dtype, block
        rot = rot or d
        self.q, self.k, self.v = (as_type(rng.standard_normal((b, n, h, d)), dtype) for h in (hq, hkv, hkv))
        self.prefix = np.asarray(prefix if prefix is not None else rng.integers(0, 50, b), np.int32)
        self.counts = None if counts is None else np.asarray(counts, np.int32)
        self.width = -(-(int(self.prefix.max()) + n) // block)
        nb = b * self.width + 2
        self.table = rng.permutation(nb)[:b * self.width].reshape(b, self.width).astype(np.int32)
        self.cache = as_type(rng.standard_normal((2, nb, block, hkv, d)), dtype)
        self.inv_freq = (theta ** (-np.arange(rot // 2) * 2.0 / rot)).astype(np.float32)
        self.axis = [i % axes for i in range(rot // 2)]
        self.interleaved, self.axes = interleaved, axes
        self.parent = None
        if tree:
            self.parent = np.array([[-1] + [int(rng.integers(max(0, j - 4), j)) for j in range(1, n)] for _ in range(b)], np.int32)
        self.positions = rng.integers(0, 100000, (axes, b, n)).astype(np.int32) if positions else None
        self.base = None if base is None else np.asarray(base, np.int32)

    def nodes(self, i):
        return self.n if self.counts is None else int(self.counts[i])

    def position(self, i, j):
        if self.positions is not None:
            return self.positions[:, i, j]
        start = int((self.base if self.base is not None else self.prefix)[i])
        return [start + (j if self.parent is None else depth_of(self.parent[i], j))] * self.axes

    def reference(self):
        half = HALF_STEP[self.dtype]
        q = np.full(self.q.shape, np.nan)
        k, v = self.cache[0].astype(np.float64), self.cache[1].astype(np.float64)
        tq, tk = np.zeros_like(q), np.zeros_like(k)
        for i in range(self.b):
            for j in range(self.nodes(i)):
                pos = self.position(i, j)
                q[i, j], size = rotary_reference(self.q[i, j], pos, self.inv_freq, self.axis, self.interleaved)
                tq[i, j] = (size > 0) * (half * np.abs(q[i, j]) + 2 ** -20 * size)
                t = int(self.prefix[i]) + j
                at = (self.table[i, t // self.block], t % self.block)
                k[at], size = rotary_reference(self.k[i, j], pos, self.inv_freq, self.axis, self.interleaved)
                tk[at] = (size > 0) * (half * np.abs(k[at]) + 2 ** -20 * size)
                v[at] = self.v[i, j]
        return q, k, v, tq, tk

    def run(self, q_out="new", **kw):
        dq, dk, dv = (to_gpu(x, self.dtype) for x in (self.q, self.k, self.v))
        ck, cv = to_gpu(self.cache[0], self.dtype), to_gpu(self.cache[1], self.dtype)
        out = torch.full_like(dq, float("nan")) if q_out == "new" else dq if q_out == "same" else None
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        opt = lambda x: None if x is None else to_gpu(x)  # noqa: E731
        a = dict(q=dq, q_out=out, parent_idx=opt(self.parent), positions=opt(self.positions),
                 position_base=opt(self.base), axis_of_pair=self.axis if self.axes > 1 else None,
                 interleaved=self.interleaved, node_counts=opt(self.counts), dev_status=status)
        a.update(kw)
        res = tv.rotary_write(dk, dv, to_gpu(self.inv_freq), ck, cv, to_gpu(self.table), to_gpu(self.prefix), **a)
        torch.cuda.synchronize()
        return res, ck, cv, int(status.item())

    def check(self, **kw):
        q, k, v, tq, tk = self.reference()
        got_q, ck, cv, status = self.run(**kw)
        assert status == 0
        got_q, ck, cv = (x.float().cpu().numpy() for x in (got_q, ck, cv))
        for i in range(self.b):
            n = self.nodes(i)
            assert (np.abs(got_q[i, :n] - q[i, :n]) <= tq[i, :n]).all()
            if kw.get("q_out") != "same":
                assert np.isnan(got_q[i, n:]).all()
            else:
                np.testing.assert_array_equal(got_q[i, n:], self.q[i, n:])
        assert (np.abs(ck - k) <= tk).all()  # zero where nothing was written
        np.testing.assert_array_equal(cv, v)


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("d,rot", [(128, 128), (64, 64), (128, 64), (96, 32), (256, 256), (16, 16), (80, 80), (48, 16)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_types_dims_and_pairings(dtype, d, rot, interleaved):
    Step(d + rot, 2, 5, 6, 2, d, dtype, rot=rot, interleaved=interleaved).check()


@pytest.mark.parametrize("hq,hkv", [(1, 1), (40, 8), (64, 8), (9, 3), (128, 1), (200, 100)])
def test_heads(hq, hkv):
    Step(hq, 2, 3, hq, hkv, 64, "bf16").check()


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("counts", [None, [9, 0, 1, 5]])
def test_trees(interleaved, counts):
    Step(1, 4, 9, 8, 2, 64, "bf16", tree=True, counts=counts, interleaved=interleaved).check()
    Step(2, 4, 9, 8, 2, 64, "f32", tree=True, counts=counts, interleaved=interleaved, base=[7, 100000, 0, 31]).check()


def test_a_deep_tree_and_a_chain_agree():
    s = Step(3, 1, 128, 4, 2, 64, "f32", tree=True)
    s.parent[0] = np.arange(-1, 127)
    chain = s.run(parent_idx=None)
    tree = s.run()
    for a, b in zip(chain[:3], tree[:3]):
        assert torch.equal(a, b)
    s.check()


@pytest.mark.parametrize("axes", [1, 2, 3, 4])
def test_axes(axes):
    Step(4, 2, 21, 4, 2, 128, "bf16", axes=axes, positions=True).check()
    Step(5, 2, 21, 4, 2, 64, "f32", axes=axes, positions=True, interleaved=True, rot=32).check()
    Step(6, 2, 7, 4, 2, 64, "f32", axes=axes, tree=True).check()  # the same position on every axis


def test_far_positions():
    s = Step(7, 2, 3, 4, 2, 128, "f32", positions=True, theta=5e5)
    s.positions[:] = np.array([2 ** 31 - 1, 131071, -5, 0, -2 ** 31, 1000003]).reshape(1, 2, 3)
    s.check()


@pytest.mark.parametrize("block", [1, 7, 16, 64])
def test_block_sizes(block):
    Step(8, 3, 33, 2, 1, 64, "bf16", block=block).check()


def test_one_token_and_a_long_prompt():
    Step(9, 1, 1, 32, 8, 128, "bf16", prefix=[0]).check()
    Step(10, 1, 3001, 2, 1, 64, "f16", prefix=[77]).check()


def test_batches_of_many_sequences():
    rng = np.random.default_rng(18)
    Step(18, 700, 3, 2, 1, 16, "bf16", tree=True, counts=rng.integers(0, 4, 700)).check()


def test_a_tree_of_1024_nodes():
    s = Step(19, 1, 1024, 1, 1, 16, "f32", tree=True)
    s.parent[0, 700:] = np.arange(699, 1023)  # its tail a chain
    s.check()


def test_in_place_queries_and_no_queries():
    Step(11, 2, 6, 8, 2, 128, "bf16", counts=[6, 3]).check(q_out="same")
    s = Step(12, 2, 6, 8, 2, 128, "bf16")
    _, k, v, _, tk = s.reference()
    res, ck, cv, status = s.run(q=None, q_out=None)
    assert res is None and status == 0
    assert (np.abs(ck.float().cpu().numpy() - k) <= tk).all()
    np.testing.assert_array_equal(cv.float().cpu().numpy(), v)


def test_strided_rows_and_caches():
    s = Step(13, 3, 5, 8, 2, 64, "bf16")
    q, k, v, tq, tk = s.reference()
    fused = torch.cat([to_gpu(x, "bf16") for x in (s.q, s.k, s.v)], dim=2)  # one projection's output
    both = torch.stack([to_gpu(s.cache[0], "bf16"), to_gpu(s.cache[1], "bf16")], dim=1)
    ck, cv = both[:, 0].transpose(1, 2).contiguous().transpose(1, 2), both[:, 1].transpose(1, 2).contiguous().transpose(1, 2)
    out = tv.rotary_write(fused[:, :, 8:10], fused[:, :, 10:], to_gpu(s.inv_freq), ck, cv, to_gpu(s.table),
                          to_gpu(s.prefix), q=fused[:, :, :8])
    assert (np.abs(out.float().cpu().numpy() - q) <= tq).all()
    assert (np.abs(ck.float().cpu().numpy() - k) <= tk).all()
    np.testing.assert_array_equal(cv.float().cpu().numpy(), v)
    # one token per sequence: its rows lie a sequence's stride apart
    s = Step(14, 3, 1, 8, 2, 64, "bf16")
    q, k, v, tq, tk = s.reference()
    fused = torch.cat([to_gpu(x, "bf16") for x in (s.q, s.k, s.v)], dim=2)
    ck, cv = to_gpu(s.cache[0], "bf16"), to_gpu(s.cache[1], "bf16")
    out = tv.rotary_write(fused[:, :, 8:10], fused[:, :, 10:], to_gpu(s.inv_freq), ck, cv, to_gpu(s.table),
                          to_gpu(s.prefix), q=fused[:, :, :8])
    assert (np.abs(out.float().cpu().numpy() - q) <= tq).all()
    assert (np.abs(ck.float().cpu().numpy() - k) <= tk).all()


@pytest.mark.parametrize("what", ["count", "span", "prefix", "block", "tree", "root"])
def test_bad_nodes_get_nan_and_leave_the_cache(what):
    s = Step(15, 3, 6, 4, 2, 64, "bf16", tree=True, counts=[6, 6, 6], prefix=[16, 30, 10], block=16)
    q, k, v, tq, tk = s.reference()
    bad = set(range(6))
    code = tv.TV_ERR_INVALID_ARG
    first = s.prefix[1]
    if what == "count":
        s.counts[1] = 7
    elif what == "span":
        s.prefix[1] = s.width * 16 - 5
    elif what == "prefix":
        s.prefix[1] = -1
    elif what == "block":  # nodes 0 and 1 lie in the block before
        s.table = s.table.copy()
        keep = s.table[1, 2]
        s.table[1, 2] = 10 ** 6
        bad, code = {2, 3, 4, 5}, tv.TV_ERR_BLOCK_TABLE
    elif what == "tree":
        s.parent[1] = [-1, 0, 3, 0, 2, 3]  # node 2's parent comes after it, node 4 hangs on node 2
        bad, code = {2, 4}, tv.TV_ERR_TREE
    else:
        s.parent[1, 0] = 0
        code = tv.TV_ERR_TREE
    got, ck, cv, status = s.run()
    assert status == code
    got, ck, cv = (x.float().cpu().numpy() for x in (got, ck, cv))
    for j in range(6):
        t = int(first) + j
        if j in bad:
            assert np.isnan(got[1, j]).all()
            if what != "block":
                at = (s.table[1, t // 16], t % 16)
                np.testing.assert_array_equal(ck[at], s.cache[0][at])
                np.testing.assert_array_equal(cv[at], s.cache[1][at])
            else:
                np.testing.assert_array_equal(ck[keep], s.cache[0][keep])
        elif what != "tree" or j in (0, 1, 3):
            if what != "tree":
                assert (np.abs(got[1, j] - q[1, j]) <= tq[1, j]).all()
            assert np.isfinite(got[1, j]).all()
    for i in (0, 2):
        assert (np.abs(got[i] - q[i]) <= tq[i]).all()


def test_streams_and_capture():
    s = Step(16, 2, 9, 8, 2, 64, "bf16", tree=True)
    first = s.run()
    side = torch.cuda.Stream()
    for stream in (side, side.cuda_stream):
        again = s.run(stream=stream)
        for a, b in zip(first[:3], again[:3]):
            assert torch.equal(a, b)
    dq, dk, dv = (to_gpu(x, "bf16") for x in (s.q, s.k, s.v))
    ck, cv = to_gpu(s.cache[0], "bf16"), to_gpu(s.cache[1], "bf16")
    args = (to_gpu(s.inv_freq), ck, cv, to_gpu(s.table), to_gpu(s.prefix))
    par = to_gpu(s.parent)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = tv.rotary_write(dk, dv, *args, q=dq, parent_idx=par)
    for _ in range(2):
        ck.zero_()
        out.zero_()
        g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, first[0])


def test_wrapper_refusals():
    s = Step(17, 2, 3, 4, 2, 64, "bf16")
    dq, dk, dv = (to_gpu(x, "bf16") for x in (s.q, s.k, s.v))
    ck, cv = to_gpu(s.cache[0], "bf16"), to_gpu(s.cache[1], "bf16")
    f, table, prefix = to_gpu(s.inv_freq), to_gpu(s.table), to_gpu(s.prefix)
    pos = torch.zeros(2, 2, 3, dtype=torch.int32, device="cuda")
    bad = [
        (dict(k=dk.half()), TypeError), (dict(k=dk[:1]), Exception), (dict(v=dv[:, :2]), TypeError),
        (dict(f=f.double()), TypeError), (dict(f=f[:-1].contiguous()), tv.TreeVerifyError),
        (dict(f=torch.cat([f, f])), tv.TreeVerifyError), (dict(f=torch.ones(200, device="cuda")), ValueError),
        (dict(prefix=prefix.long()), TypeError), (dict(q=dq.float()), TypeError), (dict(q=dq[:, :2]), TypeError),
        (dict(q=dq, q_out=dq[:, :, :2]), ValueError), (dict(q_out=dq), Exception), (dict(k=dk.transpose(0, 1)), Exception),
        (dict(axis_of_pair=[0] * 31), ValueError), (dict(axis_of_pair=[0] * 31 + [2], positions=pos), ValueError),
        (dict(positions=pos.float()), TypeError), (dict(positions=pos[:, :1]), ValueError),
        (dict(parent_idx=prefix), ValueError), (dict(node_counts=table), ValueError), (dict(k=dk.cpu()), ValueError),
        (dict(axis_of_pair=[4] * 32), tv.TreeVerifyError),
    ]
    for kw, error in bad:
        a = dict(k=dk, v=dv, f=f, prefix=prefix)
        a.update({x: kw[x] for x in kw if x in a})
        rest = {x: kw[x] for x in kw if x not in a}
        with pytest.raises(error):
            tv.rotary_write(a["k"], a["v"], a["f"], ck, cv, table, a["prefix"], **rest)
    torch.cuda.synchronize()

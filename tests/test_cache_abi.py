"""The calls on the paged cache: refusals on the host before anything is launched
(no GPU needed), plans, and the 64-bit references against closed forms."""
import ctypes

import numpy as np
import pytest
import torch

import tree_speculative_decoding_07_b200 as tv
from cache_cases import Cache, as_type, decode_reference, evict_reference, rotary_reference

A = 256  # a non-null, aligned dummy address: nothing is launched on these paths


def _desc(**kw):
    base = dict(batch=2, num_q_heads=8, num_kv_heads=2, head_dim=128, block_size=16, max_blocks_per_seq=9,
                num_blocks=20, dtype=tv.TV_BF16, softmax_scale=0.0, max_kv_len=0, block_stride=0, token_stride=0,
                head_stride=0, q_stride=0, weight_stride=0)
    base.update(kw)
    return tv.TvCacheDesc(**base)


def _rot(**kw):
    base = dict(num_nodes=4, rotary_dim=128, interleaved=0, num_axes=1, q_stride=0, k_stride=0, v_stride=0,
                node_counts=None)
    base.update(kw)
    return tv.TvRotaryDesc(**base)


BAD_DESCS = [
    (dict(batch=0), tv.TV_ERR_INVALID_ARG),
    (dict(num_q_heads=7), tv.TV_ERR_INVALID_ARG),
    (dict(num_kv_heads=0), tv.TV_ERR_INVALID_ARG),
    (dict(head_dim=0), tv.TV_ERR_INVALID_ARG),
    (dict(head_dim=40), tv.TV_ERR_UNSUPPORTED),
    (dict(head_dim=272), tv.TV_ERR_UNSUPPORTED),
    (dict(block_size=0), tv.TV_ERR_INVALID_ARG),
    (dict(max_blocks_per_seq=0), tv.TV_ERR_INVALID_ARG),
    (dict(num_blocks=0), tv.TV_ERR_INVALID_ARG),
    (dict(dtype=3), tv.TV_ERR_INVALID_ARG),
    (dict(softmax_scale=-1.0), tv.TV_ERR_INVALID_ARG),
    (dict(softmax_scale=float("nan")), tv.TV_ERR_INVALID_ARG),
    (dict(softmax_scale=float("inf")), tv.TV_ERR_INVALID_ARG),
    (dict(max_kv_len=-1), tv.TV_ERR_INVALID_ARG),
    (dict(max_kv_len=145), tv.TV_ERR_INVALID_ARG),
    (dict(num_q_heads=258, num_kv_heads=2), tv.TV_ERR_UNSUPPORTED),
    (dict(max_blocks_per_seq=1 << 27), tv.TV_ERR_UNSUPPORTED),
    (dict(block_stride=4096, token_stride=256), tv.TV_ERR_INVALID_ARG),
    (dict(block_stride=4096, token_stride=256, head_stride=-128), tv.TV_ERR_INVALID_ARG),
    (dict(block_stride=4096, token_stride=257, head_stride=128), tv.TV_ERR_INVALID_ARG),
    (dict(weight_stride=143), tv.TV_ERR_INVALID_ARG),
    (dict(q_stride=1023), tv.TV_ERR_INVALID_ARG),
    (dict(q_stride=1028), tv.TV_ERR_INVALID_ARG),
]


def _decode(d, q=A, k=A, v=A, table=A, lens=A, out=2 * A, lse=A, w=None, ws=A, size=1 << 40):
    return tv.tv_decode_attention(d, q, k, v, table, lens, out, lse, w, ws, size, None, stream=0)


def _evict(d, budget=8, sink=1, recent=2, k=A, v=A, table=A, lens=A, w=A, dst=None, wo=None, kept=A, new=2 * A):
    return tv.tv_evict_cache(d, budget, sink, recent, k, v, table, lens, w, dst, wo, kept, new, None, stream=0)


def _rotary(d, r, q=A, k=A, v=A, f=A, par=None, pos=None, base=None, pre=A, table=A, qo=2 * A, ck=A, cv=A):
    return tv.tv_rotary_write(d, r, q, k, v, f, par, pos, base, pre, table, qo, ck, cv, None, stream=0)


@pytest.mark.parametrize("kw,status", BAD_DESCS)
def test_bad_descriptors_are_refused(kw, status):
    d = _desc(**kw)
    assert _decode(d) == status
    assert _evict(d) == status
    assert _rotary(d, _rot(rotary_dim=min(128, max(16, d.head_dim)))) == status
    assert tv.tv_decode_attention_workspace_size(d) == 0


def test_decode_refuses_bad_arguments():
    d = _desc()
    for name in ("q", "k", "v", "table", "lens", "out"):
        assert _decode(d, **{name: None}) == tv.TV_ERR_INVALID_ARG
    for name in ("q", "k", "v", "out"):
        assert _decode(d, **{name: A + 8}) == tv.TV_ERR_INVALID_ARG
    assert _decode(d, q=A, out=A) == tv.TV_ERR_INVALID_ARG
    # short work needs a workspace for the weights only, equal stretches always one
    assert tv.tv_decode_attention_workspace_size(d) == 0
    long = _desc(max_blocks_per_seq=900)
    for x, w in ((d, A), (long, None), (long, A)):
        need = tv.tv_decode_attention_workspace_size(x, w is not None)
        assert need > 0 and need % 256 == 0
        assert _decode(x, w=w, size=need - 1) == tv.TV_ERR_WORKSPACE
        assert _decode(x, w=w, ws=None) == tv.TV_ERR_WORKSPACE
        assert _decode(x, w=w, ws=A + 128) == tv.TV_ERR_WORKSPACE
    assert tv.tv_decode_attention_workspace_size(long, True) > tv.tv_decode_attention_workspace_size(long)
    for dim in (16, 80, 192):
        assert _decode(_desc(head_dim=dim)) == tv.TV_ERR_UNSUPPORTED
    # more tiles than the line's 32-bit numbers hold
    assert _decode(_desc(batch=1 << 14, num_q_heads=8, num_kv_heads=8, max_blocks_per_seq=1 << 20,
                         num_blocks=1 << 20)) == tv.TV_ERR_UNSUPPORTED


def test_decode_plans():
    for dtype in (tv.TV_BF16, tv.TV_F16, tv.TV_F32):
        for dim in (64, 96, 128, 256):
            for g in (1, 3, 8, 12, 40):
                d = _desc(dtype=dtype, head_dim=dim, num_q_heads=2 * g)
                p = tv.tv_decode_attention_plan(d, True)
                assert p.workspace_bytes == tv.tv_decode_attention_workspace_size(d, True)
                assert 1 <= p.smem_bytes <= 227 * 1024 and p.grid_ctas >= 1 and p.launches in (1, 2)
                assert p.heads_per_unit in (4, 8, 16)
    small = tv.tv_decode_attention_plan(_desc(batch=1, max_kv_len=16), False)
    assert (small.grid_ctas, small.cluster_ctas, small.launches) == (2, 1, 1)
    large = tv.tv_decode_attention_plan(_desc(batch=1, max_blocks_per_seq=9000), False)
    assert large.cluster_ctas == 0 and large.launches == 2
    plan = tv.TvDecodePlan()
    assert tv.lib().tv_decode_attention_plan(ctypes.byref(_desc()), 0, None) == tv.TV_ERR_INVALID_ARG
    assert tv.lib().tv_decode_attention_plan(None, 0, ctypes.byref(plan)) == tv.TV_ERR_INVALID_ARG
    with pytest.raises(tv.TreeVerifyError):
        tv.tv_decode_attention_plan(_desc(batch=0))


def test_evict_refuses_bad_arguments():
    d = _desc()
    for kw in (dict(budget=0), dict(sink=-1), dict(recent=-1), dict(budget=8, sink=4, recent=5),
               dict(budget=2 ** 31 - 1, sink=2 ** 31 - 1, recent=2 ** 31 - 1)):
        assert _evict(d, **kw) == tv.TV_ERR_INVALID_ARG
    for name in ("k", "v", "table", "lens", "w", "kept", "new"):
        assert _evict(d, **{name: None}) == tv.TV_ERR_INVALID_ARG
    assert _evict(d, k=A + 8) == tv.TV_ERR_INVALID_ARG
    assert _evict(d, lens=A, new=A) == tv.TV_ERR_INVALID_ARG
    assert _evict(d, table=A, dst=A) == tv.TV_ERR_INVALID_ARG
    long = _desc(max_blocks_per_seq=tv.TV_EVICT_MAX_LEN // 16 + 1)
    assert _evict(long) == tv.TV_ERR_UNSUPPORTED
    assert _evict(d, budget=2 ** 30) == tv.TV_ERR_UNSUPPORTED


@pytest.mark.parametrize("kw,status", [
    (dict(num_nodes=0), tv.TV_ERR_INVALID_ARG),
    (dict(rotary_dim=0), tv.TV_ERR_INVALID_ARG),
    (dict(rotary_dim=144), tv.TV_ERR_INVALID_ARG),
    (dict(rotary_dim=40), tv.TV_ERR_UNSUPPORTED),
    (dict(interleaved=2), tv.TV_ERR_INVALID_ARG),
    (dict(num_axes=0), tv.TV_ERR_INVALID_ARG),
    (dict(num_axes=5), tv.TV_ERR_UNSUPPORTED),
    (dict(q_stride=1016), tv.TV_ERR_INVALID_ARG),
    (dict(k_stride=260), tv.TV_ERR_INVALID_ARG),
    (dict(v_stride=128), tv.TV_ERR_INVALID_ARG),
])
def test_rotary_refuses_bad_descriptors(kw, status):
    assert _rotary(_desc(), _rot(**kw)) == status


def test_rotary_refuses_bad_arguments():
    d = _desc()
    for name in ("k", "v", "f", "pre", "table", "ck", "cv", "q", "qo"):  # q without q_out and the other way round
        assert _rotary(d, _rot(), **{name: None}) == tv.TV_ERR_INVALID_ARG
    for name in ("q", "k", "v", "qo", "ck", "cv"):
        assert _rotary(d, _rot(), **{name: A + 8}) == tv.TV_ERR_INVALID_ARG
    assert _rotary(d, _rot(q_stride=2048), q=A, qo=A) == tv.TV_ERR_INVALID_ARG
    assert _rotary(d, _rot(num_nodes=1025), par=A) == tv.TV_ERR_UNSUPPORTED
    r = _rot(num_axes=2)
    r.axis_of_pair[63] = 2
    assert _rotary(d, r) == tv.TV_ERR_INVALID_ARG
    assert tv.lib().tv_rotary_write(ctypes.byref(d), None, *([None] * 14)) == tv.TV_ERR_INVALID_ARG


def test_struct_layout_matches_the_header(tmp_path):
    import os
    import subprocess
    structs = {"tv_cache_desc": tv.TvCacheDesc, "tv_decode_plan": tv.TvDecodePlan, "tv_rotary_desc": tv.TvRotaryDesc}
    lines = ["#include <stdio.h>", "#include <stddef.h>", '#include "treeverify.h"', "int main(void) {"]
    for cname, cls in structs.items():
        lines.append(f'printf("{cname} size %zu\\n", sizeof({cname}));')
        for fname, _ in cls._fields_:
            lines.append(f'printf("{cname} {fname} %zu\\n", offsetof({cname}, {fname}));')
    lines += ['printf("consts evict_max %d\\n", TV_EVICT_MAX_LEN);', 'printf("consts f16 %d\\n", TV_F16);',
              "return 0;", "}"]
    src, exe = tmp_path / "layout.c", tmp_path / "layout"
    src.write_text("\n".join(lines))
    include = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include")
    subprocess.check_call(["gcc", "-std=c11", "-I", include, "-o", str(exe), str(src)])
    got = {tuple(x.split()[:2]): int(x.split()[2])
           for x in subprocess.check_output([str(exe)], text=True).splitlines()}
    for cname, cls in structs.items():
        assert got[(cname, "size")] == ctypes.sizeof(cls)
        for fname, _ in cls._fields_:
            assert got[(cname, fname)] == getattr(cls, fname).offset, (cname, fname)
    assert got[("consts", "evict_max")] == tv.TV_EVICT_MAX_LEN and got[("consts", "f16")] == tv.TV_F16


def test_wrappers_refuse_host_tensors_and_bad_shapes():
    c = torch.zeros(4, 16, 2, 64)
    table, lens = torch.zeros(1, 2, dtype=torch.int32), torch.ones(1, dtype=torch.int32)
    q = torch.zeros(1, 4, 64)
    with pytest.raises(ValueError, match="CUDA"):
        tv.decode_attention(q, c, c, table, lens)
    with pytest.raises(ValueError, match="CUDA"):
        tv.evict_cache(c, c, table, lens, torch.zeros(1, 2, 32), 8)
    with pytest.raises(ValueError, match="CUDA"):
        tv.rotary_write(torch.zeros(1, 1, 2, 64), torch.zeros(1, 1, 2, 64), torch.ones(32), c, c, table, lens)
    with pytest.raises(TypeError):
        tv.cache_desc(c.double(), c.double(), table)
    with pytest.raises(TypeError):
        tv.cache_desc(c, c[:3], table)
    with pytest.raises(TypeError):
        tv.cache_desc(c, c, table.long())
    with pytest.raises(ValueError, match="overlap"):
        tv.cache_desc(c[:1].expand(4, 16, 2, 64), c[:1].expand(4, 16, 2, 64), table)
    with pytest.raises(ValueError, match="strides"):
        tv.cache_desc(c, c.transpose(1, 2).contiguous().transpose(1, 2), table)
    d = tv.cache_desc(c.transpose(1, 2).contiguous().transpose(1, 2), c.transpose(1, 2).contiguous().transpose(1, 2),
                      table)
    assert (d.block_stride, d.token_stride, d.head_stride) == (2048, 64, 1024)
    assert tv.cache_desc(c, c, table).block_stride == 0


def test_wrappers_refuse_expanded_rows():
    """A stride of 0 between sequences or nodes is an expanded tensor's; in the descriptors 0 means contiguous,
    so passing it on would read past the one row that there is."""
    c = torch.zeros(4, 16, 2, 64)
    table, lens = torch.zeros(2, 2, dtype=torch.int32), torch.ones(2, dtype=torch.int32)
    one_q = torch.zeros(1, 4, 64)
    for q in (one_q.expand(2, 4, 64), torch.zeros(320).as_strided((2, 4, 64), (64, 64, 1))):
        with pytest.raises(ValueError, match="q: .*overlap"):
            tv.decode_attention(q, c, c, table, lens)
    with pytest.raises(ValueError, match="heads"):
        tv.decode_attention(torch.zeros(2, 1, 64).expand(2, 4, 64), c, c, table, lens)
    freq = torch.ones(32)

    def rows(b, n, h=2):
        return torch.zeros(b, n, h, 64)

    for b, n in ((2, 1), (1, 3), (2, 3)):
        tab, pre = torch.zeros(b, 2, dtype=torch.int32), torch.zeros(b, dtype=torch.int32)
        whole, q = rows(b, n), rows(b, n, 4)
        expanded = [rows(1, 1).expand(b, n, 2, 64)]
        if b > 1 and n > 1:
            expanded += [rows(1, n).expand(b, n, 2, 64), rows(b, 1).expand(b, n, 2, 64)]
        for x in expanded:
            for k, v, name in ((x, whole, "k"), (whole, x, "v")):
                with pytest.raises(ValueError, match=name + ": .*(overlap|apart)"):
                    tv.rotary_write(k, v, freq, c, c, tab, pre, q=q)
        with pytest.raises(ValueError, match="q: .*(overlap|apart)"):
            tv.rotary_write(whole, whole, freq, c, c, tab, pre, q=rows(1, 1, 4).expand(b, n, 4, 64))
        with pytest.raises(ValueError, match="CUDA"):  # the same call on rows of their own gets past these checks
            tv.rotary_write(whole, whole, freq, c, c, tab, pre, q=q)
    # a single sequence's stride says nothing
    with pytest.raises(ValueError, match="CUDA"):
        tv.decode_attention(torch.zeros(1, 4, 64).expand(1, 4, 64), c, c, table[:1], lens[:1])


def test_wrappers_refuse_empty_tensors():
    """An empty tensor has no address, which the C calls take for an argument that was not given."""
    c = torch.zeros(4, 16, 2, 64)
    table, lens = torch.zeros(1, 2, dtype=torch.int32), torch.ones(1, dtype=torch.int32)
    q, k = torch.zeros(1, 4, 64), torch.zeros(1, 1, 2, 64)
    none, empty = torch.zeros(1, 2, 0), torch.zeros(0, dtype=torch.int32)
    with pytest.raises(ValueError, match="attn_weights"):
        tv.decode_attention(q, c, c, table, lens, attn_weights=none)
    with pytest.raises(ValueError, match="weights"):
        tv.evict_cache(c, c, table, lens, none, 8)
    with pytest.raises(ValueError, match="dev_status"):
        tv.decode_attention(q, c, c, table, lens, dev_status=empty)
    with pytest.raises(ValueError, match="dev_status"):
        tv.evict_cache(c, c, table, lens, torch.zeros(1, 2, 32), 8, dev_status=empty)
    with pytest.raises(ValueError, match="dev_status"):
        tv.rotary_write(k, k, torch.ones(32), c, c, table, lens, dev_status=empty)


def test_writers_refuse_one_cache_for_keys_and_values():
    """Rows of K and of V are written by different threads: in one cache their order would be left to chance."""
    d = _desc()
    assert _evict(d, k=A, v=A) == tv.TV_ERR_INVALID_ARG
    assert _rotary(d, _rot(), ck=A, cv=A) == tv.TV_ERR_INVALID_ARG
    assert _rotary(d, _rot(), q=None, qo=None, ck=A, cv=A) == tv.TV_ERR_INVALID_ARG


def test_writers_refuse_bad_arguments_with_two_caches():
    """Each refusal by itself, not for the caches' being one."""
    two = dict(k=A, v=3 * A)
    for kw, status in BAD_DESCS:
        d = _desc(**kw)
        assert _evict(d, **two) == status
        assert _rotary(d, _rot(rotary_dim=min(128, max(16, d.head_dim))), cv=3 * A) == status
    d = _desc()
    for kw in (dict(budget=0), dict(sink=-1), dict(recent=-1), dict(budget=8, sink=4, recent=5),
               dict(table=None), dict(lens=None), dict(w=None), dict(kept=None), dict(new=None), dict(new=A),
               dict(k=None), dict(v=None), dict(k=A + 8), dict(v=A + 8), dict(dst=A)):
        assert _evict(d, **{**two, **kw}) == tv.TV_ERR_INVALID_ARG
    for kw in (dict(k=None), dict(v=None), dict(f=None), dict(pre=None), dict(table=None), dict(ck=None), dict(q=None),
               dict(qo=None), dict(q=A + 8), dict(k=A + 8), dict(v=A + 8), dict(qo=A + 8), dict(ck=A + 8)):
        assert _rotary(d, _rot(), cv=3 * A, **kw) == tv.TV_ERR_INVALID_ARG
    for kw in (dict(num_nodes=0), dict(rotary_dim=0), dict(rotary_dim=144), dict(interleaved=2), dict(num_axes=0),
               dict(q_stride=1016), dict(k_stride=260), dict(v_stride=128)):
        assert _rotary(d, _rot(**kw), cv=3 * A) == tv.TV_ERR_INVALID_ARG
    assert _rotary(d, _rot(q_stride=2048), q=A, qo=A, cv=3 * A) == tv.TV_ERR_INVALID_ARG


def test_every_wrapper_checks_the_caches_alike():
    """Types, shapes, strides and overlaps of the caches and the table, through each call that takes them."""
    c = torch.zeros(4, 16, 2, 64)
    table, lens = torch.zeros(1, 2, dtype=torch.int32), torch.ones(1, dtype=torch.int32)
    heads_first = c.transpose(1, 2).contiguous().transpose(1, 2)
    calls = [
        lambda k, v, t: tv.cache_desc(k, v, t, 4),
        lambda k, v, t: tv.decode_attention(torch.zeros(1, 4, 64, dtype=k.dtype), k, v, t, lens),
        lambda k, v, t: tv.evict_cache(k, v, t, lens, torch.zeros(1, 2, 32), 8),
        lambda k, v, t: tv.rotary_write(*[torch.zeros(1, 1, 2, 64, dtype=k.dtype)] * 2, torch.ones(32), k, v, t, lens),
    ]
    last = torch.zeros(4, 16, 2, 128)[..., ::2]
    bad = [(c.double(), c.double(), table, TypeError, "dtype"), (c, c[:3], table, TypeError, "one type"),
           (c, c.half(), table, TypeError, "one type"), (c[0], c[0], table, TypeError, "one type"),
           (c, c, table.long(), TypeError, "block_table"), (c, c, table[0], TypeError, "block_table"),
           (c, c, table.expand(3, 2)[:, :1], TypeError, "block_table"),
           (c[:1].expand(4, 16, 2, 64), c[:1].expand(4, 16, 2, 64), table, ValueError, "k_cache: rows overlap"),
           (c, c[:, :1].expand(4, 16, 2, 64), table, ValueError, "v_cache: rows overlap"),
           (c[:, :, :1].expand(4, 16, 2, 64), c, table, ValueError, "k_cache: rows overlap"),
           (c, heads_first, table, ValueError, "same strides"), (last, last, table, ValueError, "contiguous")]
    for call in calls:
        for k, v, t, error, match in bad:
            with pytest.raises(error, match=match):
                call(k, v, t)
    for k in (c, heads_first):
        for call in calls[1:]:
            with pytest.raises(ValueError, match="CUDA"):
                call(k, k, table)
    d = tv.cache_desc(heads_first, heads_first, table, softmax_scale=0.5, max_kv_len=7)
    assert (d.batch, d.num_q_heads, d.num_kv_heads, d.head_dim, d.block_size, d.max_blocks_per_seq, d.num_blocks,
            d.dtype, d.softmax_scale, d.max_kv_len) == (1, 2, 2, 64, 16, 2, 4, tv.TV_F32, 0.5, 7)
    for kw in (dict(num_q_heads=-1), dict(num_q_heads=1 << 40), dict(max_kv_len=1 << 40)):
        with pytest.raises(ValueError, match="range"):
            tv.cache_desc(c, c, table, **kw)


def test_references_against_closed_forms():
    c = Cache(0, [1, 40], 2, 64, "f32")
    q = as_type(c.rng.standard_normal((2, 4, 64)), "f32")
    (out, lse, w), _ = decode_reference(c, q, np.zeros((2, 2, 48), np.float32))
    # a single token: its value, weight 1 for each of the two query heads of a KV head
    np.testing.assert_allclose(out[0, 3], c.rows(c.v, 0, 1)[0], rtol=1e-12)
    assert w[0, 0, 0] == 2 and (w[0, :, 1:] == 0).all()
    np.testing.assert_allclose(w[1].sum(axis=1), 2, rtol=1e-12)
    k = torch.from_numpy(np.stack([c.rows(c.k, 1, h // 2) for h in range(4)]))
    v = torch.from_numpy(np.stack([c.rows(c.v, 1, h // 2) for h in range(4)]))
    ref = torch.nn.functional.scaled_dot_product_attention(torch.from_numpy(q[1]).double()[:, None], k, v)[:, 0]
    np.testing.assert_allclose(out[1], ref.numpy(), rtol=1e-10)
    # eviction: worked by hand (ties go to the lower position, NaN is lowest)
    c = Cache(1, [7], 1, 16, "f32", block=4)
    wt = np.array([[[0.1, 2.0, np.nan, 2.0, 2.0, 0.5, 0.0, 9.0]]], np.float32)
    k, v, wo, kept, new = evict_reference(c, wt, 4, 1, 1)
    assert kept.tolist() == [[[0, 1, 3, 6]]] and new.tolist() == [4]
    assert wo[0, 0].tolist() == [np.float32(0.1), 2, 2, 0, 0, 0, 0, 9]
    np.testing.assert_array_equal(c.rows(k, 0, 0, 4), c.rows(c.k, 0, 0)[[0, 1, 3, 6]])
    # rotation: a quarter turn, and the length of every pair is kept
    y, _ = rotary_reference(np.array([[1.0, 2.0, 3.0, 4.0]]), [1], [np.pi / 2, 0.0], [0, 0], False)
    np.testing.assert_allclose(y, [[-3, 2, 1, 4]], atol=1e-15)
    y, _ = rotary_reference(np.array([[1.0, 2.0, 3.0, 4.0]]), [1, 3], [np.pi / 2, np.pi / 2], [0, 1], True)
    np.testing.assert_allclose(y, [[-2, 1, 4, -3]], atol=1e-12)

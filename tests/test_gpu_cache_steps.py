"""The three calls together, as a draft model uses them: each step writes its rotated
rows, attends to the cache and sums the weights; every few steps the cache is cut
back to a budget, and the positions go on from the true ones.  Against dense
64-bit arithmetic on lists of rows, with the library's choice of kept tokens
checked against the sums that it had."""
import numpy as np
import pytest
import torch

import tree_speculative_decoding_07_b200 as tv
from cache_cases import HALF_STEP, as_type, decode_bounds, rotary_reference, to_gpu

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("captured", [False, True])
def test_generation_with_a_budget(dtype, captured):
    rng = np.random.default_rng(0)
    B, hq, hkv, d, block, budget, sink, recent, every, steps = 3, 8, 2, 64, 16, 48, 2, 8, 6, 25
    prompt = [40, 7, 63]
    width = -(-(max(max(prompt), budget) + every + 2) // block)
    nb = B * width
    table = rng.permutation(nb).reshape(B, width).astype(np.int32)
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    ck = torch.full((nb, block, hkv, d), float("nan"), dtype=dt, device="cuda")
    cv = torch.full_like(ck, float("nan"))
    freq = (1e4 ** (-np.arange(d // 2) * 2.0 / d)).astype(np.float32)
    dtab, dfreq = to_gpu(table), to_gpu(freq)
    weights = torch.zeros(B, hkv, width * block, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")

    # the prompts, ragged, written in one call
    n = max(prompt)
    k0, v0 = (as_type(rng.standard_normal((B, n, hkv, d)), dtype) for _ in range(2))
    counts = np.array(prompt, np.int32)
    zero = torch.zeros(B, dtype=torch.int32, device="cuda")
    tv.rotary_write(to_gpu(k0, dtype), to_gpu(v0, dtype), dfreq, ck, cv, dtab, zero, node_counts=to_gpu(counts),
                    dev_status=status)

    def rows_now(lens):  # the cache as lists of rows, read back
        k, v = ck.float().cpu().numpy(), cv.float().cpu().numpy()
        t = [np.arange(x) for x in lens]
        return ([k[table[b][t[b] // block], t[b] % block] for b in range(B)],
                [v[table[b][t[b] // block], t[b] % block] for b in range(B)])

    half = HALF_STEP[dtype]
    keys, values = rows_now(prompt)
    for b in range(B):
        for j in range(prompt[b]):
            ref, size = rotary_reference(k0[b, j], [j], freq, [0] * (d // 2), False)
            assert (np.abs(keys[b][j] - ref) <= half * np.abs(ref) + 2 ** -20 * size).all()
            np.testing.assert_array_equal(values[b][j], v0[b, j])

    lens, true_pos = np.array(prompt), np.array(prompt)
    q_in = torch.empty(B, 1, hq, d, dtype=dt, device="cuda")
    k_in, v_in = torch.empty(B, 1, hkv, d, dtype=dt, device="cuda"), torch.empty(B, 1, hkv, d, dtype=dt, device="cuda")
    dlens, dnext = to_gpu(lens.astype(np.int32)), to_gpu((lens + 1).astype(np.int32))
    dpos = to_gpu(true_pos.astype(np.int32))

    def step():
        q = tv.rotary_write(k_in, v_in, dfreq, ck, cv, dtab, dlens, q=q_in, position_base=dpos, dev_status=status)
        return q, *tv.decode_attention(q[:, 0], ck, cv, dtab, dnext, attn_weights=weights, dev_status=status)

    graph = None
    if captured:
        keep = ck.clone(), cv.clone()
        q_in.zero_(), k_in.zero_(), v_in.zero_()
        step()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            res = step()
        ck.copy_(keep[0]), cv.copy_(keep[1]), weights.zero_()
    sums = np.zeros((B, hkv, width * block))
    slack = np.zeros_like(sums)
    for i in range(steps):
        q, k, v = (as_type(rng.standard_normal((B, 1, h, d)), dtype) for h in (hq, hkv, hkv))
        q_in.copy_(to_gpu(q)), k_in.copy_(to_gpu(k)), v_in.copy_(to_gpu(v))
        dlens.copy_(to_gpu(lens.astype(np.int32))), dnext.copy_(dlens + 1), dpos.copy_(to_gpu(true_pos.astype(np.int32)))
        if graph is not None:
            graph.replay()
        else:
            res = step()
        torch.cuda.synchronize()
        rq, out, lse = (x.float().cpu().numpy() for x in res)
        lens, true_pos = lens + 1, true_pos + 1
        keys, values = rows_now(lens)
        for b in range(B):
            ref, size = rotary_reference(k[b, 0], [true_pos[b] - 1], freq, [0] * (d // 2), False)
            assert (np.abs(keys[b][-1] - ref) <= half * np.abs(ref) + 2 ** -20 * size).all()
            for h in range(hq):
                kk, vv = keys[b][:, h // 4].astype(np.float64), values[b][:, h // 4].astype(np.float64)
                s = kk @ rq[b, 0, h].astype(np.float64) / np.sqrt(d)
                p = np.exp(s - s.max())
                p /= p.sum()
                ds, rel = decode_bounds((np.abs(kk) @ np.abs(rq[b, 0, h])).max() / np.sqrt(d), len(s), d)
                o = p @ vv
                assert (np.abs(out[b, h] - o) <= rel * (p @ np.abs(vv)) + half * np.abs(o) * (1 + rel)).all()
                sums[b, h // 4, :len(s)] += p
                slack[b, h // 4, :len(s)] += rel * p + 2 ** -23 * sums[b, h // 4, :len(s)]
        assert (np.abs(weights.cpu().numpy() - sums) <= slack).all()
        if (i + 1) % every == 0:
            had = weights.cpu().numpy()
            new, kept = tv.evict_cache(ck, cv, dtab, dnext, weights, budget, sink, recent, weights_out=weights,
                                       dev_status=status)
            kept = kept.cpu().numpy()
            assert new.cpu().tolist() == [min(int(x), budget) for x in lens]
            keys2, values2 = rows_now(new.cpu().tolist())
            for b in range(B):
                m, L = int(new[b]), int(lens[b])
                for h in range(hkv):
                    want = np.arange(L)
                    if L > budget:
                        mid = had[b, h, sink:L - recent]
                        best = np.argsort(-mid, kind="stable")[:budget - sink - recent]
                        want = np.sort(np.concatenate([np.arange(sink), best + sink, np.arange(L - recent, L)]))
                    np.testing.assert_array_equal(kept[b, h, :m], want)
                    np.testing.assert_array_equal(keys2[b][:, h], keys[b][want, h])
                    np.testing.assert_array_equal(values2[b][:, h], values[b][want, h])
                    for x in (sums, slack):
                        x[b, h, :L] = np.concatenate([x[b, h, want], np.zeros(L - m)])
            lens = np.minimum(lens, budget)
    assert int(status.item()) == 0
    assert (lens <= budget + every).all() and (true_pos == np.array(prompt) + steps).all()


def test_a_tree_is_written_and_verified_on_an_evicted_cache():
    """The target's side: after an eviction, a draft tree's rotated rows join the cache and the
    tree attends to them; a chain of one node agrees with the single-token call."""
    rng = np.random.default_rng(1)
    B, N, hq, hkv, d, block, L, budget = 2, 5, 8, 2, 128, 16, 200, 90
    width = -(-(L + N) // block)
    nb = B * width
    table = to_gpu(rng.permutation(nb).reshape(B, width).astype(np.int32))
    ck, cv = (to_gpu(rng.standard_normal((nb, block, hkv, d)).astype(np.float32), "bf16") for _ in range(2))
    lens = torch.full((B,), L, dtype=torch.int32, device="cuda")
    w = torch.rand(B, hkv, width * block, device="cuda")
    new, _ = tv.evict_cache(ck, cv, table, lens, w, budget, 4, 16, weights_out=w)
    parent = to_gpu(np.array([[-1, 0, 1, 0, 3]] * B, np.int32))  # two drafts of two tokens
    freq = to_gpu((1e4 ** (-np.arange(d // 2) * 2.0 / d)).astype(np.float32))
    q, k, v = (to_gpu(rng.standard_normal((B, N, h, d)).astype(np.float32), "bf16") for h in (hq, hkv, hkv))
    rq = tv.rotary_write(k, v, freq, ck, cv, table, new, q=q, parent_idx=parent, position_base=lens)
    tree = tv.tree_attention(rq, ck, cv, table, new, parent)

    def near(node, length, k_cache, v_cache):
        """Each output is rounded to bf16 (half a step, 2^-8 of it).  The tree kernel also rounds
        its weights (2^-8 of each, so 2^-8 of the weights times |v|) and its splits' results
        (2^-8 of those, no more than the weights times |v|)."""
        one, _ = tv.decode_attention(rq[:, node], k_cache, v_cache, table, length)
        size, _ = tv.decode_attention(rq[:, node], k_cache, v_cache.abs(), table, length)
        a, b = tree[:, node].float(), one.float()
        assert ((a - b).abs() <= 2 ** -8 * (a.abs() + b.abs() + 2 * (1 + 2 ** -8) * size.float())).all()

    near(0, new + 1, ck, cv)
    # node 2's path is 0, 1, 2: the same rows in a cache of their own, as a chain's last token
    depth = {2: [0, 1, 2], 4: [0, 3, 4]}
    for node, path in depth.items():
        ck2, cv2 = ck.clone(), cv.clone()
        tv.rotary_write(k[:, path].contiguous(), v[:, path].contiguous(), freq, ck2, cv2, table, new, position_base=lens)
        near(node, new + 3, ck2, cv2)

"""The cases that the cache operators are measured at, and their plain forms.

Three operators work on one paged key-value cache: ``rotary_write`` rotates a
step's queries and keys by their positions and writes keys and values into the
cache, ``decode_attention`` lets one new token of each sequence attend to it
(and adds the attention weights up, per cached token), ``evict_cache`` keeps
each KV head's cache to a budget by those sums.

``own`` chooses between the plain torch forms and the library's calls.
"""
import math
import random

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


# ------------------------------------------------------------------ the cases

def listed():
    return [
        # the smallest call: a small fp32 draft model's token, short context (latency)
        dict(name="decode-tiny", op="decode", batch=1, lo=128, hi=128, heads=8, kv_heads=2, dim=64, block=16,
             dtype="f32", weights=True),
        # one sequence of an 8B-shaped model (32 / 8 heads) at 4K context
        dict(name="decode-4k", op="decode", batch=1, lo=4096, hi=4096, heads=32, kv_heads=8, dim=128, block=16,
             dtype="bf16", weights=False),
        # a batch of a 70B-shaped model's layer (64 / 8 heads), summing weights for the eviction
        dict(name="decode-batch-8k", op="decode", batch=8, lo=8192, hi=8192, heads=64, kv_heads=8, dim=128, block=16,
             dtype="bf16", weights=True),
        # mixed serving: every sequence at a length of its own
        dict(name="decode-mixed", op="decode", batch=32, lo=512, hi=32768, heads=32, kv_heads=8, dim=128, block=16,
             dtype="bf16", weights=False),
        # one very long context in half precision, weights kept
        dict(name="decode-128k", op="decode", batch=1, lo=131072, hi=131072, heads=64, kv_heads=8, dim=128, block=16,
             dtype="f16", weights=True),
        # a draft's cache halved where it lies
        dict(name="evict-4k", op="evict", batch=1, lo=4096, hi=4096, kv_heads=8, dim=128, block=16, dtype="bf16",
             budget=2048, sink=4, recent=256, in_place=True),
        # a batch at an odd length, kept rows copied into blocks of their own
        dict(name="evict-batch-8k", op="evict", batch=8, lo=8190, hi=8190, kv_heads=8, dim=128, block=16, dtype="bf16",
             budget=4001, sink=4, recent=512, in_place=False),
        # a long document cut to an eighth after its prompt
        dict(name="evict-128k", op="evict", batch=1, lo=131072, hi=131072, kv_heads=8, dim=128, block=16, dtype="f16",
             budget=16384, sink=16, recent=1024, in_place=False),
        # mixed serving: many short caches are already below the budget
        dict(name="evict-mixed", op="evict", batch=32, lo=512, hi=32768, kv_heads=8, dim=128, block=16, dtype="bf16",
             budget=4096, sink=4, recent=1024, in_place=True),
        # the rows of one 64-node draft tree (position = prefix + depth)
        dict(name="rotary-tree", op="rotary", batch=1, nodes=64, ragged=False, tree=True, prefix=4096, heads=32,
             kv_heads=8, dim=128, rot=128, interleaved=False, axes=1, split="sections", block=16, dtype="bf16"),
        # ragged trees of a mixed batch, half of each head rotated, neighbouring pairs
        dict(name="rotary-trees", op="rotary", batch=64, nodes=32, ragged=True, tree=True, prefix=32000, heads=32,
             kv_heads=8, dim=128, rot=64, interleaved=True, axes=1, split="sections", block=16, dtype="f16"),
        # a prompt with an image in it: time, height and width axes
        dict(name="rotary-prompt", op="rotary", batch=1, nodes=16384, ragged=False, tree=False, prefix=0, heads=32,
             kv_heads=8, dim=128, rot=128, interleaved=False, axes=3, split="woven", block=16, dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["decode", "evict", "rotary"])
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    dim = rng.choice([64, 96, 128, 128, 256])
    kv_heads = rng.choice([1, 2, 4, 8, 8])
    block = rng.choice([16, 16, 32, 64, 20])
    row = kv_heads * dim * (4 if dtype == "f32" else 2)
    case = dict(op=op, dtype=dtype, dim=dim, kv_heads=kv_heads, block=block)
    if op in ("decode", "evict"):
        batch = _log(rng, 1, 64)
        # the whole cache stays below the largest listed one's
        hi = _log(rng, 16, min(131072, (1 << 30) // (row * batch)))
        case.update(batch=batch, lo=_log(rng, 1, hi), hi=hi)
    if op == "decode":
        case.update(heads=kv_heads * rng.choice([1, 2, 3, 4, 7, 8, 16]), weights=rng.random() < 0.5)
    elif op == "evict":
        budget = _log(rng, 8, max(8, case["hi"]))
        sink = rng.randint(0, min(16, budget // 2))
        case.update(budget=budget, sink=sink, recent=rng.randint(0, (budget - sink) // 2),
                    in_place=rng.random() < 0.5)
    else:
        tree = rng.random() < 0.5
        batch = _log(rng, 1, 64)
        nodes = _log(rng, 1, 128) if tree else _log(rng, 1, 16384 // batch)
        axes = rng.choice([1, 1, 3, 4])
        case.update(batch=batch, nodes=nodes, ragged=rng.random() < 0.5, tree=tree, prefix=rng.randint(0, 131072 // batch),
                    heads=kv_heads * rng.choice([1, 2, 4, 7]), rot=rng.choice([dim, dim, dim // 2]),
                    interleaved=rng.random() < 0.5, axes=axes, split=rng.choice(["sections", "woven"]))
    return case


def _lens(case):
    """The sequences' lengths: the case's own, whatever the seed."""
    r = random.Random("%d %d %d" % (case["batch"], case["lo"], case["hi"]))
    return [r.randint(case["lo"], case["hi"]) for _ in range(case["batch"])]


def _counts(case):
    """The number of nodes of each sequence."""
    if not case["ragged"]:
        return [case["nodes"]] * case["batch"]
    r = random.Random("%d %d" % (case["batch"], case["nodes"]))
    return [r.randint(1, case["nodes"]) for _ in range(case["batch"])]


def work(case):
    es = 4 if case["dtype"] == "f32" else 2
    hkv, d = case["kv_heads"], case["dim"]
    if case["op"] == "decode":
        total, hq, b = sum(_lens(case)), case["heads"], case["batch"]
        moved = 2 * total * hkv * d * es + 2 * b * hq * d * es + 4 * b * hq + 4 * total // case["block"] + 4 * b
        return dict(bytes=moved + (8 * total * hkv if case["weights"] else 0), flops=4 * total * hq * d)
    if case["op"] == "evict":
        lens = _lens(case)
        cut = [n for n in lens if n > case["budget"]]
        # rows that stay where they are (all of a short cache in place, the sink) need not move
        rows = len(cut) * (case["budget"] - case["sink"]) if case["in_place"] else sum(min(n, case["budget"]) for n in lens)
        moved = 4 * rows * hkv * d * es + 8 * sum(lens) * hkv + 4 * case["batch"] * (hkv * case["budget"] + 2)
        return dict(bytes=moved, flops=sum(lens) * hkv)
    n, hq = sum(_counts(case)), case["heads"]
    moved = n * ((2 * hq + 4 * hkv) * d * es + 4 * case["axes"])
    return dict(bytes=moved, flops=n * (hq + hkv) * case["rot"] * 3)


# ------------------------------------------------------------------ the inputs

def _table(gen, batch, per_seq, first):
    """Block tables with the physical blocks in no order, from block `first` on."""
    ids = torch.randperm(batch * per_seq, generator=gen, device="cuda").to(torch.int32) + first
    return ids.reshape(batch, per_seq).contiguous()


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    dt, hkv, d, bs, b = TYPES[case["dtype"]], case["kv_heads"], case["dim"], case["block"], case["batch"]

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device="cuda", dtype=torch.float32).to(dt)

    def cache(blocks):
        # in pieces: a long cache's fp32 draws need not all be there at once
        c = torch.empty(blocks, bs, hkv, d, device="cuda", dtype=dt)
        step = max(1, (1 << 27) // (bs * hkv * d))
        for i in range(0, blocks, step):
            c[i:i + step] = normal(min(step, blocks - i), bs, hkv, d)
        return c

    s = dict(case=case)
    if case["op"] in ("decode", "evict"):
        lens = _lens(case)
        per_seq = -(-max(lens) // bs)
        s["table"] = _table(gen, b, per_seq, 0)
        s["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
        blocks = b * per_seq
    if case["op"] == "decode":
        s["k"], s["v"] = cache(blocks), cache(blocks)
        s["q"] = normal(b, case["heads"], d)
        # what earlier tokens left: heavy-tailed sums
        s["weights"] = torch.randn(b, hkv, per_seq * bs, generator=gen, device="cuda").mul_(1.5).exp_() if case["weights"] else None
    elif case["op"] == "evict":
        w = torch.randn(b, hkv, per_seq * bs, generator=gen, device="cuda").mul_(2).exp_()
        # tokens that no query has looked at have sums of zero: ties
        s["weights"] = torch.where(torch.rand(w.shape, generator=gen, device="cuda") < 0.05, torch.zeros_like(w), w)
        s["weights_out"] = torch.zeros_like(w)
        s["dst"] = None
        if not case["in_place"]:
            width = -(-min(max(lens), case["budget"]) // bs)
            s["dst"] = torch.zeros(b, per_seq, dtype=torch.int32, device="cuda")
            s["dst"][:, :width] = _table(gen, b, width, blocks)
            blocks += b * width
        s["k"], s["v"] = cache(blocks), cache(blocks)
        n = [min(x, case["budget"]) for x in lens]
        at = [(i, r) for i, x in enumerate(n) for r in range(x)]
        s["rows"] = torch.tensor(at, dtype=torch.int64, device="cuda").T.contiguous()
    else:
        n, hq, rot, axes = case["nodes"], case["heads"], case["rot"], case["axes"]
        counts = _counts(case)
        s["counts"] = torch.tensor(counts, dtype=torch.int32, device="cuda") if case["ragged"] else None
        prefix = torch.randint(case["prefix"] // 2, case["prefix"] + 1, (b,), generator=gen, device="cuda", dtype=torch.int32)
        s["prefix"] = prefix
        per_seq = -(-(case["prefix"] + n) // bs)
        s["table"] = _table(gen, b, per_seq, 0)
        # zeros: the rows are this call's own output
        s["k"], s["v"] = (torch.zeros(b * per_seq, bs, hkv, d, device="cuda", dtype=dt) for _ in range(2))
        # one fused projection's output: q, k and v lie side by side in a node's row
        qkv = normal(b, n, hq + 2 * hkv, d)
        s["q_in"], s["k_in"], s["v_in"] = qkv[:, :, :hq], qkv[:, :, hq:hq + hkv], qkv[:, :, hq + hkv:]
        s["inv_freq"] = (500000.0 ** (-torch.arange(0, rot // 2, device="cuda", dtype=torch.float64) * 2 / rot)).float()
        pairs = rot // 2
        if case["split"] == "sections":
            s["axis"] = [i * axes // pairs for i in range(pairs)]
        else:
            s["axis"] = [i % axes for i in range(pairs)]
        s["axis_dev"] = torch.tensor(s["axis"], dtype=torch.int64, device="cuda")
        i = torch.arange(n, device="cuda")
        s["parent"] = None
        if case["tree"]:
            back = (torch.rand(b, n, generator=gen, device="cuda") * torch.clamp(i, max=4)).long()
            s["parent"] = (i - 1 - back).to(torch.int32)
        s["positions"] = None
        if axes > 1 and not case["tree"]:
            # text, then an image of some rows and columns, then text again
            first, last, wide = n // 4, n - n // 4, max(1, int(math.sqrt(n / 2)))
            r = torch.clamp(i - first, 0, max(0, last - first - 1))
            inside = (i >= first) & (i < last)
            after = torch.where(i >= last, i - last + wide + first, i)
            grid = torch.stack([torch.zeros_like(r), r // wide, r % wide, r % 7][:axes])
            pos = torch.where(inside, first + grid, after.expand(axes, n))
            s["positions"] = (pos[:, None, :] + prefix[None, :, None]).to(torch.int32).contiguous()
        at = [(i_, j) for i_, c in enumerate(counts) for j in range(c)]
        s["rows"] = torch.tensor(at, dtype=torch.int64, device="cuda").T.contiguous()
        s["q_out"] = torch.zeros(b, n, hq, d, device="cuda", dtype=dt)
    return s


# ------------------------------------------------------------------ one pass

def run(s):
    op = s["case"]["op"]
    if op == "decode":
        return _decode_own(s) if own else _decode(s)
    if op == "evict":
        return _evict_own(s) if own else _evict(s)
    return _rotary_own(s) if own else _rotary(s)


def _decode(s):
    q, k, v, table, lens = s["q"], s["k"], s["v"], s["table"], s["lens"]
    b, hq, d = q.shape
    hkv = k.shape[2]
    kk = k[table.long()].reshape(b, -1, hkv, d).permute(0, 2, 1, 3).float()
    vv = v[table.long()].reshape(b, -1, hkv, d).permute(0, 2, 1, 3).float()
    scores = (q.float().reshape(b, hkv, hq // hkv, d) * d ** -0.5) @ kk.transpose(2, 3)
    seen = torch.arange(kk.shape[2], device=q.device) < lens[:, None]
    scores = torch.where(seen[:, None, None, :], scores, -torch.inf)
    top = scores.amax(dim=3, keepdim=True)
    e = torch.exp(scores - top)
    total = e.sum(dim=3, keepdim=True)
    p = e / total
    out = (p @ vv).reshape(b, hq, d).to(q.dtype)
    lse = (top + torch.log(total)).reshape(b, hq)
    if s["weights"] is None:
        return out, lse
    s["weights"] += p.sum(dim=2)
    return out, lse, s["weights"]


def _decode_own(s):
    import tree_speculative_decoding_07_b200 as tv
    out, lse = tv.decode_attention(s["q"], s["k"], s["v"], s["table"], s["lens"], attn_weights=s["weights"])
    return (out, lse) if s["weights"] is None else (out, lse, s["weights"])


def _evict(s):
    case, w, lens, table = s["case"], s["weights"], s["lens"], s["table"].long()
    budget, bs = case["budget"], case["block"]
    b, hkv, width = w.shape
    t = torch.arange(width, device=w.device)
    n = lens.long()[:, None]
    short = n <= budget
    always = (t < case["sink"]) | (t >= n - case["recent"]) | short
    rank = torch.where((t >= n)[:, None], -torch.inf, torch.where(always[:, None], torch.inf, w))
    order = torch.sort(rank, dim=2, descending=True, stable=True).indices[:, :, :budget]
    if width < budget:
        order = torch.nn.functional.pad(order, (0, budget - width), value=width)
    kept_n = torch.clamp(n, max=budget)
    r = torch.arange(budget, device=w.device)
    kept = torch.sort(torch.where((r < kept_n)[:, None], order, width), dim=2).values
    # the weights go along; the rest of each row's old length is cleared
    rows_w = torch.where(kept < width, torch.gather(w, 2, kept.clamp(max=width - 1)), 0.0)
    new_w = torch.nn.functional.pad(rows_w, (0, max(0, width - budget)))[:, :, :width]
    s["weights_out"].copy_(torch.where((t < n)[:, None], new_w, s["weights_out"]))
    # the rows, all of them read before any is written
    at_b, at_r = s["rows"]
    src = kept[at_b, :, at_r]
    head = torch.arange(hkv, device=w.device)
    sb, ss = table[at_b[:, None], src // bs], src % bs
    to = table if s["dst"] is None else s["dst"].long()
    db, ds = to[at_b, at_r // bs][:, None], (at_r % bs)[:, None]
    k_rows, v_rows = s["k"][sb, ss, head], s["v"][sb, ss, head]
    s["k"][db, ds, head] = k_rows
    s["v"][db, ds, head] = v_rows
    kept = torch.where((r < kept_n)[:, None], kept, -1).to(torch.int32)
    return s["k"], s["v"], s["weights_out"], kept, kept_n[:, 0].to(torch.int32)


def _evict_own(s):
    import tree_speculative_decoding_07_b200 as tv
    case = s["case"]
    new_lens, kept = tv.evict_cache(s["k"], s["v"], s["table"], s["lens"], s["weights"], case["budget"],
                                    sink=case["sink"], recent=case["recent"], dst_block_table=s["dst"],
                                    weights_out=s["weights_out"])
    return s["k"], s["v"], s["weights_out"], kept, new_lens


def _turn(x, cos, sin, rot, interleaved):
    x = x.float()
    if interleaved:
        a, c = x[..., 0:rot:2], x[..., 1:rot:2]
        y = torch.stack([a * cos - c * sin, a * sin + c * cos], dim=-1).flatten(-2)
    else:
        a, c = x[..., :rot // 2], x[..., rot // 2:rot]
        y = torch.cat([a * cos - c * sin, a * sin + c * cos], dim=-1)
    return torch.cat([y, x[..., rot:]], dim=-1)


def _rotary(s):
    case, bs = s["case"], s["case"]["block"]
    b, n = s["q_in"].shape[:2]
    at_b, at_j = s["rows"]
    if s["positions"] is not None:
        pos = s["positions"][:, at_b, at_j].T.double()[:, s["axis_dev"]]
    else:
        depth = torch.arange(n, device="cuda").expand(b, n)
        if s["parent"] is not None:
            # the depth is the number of steps to the root; each round doubles the steps taken
            up = s["parent"].long()
            depth = (up >= 0).long()
            for _ in range(7):
                more = torch.where(up >= 0, torch.gather(depth, 1, up.clamp(min=0)), 0)
                up = torch.where(up >= 0, torch.gather(up, 1, up.clamp(min=0)), -1)
                depth = depth + more
        pos = (s["prefix"].long()[:, None] + depth)[at_b, at_j].double()[:, None]
    angle = pos * s["inv_freq"].double()
    cos, sin = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]
    dt = s["q_in"].dtype
    s["q_out"][at_b, at_j] = _turn(s["q_in"][at_b, at_j], cos, sin, case["rot"], case["interleaved"]).to(dt)
    place = s["prefix"].long()[at_b] + at_j
    block, slot = s["table"].long()[at_b, place // bs], place % bs
    s["k"][block, slot] = _turn(s["k_in"][at_b, at_j], cos, sin, case["rot"], case["interleaved"]).to(dt)
    s["v"][block, slot] = s["v_in"][at_b, at_j]
    return s["q_out"], s["k"], s["v"]


def _rotary_own(s):
    import tree_speculative_decoding_07_b200 as tv
    tv.rotary_write(s["k_in"], s["v_in"], s["inv_freq"], s["k"], s["v"], s["table"], s["prefix"], q=s["q_in"],
                    q_out=s["q_out"], parent_idx=s["parent"], positions=s["positions"],
                    axis_of_pair=s["axis"] if s["case"]["axes"] > 1 else None,
                    interleaved=s["case"]["interleaved"], node_counts=s["counts"])
    return s["q_out"], s["k"], s["v"]


# ------------------------------------------------------------------ in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "decode":
        return _exact_decode(case, s)
    if case["op"] == "evict":
        return _exact_evict(case, s)
    return _exact_rotary(case, s)


def _exact_decode(case, s):
    bs, d, g = case["block"], case["dim"], case["heads"] // case["kv_heads"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.zeros(s["q"].shape[:2], dtype=torch.float64, device="cuda")
    weights = None if s["weights"] is None else s["weights"].double()
    for i, n in enumerate(_lens(case)):
        blocks = s["table"][i, :-(-n // bs)].long()
        for h in range(case["kv_heads"]):
            keys = s["k"][blocks, :, h].reshape(-1, d)[:n].double()
            values = s["v"][blocks, :, h].reshape(-1, d)[:n].double()
            logits = s["q"][i, h * g:(h + 1) * g].double() @ keys.T / math.sqrt(d)
            out[i, h * g:(h + 1) * g] = torch.softmax(logits, dim=1) @ values
            lse[i, h * g:(h + 1) * g] = torch.logsumexp(logits, dim=1)
            if weights is not None:
                weights[i, h, :n] += torch.softmax(logits, dim=1).sum(dim=0)
    return (out, lse) if weights is None else (out, lse, weights)


def _exact_evict(case, s):
    bs, budget = case["block"], case["budget"]
    k, v, w_out = s["k"].double(), s["v"].double(), s["weights_out"].double()
    kept_all = torch.full((case["batch"], case["kv_heads"], budget), -1, dtype=torch.int32, device="cuda")
    for i, n in enumerate(_lens(case)):
        for h in range(case["kv_heads"]):
            if n <= budget:
                kept = torch.arange(n, device="cuda")
            else:
                middle = s["weights"][i, h, case["sink"]:n - case["recent"]]
                best = torch.argsort(middle, descending=True, stable=True)[:budget - case["sink"] - case["recent"]]
                kept = torch.cat([torch.arange(case["sink"], device="cuda"), torch.sort(best).values + case["sink"],
                                  torch.arange(n - case["recent"], n, device="cuda")])
            m = kept.numel()
            kept_all[i, h, :m] = kept.to(torch.int32)
            w_out[i, h, :n] = 0
            w_out[i, h, :m] = s["weights"][i, h, kept].double()
            src = s["table"][i].long()[kept // bs]
            r = torch.arange(m, device="cuda")
            dst = (s["table"] if s["dst"] is None else s["dst"])[i].long()[r // bs]
            k[dst, r % bs, h] = s["k"][src, kept % bs, h].double()
            v[dst, r % bs, h] = s["v"][src, kept % bs, h].double()
    new = torch.tensor([min(n, budget) for n in _lens(case)], dtype=torch.int32, device="cuda")
    return k, v, w_out, kept_all, new


def _exact_rotary(case, s):
    rot, bs = case["rot"], case["block"]
    q, k, v = s["q_out"].double(), s["k"].double(), s["v"].double()
    freq = s["inv_freq"].double()
    for i, n in enumerate(_counts(case)):
        if s["positions"] is not None:
            pos = s["positions"][s["axis_dev"], i, :n].double().T
        else:
            depth = list(range(n))
            if s["parent"] is not None:
                for j, up in enumerate(s["parent"][i, :n].tolist()):
                    depth[j] = 0 if j == 0 else depth[up] + 1
            pos = (torch.tensor(depth, device="cuda", dtype=torch.float64) + float(s["prefix"][i]))[:, None]
        turn = torch.polar(torch.ones((), dtype=torch.float64, device="cuda"), pos * freq)[:, None, :]

        def rotate(x):
            x = x.double().clone()
            first = torch.arange(rot // 2, device="cuda") * (2 if case["interleaved"] else 1)
            second = first + (1 if case["interleaved"] else rot // 2)
            z = torch.complex(x[..., first], x[..., second]) * turn
            x[..., first], x[..., second] = z.real, z.imag
            return x

        q[i, :n] = rotate(s["q_in"][i, :n])
        place = int(s["prefix"][i]) + torch.arange(n, device="cuda")
        block = s["table"][i].long()[place // bs]
        k[block, place % bs] = rotate(s["k_in"][i, :n])
        v[block, place % bs] = s["v_in"][i, :n].double()
    return q, k, v

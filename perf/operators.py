"""Cases and plain forms of the token-sequence operators: sliding-window
attention with sinks (forward, training, single tokens), the 8-bit key/value
cache's write and read-back, and attention over that cache.

``run`` computes an operator in elementary torch operations in fp32, or, with
``own`` set, through this package's public calls.  ``exact`` is the operator's
definition in fp64, computed another way.  Head counts (16, 24) and head dims
(64, 128) are those of the package's own workloads.
"""
import random

import torch

own = False

QMAX = {"e4m3": 448.0, "int8": 127.0}
SCALE_FLOOR = 2.0 ** -100  # the smallest scale a block of the cache has
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


# ------------------------------------------------------------------ cases
def listed():
    return [
        # prompts of several requests packed behind one another, each of its own length
        dict(name="prefill packed", op="forward", dtype="bf16", batch=6, heads=24, kv_heads=8, d=128, packed=True,
             q_len=2048, kv_len=2048, same=True, lens=3, window=1024, sinks=4, rows_last=False),
        # one chunk of two long prompts against the keys before it; rows outside heads, as a projection leaves them
        dict(name="prefill chunk", op="forward", dtype="fp16", batch=2, heads=16, kv_heads=4, d=64, packed=False,
             q_len=500, kv_len=8191, same=False, lens=0, window=2048, sinks=16, rows_last=True),
        # one new token of eight requests: the smallest call of the window's forward
        dict(name="token", op="forward", dtype="bf16", batch=8, heads=24, kv_heads=8, d=128, packed=False,
             q_len=1, kv_len=4097, same=False, lens=0, window=1024, sinks=4, rows_last=False),
        # a training step's attention, a key head for each query head, no sinks
        dict(name="train d64", op="train", dtype="bf16", batch=2, heads=16, kv_heads=16, d=64, packed=False,
             q_len=4096, kv_len=4096, same=True, lens=0, window=512, sinks=0, rows_last=False),
        # the longest training sequence, shared key heads, an odd length
        dict(name="train long d128", op="train", dtype="fp16", batch=1, heads=24, kv_heads=8, d=128, packed=False,
             q_len=8190, kv_len=8190, same=True, lens=0, window=2048, sinks=4, rows_last=True),
        # short documents packed into one training row
        dict(name="train packed", op="train", dtype="bf16", batch=9, heads=16, kv_heads=8, d=128, packed=True,
             q_len=701, kv_len=701, same=True, lens=5, window=256, sinks=64, rows_last=False),
        # one token of every running request goes into the cache
        dict(name="cache append", op="store", dtype="bf16", batch=64, kv_heads=8, d=128, format="e4m3", block=16,
             page=64, before=2000, count=1, lens=7),
        # prompts go into the cache and are read back for the next chunk's attention
        dict(name="cache prompts", op="store", dtype="bf16", batch=8, kv_heads=8, d=128, format="int8", block=64,
             page=128, before=0, count=4096, lens=11),
        # a chunk that begins inside a block already in the cache
        dict(name="cache chunk d64", op="store", dtype="fp16", batch=16, kv_heads=4, d=64, format="e4m3", block=32,
             page=32, before=777, count=513, lens=13),
        # one request, one token: latency
        dict(name="decode one", op="decode", dtype="bf16", batch=1, heads=24, kv_heads=8, d=128, format="e4m3",
             block=16, page=64, q_len=1, kv_len=1031, lens=0, window=0, sinks=0),
        # a full server: ragged long contexts
        dict(name="decode many", op="decode", dtype="bf16", batch=64, heads=24, kv_heads=8, d=128, format="e4m3",
             block=64, page=128, q_len=1, kv_len=8192, lens=17, window=0, sinks=0),
        # a few drafted tokens at a time, a window with sinks over long contexts
        dict(name="decode window d64", op="decode", dtype="fp16", batch=32, heads=16, kv_heads=4, d=64, format="int8",
             block=32, page=64, q_len=4, kv_len=20000, lens=19, window=4096, sinks=4),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(["forward", "train", "store", "decode"])
    d = rng.choice([64, 128])
    dtype = rng.choice(["bf16", "fp16"])
    kv_heads = rng.choice([2, 4, 8])
    heads = kv_heads * rng.choice([1, 2, 3, 4])
    lens = rng.randrange(1, 10 ** 6)
    if op in ("forward", "train"):
        packed = rng.random() < 0.5
        batch = _log_int(rng, 2, 9) if packed else _log_int(rng, 1, 3)
        kv_len = _log_int(rng, 60, 1100) if packed else _log_int(rng, 200, 5000)
        same = op == "train" or packed or rng.random() < 0.5
        q_len = kv_len if same else _log_int(rng, 1, kv_len)
        return dict(op=op, dtype=dtype, batch=batch, heads=heads, kv_heads=kv_heads, d=d, packed=packed, q_len=q_len,
                    kv_len=kv_len, same=same, lens=lens if packed else 0, window=_log_int(rng, 32, 3000),
                    sinks=rng.choice([0, 1, 4, 16, 64, 130]), rows_last=not packed and rng.random() < 0.5)
    fmt = rng.choice(["e4m3", "int8"])
    block = rng.choice([16, 32, 64, 128])
    page = block * rng.choice([1, 2, 4])
    if op == "store":
        count = rng.choice([1, _log_int(rng, 2, 3000)])
        return dict(op=op, dtype=dtype, batch=_log_int(rng, 1, 48) if count < 500 else _log_int(rng, 1, 8),
                    kv_heads=kv_heads, d=d, format=fmt, block=block, page=page,
                    before=rng.choice([0, _log_int(rng, 1, 2000)]), count=count, lens=lens)
    kv_len = _log_int(rng, 100, 20000)
    return dict(op=op, dtype=dtype, batch=_log_int(rng, 1, max(1, min(64, 200000 // kv_len))), heads=heads,
                kv_heads=kv_heads, d=d, format=fmt, block=block, page=page, q_len=rng.choice([1, 1, 2, 5, 8]),
                kv_len=kv_len, lens=lens, window=rng.choice([0, _log_int(rng, 64, 5000)]),
                sinks=rng.choice([0, 4, 64]))


def _lengths(case, longest):
    """One length per sequence: all the longest, or drawn from `lens` with at least one of them the longest."""
    n = case["batch"]
    if not case["lens"]:
        return [longest] * n
    r = random.Random(case["lens"])
    got = [max(1, int(longest * (0.2 + 0.8 * r.random()))) for _ in range(n)]
    got[r.randrange(n)] = longest
    return got


def _store_counts(case):
    """(tokens before, new tokens) of each sequence of a store case; a short sequence has tokens before it."""
    before = _lengths(case, case["before"]) if case["before"] else [0] * case["batch"]
    return before, _lengths(dict(case, lens=case["lens"] + 1), case["count"])


# ------------------------------------------------------------------ inputs
def _normal(shape, g, dtype):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).to(dtype)


def _starts(lens):
    return torch.tensor([0] + lens, dtype=torch.int32).cumsum(0).to(torch.int32).cuda()


def _pages(case, lens, g):
    """A page table in shuffled order, one page more than the sequences need, absent pages -1."""
    page, n = case["page"], [-(-x // case["page"]) for x in lens]
    order = torch.randperm(sum(n) + 1, generator=g, device="cuda").to(torch.int32)
    table = torch.full((len(n), max(n)), -1, dtype=torch.int32, device="cuda")
    at = 0
    for i, m in enumerate(n):
        table[i, :m] = order[at:at + m]
        at += m
    return table, sum(n) + 1


def _codes(x, scale, fmt):
    """x / scale in 8 bits: x times the reciprocal of scale, rounded to nearest even, no further than the largest code."""
    y = (x * (1.0 / scale)).clamp(-QMAX[fmt], QMAX[fmt])
    return y.to(torch.float8_e4m3fn) if fmt == "e4m3" else y.round().to(torch.int8)


def _filled(case, pages, g):
    """Codes and scales of a cache that holds normal keys and values in every page."""
    x = torch.randn((pages, case["kv_heads"], case["page"] // case["block"], case["block"], case["d"]), generator=g,
                    device="cuda")
    scale = (x.abs().amax((-1, -2)) / QMAX[case["format"]]).clamp_min(SCALE_FLOOR)
    codes = _codes(x, scale[..., None, None], case["format"])
    return codes.reshape(pages, case["kv_heads"], case["page"], case["d"]), scale


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dtype, s = TYPES[case["dtype"]], dict(case=case)
    if case["op"] in ("forward", "train"):
        if case["packed"]:
            s["q_lens"] = s["kv_lens"] = lens = _lengths(case, case["q_len"])
            s["cu"] = _starts(lens)
            s["seq"] = torch.repeat_interleave(torch.arange(len(lens)), torch.tensor(lens)).cuda()
            s["row"] = torch.cat([torch.arange(n) for n in lens]).cuda()
            b, nq, nk = 1, sum(lens), sum(lens)
        else:
            b, nq, nk = case["batch"], case["q_len"], case["kv_len"]

        def make(heads, n):
            if case["rows_last"]:
                return _normal((b, n, heads, case["d"]), g, dtype).transpose(1, 2)
            return _normal((b, heads, n, case["d"]), g, dtype)

        s["q"], s["k"], s["v"] = make(case["heads"], nq), make(case["kv_heads"], nk), make(case["kv_heads"], nk)
        if case["op"] == "train":
            s["do"] = make(case["heads"], nq)
            for n in "qkv":
                s[n].requires_grad_()
        return s
    if case["op"] == "store":
        before, count = _store_counts(case)
        after = [a + c for a, c in zip(before, count)]
        s["table"], pages = _pages(case, after, g)
        s["start"] = torch.tensor(before, dtype=torch.int32, device="cuda")
        s["count"] = torch.tensor(count, dtype=torch.int32, device="cuda")
        shape = (case["batch"], case["kv_heads"], case["count"], case["d"])
        s["k"], s["v"] = _normal(shape, g, dtype), _normal(shape, g, dtype)
    else:
        lens = _lengths(case, case["kv_len"])
        s["table"], pages = _pages(case, lens, g)
        s["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
        s["q"] = _normal((case["batch"], case["heads"], case["q_len"], case["d"]), g, dtype)
    (s["kc"], s["ks"]), (s["vc"], s["vs"]) = _filled(case, pages, g), _filled(case, pages, g)
    if own:
        from sparse_local_attention_b200 import KVCache
        s["cache"] = KVCache.from_tensors(s["kc"], s["vc"], s["ks"], s["vs"])
    return s


# ------------------------------------------------------------------ plain forms
def _visible(qpos, kpos, window, sinks):
    """Keys a query sees: none after it, the last `window` up to it (0: all), and the first `sinks`."""
    m = kpos <= qpos
    return m & ((kpos > qpos - window) | (kpos < sinks)) if window else m


def _window_mask(s):
    c = s["case"]
    if c["packed"]:
        m = _visible(s["row"][:, None], s["row"][None, :], c["window"], c["sinks"])
        return m & (s["seq"][:, None] == s["seq"][None, :])
    q = torch.arange(c["q_len"], device="cuda") + (c["kv_len"] - c["q_len"])
    return _visible(q[:, None], torch.arange(c["kv_len"], device="cuda")[None, :], c["window"], c["sinks"])


def _softmax(scores, mask):
    """(probabilities, log of the sum) over the last axis where mask; zero and -inf where it leaves nothing."""
    scores = scores.masked_fill(~mask, float("-inf"))
    top = scores.amax(-1, keepdim=True)
    p = torch.exp(scores - torch.where(top.isinf(), torch.zeros_like(top), top))
    total = p.sum(-1, keepdim=True)
    return p / torch.where(total == 0, torch.ones_like(total), total), (top + torch.log(total))[..., 0]


def _grouped(x, kv_heads):
    return x.float().unflatten(1, (kv_heads, x.shape[1] // kv_heads))


def _plain_window(s):
    c, scale = s["case"], s["case"]["d"] ** -0.5
    q, k, v = _grouped(s["q"], c["kv_heads"]), s["k"].float()[:, :, None], s["v"].float()[:, :, None]
    p, lse = _softmax(q @ k.transpose(-1, -2) * scale, _window_mask(s))
    o = p @ v
    out = dict(o=o.flatten(1, 2).to(s["q"].dtype))
    if c["op"] == "forward":
        out["lse"] = lse.flatten(1, 2)
        return out
    do = _grouped(s["do"], c["kv_heads"])
    out["dv"] = (p.transpose(-1, -2) @ do).sum(2).to(s["q"].dtype)
    ds = do @ v.transpose(-1, -2)
    ds -= (do * o).sum(-1, keepdim=True)
    ds *= p
    out["dq"] = (ds @ k * scale).flatten(1, 2).to(s["q"].dtype)
    out["dk"] = (ds.transpose(-1, -2) @ q * scale).sum(2).to(s["q"].dtype)
    return out


def _gathered(codes, scale, table):
    """The values of each sequence's pages behind one another: [batch, kv_heads, tokens, d] in fp32."""
    block = codes.shape[2] // scale.shape[2]
    t = table.clamp_min(0).long()
    x = codes[t].float() * scale[t].repeat_interleave(block, -1)[..., None]
    return x.transpose(1, 2).flatten(2, 3)


def _scattered(x, codes, table):
    """[batch, kv_heads, tokens, ...] back into pages of `codes`' shape, where the table has a page."""
    per = codes.shape[2]
    y = x.unflatten(2, (table.shape[1], per)).transpose(1, 2)
    codes[table[table >= 0].long()] = y[table >= 0]


def _plain_store(s):
    c = s["case"]
    fmt, block, span = c["format"], c["block"], s["table"].shape[1] * c["page"]
    at = torch.arange(span, device="cuda")[None, :] - s["start"][:, None]  # row of k, v of each token of a sequence
    new = ((at >= 0) & (at < s["count"][:, None]))[:, None, :]
    have = (at < 0).unflatten(1, (-1, block))[:, None, :, 0]  # blocks that hold earlier tokens
    touched = new.unflatten(2, (-1, block)).any(-1)
    row = at.clamp(0, c["count"] - 1)[:, None, :, None].expand(-1, c["kv_heads"], -1, c["d"])
    out, blocks = {}, s["ks"].shape[2]
    tb = s["table"].clamp_min(0).long()
    for n in ("k", "v"):
        codes, scales = s[n + "c"], s[n + "s"]
        x = torch.where(new[..., None], s[n].float().gather(2, row), 0.0)
        amax = x.abs().amax(-1).unflatten(2, (-1, block)).amax(-1)
        old = scales[tb].transpose(1, 2).flatten(2, 3)
        was = torch.where(have, old, 0.0)
        fresh = torch.maximum(was, (amax / QMAX[fmt]).clamp_min(SCALE_FLOOR))
        fresh = torch.where(touched, fresh, old)
        wide = fresh.repeat_interleave(block, 2)[..., None]
        held = codes[tb].transpose(1, 2).flatten(2, 3).float()
        moved = _codes(held * old.repeat_interleave(block, 2)[..., None], wide, fmt)
        grown = (touched & have & (fresh > old)).repeat_interleave(block, 2)[..., None]
        kept = torch.where(grown, moved.float(), held)
        done = torch.where(new[..., None], _codes(x, wide, fmt).float(), kept)
        _scattered(done.to(codes.dtype), codes, s["table"])
        _scattered(fresh, scales, s["table"])
        out[n] = torch.where(new[..., None], done * wide, 0.0)
        out[n] = out[n].gather(2, _back(s)).to(s[n].dtype) * _there(s)
        out[n + "_scale"] = scales
    return out


def _back(s):
    """Tokens start .. start + count of each sequence, as indices of a gather along the tokens."""
    c = s["case"]
    i = s["start"][:, None].long() + torch.arange(c["count"], device="cuda")
    i = i.clamp_max(s["table"].shape[1] * c["page"] - 1)
    return i[:, None, :, None].expand(-1, c["kv_heads"], -1, c["d"])


def _there(s):
    return (torch.arange(s["case"]["count"], device="cuda") < s["count"][:, None])[:, None, :, None]


def _plain_decode(s):
    c = s["case"]
    k, v = (_gathered(s[n + "c"], s[n + "s"], s["table"])[:, :, None] for n in "kv")
    q = _grouped(s["q"], c["kv_heads"])
    qpos = (s["lens"][:, None] - c["q_len"] + torch.arange(c["q_len"], device="cuda"))[:, None, None, :, None]
    mask = _visible(qpos, torch.arange(k.shape[3], device="cuda"), c["window"], c["sinks"])
    p, lse = _softmax(q @ k.transpose(-1, -2) * c["d"] ** -0.5, mask)
    return dict(o=(p @ v).flatten(1, 2).to(s["q"].dtype), lse=lse.flatten(1, 2))


# ------------------------------------------------------------------ one pass
def run(s):
    c = s["case"]
    if not own:
        with torch.no_grad():
            return {"forward": _plain_window, "train": _plain_window, "store": _plain_store,
                    "decode": _plain_decode}[c["op"]](s)
    from sparse_local_attention_b200 import sliding_window_attention, window_forward
    if c["op"] in ("forward", "train"):
        seqs = dict(cu_q=s["cu"], cu_kv=s["cu"], max_q=c["q_len"], max_kv=c["kv_len"]) if c["packed"] else {}
        if c["op"] == "forward":
            o, lse = window_forward(s["q"], s["k"], s["v"], c["window"], c["sinks"], **seqs)
            return dict(o=o, lse=lse)
        o = sliding_window_attention(s["q"], s["k"], s["v"], c["window"], c["sinks"], **seqs)
        dq, dk, dv = torch.autograd.grad(o, (s["q"], s["k"], s["v"]), s["do"])
        return dict(o=o.detach(), dq=dq, dk=dk, dv=dv)
    cache = s["cache"]
    if c["op"] == "store":
        cache.write(s["k"], s["v"], s["table"], s["start"], s["count"])
        k, v = cache.read(s["table"], s["start"], s["count"], c["count"], s["k"].dtype)
        return dict(k=k, v=v, k_scale=cache.k_scale, v_scale=cache.v_scale)
    o, lse = cache.attention(s["q"], s["table"], s["lens"], c["window"], c["sinks"])
    return dict(o=o, lse=lse)


# ------------------------------------------------------------------ what a pass cannot do without
def _seen(qpos, window, sinks):
    """Number of keys that a query at qpos sees."""
    if qpos < 0:
        return 0
    if not window or window > qpos:
        return qpos + 1
    return window + min(sinks, qpos - window + 1)


def _pairs_keys(nq, nk, window, sinks):
    """(query, key) pairs and keys seen by anyone, of one sequence."""
    first = nk - nq
    pairs = sum(_seen(first + i, window, sinks) for i in range(nq))
    low = max(0, max(first, 0) - window + 1) if window else 0
    return pairs, (nk - low + min(sinks, low)) if nq and nk else 0


def work(case):
    c, d = case, case["d"]
    if c["op"] == "store":
        before, count = _store_counts(c)
        n = sum(count) * c["kv_heads"] * 2  # rows of keys and values
        scales = sum(-(-(a + x) // c["block"]) - a // c["block"] for a, x in zip(before, count)) * c["kv_heads"] * 2
        # read the new rows, write codes and scales, read both back, write the rows
        return {"bytes": n * d * (2 + 1 + 1 + 2) + scales * 8, "flops": 3 * n * d}
    if c["op"] == "decode":
        lens = _lengths(c, c["kv_len"])
        pk = [_pairs_keys(c["q_len"], n, c["window"], c["sinks"]) for n in lens]
        keys, rows = sum(k for _, k in pk), c["batch"] * c["heads"] * c["q_len"]
        b = 2 * keys * c["kv_heads"] * (d + 4 / c["block"]) + rows * (4 * d + 4)
        return {"bytes": b, "flops": 4 * d * c["heads"] * sum(p for p, _ in pk)}
    lens = _lengths(c, c["q_len"]) if c["packed"] else [c["q_len"]] * c["batch"]
    pk = [_pairs_keys(n, n if c["packed"] else c["kv_len"], c["window"], c["sinks"]) for n in lens]
    pairs, keys, rows = sum(p for p, _ in pk), sum(k for _, k in pk) * c["kv_heads"], sum(lens) * c["heads"]
    if c["op"] == "forward":
        return {"bytes": rows * (4 * d + 4) + keys * 4 * d, "flops": 4 * d * pairs * c["heads"]}
    # q, o, do, dq and k, v, dk, dv once each; two products forward, five back
    return {"bytes": rows * 8 * d + keys * 8 * d, "flops": 14 * d * pairs * c["heads"]}


# ------------------------------------------------------------------ the definition in 64 bits
def _exact_rows(q, k, v, first, window, sinks, do=None):
    """One head of one sequence, the queries at first, first + 1, ...: sums over each query's own list of keys, in
    chunks of queries.  k, v: [keys, d]; q: [heads of the group, queries, d]."""
    hq, nq, d = q.shape
    nk, scale = k.shape[0], d ** -0.5
    o, lse = torch.zeros_like(q), torch.full((hq, nq), float("-inf"), dtype=torch.float64, device=q.device)
    dq, dk, dv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    for a in range(0, nq, 512):
        b = min(nq, a + 512)
        last = first + b - 1
        if last < 0 or nk == 0:
            continue
        lo = max(0, first + a - window + 1) if window else 0
        keys = torch.cat([torch.arange(min(sinks, lo)), torch.arange(lo, min(last, nk - 1) + 1)]).to(q.device)
        pos = torch.arange(first + a, first + b, device=q.device)[:, None]
        hidden = (keys > pos) | ((pos - keys >= window) & (keys >= sinks) if window else keys > pos)
        x = torch.einsum("hqd,kd->hqk", q[:, a:b], k[keys]) * scale
        x[:, hidden] = float("-inf")
        z = torch.logsumexp(x, -1)
        lse[:, a:b] = z
        p = torch.where(hidden, 0.0, torch.exp(x - torch.where(z.isinf(), 0.0, z)[..., None]))
        o[:, a:b] = torch.einsum("hqk,kd->hqd", p, v[keys])
        if do is not None:
            g = do[:, a:b]
            dv.index_add_(0, keys, torch.einsum("hqk,hqd->kd", p, g))
            dp = torch.einsum("hqd,kd->hqk", g, v[keys])
            ds = p * (dp - (p * dp).sum(-1, keepdim=True)) * scale
            dq[:, a:b] = torch.einsum("hqk,kd->hqd", ds, k[keys])
            dk.index_add_(0, keys, torch.einsum("hqk,hqd->kd", ds, q[:, a:b]))
    return o, lse, dq, dk, dv


def _exact_window(case, s):
    c, group = case, case["heads"] // case["kv_heads"]
    q, k, v = (s[n].detach().double() for n in "qkv")
    do = s["do"].double() if c["op"] == "train" else None
    got = [torch.zeros_like(q), torch.zeros(q.shape[:3], dtype=torch.float64, device="cuda"), torch.zeros_like(q),
           torch.zeros_like(k), torch.zeros_like(v)]
    at = 0
    for i in range(c["batch"]):
        b = 0 if c["packed"] else i
        nq, nk = (s["q_lens"][i], s["kv_lens"][i]) if c["packed"] else (c["q_len"], c["kv_len"])
        r = slice(at, at + nq) if c["packed"] else slice(0, nq)
        rk = slice(at, at + nk) if c["packed"] else slice(0, nk)
        at += nq if c["packed"] else 0
        for h in range(c["kv_heads"]):
            hs = slice(h * group, (h + 1) * group)
            o, lse, dq, dk, dv = _exact_rows(q[b, hs, r], k[b, h, rk], v[b, h, rk], nk - nq, c["window"], c["sinks"],
                                             None if do is None else do[b, hs, r])
            got[0][b, hs, r], got[1][b, hs, r], got[2][b, hs, r] = o, lse, dq
            got[3][b, h, rk], got[4][b, h, rk] = dk, dv
    if do is None:
        return dict(o=got[0], lse=got[1])
    return dict(o=got[0], dq=got[2], dk=got[3], dv=got[4])


def _to_codes64(x, fmt):
    """The nearest code of each value, ties to even, in fp64."""
    if fmt == "int8":
        return x.round().clamp(-127, 127)
    step = 2.0 ** (torch.frexp(x.abs().clamp_min(2.0 ** -6))[1] - 4).double()  # e4m3: 3 bits behind the leading one
    return ((x / step).round() * step).clamp(-448, 448)


def _exact_store(case, s):
    c, fmt, block = case, case["format"], case["block"]
    before, count = _store_counts(c)
    out = {n: torch.zeros(s[n].shape, dtype=torch.float64, device="cuda") for n in "kv"}
    for n in "kv":
        scales = s[n + "s"].double()
        for i in range(c["batch"]):
            a, m = before[i], count[i]
            t, x = s["table"][i].tolist(), s[n][i, :, :m].double()
            for j in range(a // block, (a + m - 1) // block + 1):
                lo, hi = max(a, j * block), min(a + m, (j + 1) * block)
                part = x[:, lo - a:hi - a]
                page, slot = t[j * block // c["page"]], (j * block % c["page"]) // block
                fresh = (part.abs().amax((-1, -2)) / QMAX[fmt]).clamp_min(SCALE_FLOOR)
                if a > j * block:
                    fresh = torch.maximum(fresh, scales[page, :, slot])
                scales[page, :, slot] = fresh
                out[n][i, :, lo - a:hi - a] = _to_codes64(part / fresh[:, None, None], fmt) * fresh[:, None, None]
        out[n + "_scale"] = scales
    return out


def _exact_decode(case, s):
    c, group = case, case["heads"] // case["kv_heads"]
    o = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.zeros(s["q"].shape[:3], dtype=torch.float64, device="cuda")
    for i, n in enumerate(_lengths(c, c["kv_len"])):
        t = s["table"][i, :-(-n // c["page"])].long()
        for h in range(c["kv_heads"]):
            hs = slice(h * group, (h + 1) * group)
            kv = [(s[x + "c"][t, h].double() * s[x + "s"][t, h].double().repeat_interleave(c["block"], 1)[..., None])
                  .reshape(-1, c["d"])[:n] for x in "kv"]
            o[i, hs], lse[i, hs] = _exact_rows(s["q"][i, hs].double(), *kv, n - c["q_len"], c["window"], c["sinks"])[:2]
    return dict(o=o, lse=lse)


def exact(case, seed):
    s = prepare(case, seed)
    with torch.no_grad():
        if case["op"] in ("forward", "train"):
            return _exact_window(case, s)
        return (_exact_store if case["op"] == "store" else _exact_decode)(case, s)

"""The 8-bit key/value cache: write and read-back bit for bit against the
definition, attention over it against fp64, a serving run of them together,
and refusals."""
import ctypes

import pytest
import torch

import seq_ref
from sparse_local_attention_b200 import KVCache, sta, window_forward
from sparse_local_attention_b200.kv_cache import _Cache

BF16, FP16, E4M3, INT8 = torch.bfloat16, torch.float16, torch.float8_e4m3fn, torch.int8


def randn(*shape, seed, dtype):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).to(dtype)


def tables(batch, pages_per, seed=0, spare=2):
    order = torch.randperm(batch * pages_per + spare, generator=torch.Generator().manual_seed(seed)).to(torch.int32)
    return order[:batch * pages_per].view(batch, pages_per).clone(), batch * pages_per + spare


class Pair:
    """A device cache and its host model."""

    def __init__(self, pages, kv_heads, page, d, block, dtype):
        self.cache = KVCache(pages, kv_heads, page, d, block=block, dtype=dtype)
        self.host = [t.cpu() for t in (self.cache.k, self.cache.v, self.cache.k_scale, self.cache.v_scale)]

    def write(self, k, v, table, start, count=None):
        dev = [None if t is None else t.cuda() for t in (k, v, table, start, count)]
        self.cache.write(*dev, check=True)
        seq_ref.cache_write(self.host[0], self.host[2], k, table, start, count)
        seq_ref.cache_write(self.host[1], self.host[3], v, table, start, count)
        self.same()

    def same(self):
        c = self.cache
        for name, got, want in (("k_scale", c.k_scale, self.host[2]), ("v_scale", c.v_scale, self.host[3]),
                                ("k", c.k, self.host[0]), ("v", c.v, self.host[1])):
            assert torch.equal(got.cpu().view(torch.uint8), want.view(torch.uint8)), name


def ints(*x):
    return torch.tensor(x, dtype=torch.int32)


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", [E4M3, INT8], ids=["e4m3", "int8"])
@pytest.mark.parametrize("d,block,page,kv_heads,dtype", [(128, 16, 64, 2, BF16), (64, 64, 64, 3, FP16),
                                                         (128, 128, 256, 1, FP16), (64, 32, 96, 2, BF16)])
def test_write_and_read(fmt, d, block, page, kv_heads, dtype):
    """Prompts, chunks that begin inside a block, single tokens that raise a
    block's scale, ragged counts; then everything read back."""
    table, pages = tables(3, 4, seed=d + block)
    p = Pair(pages, kv_heads, page, d, block, fmt)
    span = 4 * page
    lens = [0, 0, 0]
    for step, counts in enumerate(([37, 1, span // 2], [block, 0, 5], [1, 2, 0], [1, block - 1, span // 2 - 5], [9, 1, 0])):
        n = max(max(counts), 1)
        k, v = (randn(3, kv_heads, n, d, seed=10 * step + i, dtype=dtype) * (1 + step) for i in (0, 1))
        counts = [min(c, span - a) for c, a in zip(counts, lens)]
        p.write(k, v, table, ints(*lens), ints(*counts))
        lens = [a + c for a, c in zip(lens, counts)]
    # counts past `rows` and below zero are cut; no count: all rows
    p.write(randn(3, kv_heads, 3, d, seed=90, dtype=dtype), randn(3, kv_heads, 3, d, seed=91, dtype=dtype), table, ints(0, 16, 5),
            ints(100, -4, 2))
    p.write(randn(3, kv_heads, 2, d, seed=92, dtype=dtype), randn(3, kv_heads, 2, d, seed=93, dtype=dtype), table, ints(3, 0, -1))
    start, rows = ints(0, 3, 7), span
    count = ints(*[max(0, n - s) for n, s in zip(lens, start.tolist())])
    k = torch.full((3, kv_heads, rows, d), 5.0, dtype=dtype, device="cuda")
    v = torch.full_like(k, 5.0).transpose(1, 2).contiguous().transpose(1, 2)
    p.cache.read(table.cuda(), start.cuda(), count.cuda(), rows, dtype, k=k, v=v, check=True)
    for b in range(3):
        s, n = int(start[b]), int(count[b])
        for got, codes, scales in ((k, p.host[0], p.host[2]), (v, p.host[1], p.host[3])):
            want = seq_ref.cache_values(codes, scales, table, b, s + n)[0][:, s:]
            # the product of code and scale rounds to fp32 and then to the type
            assert ((got[b, :, :n].double().cpu() - want).abs() <= want.abs() * (seq_ref.unit(dtype) + 2.0 ** -24)
                    + torch.finfo(dtype).smallest_normal * seq_ref.unit(dtype) * 2).all()
            assert bool((got[b, :, n:] == 5.0).all())
    k2, v2 = p.cache.read(table.cuda(), start.cuda(), count.cuda(), rows, dtype)
    for b in range(3):
        n = int(count[b])
        assert torch.equal(k2[b, :, :n], k[b, :, :n]) and not k2[b, :, n:].any() and torch.equal(v2[b, :, :n], v[b, :, :n])
    p.same()


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", [E4M3, INT8], ids=["e4m3", "int8"])
def test_values_a_block_can_meet(fmt):
    """All zero, tiny, huge, infinite and NaN rows; a block whose scale stays when smaller rows follow."""
    table = ints(1, 0).view(1, 2)
    for dtype in (BF16, FP16):
        p = Pair(2, 2, 32, 64, 16, fmt)
        big = torch.finfo(dtype).max
        x = randn(1, 2, 5, 64, seed=1, dtype=dtype)
        for i, f in enumerate((0.0, 1e-30, 1e-3, 1.0, 100.0, 0.01)):
            p.write((x.float() * f).to(dtype), (x.float() * (f and 1 / f)).clamp(-big, big).to(dtype), table, ints(5 * i))
        bad = x.clone()
        bad[0, 0, 0, 3], bad[0, 0, 1, 0], bad[0, 1, 2, 7], bad[0, 1, 4, 63] = float("inf"), float("nan"), float("-inf"), big
        p.write(bad, -bad, table, ints(30))
        p.write(torch.full_like(x, float("nan")), x, table, ints(0))
        assert bool(p.cache.k_scale.isfinite().all()) and bool((p.cache.k_scale[1, :, 0] == 2.0 ** -100).all())


@pytest.mark.gpu
def test_absent_pages_and_strides():
    """Entries outside [0, pages) and tokens past the table are not written
    and not read; strided rows give what contiguous ones give."""
    table = torch.tensor([[2, -1, 0, 9], [1, 7, 10 ** 9, -3]], dtype=torch.int32)
    p, q = Pair(4, 2, 16, 64, 16, INT8), Pair(4, 2, 16, 64, 16, INT8)
    k, v = randn(2, 2, 80, 64, seed=1, dtype=BF16), randn(2, 2, 80, 64, seed=2, dtype=BF16)
    p.write(k, v, table, ints(5, 0))
    wide = torch.zeros(2, 80, 2, 72, dtype=BF16).transpose(1, 2)
    wide[..., 8:] = k
    q.write(wide[..., 8:], v.transpose(1, 2).contiguous().transpose(1, 2), table, ints(5, 0))
    assert torch.equal(p.cache.k, q.cache.k) and torch.equal(p.cache.v_scale, q.cache.v_scale)
    out, _ = p.cache.read(table.cuda(), ints(0, 0).cuda(), None, 100, BF16, check=True)
    for b in range(2):
        want, there = seq_ref.cache_values(p.host[0], p.host[2], table, b, 100)
        if b == 0:
            there[:5] = True  # written as zero codes of a new cache
        assert not out[b].cpu()[:, ~there].any()
        assert ((out[b].double().cpu() - want).abs() <= want.abs() * 2.0 ** -7).all()
    far = ints(2 ** 31 - 1, 2 ** 31 - 100)
    p.write(k[:, :, :3], v[:, :, :3], table, far)
    p.cache.read(table.cuda(), far.cuda(), None, 3, BF16, check=True)


def filled(batch, lens, kv_heads, page, d, block, fmt, seed=0):
    per = -(-max(max(lens), 1) // page)
    table, pages = tables(batch, per, seed=seed)
    p = Pair(pages, kv_heads, page, d, block, fmt)
    n = max(max(lens), 1)
    p.write(randn(batch, kv_heads, n, d, seed=seed + 1, dtype=BF16), randn(batch, kv_heads, n, d, seed=seed + 2, dtype=BF16),
            table, ints(*[0] * batch), ints(*lens))
    return p, table


def attend_and_check(p, table, lens, q, window, sinks, scale=0.0, **kw):
    o, lse = p.cache.attention(q.cuda(), table.cuda(), ints(*lens).cuda(), window, sinks, scale, check=True, **kw)
    for b, n in enumerate(lens):
        n = min(max(n, 0), table.shape[1] * p.host[0].shape[2])
        k, there = seq_ref.cache_values(p.host[0], p.host[2], table, b, n)
        v, _ = seq_ref.cache_values(p.host[1], p.host[3], table, b, n)
        mask = seq_ref.mask_of(q.shape[2], n, window, sinks) & there
        # P is rounded to a 16-bit type of at least bf16's precision, whatever q's; in fp16 times at least 2^7 for a
        # row's largest, so half a step of its smallest numbers, 2^-25, stands for at most 2^-32
        want = seq_ref.attention(q[b], k, v, mask, scale or q.shape[3] ** -0.5, p_floor=2.0 ** -32)
        o_bound = want["o"][1] - seq_ref.unit(BF16) * want["o"][0].abs() + seq_ref.unit(q.dtype) * want["o"][0].abs()
        seq_ref.check(o[b], (want["o"][0], o_bound), f"o of sequence {b}")
        seq_ref.check(lse[b], want["lse"], f"lse of sequence {b}")
    return o, lse


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", [E4M3, INT8], ids=["e4m3", "int8"])
@pytest.mark.parametrize("heads,kv_heads,q_len,d,block,page,window,sinks,lens,dtype", [
    (1, 1, 1, 64, 16, 16, 0, 0, [1, 2, 0], BF16),
    (8, 2, 1, 128, 16, 64, 0, 0, [300, 17, 1000], BF16),
    (6, 2, 3, 64, 32, 96, 0, 0, [40, 2, 777], FP16),           # fewer tokens than queries: rows that see nothing
    (12, 2, 4, 128, 64, 64, 50, 3, [500, 48, 1], FP16),        # 24 rows of a key head
    (16, 1, 5, 64, 128, 256, 200, 130, [3000, 260, 129], BF16),  # 80 rows of a key head
    (3, 3, 1, 128, 16, 48, 1, 0, [100, 33, 16], BF16),         # a window of one
    (4, 4, 130, 64, 32, 32, 70, 9, [400, 130, 100], BF16),     # more rows than a tile
    (4, 1, 1, 128, 64, 128, 0, 0, [20000, 64, 8191], BF16),    # long: split over the GPU
], ids=str)
def test_attention_over_the_cache(fmt, heads, kv_heads, q_len, d, block, page, window, sinks, lens, dtype):
    p, table = filled(3, lens, kv_heads, page, d, block, fmt, seed=sum(lens))
    attend_and_check(p, table, lens, randn(3, heads, q_len, d, seed=7, dtype=dtype), window, sinks)


@pytest.mark.gpu
def test_attention_where_pages_are_absent_or_shared():
    """Evicted pages behind the window are not missed, absent ones inside it
    are not seen, sequences may share pages, lengths are cut to the table, and
    what lies in a page behind a sequence's end reaches nothing."""
    lens = [400, 390]
    p, table = filled(2, lens, 2, 32, 64, 16, E4M3, seed=3)
    q = randn(2, 4, 2, 64, seed=8, dtype=BF16)
    full, _ = attend_and_check(p, table, lens, q, 100, 4)
    gone = table.clone()
    gone[:, 1:9] = -1
    o, _ = attend_and_check(p, gone, lens, q, 100, 4)
    assert torch.equal(o, full)
    gone[:, 10] = 10 ** 6
    attend_and_check(p, gone, lens, q, 100, 4)
    shared = table.clone()
    shared[1, :6] = shared[0, :6]
    attend_and_check(p, shared, lens, q, 0, 0)
    attend_and_check(p, table, [10 ** 6, -3], q, 0, 0)
    attend_and_check(p, torch.full_like(table, -1), lens, q, 0, 0)
    # NaN codes and scales behind the end
    for t in (p.cache.k, p.cache.v):
        t.view(torch.uint8)[int(table[0, 12]), :, 16:] = 0x7F
    for t in (p.cache.k_scale, p.cache.v_scale):
        t[int(table[0, 12]), :, 1] = float("nan")
    o, lse = p.cache.attention(q.cuda(), table.cuda(), ints(*lens).cuda(), 100, 4)
    assert torch.equal(o, full)


@pytest.mark.gpu
def test_attention_large_scores_layouts_and_lse():
    """Peaked scores, queries far above 1 (bf16) and rows outside heads; lse may be left out."""
    p, table = filled(2, [513, 700], 2, 64, 128, 64, INT8, seed=11)
    q = randn(2, 6, 2, 128, seed=12, dtype=BF16)
    attend_and_check(p, table, [513, 700], (q.float() * 30).to(BF16), 0, 0)
    attend_and_check(p, table, [513, 700], (q.float() * 3e4).to(BF16), 0, 0, scale=1e-5)
    o, _ = attend_and_check(p, table, [513, 700], q, 100, 2, scale=0.5)
    last = q.cuda().transpose(1, 2).contiguous().transpose(1, 2)
    out = torch.zeros_like(last)
    o2, none = p.cache.attention(last, table.cuda(), ints(513, 700).cuda(), 100, 2, 0.5, o=out, want_lse=False)
    assert none is None and o2 is out and torch.equal(out, o)


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", [E4M3, INT8], ids=["e4m3", "int8"])
def test_serving_run(fmt):
    """A prompt's attention, its keys into the cache, then token after token:
    write, attend.  Each token's output is that of 16-bit attention over the
    values read back, captured and replayed as one graph step too."""
    heads, kv_heads, d, window, sinks, prompt, steps = 8, 2, 128, 150, 4, 333, 20
    table, pages = tables(2, 6, seed=1)
    p = Pair(pages, kv_heads, 64, d, 16, fmt)
    k, v = (randn(2, kv_heads, prompt + steps, d, seed=i, dtype=BF16) for i in (1, 2))
    q = randn(2, heads, prompt + steps, d, seed=3, dtype=BF16)
    start = ints(0, 0)
    p.write(k[:, :, :prompt], v[:, :, :prompt], table, start)
    td = table.cuda()
    lens, one_q, one_k, one_v = ints(prompt, prompt).cuda(), *(torch.zeros(2, h, 1, d, dtype=BF16, device="cuda") for h in (heads, kv_heads, kv_heads))
    o = torch.zeros(2, heads, 1, d, dtype=BF16, device="cuda")
    saved = [t.clone() for t in (p.cache.k, p.cache.v, p.cache.k_scale, p.cache.v_scale)]

    def step():
        p.cache.write(one_k, one_v, td, lens)
        lens.add_(1)
        p.cache.attention(one_q, td, lens, window, sinks, o=o, want_lse=False)

    eager = []
    for t in range(prompt, prompt + steps):
        for dst, src in ((one_q, q), (one_k, k), (one_v, v)):
            dst.copy_(src[:, :, t:t + 1])
        step()
        eager.append(o.clone())
        kr, vr = p.cache.read(td, torch.zeros_like(lens), lens, t + 1, BF16, check=True)
        want, _ = window_forward(one_q, kr, vr, window, sinks)
        # both round P (2^-9 each on average, 2^-8 at most), the values read back (2^-8) and O
        assert (o.double() - want.double()).abs().max() <= 5 * 2.0 ** -8 * vr.double().abs().max()
    for t, s in zip((p.cache.k, p.cache.v, p.cache.k_scale, p.cache.v_scale), saved):
        t.copy_(s)
    lens.fill_(prompt)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i, t in enumerate(range(prompt, prompt + steps)):
        for dst, src in ((one_q, q), (one_k, k), (one_v, v)):
            dst.copy_(src[:, :, t:t + 1])
        graph.replay()
        assert torch.equal(o, eager[i])


@pytest.mark.gpu
def test_two_graphs_and_streams_at_once():
    p, table = filled(2, [5000, 4000], 2, 64, 128, 64, E4M3, seed=5)
    td, lens = table.cuda(), ints(5000, 4000).cuda()
    qs = [randn(2, 8, 1, 128, seed=20 + i, dtype=BF16).cuda() for i in range(2)]
    want = [p.cache.attention(x, td, lens)[0] for x in qs]
    pool = torch.cuda.graph_pool_handle()
    graphs, outs = [], []
    for x in qs:
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, pool=pool):
            outs.append(p.cache.attention(x, td, lens)[0])
        graphs.append(g)
    for i in (0, 1, 1, 0):
        graphs[i].replay()
        torch.cuda.synchronize()
        assert torch.equal(outs[i], want[i])
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[p.cache.attention(qs[i], td, lens, stream=streams[i])[0] for _ in range(8)] for i in range(2)]
    torch.cuda.synchronize()
    assert all(torch.equal(x, want[i]) for i in range(2) for x in got[i])


# ------------------------------------------------------------------ refusals (no GPU)
def cache(**kw):
    base = dict(pages=4, kv_heads=2, page_size=64, block=32, head_dim=64, type=2, k=4096, v=4096, k_scale=4096, v_scale=4096)
    base.update(kw)
    return _Cache(*[base[n] for n, _ in _Cache._fields_])


@pytest.mark.parametrize("kw,status", [
    (dict(pages=0), 2), (dict(page_size=40), 2), (dict(kv_heads=0), 2), (dict(head_dim=80), 3), (dict(type=0), 3),
    (dict(block=8), 3), (dict(block=256, page_size=256), 3), (dict(pages=1 << 20, page_size=1 << 12), 2),
])
def test_bad_caches_are_refused(kw, status):
    L, c = sta.lib(), cache(**kw)
    row = sta._Rows(4096, 1024, 512, 64)
    assert L.sta_cache_attention(ctypes.byref(c), 1, 4, 1, 0, 0, 0.0, 0, row, row, None, 4096, 3, 4096, None, 0) == status
    assert L.sta_cache_write(ctypes.byref(c), 1, 1, row, row, 0, 4096, 3, 4096, None, None, 0) == status
    assert L.sta_cache_read(ctypes.byref(c), 1, 1, row, row, 0, 4096, 3, 4096, None, None, 0) == status


def test_bad_cache_calls_are_refused_before_anything_is_enqueued():
    L, c = sta.lib(), cache()
    row = lambda ptr=4096, r=64: sta._Rows(ptr, 1024, 512, r)  # noqa: E731
    for call in (L.sta_cache_write, L.sta_cache_read):
        move = lambda k=row(), rows=2, typ=0, table=4096, start=4096, flags=0: call(  # noqa: E731
            ctypes.byref(c), 1, rows, k, row(), typ, table, 3, start, None, None, flags)
        assert move(k=None) == 1 and move(table=None) == 1 and move(start=None) == 1 and move(flags=4) == 1
        assert move(rows=-1) == 2 and move(typ=2) == 3 and move(k=row(ptr=4100)) == 4 and move(k=row(r=68)) == 4
    att = lambda q=row(), scale=0.0, typ=0, lengths=4096, flags=0, batch=1, heads=4, n=1, w=0, sinks=0, pages=3, c=c: (  # noqa: E731
        L.sta_cache_attention(ctypes.byref(c), batch, heads, n, w, sinks, scale, typ, q, row(), None, 4096, pages, lengths,
                              None, flags))
    assert att(q=None) == 1 and att(lengths=None) == 1 and att(scale=float("nan")) == 1 and att(flags=2) == 1
    assert att(w=-1) == 1 and att(sinks=-1) == 1
    assert att(batch=0) == 2 and att(heads=3) == 2 and att(n=-1) == 2 and att(pages=0) == 2 and att(pages=1 << 26) == 2
    assert att(typ=3) == 3 and att(q=row(ptr=8)) == 4 and att(c=cache(k_scale=4)) == 4


def test_binding_refusals():
    z = torch.zeros(2, 2, 32, 64, dtype=INT8)
    s = torch.zeros(2, 2, 2)
    with pytest.raises(ValueError):
        KVCache.from_tensors(z, z, s, s)  # host tensors
    with pytest.raises(ValueError):
        KVCache(2, 2, 30, 64, block=16, device="cpu")
    with pytest.raises(ValueError):
        KVCache(2, 2, 32, 64, block=16, dtype=BF16, device="cpu")


@pytest.mark.parametrize("kw", [dict(block=8), dict(block=48, page_size=96), dict(block=256, page_size=256), dict(head_dim=96),
                                dict(head_dim=0), dict(pages=0), dict(kv_heads=0), dict(page_size=0),
                                dict(pages=2 ** 20, page_size=2 ** 12)], ids=str)
def test_caches_that_no_call_takes_are_refused(kw):
    """Before anything is allocated."""
    with pytest.raises(ValueError) as e:
        KVCache(**{**dict(pages=2, kv_heads=2, page_size=32, head_dim=64, block=16, device="meta"), **kw})
    assert "on meta" not in str(e.value)  # the sizes, not the device of tensors that were made


@pytest.mark.gpu
def test_tensors_that_no_call_takes_are_refused():
    make = lambda *shape: torch.zeros(shape, dtype=INT8, device="cuda")  # noqa: E731
    scales = lambda *shape: torch.zeros(shape, device="cuda")  # noqa: E731
    for codes, blocks in (((2, 2, 32, 96), 2), ((2, 2, 32, 64), 4), ((0, 2, 32, 64), 2), ((2, 2, 48, 64), 1)):
        k, s = make(*codes), scales(*codes[:2], blocks)
        with pytest.raises(ValueError):
            KVCache.from_tensors(k, k.clone(), s, s.clone())
    k, s = make(2, 2, 32, 64), scales(2, 2, 2)
    for args in ((k, None, s, s), (k, k, None, s), (k, k, s, None), (None, k, s, s)):
        with pytest.raises((TypeError, ValueError)):
            KVCache.from_tensors(*args)
    odd = torch.zeros(2 * 2 * 32 * 64 + 1, dtype=INT8, device="cuda")[1:].view(2, 2, 32, 64)
    with pytest.raises(ValueError):
        KVCache.from_tensors(odd, k, s, s)


@pytest.mark.gpu
def test_binding_refusals_on_device():
    c = KVCache(4, 2, 32, 64, block=16)
    x = torch.zeros(1, 2, 3, 64, dtype=BF16, device="cuda")
    q = torch.zeros(1, 4, 1, 64, dtype=BF16, device="cuda")
    t, n = torch.zeros(1, 2, dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    for args in ((x, x.half(), t, n), (x[:, :1], x[:, :1], t, n), (x.float(), x.float(), t, n), (x, x, t.long(), n),
                 (x, x, t, n.cpu()), (x, x, t[0], n), (x, x, t, None), (x, x, t, n, n.long()), (x.cpu(), x, t, n)):
        with pytest.raises(ValueError):
            c.write(*args)
    for args in ((t, n, None, 3, torch.float32), (t, n, None, 3, BF16, x.half()), (t.cpu(), n, None, 3), (t, None, None, 3)):
        with pytest.raises(ValueError):
            c.read(*args)
    for args in ((q.float(), t, n), (q[..., :32], t, n), (q, t.long(), n), (q, t, n.long()), (q, t, None), (q[0], t, n)):
        with pytest.raises(ValueError):
            c.attention(*args)
    for args, status in (((q[:, :3], t, n), 2), ((q, t, n, -1), 1), ((q, t, n, 4, -1), 1), ((q, t, n, 0, 0, float("inf")), 1)):
        with pytest.raises(sta.StaError) as e:
            c.attention(*args)
        assert e.value.status == status
    o, lse = c.attention(q[:, :, :0], t, n)
    assert o.shape == (1, 4, 0, 64) and lse.shape == (1, 4, 0)
    c.write(x[:, :, :0], x[:, :, :0], t, n)
    k = torch.zeros(2, 2, 32, 64, dtype=INT8, device="cuda")
    s = torch.zeros(2, 2, 2, device="cuda")
    for args in ((k, k.view(E4M3), s, s), (k, k, s[..., :1], s), (k, k, s.half(), s), (k[0], k[0], s, s), (k, k, s[:1], s[:1])):
        with pytest.raises(ValueError):
            KVCache.from_tensors(*args)


@pytest.mark.gpu
def test_a_cache_keeps_its_tensors():
    """The calls use the tensors' addresses, so that no other tensor can take their place."""
    c = KVCache(2, 1, 16, 64, block=16)
    for name in ("k", "v", "k_scale", "v_scale"):
        with pytest.raises(AttributeError):
            setattr(c, name, torch.zeros_like(getattr(c, name)))


@pytest.mark.gpu
@pytest.mark.parametrize("kw", [dict(window=2 ** 32 + 3), dict(sinks=2 ** 32)])
def test_numbers_past_32_bits_are_refused(kw):
    c = KVCache(2, 1, 16, 64, block=16)
    with pytest.raises(ValueError, match="32-bit"):
        c.attention(torch.zeros(1, 2, 1, 64, dtype=BF16, device="cuda"), ints(0).view(1, 1).cuda(), ints(3).cuda(), **kw)


@pytest.mark.gpu
@pytest.mark.parametrize("batch", [80, 256, 300])
def test_many_sequences_of_uneven_lengths(batch):
    """More sequences than the GPU holds at once, of lengths from none to all of
    the table, equal ones among them: each as if alone."""
    g = torch.Generator().manual_seed(batch)
    lens = torch.randint(0, 641, (batch,), generator=g)
    lens[1::3], lens[7] = 500, 640
    p, table = filled(batch, lens.tolist(), 4, 64, 64, 64, INT8, seed=batch)
    attend_and_check(p, table, lens.tolist(), randn(batch, 8, 1, 64, seed=1, dtype=FP16), 0, 0)


@pytest.mark.gpu
def test_many_long_sequences_over_shared_pages():
    """Long sequences of uneven lengths, each split over two blocks, that share their pages."""
    p, one = filled(1, [4224], 2, 64, 64, 64, E4M3, seed=21)
    lens = torch.randint(0, 4225, (80,), generator=torch.Generator().manual_seed(22))
    lens[5], lens[6] = 4224, 0
    attend_and_check(p, one.expand(80, -1).contiguous(), lens.tolist(), randn(80, 4, 1, 64, seed=23, dtype=BF16), 0, 3)


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", [E4M3, INT8], ids=["e4m3", "int8"])
def test_rows_behind_the_count_are_zeros_whatever_the_page_holds(fmt):
    p, table = filled(2, [40, 64], 2, 64, 64, 16, fmt, seed=31)
    want = p.cache.read(table.cuda(), ints(0, 3).cuda(), ints(33, 20).cuda(), 60)
    for t in (p.cache.k, p.cache.v):
        t.view(torch.uint8)[int(table[0, 0]), :, 33:] = 0x7F
        t.view(torch.uint8)[int(table[1, 0]), :, 23:] = 0x7F
    for t in (p.cache.k_scale, p.cache.v_scale):
        t[int(table[0, 0]), :, 3] = float("nan")
        t[int(table[1, 0]), :, 2:] = float("inf")
    got = p.cache.read(table.cuda(), ints(0, 3).cuda(), ints(33, 20).cuda(), 60, check=True)
    for a, b in zip(want, got):
        assert torch.equal(a, b) and not b[0, :, 33:].any() and not b[1, :, 20:].any() and b[0, :, :33].any()


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", [E4M3, INT8], ids=["e4m3", "int8"])
def test_offsets_past_32_bits(fmt):
    """The last pages of a cache of more than 4 GB hold and give what those of a small one do."""
    pages, kv_heads, page, d = 33000, 8, 128, 128
    codes = torch.empty(pages, kv_heads, page, d, dtype=torch.uint8, device="cuda").view(fmt)
    scales = [torch.zeros(pages, kv_heads, page // 16, device="cuda") for _ in range(2)]
    assert codes.numel() > 2 ** 32
    large = KVCache.from_tensors(codes, torch.empty_like(codes), *scales)
    small = KVCache(3, kv_heads, page, d, block=16, dtype=fmt)
    k, v, q = (randn(1, h, n, d, seed=41 + i, dtype=BF16).cuda() for i, (h, n) in enumerate(((8, 300), (8, 300), (16, 2))))
    results = []
    for cache, first in ((small, 0), (large, pages - 3)):
        table = (torch.arange(3, dtype=torch.int32)[None] + first).cuda()
        cache.write(k, v, table, ints(0).cuda(), check=True)
        cache.write(k[:, :, :1] * 3, v[:, :, :1] * 3, table, ints(300).cuda(), check=True)
        results.append([*cache.read(table, ints(0).cuda(), None, 301, BF16, check=True),
                        *cache.attention(q, table, ints(301).cuda(), 200, 4, check=True),
                        cache.k[first:first + 3].view(torch.uint8), cache.k_scale[first:first + 3]])
    (*same, small_k, _), (*other, large_k, _) = results
    for a, b in zip(same, other):
        assert torch.equal(a, b)
    assert torch.equal(small_k[:2], large_k[:2]) and torch.equal(results[0][-1], results[1][-1])


def attend_unequal(p, table, lens, q, window, sinks, **kw):
    """attend_and_check for values of any scales: a row's P times its block's scale
    of values is rounded to fp16 at 2^7 or more for the largest such product, so
    half a step of the smallest numbers, 2^-25, stands for 2^-32 of it, times the
    code.  O is rounded to q's type: at least half a step of its smallest numbers."""
    o, lse = p.cache.attention(q.cuda(), table.cuda(), ints(*lens).cuda(), window, sinks, check=True, **kw)
    c, g = p.cache, q.shape[1] // p.cache.kv_heads
    for b, n in enumerate(lens):
        k, there = seq_ref.cache_values(p.host[0], p.host[2], table, b, n)
        v, _ = seq_ref.cache_values(p.host[1], p.host[3], table, b, n)
        scale = p.host[3][table[b].long()].transpose(0, 1).flatten(1).double().repeat_interleave(c.block, 1)[:, :n]
        mask = seq_ref.mask_of(q.shape[2], n, window, sinks) & there
        want = seq_ref.attention(q[b], k, v, mask, q.shape[3] ** -0.5)
        kd, vd, sd = (t.repeat_interleave(g, 0) for t in (k, v, scale))
        x = (q[b].double() @ kd.mT * q.shape[3] ** -0.5).masked_fill(~mask, float("-inf"))
        w = torch.softmax(x, -1).nan_to_num(0.0) * sd.abs()[:, None]
        floor = 2.0 ** -32 * w.amax(-1, keepdim=True) * ((mask / sd.abs()[:, None].clamp_min(2.0 ** -100)) @ vd.abs())
        o_want, o_bound = want["o"]
        tiny = torch.finfo(q.dtype).smallest_normal * seq_ref.unit(q.dtype)
        o_bound = o_bound + (seq_ref.unit(q.dtype) - seq_ref.unit(BF16)) * o_want.abs() + floor + tiny
        seq_ref.check(o[b], (o_want, o_bound), f"o of sequence {b}")
        seq_ref.check(lse[b], want["lse"], f"lse of sequence {b}")
    return o, lse


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", [E4M3, INT8], ids=["e4m3", "int8"])
@pytest.mark.parametrize("heads,q_len,d", [(2, 1, 128), (8, 4, 64), (4, 1, 64)])
@pytest.mark.parametrize("up,block_at", [(12, 3), (24, 0), (24, 9), (34, 3), (60, 5)])
def test_values_beside_a_block_of_a_much_larger_scale(fmt, heads, q_len, d, up, block_at):
    """One block's values are 2^up times the others', and its keys get next to no
    weight (or its tokens are not seen): the others' contribution stays."""
    lens = [400]
    table, pages = tables(1, 13, seed=4)
    p = Pair(pages, 2, 32, d, 16, fmt)
    k, v = (randn(1, 2, 400, d, seed=60 + i, dtype=BF16) for i in (0, 1))
    q = randn(1, heads, q_len, d, seed=62, dtype=BF16)
    q[..., 0], k[..., 0] = 16.0, 0.0
    rows = slice(16 * block_at, 16 * block_at + 16)
    v[:, :, rows] *= 2.0 ** up
    k[:, :, rows, 0] = -min(up + 8, 60) * 0.6931 * d ** 0.5 / 16  # weight 2^-(up + 8), up to 2^-60
    p.write(k, v, table, ints(0), ints(400))
    attend_unequal(p, table, lens, q, 0, 0)
    attend_unequal(p, table, lens, q, 90, 16 * block_at + 3)  # some of the block's tokens are seen, or none


@pytest.mark.gpu
def test_an_outlier_reaches_only_rows_that_see_its_block():
    """Rows that do not see any token of an outlier's block (behind their
    positions, or before their window) keep their precision beside rows that do."""
    table, pages = tables(1, 4, seed=5)
    k, v = (randn(1, 1, 64, 64, seed=70 + i, dtype=BF16) for i in (0, 1))
    q = randn(1, 2, 20, 64, seed=72, dtype=BF16)  # positions 44 .. 63
    for token, window in ((50, 40), (17, 20)):
        p = Pair(pages, 1, 16, 64, 16, E4M3)
        vb = v.clone()
        vb[:, :, token] = 2.0 ** 60
        p.write(k, vb, table, ints(0))
        attend_unequal(p, table, [64], q, window, 0)


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", [E4M3, INT8], ids=["e4m3", "int8"])
def test_scores_far_below_zero(fmt):
    """Equal scores below -2^116 for all keys: O is the mean of the values."""
    table, pages = tables(1, 2, seed=6)
    p = Pair(pages, 1, 16, 64, 16, fmt)
    k, v = torch.zeros(1, 1, 20, 64, dtype=BF16), randn(1, 1, 20, 64, seed=81, dtype=BF16)
    q = torch.zeros(1, 2, 1, 64, dtype=BF16)
    q[..., 3], k[..., 3] = 2.0 ** 60, -2.0 ** 60
    p.write(k, v, table, ints(0))
    o, lse = p.cache.attention(q.cuda(), table.cuda(), ints(20).cuda(), check=True)
    values, _ = seq_ref.cache_values(p.host[1], p.host[3], table, 0, 20)
    want, mag = values.mean(1), values.abs().mean(1)
    for h in range(2):
        seq_ref.check(o[0, h], (want, mag * (2.0 ** -11 + 2.0 ** -20) + want.abs() * 2.0 ** -8), "o")
    assert ((lse.double().cpu() + 2.0 ** 117).abs() <= 2.0 ** (117 - 7)).all()  # k is rounded in the cache


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", [E4M3, INT8], ids=["e4m3", "int8"])
@pytest.mark.parametrize("q_len,d,lens", [(1, 128, [300]), (6, 64, [300]), (1, 64, [3000])])
def test_scales_of_zero_of_either_sign_and_far_apart(fmt, q_len, d, lens):
    """Pages never written (scale 0), blocks of zeros (2^-100), scales below zero
    and of 2^30 beside one another, in any order."""
    per = -(-lens[0] // 32)
    table, pages = tables(1, per, seed=9)
    p = Pair(pages, 2, 32, d, 16, fmt)
    q = randn(1, 4, q_len, d, seed=90, dtype=BF16)
    o, lse = attend_unequal(p, table, lens, q, 0, 0)  # a new cache: zeros with equal weights
    assert not o.any()
    k, v = (randn(1, 2, lens[0], d, seed=91 + i, dtype=BF16) for i in (0, 1))
    v[:, :, 16:48], v[:, :, 96:112] = 0.0, 2.0 ** 30
    p.write(k, v, table, ints(0))
    for scales in (p.host[3], p.cache.v_scale):
        scales[int(table[0, 5])], scales[int(table[0, 2]), :, 1] = 0.0, 0.0
        scales[int(table[0, 1])] *= -1
    p.cache.k_scale[int(table[0, 4])] *= -1
    p.host[2][int(table[0, 4])] *= -1
    for window in (0, 90):
        attend_unequal(p, table, lens, q, window, 40)

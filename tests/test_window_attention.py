"""Sliding-window attention with sinks: forward and backward against the fp64
definition, over types, head layouts, lengths, strides and masks; packed
sequences; graphs, streams and refusals."""
import ctypes

import pytest
import torch

import seq_ref
from sparse_local_attention_b200 import sliding_window_attention, sta, window, window_backward, window_forward
from sparse_local_attention_b200.window import _WindowProblem

BF16, FP16 = torch.bfloat16, torch.float16


def randn(*shape, seed, dtype, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale).to(dtype)


def make(heads, kv_heads, nq, nk, d, dtype, batch=1, seed=0, do_scale=1.0):
    return (randn(batch, heads, nq, d, seed=seed, dtype=dtype), randn(batch, kv_heads, nk, d, seed=seed + 1, dtype=dtype),
            randn(batch, kv_heads, nk, d, seed=seed + 2, dtype=dtype),
            randn(batch, heads, nq, d, seed=seed + 3, dtype=dtype, scale=do_scale))


def compare(q, k, v, do, window, sinks, scale=0.0, backward=True):
    """Device results of a dense batch against the definition, sequence by sequence."""
    qd, kd, vd, dod = (t.cuda() for t in (q, k, v, do))
    o, lse = window_forward(qd, kd, vd, window, sinks, scale, check=True)
    grads = window_backward(qd, kd, vd, o, lse, dod, window, sinks, scale, check=True) if backward else ()
    mask = seq_ref.mask_of(q.shape[2], k.shape[2], window, sinks)
    for b in range(q.shape[0]):
        want = seq_ref.attention(q[b], k[b], v[b], mask, scale or q.shape[3] ** -0.5, do[b] if backward else None, q.dtype,
                                 float(do.double().norm(dim=-1).max()) if do.numel() else 0.0)
        for name, got in zip(("o", "lse", "dq", "dk", "dv"), (o, lse, *grads)):
            seq_ref.check(got[b], want[name], f"{name} of sequence {b}")
    return (o, lse, *grads)


CASES = [
    # heads, kv_heads, nq, nk, d, window, sinks
    (1, 1, 1, 1, 64, 1, 0),
    (4, 2, 1, 300, 128, 100, 4),       # one token
    (6, 2, 3, 1000, 64, 0, 0),         # a few tokens, no window
    (2, 2, 128, 128, 64, 0, 0),        # one whole tile
    (3, 1, 127, 127, 128, 50, 3),      # one row short of a tile, an odd group
    (2, 1, 129, 129, 64, 128, 1),      # one row past a tile
    (4, 4, 260, 260, 128, 1, 0),       # every row sees itself alone
    (2, 2, 300, 700, 64, 77, 130),     # sinks past one tile, keys before the queries
    (5, 5, 513, 513, 128, 256, 200),   # sinks that meet the window
    (2, 1, 200, 64, 64, 30, 4),        # more queries than keys: rows that see nothing
    (8, 1, 333, 901, 128, 300, 16),    # one key head for all
    (2, 2, 640, 640, 64, 10000, 5),    # a window longer than the sequence
    (2, 2, 70, 0, 64, 10, 2),          # no keys
    (4, 4, 1500, 1500, 64, 96, 700),   # sinks over many tiles
    # more blocks than SMs: two blocks of a key head share their keys
    (48, 16, 200, 333, 64, 77, 5),
    (40, 8, 260, 260, 128, 1000, 0),
    (32, 32, 300, 300, 128, 100, 130),
]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF16, FP16], ids=["bf16", "fp16"])
@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c)))
def test_against_the_definition(case, dtype):
    heads, kv_heads, nq, nk, d, window, sinks = case
    compare(*make(heads, kv_heads, nq, nk, d, dtype, batch=2, seed=nq + nk), window, sinks)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,do_scale,q_scale", [(FP16, 1e-3, 1.0), (BF16, 1e-6, 1.0), (FP16, 30.0, 4.0), (BF16, 1e4, 6.0)])
def test_small_and_large_values(dtype, do_scale, q_scale):
    """Gradients far below 1 keep their relative precision; peaked and large scores do not overflow."""
    q, k, v, do = make(4, 2, 600, 600, 128, dtype, seed=5, do_scale=do_scale)
    compare((q.float() * q_scale).to(dtype), k, v, do, 500, 4)


@pytest.mark.gpu
def test_scale_and_equal_scores():
    q, k, v, do = make(2, 2, 400, 400, 64, BF16, seed=9)
    compare(q, k, v, do, 90, 7, scale=0.37)
    # equal scores: O is the mean of the visible values, the sum of P is exact
    o, lse, *_ = compare(torch.zeros_like(q), k, v, do, 90, 7)
    n = seq_ref.mask_of(400, 400, 90, 7).sum(-1).double()
    assert (lse[0, 0].double().cpu() - n.log()).abs().max() < 1e-5


@pytest.mark.gpu
def test_gradients_against_differences():
    """dq, dk, dv along random directions against central differences of the fp64 definition."""
    q, k, v, do = make(4, 2, 150, 150, 64, FP16, seed=21)
    mask, scale = seq_ref.mask_of(150, 150, 40, 6), 64 ** -0.5
    _, _, dq, dk, dv = compare(q, k, v, do, 40, 6)

    def loss(q, k, v):
        return (seq_ref.attention(q[0], k[0], v[0], mask, scale)["o"][0] * do[0].double()).sum()

    for i, (x, g) in enumerate(((q, dq), (k, dk), (v, dv))):
        r = torch.randn(x.shape, generator=torch.Generator().manual_seed(i), dtype=torch.float64)
        args = [t.double() for t in (q, k, v)]
        h = 1e-5
        up, down = list(args), list(args)
        up[i], down[i] = args[i] + h * r, args[i] - h * r
        want = (loss(*up) - loss(*down)) / (2 * h)
        g64 = g.double().cpu()
        # each element within a few roundings of fp16 (2^-11): the sum within their root mean square
        assert abs((g64 * r).sum() - want) <= 8 * 2.0 ** -11 * (g64 * r).norm() + 1e-6, i


def packed(lens_q, lens_k, heads, kv_heads, d, dtype, tail=37, seed=0):
    tot_q, tot_k = sum(lens_q) + tail, sum(lens_k) + tail
    q, k, v, do = (t for t in (randn(1, heads, tot_q, d, seed=seed, dtype=dtype), randn(1, kv_heads, tot_k, d, seed=seed + 1, dtype=dtype),
                               randn(1, kv_heads, tot_k, d, seed=seed + 2, dtype=dtype), randn(1, heads, tot_q, d, seed=seed + 3, dtype=dtype)))
    cu = [torch.tensor([0] + list(x), dtype=torch.int32).cumsum(0).to(torch.int32) for x in (lens_q, lens_k)]
    return q, k, v, do, *cu


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,d", [(BF16, 128), (FP16, 64)])
@pytest.mark.parametrize("lens_q,lens_k,window,sinks", [
    ([5, 128, 1, 0, 300, 129], None, 64, 4),
    ([1, 1, 1], [200, 0, 513], 100, 2),       # single tokens
    ([130, 2, 257], [130, 700, 300], 0, 0),   # chunks with earlier keys
    ([20, 200], [7, 40], 1000, 3),            # more queries than keys
], ids=["mixed", "tokens", "chunks", "empty rows"])
@pytest.mark.parametrize("bounds", [True, False], ids=["bounds", "no bounds"])
def test_packed_sequences(dtype, d, lens_q, lens_k, window, sinks, bounds):
    """Each sequence as if alone.  What lies between and behind sequences
    (NaN here) reaches nothing, and rows behind the last one stay as they were."""
    lens_k = lens_k or lens_q
    q, k, v, do, cu_q, cu_k = packed(lens_q, lens_k, 6, 2, d, dtype, seed=sum(lens_q))
    for t, n in ((q, sum(lens_q)), (k, sum(lens_k)), (v, sum(lens_k)), (do, sum(lens_q))):
        t[:, :, n:] = float("nan")
    qd, kd, vd, dod, cq, ck = (t.cuda() for t in (q, k, v, do, cu_q, cu_k))
    kw = dict(cu_q=cq, cu_kv=ck, check=True, **(dict(max_q=max(lens_q), max_kv=max(lens_k)) if bounds else {}))
    o, lse = torch.full_like(qd, 7.0), torch.full(q.shape[:3], 7.0).cuda()
    window_forward(qd, kd, vd, window, sinks, o=o, lse=lse, **kw)
    dq, dk, dv = torch.full_like(qd, 7.0), torch.full_like(kd, 7.0), torch.full_like(vd, 7.0)
    window_backward(qd, kd, vd, o, lse, dod, window, sinks, dq=dq, dk=dk, dv=dv, **kw)
    for b in range(len(lens_q)):
        rq, rk = slice(int(cu_q[b]), int(cu_q[b + 1])), slice(int(cu_k[b]), int(cu_k[b + 1]))
        mask = seq_ref.mask_of(lens_q[b], lens_k[b], window, sinks)
        want = seq_ref.attention(q[0, :, rq], k[0, :, rk], v[0, :, rk], mask, d ** -0.5, do[0, :, rq], dtype,
                                 float(do[0, :, :sum(lens_q)].double().norm(dim=-1).max()))
        for name, got, r in (("o", o, rq), ("lse", lse, rq), ("dq", dq, rq), ("dk", dk, rk), ("dv", dv, rk)):
            seq_ref.check(got[0, :, r], want[name], f"{name} of sequence {b}")
    for t, n in ((o, sum(lens_q)), (lse, sum(lens_q)), (dq, sum(lens_q)), (dk, sum(lens_k)), (dv, sum(lens_k))):
        assert bool((t[:, :, n:] == 7.0).all())
    # outputs that the call makes: zero (-inf) there
    o2, lse2 = window_forward(qd, kd, vd, window, sinks, **kw)
    n = sum(lens_q)
    assert torch.equal(o2[:, :, :n], o[:, :, :n]) and torch.equal(lse2[:, :, :n], lse[:, :, :n])
    assert bool((o2[:, :, n:] == 0).all()) and bool((lse2[:, :, n:] == float("-inf")).all())


@pytest.mark.gpu
@pytest.mark.parametrize("d,dtype,n", [(64, FP16, 150), (128, BF16, 100)])
def test_packed_tokens_of_many_uneven_sequences(d, dtype, n):
    """A token each of more sequences than the GPU holds at once, of uneven lengths."""
    g = torch.Generator().manual_seed(n)
    lens_k = torch.randint(0, 600, (n,), generator=g)
    lens_k[3], lens_k[::4] = 600, 333
    q, k, v, _, cu_q, cu_k = packed([1] * n, lens_k.tolist(), 8, 4, d, dtype, seed=n)
    o, lse = window_forward(*(t.cuda() for t in (q, k, v)), 450, 5, cu_q=cu_q.cuda(), cu_kv=cu_k.cuda(), max_q=1, max_kv=600,
                            check=True)
    for b in range(n):
        rk = slice(int(cu_k[b]), int(cu_k[b + 1]))
        want = seq_ref.attention(q[0, :, b:b + 1], k[0, :, rk], v[0, :, rk], seq_ref.mask_of(1, int(lens_k[b]), 450, 5),
                                 d ** -0.5, dtype=dtype)
        seq_ref.check(o[0, :, b:b + 1], want["o"], f"o of sequence {b}")
        seq_ref.check(lse[0, :, b:b + 1], want["lse"], f"lse of sequence {b}")


@pytest.mark.gpu
def test_packed_bounds_cut_and_bad_starts_are_dropped():
    """max_q below a length computes the sequence's first max_q rows against its
    first max_kv keys; starts outside the tensor are cut to it."""
    q, k, v, do, cu, _ = packed([200, 90], [200, 90], 2, 2, 64, BF16, tail=0, seed=3)
    qd, kd, vd = (t.cuda() for t in (q, k, v))
    o = torch.full_like(qd, 7.0)
    window_forward(qd, kd, vd, 50, 4, cu_q=cu.cuda(), cu_kv=cu.cuda(), max_q=100, max_kv=100, o=o, check=True)
    want = seq_ref.attention(q[0, :, :100], k[0, :, :100], v[0, :, :100], seq_ref.mask_of(100, 100, 50, 4), 64 ** -0.5)
    seq_ref.check(o[0, :, :100], want["o"], "o")
    assert bool((o[:, :, 100:200] == 7.0).all())
    wild = torch.tensor([-5, 200, 10 ** 6], dtype=torch.int32).cuda()  # [0, 200) and [200, 290)
    o3, _ = window_forward(qd, kd, vd, 50, 4, cu_q=wild, cu_kv=wild, check=True)
    o4, _ = window_forward(qd, kd, vd, 50, 4, cu_q=cu.cuda(), cu_kv=cu.cuda(), check=True)
    assert torch.equal(o3, o4)


@pytest.mark.gpu
@pytest.mark.parametrize("cu", [[3, 5, 5], [7]], ids=["two", "none"])
def test_packed_sequences_without_keys_leave_the_other_rows(cu):
    """Key tensors without a row, and no sequence at all: rows of sequences are
    empty ones, rows outside stay as they were in tensors that are passed in."""
    q, k, v, do = (t.cuda() for t in make(4, 2, 9, 0, 64, BF16))
    cu_q = torch.tensor(cu, dtype=torch.int32).cuda()
    seqs = dict(cu_q=cu_q, cu_kv=torch.zeros_like(cu_q))
    o, lse, dq = torch.full_like(q, 7.0), torch.full((1, 4, 9), 7.0, device="cuda"), torch.full_like(q, 7.0)
    window_forward(q, k, v, 5, 1, o=o, lse=lse, check=True, **seqs)
    _, dk, dv = window_backward(q, k, v, o, lse, do, 5, 1, dq=dq, check=True, **seqs)
    assert dk.shape == k.shape and dv.shape == v.shape
    inside = torch.zeros(9, dtype=torch.bool)
    inside[cu[0]:cu[-1]] = True
    for t, empty in ((o, 0.0), (lse, float("-inf")), (dq, 0.0)):
        assert (t[:, :, inside] == empty).all() and (t[:, :, ~inside] == 7.0).all()
    q.requires_grad_()
    out = sliding_window_attention(q, k, v, 5, 1, **seqs)
    out.backward(do)
    assert not out.any() and not q.grad.any()


@pytest.mark.gpu
@pytest.mark.parametrize("heads,kv_heads,d,dtype,max_n", [(2, 1, 64, BF16, 0), (6, 3, 128, FP16, 0), (2, 2, 128, BF16, 70)])
@pytest.mark.parametrize("cu", [[40, 41, 41, 300, 433], [0, 16], [470, 500], [9, 9], [-7, 200, 10 ** 6]],
                         ids=["gaps", "tail", "head", "empty", "wild"])
def test_new_packed_outputs_are_empty_outside_the_sequences(monkeypatch, heads, kv_heads, d, dtype, max_n, cu):
    """Rows before, behind and between sequences (cut ones) hold zeros, -inf in lse,
    whatever the memory held; the others are those of outputs that are passed in."""
    n = 500
    q, k, v, do = (t.cuda() for t in make(heads, kv_heads, n, n, d, dtype, seed=n))
    kw = dict(cu_q=torch.tensor(cu, dtype=torch.int32).cuda(), cu_kv=torch.tensor(cu, dtype=torch.int32).cuda(),
              max_q=max_n, max_kv=max_n, check=True)
    o, lse = torch.zeros_like(q), torch.full(q.shape[:3], float("-inf"), device="cuda")
    window_forward(q, k, v, 60, 4, o=o, lse=lse, **kw)
    grads = [torch.zeros_like(t) for t in (q, k, v)]
    window_backward(q, k, v, o, lse, do, 60, 4, dq=grads[0], dk=grads[1], dv=grads[2], **kw)
    monkeypatch.setattr(window, "_new", lambda like: torch.full_like(like, 7.0))
    o2, lse2 = window_forward(q, k, v, 60, 4, **kw)
    new = window_backward(q, k, v, o, lse, do, 60, 4, **kw)
    for a, b in zip((o, lse, *grads), (o2, lse2, *new)):
        assert torch.equal(a, b)


@pytest.mark.gpu
def test_bounds_written_to_before_the_backward_are_noticed():
    q, k, v, do = (t.cuda() for t in make(2, 1, 9, 9, 64, BF16))
    cu = torch.tensor([0, 4, 9], dtype=torch.int32).cuda()
    o = sliding_window_attention(q.requires_grad_(), k, v, 5, cu_q=cu, cu_kv=cu)
    cu[1] = 5
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        o.backward(do)


@pytest.mark.gpu
@pytest.mark.parametrize("kw", [dict(window=2 ** 32 + 3), dict(sinks=2 ** 32), dict(window=-2 ** 31 - 1)])
def test_numbers_past_32_bits_are_refused(kw):
    q, k, v, _ = (t.cuda() for t in make(2, 1, 9, 9, 64, BF16))
    with pytest.raises(ValueError, match="32-bit"):
        window_forward(q, k, v, **kw)


@pytest.mark.gpu
def test_hidden_keys_reach_nothing():
    """Keys that no query of the call sees hold NaN and infinities (and values
    of the type's lowest and highest)."""
    for nq, nk, window, sinks in ((40, 900, 100, 5), (1, 700, 64, 2), (300, 1200, 200, 130)):
        q, k, v, do = make(4, 2, nq, nk, 64, BF16, seed=nq)
        seen = seq_ref.mask_of(nq, nk, window, sinks).any(0)
        clean = seq_ref.attention(q[0], k[0], v[0], seq_ref.mask_of(nq, nk, window, sinks), 0.125, do[0])
        for bad in (float("nan"), float("inf"), float("-inf"), torch.finfo(BF16).min, torch.finfo(BF16).max):
            kb, vb = k.clone(), v.clone()
            kb[:, :, ~seen] = bad
            vb[:, :, ~seen] = bad
            qd, kd, vd, dod = (t.cuda() for t in (q, kb, vb, do))
            o, lse = window_forward(qd, kd, vd, window, sinks, check=True)
            dq, dk, dv = window_backward(qd, kd, vd, o, lse, dod, window, sinks, check=True)
            for name, got in (("o", o), ("lse", lse), ("dq", dq)):
                seq_ref.check(got[0], clean[name], name)
            for name, got in (("dk", dk), ("dv", dv)):
                seq_ref.check(got[0][:, seen], tuple(t[:, seen] for t in clean[name]), name)
                assert bool((got[0][:, ~seen] == 0).all()), name


@pytest.mark.gpu
@pytest.mark.parametrize("nq,nk", [(1, 257), (190, 333)])
def test_strides_orders_and_broadcasts(nq, nk):
    """Rows outside heads, slices of wider tensors, unaligned views and expanded
    inputs give what contiguous copies give."""
    q, k, v, do = (t.cuda() for t in make(4, 4, nq, nk, 64, BF16, batch=2, seed=8))
    args = (100, 3)
    o, lse = window_forward(q, k, v, *args, check=True)
    grads = window_backward(q, k, v, o, lse, do, *args, check=True)

    def last(t):  # [batch, rows, heads, d] behind the same view
        return t.transpose(1, 2).contiguous().transpose(1, 2)

    def wide(t):  # heads inside a fused projection
        w = torch.full((*t.shape[:3], 3 * t.shape[3]), float("nan"), dtype=t.dtype, device="cuda")
        w[..., 64:128] = t
        return w[..., 64:128]

    def odd(t):  # an address and strides off the kernels' alignment
        w = torch.zeros((*t.shape[:3], t.shape[3] + 3), dtype=t.dtype, device="cuda")
        w[..., 1:65] = t
        return w[..., 1:65]

    for f in (last, wide, odd):
        qf, kf, vf, df = f(q), f(k), f(v), f(do)
        of, lf = window_forward(qf, kf, vf, *args, check=True)
        assert torch.equal(of, o) and torch.equal(lf, lse), f.__name__
        gf = window_backward(qf, kf, vf, f(o), lse, df, *args, check=True)
        for name, a, b in zip(("dq", "dk", "dv"), gf, grads):
            assert torch.equal(a, b), (f.__name__, name)
    # outputs of the caller's layout
    of = last(torch.zeros_like(q))
    window_forward(q, k, v, *args, o=of, check=True)
    assert torch.equal(of, o) and of.stride() == last(q).stride()
    # one key head and one batch entry broadcast over the others: gradients sum over the copies
    ke = k[:1, :1].clone().requires_grad_()
    out = sliding_window_attention(q, ke.expand_as(k), ke.expand_as(v), *args)
    (g,) = torch.autograd.grad(out, ke, do)
    kk = ke.detach().expand_as(k).contiguous()
    o2, l2 = window_forward(q, kk, kk, *args)
    _, dk2, dv2 = window_backward(q, kk, kk, o2, l2, do, *args)
    want = (dk2.float().sum((0, 1)) + dv2.float().sum((0, 1)))
    # autograd adds eight copies twice over and k's and v's parts, in bf16
    assert (g[0, 0].float() - want).abs().max() <= 12 * 2.0 ** -8 * (dk2.float().abs().sum((0, 1)) + dv2.float().abs().sum((0, 1))).max()


@pytest.mark.gpu
@pytest.mark.parametrize("nq", [1, 300])
def test_offsets_past_32_bits(nq):
    """Sequences 2^31 elements apart give what contiguous ones give."""
    big = torch.empty(2 ** 31 + 2 ** 22, dtype=BF16, device="cuda")

    def far(t, slot):
        v = big.as_strided(t.shape, (2 ** 31, *t.stride()[1:]), slot * 2 ** 18)
        return v.copy_(t)

    near = [t.cuda() for t in make(4, 2, nq, 300, 64, BF16, batch=2, seed=nq)]
    o, lse = window_forward(*near[:3], 70, 5, check=True)
    grads = window_backward(*near[:3], o, lse, near[3], 70, 5, check=True)
    q, k, v, do = (far(t, i) for i, t in enumerate(near))
    o2 = far(torch.zeros_like(o), 4)
    _, lse2 = window_forward(q, k, v, 70, 5, o=o2, check=True)
    assert torch.equal(o2, o) and torch.equal(lse2, lse)
    dq, dk, dv = (far(torch.zeros_like(t), 5 + i) for i, t in enumerate(grads))
    window_backward(q, k, v, o2, lse2, do, 70, 5, dq=dq, dk=dk, dv=dv, check=True)
    for a, b in zip(grads, (dq, dk, dv)):
        assert torch.equal(a, b)


@pytest.mark.gpu
def test_autograd_matches_the_calls_and_is_deterministic():
    q, k, v, do = (t.cuda() for t in make(6, 2, 500, 500, 128, BF16, batch=2, seed=4))
    o, lse = window_forward(q, k, v, 128, 4)
    want = window_backward(q, k, v, o, lse, do, 128, 4)
    for _ in range(2):
        leaves = [t.clone().requires_grad_() for t in (q, k, v)]
        out = sliding_window_attention(*leaves, 128, 4)
        assert torch.equal(out, o)
        for a, b in zip(torch.autograd.grad(out, leaves, do), want):
            assert torch.equal(a, b)
    with torch.no_grad():
        assert torch.equal(sliding_window_attention(*leaves, 128, 4), o)


@pytest.mark.gpu
def test_graph_streams_and_concurrent_calls():
    """A training step captures into a graph and replays with the same bits on
    new data; calls on two streams at once do not disturb each other; a call
    on a given stream allocates there."""
    sets = [[t.cuda() for t in make(4, 2, 300, 300, 64, FP16, seed=s)] for s in (1, 50)]
    args = (90, 4)
    ref = []
    for q, k, v, do in sets:
        o, lse = window_forward(q, k, v, *args, check=True)
        ref.append((o, lse, *window_backward(q, k, v, o, lse, do, *args, check=True)))
    static = [t.clone() for t in sets[0]]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, lse = window_forward(*static[:3], *args)
        got = (o, lse, *window_backward(*static[:3], o, lse, static[3], *args))
    for s in (1, 0, 1):
        for a, b in zip(static, sets[s]):
            a.copy_(b)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, ref[s]):
            assert torch.equal(a, b)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    outs = [[], []]
    for _ in range(10):
        for i, st in enumerate(streams):
            q, k, v, do = sets[i]
            o, lse = window_forward(q, k, v, *args, stream=st if i else st.cuda_stream)
            outs[i].append((o, lse, *window_backward(q, k, v, o, lse, do, *args, stream=st)))
    torch.cuda.synchronize()
    for i in range(2):
        for r in outs[i]:
            for a, b in zip(r, ref[i]):
                assert torch.equal(a, b)


@pytest.mark.gpu
def test_first_call_of_a_thread():
    """A thread whose first use of the device is one of these calls, as an autograd worker's may be."""
    import threading
    q, k, v, do = (t.cuda() for t in make(2, 1, 300, 300, 64, BF16))
    o, lse = window_forward(q, k, v, 50, 2, check=True)
    want = (o, *window_backward(q, k, v, o, lse, do, 50, 2, check=True))
    o1, lse1, grads = torch.empty_like(o), torch.empty_like(lse), [torch.empty_like(t) for t in (q, k, v)]
    ws = torch.empty(1 << 24, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    calls = (lambda: window_forward(q, k, v, 50, 2, o=o1, lse=lse1, workspace=ws),
             lambda: window_backward(q, k, v, o, lse, do, 50, 2, dq=grads[0], dk=grads[1], dv=grads[2], workspace=ws))
    failed = []
    for call in calls:
        def first(call=call):
            try:
                call()
            except Exception as e:  # noqa: BLE001
                failed.append(e)
        t = threading.Thread(target=first)
        t.start()
        t.join()
    torch.cuda.synchronize()
    assert not failed and all(torch.equal(a, b) for a, b in zip((o1, *grads), want))


@pytest.mark.gpu
def test_capture_of_leaves_with_a_live_eager_graph_is_refused():
    leaves = [t.cuda().requires_grad_() for t in make(2, 2, 64, 64, 64, BF16)[:3]]
    alive = sliding_window_attention(*leaves, 16, 2)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        graph = torch.cuda.CUDAGraph()
        graph.capture_begin()
        with pytest.raises(RuntimeError, match="still alive"):
            sliding_window_attention(*leaves, 16, 2)
        graph.capture_end()
    del alive
    grads = [torch.zeros_like(t) for t in leaves]
    torch.cuda.synchronize()
    with torch.cuda.graph(torch.cuda.CUDAGraph()):
        out = sliding_window_attention(*leaves, 16, 2)
        for g, x in zip(grads, torch.autograd.grad(out, leaves, torch.ones_like(out))):
            g.copy_(x)


# ------------------------------------------------------------------ refusals (no GPU)
def problem(**kw):
    base = dict(batch=1, heads=4, kv_heads=2, head_dim=64, q_len=10, kv_len=20, q_rows=0, kv_rows=0, window=4, sinks=1,
                type=0, scale=0.0)
    base.update(kw)
    return _WindowProblem(*[base[n] for n, _ in _WindowProblem._fields_])


@pytest.mark.parametrize("kw,status", [
    (dict(batch=0), 2), (dict(heads=3), 2), (dict(q_len=-1), 2), (dict(kv_len=1 << 30), 2),
    (dict(batch=60000, heads=4, q_len=10000), 2), (dict(head_dim=96), 3), (dict(type=2), 3), (dict(window=-1), 1),
    (dict(sinks=-2), 1), (dict(scale=float("nan")), 1), (dict(scale=float("inf")), 1), (dict(q_rows=1 << 30), 2),
])
def test_bad_problems_are_refused(kw, status):
    n = ctypes.c_size_t()
    assert sta.lib().sta_window_workspace_size(ctypes.byref(problem(**kw)), ctypes.byref(n), None) == status


def test_packed_sizes_follow_the_rows_that_are_there():
    """Bounds of all rows (none given) on many sequences: neither the workspace
    nor the limits grow with sequences times rows."""
    def size(**kw):
        n = ctypes.c_size_t()
        p = problem(heads=24, kv_heads=8, head_dim=128, window=256, sinks=0, q_rows=131072, kv_rows=131072, **kw)
        assert sta.lib().sta_window_workspace_size(ctypes.byref(p), None, ctypes.byref(n)) == 0
        return n.value

    bounded, free = size(batch=256, q_len=512, kv_len=512), size(batch=256, q_len=131072, kv_len=131072)
    # 36 bytes a row and head for the panel and D, and no more than what the parts of 300 key blocks take
    assert bounded <= free <= 24 * 131072 * 40 + 300 * 2 * 128 * 128 * 4
    assert size(batch=700, q_len=131072, kv_len=131072) < 2 ** 28
    # a dense call whose problem has packed rows needs the dense form's workspace
    p, n = problem(head_dim=128, q_len=4096, kv_len=4096, q_rows=8, kv_rows=8), ctypes.c_size_t()
    assert sta.lib().sta_window_workspace_size(ctypes.byref(p), None, ctypes.byref(n)) == 0
    row = sta._Rows(4096, 4096 * 512, 4096 * 128, 128)
    assert sta.lib().sta_window_backward(ctypes.byref(p), row, row, row, row, 4096, row, row, row, row, None, None, 4096,
                                         4 * 4096 * 36, None, 0) == 5


def test_bad_calls_are_refused_before_anything_is_enqueued():
    L, p = sta.lib(), problem()
    n = ctypes.c_size_t()
    assert L.sta_window_workspace_size(ctypes.byref(p), None, ctypes.byref(n)) == 0 and n.value > 0
    row = lambda ptr=4096, b=2560, h=640, r=64: sta._Rows(ptr, b, h, r)  # noqa: E731

    def fwd(q=row(), k=row(), v=row(), o=row(), lse=None, cu=(None, None), ws=4096, size=1 << 20, flags=0):
        return L.sta_window_forward(ctypes.byref(p), q, k, v, o, lse, *cu, ws, size, None, flags)

    assert fwd(q=None) == 1 and fwd(o=row(ptr=0)) == 1 and fwd(flags=2) == 1 and fwd(cu=(4096, None)) == 1
    assert fwd(k=row(ptr=4104)) == 4 and fwd(v=row(r=65)) == 4 and fwd(q=row(h=0)) == 1 and fwd(q=row(r=-64)) == 1
    assert fwd(ws=None) == 5 and fwd(size=16) == 5 and fwd(ws=4100) == 4

    def bwd(lse=4096, dk=row(), size=1 << 20):
        return L.sta_window_backward(ctypes.byref(p), row(), row(), row(), row(), lse, row(), row(), dk, row(), None, None,
                                     4096, size, None, 0)

    assert bwd(lse=None) == 1 and bwd(dk=None) == 1 and bwd(dk=row(ptr=8)) == 4 and bwd(size=n.value - 1) == 5


def test_a_scale_too_small_for_gradients_is_refused():
    L, n, row = sta.lib(), ctypes.c_size_t(), sta._Rows(4096, 2560, 640, 64)
    for scale, status in ((2.0 ** -101, 1), (2.0 ** -100, 5)):  # the second gets as far as the workspace
        p = problem(scale=scale)
        assert L.sta_window_workspace_size(ctypes.byref(p), None, ctypes.byref(n)) == 0
        assert L.sta_window_backward(ctypes.byref(p), row, row, row, row, 4096, row, row, row, row, None, None, 4096, 0,
                                     None, 0) == status


@pytest.mark.parametrize("at", [0, 1, 2])
def test_forward_mode_derivatives_are_refused(at):
    """A tangent would be dropped silently."""
    import torch.autograd.forward_ad as forward_ad
    x = [torch.zeros(1, 2, 8, 64, dtype=BF16) for _ in range(3)]
    with forward_ad.dual_level():
        x[at] = forward_ad.make_dual(x[at], torch.ones_like(x[at]))
        with pytest.raises(NotImplementedError, match="forward-mode"):
            sliding_window_attention(*x, 4)
        with pytest.raises(NotImplementedError, match="forward-mode"):
            sta.sliding_tile_attention(*x, 2, 2, 2, (1, 1, 1), (1, 1, 1))


def test_binding_refusals():
    q = torch.zeros(1, 2, 8, 64, dtype=BF16)
    with pytest.raises(ValueError, match="CUDA"):
        window_forward(q, q, q, 4)
    with pytest.raises(TypeError):
        window_forward([1.0], q, q, 4)
    with pytest.raises(ValueError, match="CUDA"):
        sliding_window_attention(q.requires_grad_(), q, q, 4)


@pytest.mark.gpu
def test_binding_refusals_on_device():
    q = torch.zeros(2, 4, 8, 64, dtype=BF16, device="cuda")
    cu = torch.tensor([0, 8], dtype=torch.int32, device="cuda")
    for bad in (dict(k=q.half()), dict(k=q[:1]), dict(v=q[..., :32]), dict(v=q.cpu()), dict(q=q[0]), dict(q=q.float()),
                dict(cu_q=cu), dict(cu_q=cu, cu_kv=cu), dict(o=q.half()), dict(o=q[:, :, :4]),
                dict(o=torch.zeros(2, 4, 8, 65, dtype=BF16, device="cuda")[..., 1:]), dict(lse=q.float()),
                dict(workspace=torch.zeros(8)), dict(lse=torch.zeros(2, 4, 8, device="cuda").double())):
        kw = dict(q=q, k=q, v=q, window=4)
        kw.update(bad)
        with pytest.raises(ValueError):
            window_forward(**kw)
    one = q[:1]
    for bad in (cu.long(), cu.cpu()):
        with pytest.raises(ValueError):
            window_forward(one, one, one, 4, cu_q=bad, cu_kv=bad)
    for kw, status in ((dict(window=-1), 1), (dict(sinks=-1), 1), (dict(scale=float("inf")), 1)):
        with pytest.raises(sta.StaError) as e:
            window_forward(q, q, q, **{**dict(window=4), **kw})
        assert e.value.status == status
    with pytest.raises(sta.StaError) as e:
        window_forward(q, q[:, :3], q[:, :3], 4)
    assert e.value.status == 2
    # empty tensors
    for shape in ((0, 4, 8, 64), (2, 4, 0, 64)):
        e = torch.zeros(shape, dtype=BF16, device="cuda")
        k = torch.zeros(shape[0], 4, 8, 64, dtype=BF16, device="cuda")
        o, lse = window_forward(e, k, k, 4)
        assert o.shape == e.shape and lse.shape == e.shape[:3]
        grads = window_backward(e, k, k, o, lse, e, 4)
        assert [g.shape for g in grads] == [e.shape, k.shape, k.shape] and not any(g.any() for g in grads)
@pytest.mark.gpu
def test_wait_timeout_is_reported_and_recoverable():
    q, k, v, do = (t.cuda() for t in make(2, 2, 700, 700, 128, BF16))
    o, lse = window_forward(q, k, v, 300, 4, check=True)
    good = window_backward(q, k, v, o, lse, do, 300, 4, check=True)
    try:
        sta.sta_set_wait_limit_ns(0)
        for call in (lambda: window_forward(q, k, v, 300, 4, check=True),
                     lambda: window_backward(q, k, v, o, lse, do, 300, 4, check=True)):
            with pytest.raises(sta.StaError) as e:
                call()
            assert e.value.status == 8
    finally:
        sta.sta_set_wait_limit_ns(2_000_000_000)
    o2, lse2 = window_forward(q, k, v, 300, 4, check=True)
    assert torch.equal(o2, o) and torch.equal(lse2, lse)
    for a, b in zip(window_backward(q, k, v, o, lse, do, 300, 4, check=True), good):
        assert torch.equal(a, b)


def calls_under_limits(call, limit, repeats=20):
    """`call` returns tensors: under the limit its status, or the same bits as without one."""
    good = call()
    try:
        sta.sta_set_wait_limit_ns(limit)
        for _ in range(repeats):
            try:
                got = call()
            except sta.StaError as e:
                assert e.status == 8
            else:
                assert all(torch.equal(a, b) for a, b in zip(got, good))
    finally:
        sta.sta_set_wait_limit_ns(2_000_000_000)
    assert all(torch.equal(a, b) for a, b in zip(call(), good))


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("limit", [0, 300, 1000, 3000, 10000])
def test_waits_that_run_out_anywhere_leave_no_item_behind(limit, d):
    """Limits that end waits early, in the middle or not at all, with more items
    than the GPU holds, so that items have been asked for when a wait runs out."""
    q, k, v, do = (t.cuda() for t in make(16, 8, 2000, 2000, d, BF16))
    calls_under_limits(lambda: window_forward(q, k, v, 300, 4, check=True), limit)
    o, lse = window_forward(q, k, v, 300, 4, check=True)
    calls_under_limits(lambda: window_backward(q, k, v, o, lse, do, 300, 4, check=True), limit)


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("limit", [0, 200, 1000, 3000, 10000])
def test_waits_that_run_out_anywhere_end_the_call(limit, d):
    """12 blocks take the form whose warpgroups share a block's keys and meet at its end."""
    q, k, v, _ = (t.cuda() for t in make(2, 2, 700, 700, d, BF16))
    calls_under_limits(lambda: window_forward(q, k, v, 300, 4, check=True), limit)


def integer_scores(dtype, heads, nk, d, offset, seed=0):
    """One query and nk keys of a head each whose products are integers below
    2^24, which any order of fp32 sums gives exactly: small ones, and four of
    `offset` squared (bf16 and fp16 hold it) that all keys share."""
    g = torch.Generator().manual_seed(seed)
    q, k = (torch.randint(-2, 3, (1, heads, n, d), generator=g).to(dtype) for n in (1, nk))
    q[..., :4], k[..., :4] = offset, offset
    return q, k, randn(1, heads, nk, d, seed=seed + 1, dtype=dtype), randn(1, heads, 1, d, seed=seed + 2, dtype=dtype)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,offset,scale", [(BF16, 80, 0.125), (BF16, 253, 0.125), (BF16, 3, 2e-7), (BF16, 253, 0.02),
                                                (FP16, 3, 0.125), (FP16, 500, 0.125), (FP16, 600, 0.125), (FP16, 2000, 0.125),
                                                (FP16, 3, 2e-6), (FP16, 3, 2e-7)])
def test_gradients_of_large_log_sums(dtype, offset, scale):
    """An offset that all keys share, or a small scale: |LSE / scale| up to 10^7.

    Scores x = scale S of exact S.  The log-sum-exp is off by the roundings of
    scale log2(e), its product with S, the product with log(2) and LSE / scale:
    six of 2^-24 at most, below 2^-21 |x|, and each exponential and logarithm by
    2^-20, so P is off by e = 2^-21 max |x| + 2^-20 and its own rounding u (fp16,
    held times 2^8: at least 2^-33).  D is off by the rounding of O (twice u |O|
    and e) and 2^-20 of its sum's magnitudes, dS by P's error, D's, its rounding
    (fp16: at least 2^-27 max |dO|), the results by theirs."""
    d, u = 64, seq_ref.unit(dtype)
    q, k, v, do = integer_scores(dtype, 32, 40, d, offset)
    qd, kd, vd, dod = (t.cuda() for t in (q, k, v, do))
    o, lse = window_forward(qd, kd, vd, 0, 0, scale, check=True)
    got = window_backward(qd, kd, vd, o, lse, dod, 0, 0, scale, check=True)
    q, k, v, do = (t[0].double() for t in (q, k, v, do))
    assert (q @ k.mT).abs().max() < 2 ** 24
    x = scale * (q @ k.mT)
    p = torch.softmax(x, -1)
    e = 2.0 ** -21 * x.abs().max() + 2.0 ** -20
    out, dp = p @ v, do @ v.mT
    dd = (do * out).sum(-1, keepdim=True)
    half = dtype == FP16
    dp_err = 2.0 ** -20 * (do.abs() @ v.abs().mT)
    dd_err = (do.abs() * ((p @ v.abs()) * (u + e) + u * out.abs() + 2.0 ** -20 * out.abs())).sum(-1, keepdim=True)
    ds = p * (dp - dd)
    floor = 2.0 ** -27 * float(do.norm(dim=-1).max()) if half else 0.0
    p_err = p * (u + e) + (2.0 ** -33 if half else 0.0)
    ds_err = ds.abs() * (u + e) + p * (dp_err + dd_err) + floor
    want = dict(dq=(scale * ds @ k, scale * ds_err @ k.abs()), dk=(scale * ds.mT @ q, scale * ds_err.mT @ q.abs()),
                dv=(p.mT @ do, p_err.mT @ do.abs()))
    tiny = torch.finfo(dtype).smallest_normal * u
    for g, (name, (w, b)) in zip(got, want.items()):
        seq_ref.check(g[0], (w, b + u * w.abs() + tiny), name)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF16, FP16], ids=["bf16", "fp16"])
@pytest.mark.parametrize("nq,nk,d", [(205, 64, 64), (300, 301, 128), (300, 307, 64), (400, 261, 128)])
def test_hidden_queries_reach_nothing(nq, nk, d, dtype):
    """Query rows that see nothing hold NaN and infinities, in Q and in dO; and a
    query's reach the gradients of no key behind it."""
    q, k, v, do = make(4, 2, nq, nk, d, dtype, seed=nq + nk)
    mask = seq_ref.mask_of(nq, nk, 90, 3)
    blind = ~mask.any(1)
    top = float(do[:, :, ~blind].double().norm(dim=-1).max())
    want = seq_ref.attention(q[0], k[0], v[0], mask, d ** -0.5, do[0], dtype, top)
    kd, vd = k.cuda(), v.cuda()

    def run(rows, bad):
        qb, gb = q.clone(), do.clone()
        qb[:, :, rows], gb[:, :, rows] = bad, bad
        qd, gd = qb.cuda(), gb.cuda()
        o, lse = window_forward(qd, kd, vd, 90, 3, check=True)
        return window_backward(qd, kd, vd, o, lse, gd, 90, 3, check=True)

    for bad in (float("nan"), float("inf"), float("-inf")):
        if blind.any():
            for name, got in zip(("dq", "dk", "dv"), run(blind, bad)):
                seq_ref.check(got[0], want[name], name)
        # a query whose last key is the last one of a block of 128
        row = 127 - (nk - nq)
        if row < nq and nk > 128:
            for name, got in zip(("dk", "dv"), run([row], bad)[1:]):
                assert bool(got[0, :, 128:].isfinite().all()), name


@pytest.mark.gpu
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), 6e4], ids=str)
def test_hidden_or_non_finite_gradients_do_not_scale_the_others(bad):
    """fp16 gradients are scaled by the largest row of dO: one that sees nothing,
    or is not finite itself, does not count."""
    nq, nk, d = 205, 64, 64
    q, k, v, do = make(4, 2, nq, nk, d, FP16, seed=77, do_scale=2.0 ** -12)
    mask = seq_ref.mask_of(nq, nk, 90, 3)
    blind = ~mask.any(1)
    want = seq_ref.attention(q[0], k[0], v[0], mask, d ** -0.5, do[0], FP16)
    qd, kd, vd = q.cuda(), k.cuda(), v.cuda()
    o, lse = window_forward(qd, kd, vd, 90, 3, check=True)
    gb = do.clone()
    gb[:, :, blind] = bad
    for name, got in zip(("dq", "dk", "dv"), window_backward(qd, kd, vd, o, lse, gb.cuda(), 90, 3, check=True)):
        seq_ref.check(got[0], want[name], name)
    if bad != 6e4:
        gb = do.clone()
        gb[:, :, 200] = bad
        dq = window_backward(qd, kd, vd, o, lse, gb.cuda(), 90, 3, check=True)[0]
        others = torch.arange(nq) != 200
        seq_ref.check(dq[0][:, others], tuple(t[:, others] for t in want["dq"]), "dq")


@pytest.mark.gpu
@pytest.mark.parametrize("heads,kv_heads,nq,nk,window,sinks", [
    (32, 32, 700, 700, 512, 0),   # pairs of blocks that end 128 keys apart, inside a chunk
    (32, 32, 700, 760, 100, 0),
    (32, 32, 600, 689, 0, 0),     # no window, off the chunks
    (32, 32, 700, 700, 200, 40),  # the second block's window begins inside the first chunk, behind the sinks
    (32, 32, 700, 733, 300, 64),
    (33, 11, 640, 640, 150, 7),   # pairs of heads and pairs of blocks by turns
], ids=str)
@pytest.mark.parametrize("d", [64, 128])
def test_non_finite_keys_reach_only_blocks_that_see_them(heads, kv_heads, nq, nk, window, sinks, d):
    """More blocks than the GPU has SMs, so that two of a key head share their
    keys: a row of NaN in K and V leaves every 128-row block that does not see it
    as it was."""
    q, k, v, _ = (t.cuda() for t in make(heads, kv_heads, nq, nk, d, BF16, seed=nk))
    clean = window_forward(q, k, v, window, sinks, check=True)
    mask = seq_ref.mask_of(nq, nk, window, sinks)
    for key in sorted({*range(0, nk, 13), *range(nk - nq, nk, 128), nk - 1}):  # the first behind each block, too
        kb, vb = k.clone(), v.clone()
        kb[:, :, key], vb[:, :, key] = float("nan"), float("nan")
        got = window_forward(q, kb, vb, window, sinks, check=True)
        sees = [bool(mask[i:i + 128, key].any()) for i in range(0, nq, 128)]
        rows = torch.tensor(sees).repeat_interleave(128)[:nq].cuda()
        same = all(torch.equal(a[:, :, ~rows], b[:, :, ~rows]) for a, b in zip(got, clean))
        assert same, f"key {key}"
        assert bool(got[0][:, :, mask[:, key].cuda()].isnan().all()), key


@pytest.mark.gpu
@pytest.mark.parametrize("heads,kv_heads,nq,nk", [(2, 2, 1, 5), (2, 1, 9, 9), (2, 2, 200, 200)])
def test_scores_far_below_zero(heads, kv_heads, nq, nk):
    """Equal scores of -2^117 for all keys: O is the mean of the visible values.
    The sums of nk terms are off by 2^-20, P and O by their roundings."""
    _, _, v, _ = make(heads, kv_heads, nq, nk, 64, BF16, seed=nk)
    q, k = torch.zeros(1, heads, nq, 64, dtype=BF16), torch.zeros(1, kv_heads, nk, 64, dtype=BF16)
    q[..., 3], k[..., 3] = 2.0 ** 60, -2.0 ** 60
    o, lse = window_forward(q.cuda(), k.cuda(), v.cuda(), check=True)
    seen = torch.tril(torch.ones(nq, nk, dtype=torch.float64), nk - nq)
    p = seen / seen.sum(-1, keepdim=True)
    vv = v[0].double().repeat_interleave(heads // kv_heads, 0)
    want, mag = p @ vv, p @ vv.abs()
    seq_ref.check(o[0], (want, mag * (2.0 ** -8 + 2.0 ** -20) + want.abs() * 2.0 ** -8), "o")
    assert ((lse.double().cpu() + 2.0 ** 117).abs() <= 2.0 ** (117 - 20)).all()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF16, FP16], ids=["bf16", "fp16"])
def test_many_short_documents_without_bounds(dtype):
    """Sequences times rows times heads past 2^31."""
    n, each, heads, d = 2000, 35, 16, 64
    q, k, v, do, cu, _ = packed([each] * n, [each] * n, heads, 2, d, dtype, tail=0, seed=5)
    qd, kd, vd, dod, cd = (t.cuda() for t in (q, k, v, do, cu))
    o, lse = window_forward(qd, kd, vd, 20, 2, cu_q=cd, cu_kv=cd, check=True)
    got = dict(zip(("dq", "dk", "dv"), window_backward(qd, kd, vd, o, lse, dod, 20, 2, cu_q=cd, cu_kv=cd, check=True)), o=o, lse=lse)
    mask = seq_ref.mask_of(each, each, 20, 2)
    top = float(do.double().norm(dim=-1).max())
    for b in (0, 1, 777, 1998, 1999):
        r = slice(b * each, (b + 1) * each)
        want = seq_ref.attention(q[0, :, r], k[0, :, r], v[0, :, r], mask, d ** -0.5, do[0, :, r], dtype, top)
        for name, t in got.items():
            seq_ref.check(t[0, :, r], want[name], f"{name} of sequence {b}")


@pytest.mark.gpu
def test_leaves_keep_nothing_of_the_calls():
    """A leaf can be saved, loaded and copied after a call, and a copy is not
    held back by the graphs of the one it was copied from."""
    import copy
    import io
    leaves = [t.cuda().requires_grad_() for t in make(2, 2, 64, 64, 64, BF16)[:3]]
    before = [dict(t.__dict__) for t in leaves]
    alive = sliding_window_attention(*leaves, 16, 2)
    assert [dict(t.__dict__) for t in leaves] == before
    file = io.BytesIO()
    torch.save(leaves, file)
    file.seek(0)
    assert all(torch.equal(a, b) for a, b in zip(torch.load(file, weights_only=True), leaves))
    copies = copy.deepcopy(leaves)
    torch.cuda.synchronize()
    with torch.cuda.graph(torch.cuda.CUDAGraph()):
        out = sliding_window_attention(*copies, 16, 2)
        torch.autograd.grad(out, copies, torch.ones_like(out))
    assert alive.requires_grad


@pytest.mark.gpu
@pytest.mark.parametrize("d", [0, 32])
def test_empty_tensors_of_other_head_dims_are_refused(d):
    """Without rows or columns nothing is computed, so nothing else would say so."""
    for shape in ((1, 2, 3, d), (1, 2, 0, d)):
        if shape[2] and d:
            continue
        q = torch.zeros(shape, dtype=BF16, device="cuda")
        with pytest.raises(ValueError, match="head_dim"):
            window_forward(q, q, q, 4)


@pytest.mark.gpu
def test_capture_of_views_of_leaves_with_a_live_eager_graph_is_refused():
    """Rows outside heads, halves of one tensor, a broadcast head: views of leaves
    are uses of the leaves."""
    both = torch.randn(1, 64, 4, 64, device="cuda").bfloat16().requires_grad_()
    one = torch.randn(1, 1, 64, 64, device="cuda").bfloat16().requires_grad_()

    def call():
        k, v = both.transpose(1, 2)[:, :2], both.transpose(1, 2)[:, 2:]
        return sliding_window_attention(one.expand(-1, 4, -1, -1), k, v, 16, 2)

    side = torch.cuda.Stream()
    for leaf in (both, one):
        other = one if leaf is both else both
        other.requires_grad_(False)
        alive = call()
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            graph = torch.cuda.CUDAGraph()
            graph.capture_begin()
            with pytest.raises(RuntimeError, match="still alive"):
                call()
            graph.capture_end()
        del alive
        other.requires_grad_()
    want = torch.autograd.grad(call(), (both, one), torch.ones(1, 4, 64, 64, device="cuda").bfloat16())
    ones, grads = torch.ones(1, 4, 64, 64, device="cuda").bfloat16(), [torch.zeros_like(t) for t in want]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for g, x in zip(grads, torch.autograd.grad(call(), (both, one), ones)):
            g.copy_(x)
    graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(grads, want):
        assert torch.equal(a, b)


def test_uses_are_noted_from_several_threads(monkeypatch):
    """A capture looks through the live graphs while other threads add theirs."""
    import threading

    class Graph:
        needs_input_grad = (True,)

    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: True)
    leaves = [torch.zeros(2, requires_grad=True) for _ in range(4)]
    kept, failed = [[] for _ in leaves], []

    def run(i):
        try:
            for _ in range(1500):
                kept[i].append(Graph())
                window._note_uses(kept[i][-1], (leaves[i],), i)
                if len(kept[i]) > 40:
                    del kept[i][:30]
        except Exception as e:  # noqa: BLE001
            failed.append(e)

    threads = [threading.Thread(target=run, args=(i,)) for i in range(len(leaves))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed
    with pytest.raises(RuntimeError, match="still alive"):
        window._note_uses(Graph(), (leaves[0],), 9)

"""fp64 definitions of the token-sequence operators and the error bounds their
tests use.

Bounds.  With u = finfo(type).eps / 2 (a rounding's largest relative error) and
a score error e_s (fp32 products and sums of d terms: at most 2^-20 times the
sum of their magnitudes, twice the 2^-24 d / 8 that a tree of eights gives,
plus 2^-20 for the exponential), O is off by the rounding of P (u per term),
e_s and its own rounding.  The backward's P carries e_s and the stored
log-sum-exp's error e_l, D = rowsum(dO o O) the error of the rounded O, dS its
own rounding; each propagates through sums of magnitudes, all formed below."""
import torch


def mask_of(nq, nk, window, sinks, device="cpu"):
    pos = (torch.arange(nq, device=device) + nk - nq)[:, None]
    key = torch.arange(nk, device=device)[None]
    m = key <= pos
    return m & ((key > pos - window) | (key < sinks)) if window else m


def unit(dtype):
    return torch.finfo(dtype).eps / 2


def attention(q, k, v, mask, scale, do=None, dtype=torch.bfloat16, do_top=0.0, p_floor=0.0):
    """One sequence: q [heads, nq, d], k, v [kv_heads, nk, d], mask [nq, nk].
    Returns {name: (value, bound)} in fp64.  do_top: the largest row norm of dO
    in the call, if not this sequence's.  p_floor: absolute error of a P beyond
    its relative one."""
    g, u = q.shape[0] // k.shape[0], unit(dtype)
    tiny = torch.finfo(dtype).smallest_normal * u * 2  # half a step of the smallest numbers
    q, k, v = q.double(), k.double().repeat_interleave(g, 0), v.double().repeat_interleave(g, 0)
    x = (q @ k.mT * scale).masked_fill(~mask, float("-inf"))
    mag = q.abs() @ k.abs().mT * scale
    e_s = (2.0 ** -20 * (mag + x.abs().masked_fill(~mask, 0) + 1)).masked_fill(~mask, 0)
    lse = torch.logsumexp(x, -1)
    p = torch.where(mask, torch.exp(x - torch.where(lse.isinf(), 0.0, lse)[..., None]), 0.0)
    o = p @ v
    e_l = (p * e_s).sum(-1) + 2.0 ** -22 * torch.where(lse.isinf(), 0.0, lse.abs()) + 2.0 ** -20
    pe = p * (u + e_s + e_l[..., None]) + mask * (tiny + p_floor)
    o_bound = pe @ v.abs() + u * o.abs() + tiny
    out = dict(o=(o, o_bound), lse=(lse, e_l))
    if do is None:
        return out
    do = do.double()
    dp = do @ v.mT
    dp_mag = do.abs() @ v.abs().mT
    dd = (do * o).sum(-1, keepdim=True)
    dd_err = (do.abs() * o_bound).sum(-1, keepdim=True) + 2.0 ** -15 * (do.abs() * o.abs()).sum(-1, keepdim=True)
    # the backward adds -LSE and -D to its products as two 16-bit numbers each: 2^-15 relative
    p_rel = e_s + e_l[..., None] + 2.0 ** -15 * torch.where(lse.isinf(), 0.0, lse.abs())[..., None]
    ds = p * (dp - dd)
    # fp16: dS is held times 2^(2 - e), 2^e <= max |dO_i|, so half a step of the
    # smallest numbers, 2^-25, stands for 2^-25 2^(e - 2) <= 2^-27 max |dO_i|
    floor = tiny if dtype != torch.float16 else tiny + 2.0 ** -27 * max(do_top, float(do.norm(dim=-1).max()) if do.numel() else 0.0)
    ds_err = ds.abs() * (u + p_rel) + p * (dd_err + 2.0 ** -20 * dp_mag + 2.0 ** -15 * dd.abs()) + mask * floor
    kv = lambda t: t.unflatten(0, (-1, g)).sum(1)  # noqa: E731
    pv = p * (u + p_rel) + mask * tiny
    dq, dk, dv = ds @ k * scale, kv(ds.mT @ q * scale), kv(p.mT @ do)
    out["dq"] = (dq, ds_err @ k.abs() * scale + u * dq.abs() + tiny)
    out["dk"] = (dk, kv(ds_err.mT @ q.abs() * scale) + u * dk.abs() + tiny)
    out["dv"] = (dv, kv(pv.mT @ do.abs()) + u * dv.abs() + tiny)
    return out


def check(got, want, name):
    value, bound = want
    got = got.double().cpu()
    value, bound = value.cpu(), bound.cpu()
    inf = value.isinf()
    assert torch.equal(got[inf], value[inf]), f"{name}: infinities"
    off = (got - value).abs()[~inf]
    over = off > bound[~inf]
    assert not off.isnan().any() and not over.any(), (
        f"{name}: {int(over.sum())} of {over.numel()} values off by more than their bound; worst "
        f"{float((off / bound[~inf]).nan_to_num(1e9).max()):.2f} of it")


# ------------------------------------------------------------------ the cache
QMAX = {torch.float8_e4m3fn: 448.0, torch.int8: 127.0}


def to_codes(x, dtype):
    """The nearest code of each value, in fp32 as the definition says; NaN is code 0."""
    x = torch.nan_to_num(x, nan=0.0, posinf=QMAX[dtype], neginf=-QMAX[dtype]).clamp(-QMAX[dtype], QMAX[dtype])
    return x.to(dtype) if dtype == torch.float8_e4m3fn else x.round().to(dtype)


def cache_write(codes, scales, x, table, start, count):
    """sta_cache_write of one tensor, token block by token block (host tensors, changed in place)."""
    page_size, block = codes.shape[2], codes.shape[2] // scales.shape[2]
    big = torch.finfo(x.dtype).max
    for b in range(x.shape[0]):
        n = min(max(int(count[b]), 0), x.shape[2]) if count is not None else x.shape[2]
        s0 = int(start[b])
        if s0 < 0 or n == 0:
            continue
        for j in range(s0 // block, (s0 + n - 1) // block + 1):
            i = j * block // page_size
            if i >= table.shape[1] or not 0 <= int(table[b, i]) < codes.shape[0]:
                continue
            page, at = int(table[b, i]), j * block % page_size
            lo, hi = max(s0, j * block), min(s0 + n, (j + 1) * block)
            part = x[b, :, lo - s0:hi - s0].float()
            amax = torch.nan_to_num(part.abs(), nan=0.0, posinf=big).amax((-1, -2))
            s = (amax / QMAX[codes.dtype]).clamp_min(2.0 ** -100)
            held = codes[page, :, at:at + lo - j * block]
            if lo > j * block:
                old = scales[page, :, at // block].clone()
                s = torch.maximum(s, old)
                again = to_codes(held.float() * old[:, None, None] * (1 / s)[:, None, None], codes.dtype)
                held.copy_(torch.where((s > old)[:, None, None], again.float(), held.float()).to(codes.dtype))
            codes[page, :, at + lo - j * block:at + hi - j * block] = to_codes(part * (1 / s)[:, None, None], codes.dtype)
            scales[page, :, at // block] = s


def cache_values(codes, scales, table, b, n):
    """(values [kv_heads, n, d] in fp64, present [n]) of the first n tokens of sequence b."""
    page_size, block = codes.shape[2], codes.shape[2] // scales.shape[2]
    out = torch.zeros(codes.shape[1], n, codes.shape[3], dtype=torch.float64)
    there = torch.zeros(n, dtype=torch.bool)
    for i in range(0, n, page_size):
        page = int(table[b, i // page_size]) if i // page_size < table.shape[1] else -1
        if 0 <= page < codes.shape[0]:
            m = min(page_size, n - i)
            out[:, i:i + m] = (codes[page].double() * scales[page].double().repeat_interleave(block, -1)[..., None])[:, :m]
            there[i:i + m] = True
    return out, there

"""Measured cases of the 8-bit cache operators: rotary positions, the append
that quantises into 8-bit pages, and the attention that reads them.

`run` computes each operator either in its plain form (elementary torch
operations) or, where `own` is true, with the library's calls.

  rope    y0 = x0 c - x1 s, y1 = x0 s + x1 c for the pairs of the rotated part
          of each head, c and s = magnitude * cos / sin(position * f_j)
  append  rotated keys and values of n new tokens a sequence become e4m3 codes
          with one power-of-two scale per (block of tokens, KV head); a block
          that already holds committed tokens keeps the larger scale and its
          codes are rewritten for it
  attn    grouped-query attention of n query rows a sequence over those pages
"""
import math

import torch

own = False

PAGE = 64
BF16, F16, F32 = "bf16", "fp16", "fp32"
TYPES = {BF16: torch.bfloat16, F16: torch.float16, F32: torch.float32}
E4M3 = torch.float8_e4m3fn
MIN_EXP, MAX_EXP = -100, 100       # scales of a block: 2^-100 .. 2^100

# --------------------------------------------------------------------- cases


def rope_case(**kw):
    return {"kind": "rope", "layout": "half", "scaling": "none", "factor": 1.0, "original": 0.0,
            "theta": 10000.0, "magnitude": 1.0, "inverse": False, "fused": False, **kw}


def append_case(**kw):
    return {"kind": "append", "layout": "half", "block": 64, **kw}


def attn_case(**kw):
    return {"kind": "attn", "layout": "half", "block": 64, "window": 0, **kw}


def listed():
    return [
        # the queries of one verify step of one sequence: a quarter of the pairs turned, latency only
        rope_case(name="rope_verify_b1", type=BF16, rows=5, heads=16, dim=256, span=256, n_rot=32,
                  max_pos=8192),
        # the queries of a whole long prompt, interleaved, frequencies scaled by parts for 16 x the trained length
        rope_case(name="rope_prompt_32k", type=BF16, rows=32768, heads=8, dim=256, span=256,
                  n_rot=128, layout="interleaved", scaling="parts", factor=16.0, original=8192.0,
                  magnitude=1.2772588722239782, max_pos=131072),
        # part of an odd head, taken out of wider fused rows, positions compressed; turned back
        rope_case(name="rope_part_fp32", type=F32, rows=4099, heads=12, dim=104, span=40, n_rot=20,
                  scaling="linear", factor=4.0, original=4096.0, fused=True, inverse=True, max_pos=16384),
        # the new rows of one verify step of eight sequences: a partly filled block each
        append_case(name="append_verify_b8", batch=8, n=5, kv_heads=4, dim=256, lo=4096, hi=32768, n_rot=32),
        # one prompt chunk of 64 sequences
        append_case(name="append_chunk_b64", batch=64, n=256, kv_heads=8, dim=256, lo=1024, hi=16384, n_rot=128),
        # the smallest attention call: one short sequence, one KV head
        attn_case(name="attn_verify_tiny", batch=1, n=5, q_heads=8, kv_heads=1, dim=128, lo=256,
                  hi=256, split=256, n_rot=64),
        # one sequence at 8k: few CTAs' worth of cache, latency and bandwidth
        attn_case(name="attn_verify_b1_8k", batch=1, n=5, q_heads=16, kv_heads=8, dim=256, lo=8192,
                  hi=8192, split=512, n_rot=32),
        # eight ragged sequences, eight query heads a KV head
        attn_case(name="attn_verify_b8", batch=8, n=5, q_heads=32, kv_heads=4, dim=256, lo=4096,
                  hi=32768, split=1024, n_rot=32),
        # 64 sequences on a sliding-window layer, a scale for every 16 tokens
        attn_case(name="attn_window_b64", batch=64, n=4, q_heads=16, kv_heads=8, dim=256, lo=1024,
                  hi=16384, window=1024, split=1024, block=16, n_rot=128),
        # 64 ragged sequences, one token each, on a global layer: the most bytes
        attn_case(name="attn_decode_b64", batch=64, n=1, q_heads=16, kv_heads=8, dim=256, lo=1024,
                  hi=16384, split=2048, n_rot=32),
        # one very long sequence on two KV heads: work split over the long axis
        attn_case(name="attn_verify_131k", batch=1, n=9, q_heads=8, kv_heads=2, dim=256, lo=131072,
                  hi=131072, split=1024, n_rot=32),
        # a prompt chunk over 8k of context: bound by arithmetic
        attn_case(name="attn_chunk_8k", batch=2, n=256, q_heads=32, kv_heads=4, dim=256, lo=8000,
                  hi=8192, split=2048, layout="interleaved", n_rot=128),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(("rope", "append", "attn", "attn"))
    layout = rng.choice(("half", "interleaved"))
    if kind == "rope":
        dim = rng.choice((64, 80, 104, 128, 192, 256))
        span = 2 * rng.randint(8, dim // 2)
        heads = rng.choice((1, 2, 8, 12, 16, 32))
        rows = min(_log(rng, 1, 32768), 32768 * 2048 // (heads * dim))
        scaling = rng.choice(("none", "linear", "raised", "parts"))
        return rope_case(type=rng.choice((BF16, F16, F32)), rows=rows, heads=heads, dim=dim, span=span,
                         n_rot=rng.choice((span // 2, max(1, span // 8))), layout=layout, scaling=scaling,
                         factor=1.0 if scaling == "none" else rng.uniform(1.0, 32.0),
                         original=0.0 if scaling == "none" else 8192.0,
                         theta=rng.choice((10000.0, 500000.0)), magnitude=rng.choice((1.0, 1.25)),
                         inverse=rng.random() < 0.3, fused=rng.random() < 0.4,
                         max_pos=_log(rng, 1000, 131072))
    dim = rng.choice((128, 256))
    kv_heads = rng.choice((1, 2, 4, 8))
    n_rot = rng.choice((dim // 8, dim // 2))
    block = rng.choice((16, 32, 64))
    lo = _log(rng, 1, 16384)
    if kind == "append":
        return append_case(batch=rng.randint(1, 64), n=_log(rng, 1, 256), kv_heads=kv_heads, dim=dim, lo=lo,
                           hi=lo + rng.randint(0, 16384), n_rot=n_rot, layout=layout, block=block)
    window = rng.choice((0, 0, rng.randint(1, 2048)))
    group = rng.choice((1, 2, 4, 8))
    n = rng.choice((1, rng.randint(1, 17), _log(rng, 17, 200)))
    # no more cache than the largest listed case, and no more arithmetic than the chunk
    batch = rng.randint(1, 64 if n <= 17 else 2)
    most = min(500000, int(1.3e11 / (4.0 * n * group * kv_heads * dim)))
    hi = max(1, min(lo + rng.randint(0, 16384), most // batch))
    return attn_case(batch=batch, n=n, q_heads=group * kv_heads, kv_heads=kv_heads, dim=dim,
                     lo=min(lo, hi), hi=hi, window=window, split=rng.choice((128, 256, 1024)),
                     block=block, n_rot=n_rot, layout=layout)


def _lengths(c):
    """Committed lengths of the sequences: spread over [lo, hi], the first at hi."""
    span = c["hi"] - c["lo"]
    return [c["hi"] - int(span * ((b * 0.6180339887498949) % 1.0)) for b in range(c["batch"])]


def _keys_read(c, length):
    """Keys that any row of the sequence sees."""
    end = length + c["n"]
    return end if c["window"] == 0 else min(end, c["window"] + c["n"] - 1)


def work(c):
    if c["kind"] == "rope":
        size = 4 if c["type"] == F32 else 2
        n = c["rows"] * c["heads"]
        return {"bytes": 2 * n * c["dim"] * size + 4 * c["rows"], "flops": 6 * n * c["n_rot"]}
    if c["kind"] == "append":
        n = c["batch"] * c["n"] * c["kv_heads"] * c["dim"]
        return {"bytes": 2 * n * (2 + 1), "flops": 2 * n * 3}
    keys = sum(_keys_read(c, L) for L in _lengths(c))
    rows = c["batch"] * c["n"] * c["q_heads"]
    row_keys = 0
    for L in _lengths(c):
        for i in range(c["n"]):
            row_keys += L + i + 1 if c["window"] == 0 else min(L + i + 1, c["window"])
    return {"bytes": keys * c["kv_heads"] * (2 * c["dim"] + 8.0 / c["block"]) + 4 * rows * c["dim"],
            "flops": 4 * row_keys * c["q_heads"] * c["dim"]}


# -------------------------------------------------------------------- inputs


def _frequencies(c):
    """Angle per position of each turned pair, in float64 on the host."""
    span, theta, s = c.get("span", c["dim"]), c.get("theta", 10000.0), c.get("factor", 1.0)
    scaling = c.get("scaling", "none")
    if scaling == "raised":
        theta = theta * s ** (span / (span - 2.0))
    f = theta ** (-2.0 * torch.arange(c["n_rot"], dtype=torch.float64) / span)
    if scaling == "linear":
        f = f / s
    if scaling == "parts":
        turns = c["original"] * f / (2.0 * math.pi)
        g = ((turns - 1.0) / (32.0 - 1.0)).clamp(0.0, 1.0)
        f = (1.0 - g) * f / s + g * f
    return f


class State:
    pass


def _rope_config(c):
    from speculative_decoding_verification_91_b200 import binding as B
    kinds = {"none": B.SPEC_ROPE_PLAIN, "linear": B.SPEC_ROPE_LINEAR, "raised": B.SPEC_ROPE_RAISED,
             "parts": B.SPEC_ROPE_PARTS}
    return B.SpecRope(B.SPEC_ROPE_HALF if c["layout"] == "half" else B.SPEC_ROPE_INTERLEAVED,
                      c.get("span", c["dim"]), c["n_rot"], kinds[c.get("scaling", "none")],
                      c.get("theta", 10000.0), c.get("factor", 1.0), c.get("original", 0.0), 1.0, 32.0,
                      c.get("magnitude", 1.0))


def _cache_config(c, s, split):
    from speculative_decoding_verification_91_b200 import binding as B
    return B.SpecQCache(c["dim"], c["kv_heads"], s.k.shape[0], PAGE, c["block"], split, s.k.data_ptr(),
                        s.v.data_ptr(), s.ks.data_ptr(), s.vs.data_ptr())


def _random_pages(gen, pages, heads, dim, block, amplitude):
    """Codes and scales of random pages, as an earlier append would have left them."""
    codes = torch.empty(pages, heads, PAGE, dim, dtype=E4M3, device="cuda")
    scales = torch.empty(pages, heads, PAGE // block, device="cuda")
    step = max(1, (1 << 27) // (heads * PAGE * dim))
    for p in range(0, pages, step):
        m = min(step, pages - p)
        x = torch.randn(m, heads, PAGE // block, block * dim, generator=gen, device="cuda") * amplitude
        sc = _pow2(_scale_exp(x.abs().amax(-1).double())).float()
        scales[p:p + m] = sc
        codes[p:p + m] = (x / sc[..., None]).to(E4M3).view(m, heads, PAGE, dim)
    return codes, scales


def prepare(case, seed):
    c, s = case, State()
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    s.case = c
    s.freq = _frequencies(c).cuda()
    if c["kind"] == "rope":
        rows, heads, dim = c["rows"], c["heads"], c["dim"]
        wide = heads * dim + (48 if c["fused"] else 0)
        s.x = torch.randn(rows, wide, generator=gen, device="cuda").to(TYPES[c["type"]])
        s.x = s.x[:, wide - heads * dim:].unflatten(1, (heads, dim))
        s.out = torch.empty(rows, heads, dim, dtype=s.x.dtype, device="cuda")
        s.pos = torch.randint(0, c["max_pos"], (rows,), generator=gen, device="cuda", dtype=torch.int32)
        if own:
            from speculative_decoding_verification_91_b200 import binding as B
            s.rope = _rope_config(c)
            s.dtype = {BF16: B.SPEC_BF16, F16: B.SPEC_FP16, F32: B.SPEC_FP32}[c["type"]]
        return s
    B_, n, H, D = c["batch"], c["n"], c["kv_heads"], c["dim"]
    lens = _lengths(c)
    first = [L // PAGE if c["kind"] == "append" else 0 for L in lens]
    need = [(L + n - 1) // PAGE + 1 for L in lens]
    total = sum(need) - sum(first)
    s.max_pages = max(need)
    perm = torch.randperm(total, generator=gen, device="cuda").to(torch.int32)
    s.table = torch.zeros(B_, s.max_pages, dtype=torch.int32, device="cuda")
    at = 0
    for b in range(B_):
        m = need[b] - first[b]
        s.table[b, first[b]:need[b]] = perm[at:at + m]
        at += m
    s.lens = torch.tensor(lens, dtype=torch.int32, device="cuda")
    s.batch_index = torch.arange(B_, device="cuda")
    # one page more than is mapped: no sequence's
    s.k, s.ks = _random_pages(gen, total + 1, H, D, c["block"], 0.5 if c["kind"] == "append" else 1.0)
    s.v, s.vs = _random_pages(gen, total + 1, H, D, c["block"], 0.5 if c["kind"] == "append" else 1.0)
    if c["kind"] == "append":
        s.k_new = torch.randn(B_, n, H, D, generator=gen, device="cuda").to(torch.bfloat16)
        s.v_new = torch.randn(B_, n, H, D, generator=gen, device="cuda").to(torch.bfloat16)
    else:
        s.q = (1.5 * torch.randn(B_, n, c["q_heads"], D, generator=gen, device="cuda")).to(torch.bfloat16)
        s.out = torch.empty_like(s.q)
    if own:
        from speculative_decoding_verification_91_b200 import binding as B
        from speculative_decoding_verification_91_b200.runtime import Workspace
        s.rope = _rope_config(c)
        s.cache = _cache_config(c, s, c.get("split", 0))
        if c["kind"] == "append":
            s.ws = Workspace(B.spec_qcache_write_workspace_bytes(s.cache, B_, n))
        else:
            s.ws = Workspace(B.spec_qcache_attn_workspace_bytes(s.cache, c["q_heads"], B_, n, s.max_pages,
                                                                c["window"]))
    return s


# ---------------------------------------------------------------- plain forms


def _pow2(e):
    """2^e for whole e, exactly (float64)."""
    return ((e.to(torch.int64) + 1023) << 52).view(torch.float64)


def _scale_exp(amax):
    """Least e with amax <= 448 * 2^e, within the scales' range (amax float64)."""
    m, e = torch.frexp(amax)
    e = e.to(torch.int64) - 9 + (m > 0.875).to(torch.int64)
    return torch.where(amax > 0, e, torch.full_like(e, MIN_EXP)).clamp(MIN_EXP, MAX_EXP)


def _e4m3(x):
    """x (float64) rounded to the nearest e4m3 value, ties to even, 448 at most."""
    _, e = torch.frexp(x)
    step = _pow2((e.to(torch.int64) - 1).clamp(min=-6) - 3)
    return (torch.round(x / step) * step).clamp(-448.0, 448.0)


def _turn(x, pos, freq, layout, span, magnitude, inverse):
    """x [..., rows, heads, dim] turned at pos [..., rows], in x's type; the
    angles in 64 bits."""
    n = freq.shape[0]
    ang = pos.double()[..., None, None] * freq
    cos = (torch.cos(ang) * magnitude).to(x.dtype)
    sin = (torch.sin(ang) * (-magnitude if inverse else magnitude)).to(x.dtype)
    y = x.clone()
    if layout == "half":
        x0, x1 = x[..., :n], x[..., span // 2:span // 2 + n]
        y[..., :n] = x0 * cos - x1 * sin
        y[..., span // 2:span // 2 + n] = x0 * sin + x1 * cos
    else:
        x0, x1 = x[..., 0:2 * n:2], x[..., 1:2 * n:2]
        y[..., 0:2 * n:2] = x0 * cos - x1 * sin
        y[..., 1:2 * n:2] = x0 * sin + x1 * cos
    return y


def _plain_append(pool, scales, x, s, block):
    """Codes of x [B, n, H, D] (float64) into the sequences' pages."""
    B_, n, H, D = x.shape
    L = s.lens.long()
    T = (n + block - 2) // block + 1                      # blocks that n tokens may touch
    pos = ((L // block)[:, None, None] + torch.arange(T, device=x.device)[:, None]) * block \
        + torch.arange(block, device=x.device)            # [B, T, block]
    old, new = pos < L[:, None, None], (pos >= L[:, None, None]) & (pos < (L + n)[:, None, None])
    touched = new.any(-1)                                 # [B, T]
    at = s.batch_index[:, None].expand(B_, T)
    page = s.table[at, (pos[..., 0] // PAGE).clamp(max=s.max_pages - 1)].long()
    page = torch.where(touched, page, torch.full_like(page, pool.shape[0] - 1))
    slot = pos % PAGE
    sub = slot[..., 0] // block
    slot = torch.where(touched[..., None], slot, torch.arange(block, device=x.device))
    sub = torch.where(touched, sub, torch.zeros_like(sub))
    have = pool[page[..., None], :, slot].double()        # [B, T, block, H, D]
    rows = x[at[..., None], (pos - L[:, None, None]).clamp(0, n - 1)]
    rows = torch.where(new[..., None, None], rows, torch.zeros_like(rows))
    was = scales[page, :, sub].double()                   # [B, T, H]
    has_old = (old[..., 0] & touched)[..., None]
    need = _pow2(_scale_exp(rows.abs().amax(dim=(2, 4))))
    now = torch.where(has_old, torch.maximum(was, need), need)
    now = torch.where(touched[..., None], now, was)
    kept = _e4m3(have * (was / now)[:, :, None, :, None])
    codes = torch.where(new[..., None, None], _e4m3(rows / now[:, :, None, :, None]),
                        torch.where((old & touched[..., None])[..., None, None], kept, have))
    pool[page[..., None], :, slot] = codes.float().to(E4M3)
    scales[page, :, sub] = now.float()


def _plain_attention(s, c):
    B_, n, Hq, D, H = c["batch"], c["n"], c["q_heads"], c["dim"], c["kv_heads"]
    G, block, count = Hq // H, c["block"], s.max_pages
    at = s.lens.long()[:, None] + torch.arange(n, device="cuda")                   # [B, n]
    q = _turn(s.q.float(), at, s.freq, c["layout"], D, 1.0, False).view(B_, n, H, G, D)
    first = torch.zeros_like(at[:, :1])
    if c["window"]:                                       # no more pages than the window touches
        first = (at[:, :1] - c["window"] + 1).clamp(min=0) // PAGE
        count = min(count, (c["window"] + n - 2) // PAGE + 2)
    T = count * PAGE
    page = first + torch.arange(count, device="cuda")                              # [B, count]
    j = (first * PAGE + torch.arange(T, device="cuda"))[:, None]                   # [B, 1, T]
    page = s.table.gather(1, page.clamp(max=s.max_pages - 1)).long()
    kscale = s.ks[page].transpose(1, 2).reshape(B_, H, -1).repeat_interleave(block, -1)
    vscale = s.vs[page].transpose(1, 2).reshape(B_, H, -1).repeat_interleave(block, -1)
    k = s.k[page].float().transpose(1, 2).reshape(B_, H, T, D)
    score = torch.einsum("bnhgd,bhtd->bhngt", q, k) * (kscale / math.sqrt(D))[:, :, None, None]
    del k
    seen = j <= at[..., None]
    if c["window"]:
        seen &= j > at[..., None] - c["window"]
    seen = seen[:, None, :, None]
    score = score.masked_fill(~seen, -math.inf)
    top = score.amax(-1, keepdim=True)
    p = torch.exp(score - top)
    del score
    total = p.sum(-1)
    p = p * vscale[:, :, None, None]
    written = (j < (s.lens + n)[:, None, None])[..., None]                         # [B, 1, T, 1]
    v = s.v[page].float().transpose(1, 2).reshape(B_, H, T, D).masked_fill_(~written, 0.0)
    out = torch.einsum("bhngt,bhtd->bnhgd", p, v) / total.permute(0, 2, 1, 3)[..., None]
    return out.reshape(B_, n, Hq, D).to(torch.bfloat16)


# ----------------------------------------------------------------------- run


def run(s):
    c = s.case
    if own:
        return _run_own(s, c)
    if c["kind"] == "rope":
        return _turn(s.x.float(), s.pos, s.freq, c["layout"], c["span"], c["magnitude"],
                     c["inverse"]).to(s.x.dtype)
    if c["kind"] == "append":
        # in 64 bits: a code next to a rounding border must not turn on the rotation's own rounding
        at = s.lens[:, None] + torch.arange(c["n"], device="cuda")
        k = _turn(s.k_new.double(), at, s.freq, c["layout"], c["dim"], 1.0, False)
        _plain_append(s.k, s.ks, k, s, c["block"])
        _plain_append(s.v, s.vs, s.v_new.double(), s, c["block"])
        return {"k": s.k, "v": s.v, "k_scale": s.ks, "v_scale": s.vs}
    return _plain_attention(s, c)


def _run_own(s, c):
    from speculative_decoding_verification_91_b200 import binding as B
    stream = torch.cuda.current_stream().cuda_stream
    if c["kind"] == "rope":
        B.spec_rope(s.rope, s.dtype, s.x, s.x.stride(0), s.x.stride(1), s.out, s.out.stride(0),
                    s.out.stride(1), s.pos, c["rows"], c["heads"], c["dim"], int(c["inverse"]), stream)
        return s.out
    if c["kind"] == "append":
        width = c["kv_heads"] * c["dim"]
        B.spec_qcache_write(s.cache, s.rope, s.table, s.max_pages, s.lens, c["batch"], c["n"], s.k_new,
                            width, s.v_new, width, s.ws.buf, s.ws.nbytes, stream)
        return {"k": s.k, "v": s.v, "k_scale": s.ks, "v_scale": s.vs}
    B.spec_qcache_attn(s.cache, s.rope, s.q, c["q_heads"] * c["dim"], c["q_heads"], s.table, s.max_pages,
                       s.lens, c["batch"], c["n"], 0, c["n"], c["window"], 0.0, s.out, s.ws.buf,
                       s.ws.nbytes, stream)
    return s.out


# --------------------------------------------------------------------- exact


def _e4m3_table():
    """The 127 values that are not negative, by code."""
    low = [m * 2.0 ** -9 for m in range(8)]
    return torch.tensor(low + [(8 + m) * 2.0 ** (e - 10) for e in range(1, 16) for m in range(8)][:119],
                        dtype=torch.float64, device="cuda")


def _nearest(x):
    """The e4m3 value next to each x, by looking it up between its neighbours."""
    t, a = _e4m3_table(), x.abs().clamp(max=448.0)
    hi = torch.searchsorted(t, a).clamp(max=126)
    lo = (hi - 1).clamp(min=0)
    up, down = t[hi] - a, a - t[lo]
    pick = torch.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)
    return t[pick].copysign(x)


def _turned(x, pos, freq, layout, span, magnitude, inverse):
    """The rotation as a product of complex numbers, in 64 bits."""
    n, x = freq.shape[0], x.double()
    i, j = ((torch.arange(n), torch.arange(n) + span // 2) if layout == "half"
            else (2 * torch.arange(n), 2 * torch.arange(n) + 1))
    w = torch.polar(torch.full((), float(magnitude), dtype=torch.float64, device="cuda"),
                    (-1.0 if inverse else 1.0) * pos.double()[..., None, None] * freq)
    z = torch.complex(x[..., i], x[..., j]) * w
    x[..., i], x[..., j] = z.real, z.imag
    return x


def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["kind"] == "rope":
        return torch.cat([_turned(s.x[i:i + 4096], s.pos[i:i + 4096], s.freq, c["layout"], c["span"],
                                  c["magnitude"], c["inverse"]) for i in range(0, c["rows"], 4096)])
    lens = s.lens.tolist()
    n, H, D, block = c["n"], c["kv_heads"], c["dim"], c["block"]
    if c["kind"] == "append":
        got = {}
        for name, pool, scales, new in (("k", s.k, s.ks, s.k_new), ("v", s.v, s.vs, s.v_new)):
            value, sc = pool.double(), scales.double()
            for b, L in enumerate(lens):
                x = new[b]
                pos = torch.arange(L, L + n, device="cuda")
                x = _turned(x, pos, s.freq, c["layout"], D, 1.0, False) if name == "k" else x.double()
                start = L
                while start < L + n:
                    first = start // block * block
                    end = min(first + block, L + n)
                    page, slot = int(s.table[b, first // PAGE]), first % PAGE
                    part = x[start - L:end - L].transpose(0, 1)                      # [H, rows, D]
                    top = part.abs().amax(dim=(1, 2))
                    e = torch.ceil(torch.log2(top / 448.0))
                    e = e + (448.0 * 2.0 ** e < top) - (448.0 * 2.0 ** (e - 1) >= top).double()
                    now = 2.0 ** e.clamp(MIN_EXP, MAX_EXP)
                    if start > first:                      # committed tokens share the block
                        was = sc[page, :, slot // block]
                        now = torch.maximum(was, now)
                        held = value[page, :, slot:slot + start - first]
                        value[page, :, slot:slot + start - first] = _nearest(held * (was / now)[:, None, None])
                    value[page, :, slot + start - first:slot + end - first] = _nearest(part / now[:, None, None])
                    sc[page, :, slot // block] = now
                    start = end
            got[name], got[name + "_scale"] = value, sc
        return got
    G, out = c["q_heads"] // H, []
    for b, L in enumerate(lens):
        end = L + n
        first = 0 if c["window"] == 0 else max(0, L - c["window"] + 1)
        j = torch.arange(first, end, device="cuda")
        page, slot = s.table[b, j // PAGE].long(), j % PAGE
        k = s.k[page, :, slot].double() * s.ks[page, :, slot // block].double()[..., None]   # [T, H, D]
        v = s.v[page, :, slot].double() * s.vs[page, :, slot // block].double()[..., None]
        pos = torch.arange(L, end, device="cuda")
        q = _turned(s.q[b], pos, s.freq, c["layout"], D, 1.0, False)
        ahead = j[None] > pos[:, None]
        if c["window"]:
            ahead |= j[None] <= pos[:, None] - c["window"]
        heads = []
        for h in range(c["q_heads"]):
            a = (q[:, h] @ k[:, h // G].T) / math.sqrt(D)
            heads.append(torch.softmax(a.masked_fill(ahead, -math.inf), -1) @ v[:, h // G])
        out.append(torch.stack(heads, 1))
    return torch.stack(out)

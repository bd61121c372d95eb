"""The rotary operator and the 8-bit cache on the GPU against their float64
definitions, and a run of them together."""
import math

import numpy as np
import pytest
import torch

from oracle import qcache as Q
from speculative_decoding_verification_91_b200 import binding as B

pytestmark = pytest.mark.gpu

HALF_BF16, HALF_FP16, HALF_FP32 = 2.0 ** -8, 2.0 ** -11, 2.0 ** -24   # half a step, relative
SCALINGS = {"plain": B.SPEC_ROPE_PLAIN, "linear": B.SPEC_ROPE_LINEAR, "raised": B.SPEC_ROPE_RAISED,
            "parts": B.SPEC_ROPE_PARTS}
NAN_CODE = 0x7F


def rope_config(span, n_rot, layout="half", scaling="plain", theta=10000.0, factor=1.0, original=0.0, magnitude=1.0):
    return B.SpecRope(B.SPEC_ROPE_HALF if layout == "half" else B.SPEC_ROPE_INTERLEAVED, span, n_rot,
                      SCALINGS[scaling], theta, factor, original, 1.0, 32.0, magnitude)


# ------------------------------------------------------------------ spec_rope

def rope_bound(x, want, dtype, positions, freq, magnitude):
    """Rounding of the result, of the products and the sum in binary32 and of the
    cosines: each product is off by half a step of itself, twice (its factor and
    itself), the sum by half a step; angles in binary64 add position * 2^-52."""
    half = {torch.bfloat16: HALF_BF16, torch.float16: HALF_FP16, torch.float32: HALF_FP32}[dtype]
    pair = magnitude * 2 * np.abs(x).max(-1, keepdims=True)      # |x0 c| + |x1 s| at most
    angle = np.abs(positions)[:, None, None] * (freq.max() if len(freq) else 0.0) * 2.0 ** -51
    tiny = 2.0 ** -25 if dtype == torch.float16 else 0.0         # half the least fp16 step
    return half * np.abs(want) * 1.001 + pair * (4 * HALF_FP32 + angle) + tiny


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("rows,heads,dim,span,n_rot,layout,scaling", [
    (1, 1, 2, 2, 1, "half", "plain"), (5, 16, 256, 256, 32, "half", "plain"),
    (3, 2, 104, 40, 20, "interleaved", "linear"), (33, 3, 128, 128, 64, "interleaved", "parts"),
    (7, 5, 80, 78, 39, "half", "raised"), (2, 4, 96, 96, 0, "half", "plain"), (130, 1, 256, 256, 128, "half", "parts"),
    (9, 8, 192, 64, 32, "interleaved", "raised"), (4, 2, 63, 62, 31, "half", "linear"),
    (6, 3, 64, 64, 32, "half", "plain"), (6, 3, 72, 48, 20, "half", "plain"),
    (5, 3, 72, 48, 21, "interleaved", "plain")])
def test_rope(dtype, rows, heads, dim, span, n_rot, layout, scaling):
    rng = np.random.default_rng(rows * 1000 + dim)
    kw = dict(scaling=scaling, factor=1.0 if scaling == "plain" else 8.0, original=8192.0)
    freq = Q.rope_frequencies(span, n_rot, 10000.0, **kw)
    x = torch.from_numpy(rng.normal(size=(rows, heads, dim))).to(dtype).cuda()
    pos = rng.integers(0, 131072, rows).astype(np.int32)
    pos[0] = 0 if rows == 1 else 131071
    if rows > 2:
        pos[2] = -1                                   # a padding row
    for inverse in (0, 1):
        out = torch.full_like(x, 7.0)
        cfg = rope_config(span, n_rot, layout, magnitude=1.25, **kw)
        B.spec_rope(cfg, {torch.bfloat16: B.SPEC_BF16, torch.float16: B.SPEC_FP16}.get(dtype, B.SPEC_FP32), x,
                    x.stride(0), x.stride(1), out, out.stride(0), out.stride(1), torch.from_numpy(pos).cuda(), rows,
                    heads, dim, inverse)
        xs = x.double().cpu().numpy()
        want = Q.rope(xs, pos, freq, layout, span, 1.25, bool(inverse))
        want[pos < 0] = 7.0
        got = out.double().cpu().numpy()
        assert np.all(np.abs(got - want) <= rope_bound(xs, want, dtype, pos, freq, 1.25))
        used = (np.r_[0:n_rot, span // 2:span // 2 + n_rot] if layout == "half" else np.arange(2 * n_rot))
        rest = np.setdiff1d(np.arange(dim), used)
        assert np.array_equal(got[pos >= 0][..., rest], xs[pos >= 0][..., rest])


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("shift", [0, 1, 8])
def test_rope_strided_in_place_and_transposed(layout, shift):
    """A slice of fused rows in place (its neighbours untouched), and [heads][rows] order."""
    rows, heads, dim = 11, 3, 64
    rng = np.random.default_rng(shift)
    fused = torch.from_numpy(rng.normal(size=(rows, heads * dim + 24))).to(torch.bfloat16).cuda()
    x = fused[:, shift:shift + heads * dim].unflatten(1, (heads, dim))
    before = fused.clone()
    pos = torch.arange(100, 100 + rows, dtype=torch.int32).cuda()
    freq = Q.rope_frequencies(64, 24)
    xs = x.double().cpu().numpy()
    want = Q.rope(xs, pos.cpu().numpy(), freq, layout, 64)
    bound = rope_bound(xs, want, torch.bfloat16, pos.cpu().numpy(), freq, 1.0)
    cfg = rope_config(64, 24, layout)
    turned = torch.zeros(heads, rows, dim, dtype=torch.bfloat16, device="cuda")
    B.spec_rope(cfg, B.SPEC_BF16, x, x.stride(0), x.stride(1), turned, turned.stride(1), turned.stride(0), pos, rows,
                heads, dim)
    assert np.all(np.abs(turned.transpose(0, 1).double().cpu().numpy() - want) <= bound)
    B.spec_rope(cfg, B.SPEC_BF16, x, x.stride(0), x.stride(1), x, x.stride(0), x.stride(1), pos, rows, heads, dim)
    assert np.all(np.abs(x.double().cpu().numpy() - want) <= bound)
    assert torch.equal(fused[:, :shift], before[:, :shift])
    assert torch.equal(fused[:, shift + heads * dim:], before[:, shift + heads * dim:])


@pytest.mark.parametrize("layout,rows,heads,dim,span,n_rot", [
    ("half", 150001, 1, 192, 64, 32), ("interleaved", 90001, 1, 192, 64, 27), ("half", 60001, 3, 128, 128, 20)])
def test_rope_of_many_rows(layout, rows, heads, dim, span, n_rot):
    """More rows than threads side by side: each thread takes several, with padding rows among them."""
    rng = np.random.default_rng(rows)
    freq = Q.rope_frequencies(span, n_rot)
    x = torch.randn(rows, heads, dim, device="cuda").to(torch.bfloat16)
    pos = rng.integers(0, 131072, rows).astype(np.int32)
    pos[rng.integers(0, rows, 50)] = -1
    pos[-1] = 131071
    out = torch.full_like(x, 7.0)
    B.spec_rope(rope_config(span, n_rot, layout), B.SPEC_BF16, x, x.stride(0), x.stride(1), out, out.stride(0),
                out.stride(1), torch.from_numpy(pos).cuda(), rows, heads, dim)
    xs, got = x.double().cpu().numpy(), out.double().cpu().numpy()
    want = Q.rope(xs, pos, freq, layout, span)
    want[pos < 0] = 7.0
    assert np.all(np.abs(got - want) <= rope_bound(xs, want, torch.bfloat16, pos, freq, 1.0))
    inplace = x.clone()
    B.spec_rope(rope_config(span, n_rot, layout), B.SPEC_BF16, inplace, x.stride(0), x.stride(1), inplace, x.stride(0),
                x.stride(1), torch.from_numpy(pos).cuda(), rows, heads, dim)
    there = torch.from_numpy(pos >= 0).cuda()
    assert torch.equal(inplace[there], out[there]) and torch.equal(inplace[~there], x[~there])


def test_rope_passes_infinities_and_nan_of_unturned_dims_and_repeats_a_head():
    """Dims that do not turn are copied whatever they hold; a head read by stride 0 is turned into each."""
    x = torch.ones(2, 1, 16, dtype=torch.float32, device="cuda")
    x[:, :, 12], x[:, :, 13] = math.inf, math.nan
    out = torch.zeros(2, 4, 16, device="cuda")
    pos = torch.tensor([3, 1 << 30], dtype=torch.int32, device="cuda")
    B.spec_rope(rope_config(8, 4), B.SPEC_FP32, x, 16, 0, out, 64, 16, pos, 2, 4, 16)
    assert torch.all(torch.isinf(out[..., 12])) and torch.all(torch.isnan(out[..., 13]))
    want = Q.rope(np.ones((2, 1, 8)), [3, 1 << 30], Q.rope_frequencies(8, 4))
    err = np.abs(out[..., :8].double().cpu().numpy() - want)
    assert err[0].max() <= 8 * HALF_FP32 and err[1].max() <= 8 * HALF_FP32 + 2.0 ** 30 * 2.0 ** -51


def test_rope_gradient_is_the_inverse():
    """d(sum(y w))/dx = the inverse of w, against differences of the operator itself in binary32."""
    rng = np.random.default_rng(5)
    x = torch.from_numpy(rng.normal(size=(2, 1, 8))).float().cuda()
    w = torch.from_numpy(rng.normal(size=(2, 1, 8))).float().cuda()
    pos = torch.tensor([5, 77], dtype=torch.int32, device="cuda")
    cfg = rope_config(8, 3, "interleaved", magnitude=1.5)

    def turn(v, inverse=0):
        out = torch.empty_like(v)
        B.spec_rope(cfg, B.SPEC_FP32, v, 8, 8, out, 8, 8, pos, 2, 1, 8, inverse)
        return out

    grad = turn(w, 1)
    h = 2.0 ** -4                       # the map is linear: only rounding limits the difference quotient
    for i in range(8):
        step = torch.zeros_like(x)
        step[..., i] = h
        diff = ((turn(x + step) - turn(x - step)).double() * w.double()).sum(-1) / (2 * h)
        scale = float(x.abs().max() + h) * 1.5 * 2 * float(w.abs().sum(-1).max())
        assert torch.all((diff - grad[..., i].double()).abs() <= 16 * scale * HALF_FP32 / h)


# -------------------------------------------------------------------- append

class Cache:
    """Pools of random stale codes (NaN codes among them) and a block table of random pages."""

    def __init__(self, seed, lens, room, H, D, block, split=0, spare=2):
        self.rng = np.random.default_rng(seed)
        self.H, self.D, self.block = H, D, block
        need = [(max(L, 0) + room - 1) // 64 + 1 for L in lens]
        self.max_pages = max(need)
        P = sum(need) + spare
        perm = self.rng.permutation(P)
        self.table = np.zeros((len(lens), self.max_pages), dtype=np.int32)
        at = 0
        for b, m in enumerate(need):
            self.table[b, :m] = perm[at:at + m]
            at += m
        shape, sshape = (P, H, 64, D), (P, H, 64 // block)
        self.k, self.v = (self.rng.integers(0, 256, shape).astype(np.uint8) for _ in range(2))
        self.k[:, :, ::5] = NAN_CODE
        self.v[:, :, ::7] = 0xFF
        self.ks, self.vs = (np.full(sshape, 2.0 ** -3, dtype=np.float32) for _ in range(2))
        self.lens = np.array(lens, dtype=np.int32)
        self.split = split
        self.d = {n: torch.from_numpy(getattr(self, n)).cuda() for n in ("k", "v", "ks", "vs", "table", "lens")}
        self.desc = B.SpecQCache(D, H, P, 64, block, split, self.d["k"].data_ptr(), self.d["v"].data_ptr(),
                                 self.d["ks"].data_ptr(), self.d["vs"].data_ptr())

    def fill(self, amplitude=1.0):
        """The oracle's append of a random context, on both sides."""
        for b, L in enumerate(self.lens):
            if L > 0:
                for c, s in ((self.k, self.ks), (self.v, self.vs)):
                    rows = self.rng.normal(size=(L, self.H, self.D)) * amplitude
                    rows *= 2.0 ** self.rng.integers(-2, 3, (1, self.H, 1))
                    Q.append(c, s, self.block, self.table[b], 0, rows)
        self.upload()

    def upload(self):
        for n in ("k", "v", "ks", "vs"):
            self.d[n].copy_(torch.from_numpy(getattr(self, n)))

    def same(self):
        for n in ("k", "v", "ks", "vs"):
            differ = int((self.d[n].cpu().numpy() != getattr(self, n)).sum())
            assert differ == 0, (n, differ)

    def rows(self, n, heads, amplitude=1.0):
        x = self.rng.normal(size=(len(self.lens), n, heads, self.D)) * amplitude
        return torch.from_numpy(x).to(torch.bfloat16).cuda()


def workspace(nbytes):
    ws = torch.empty(nbytes, dtype=torch.uint8, device="cuda")
    B.spec_workspace_init(ws, nbytes)
    return ws


def turned(x, L, freq, layout, span, magnitude=1.0, offset=0):
    """The device's bf16 rows [n, heads, D] turned in float64."""
    pos = np.arange(L + offset, L + offset + x.shape[0])
    return Q.rope(x.double().cpu().numpy(), pos, freq, layout, span, magnitude)


WRITES = [
    # lens, n, H, D, block, layout, span, n_rot
    ([0], 1, 1, 128, 16, "half", 128, 64), ([63, 64, 65, 0], 5, 2, 128, 16, "half", 128, 16),
    ([5, 70, 127], 17, 3, 256, 32, "interleaved", 256, 128), ([10, 60, 130], 200, 1, 128, 64, "interleaved", 64, 32),
    ([31, 48, 1000], 3, 8, 256, 64, "half", 256, 32), ([100], 300, 2, 256, 16, "half", 192, 96),
    ([15, 16, 17], 16, 2, 128, 16, "interleaved", 40, 3)]


@pytest.mark.parametrize("case", range(len(WRITES)))
@pytest.mark.parametrize("amplitude", [0.25, 40.0])
def test_write_stores_the_nearest_codes(case, amplitude):
    """Codes and scales exactly; every other byte of the pools as it was.  40: the
    committed codes of partly filled blocks are rewritten for a larger scale."""
    lens, n, H, D, block, layout, span, n_rot = WRITES[case]
    c = Cache(case, lens, n, H, D, block)
    c.fill()
    k, v = c.rows(n, H, amplitude), c.rows(n, H, amplitude)
    freq = Q.rope_frequencies(span, n_rot)
    for b, L in enumerate(lens):
        Q.append(c.k, c.ks, block, c.table[b], L, turned(k[b], L, freq, layout, span, 1.125))
        Q.append(c.v, c.vs, block, c.table[b], L, v[b].double().cpu().numpy())
    ws = workspace(B.spec_qcache_write_workspace_bytes(c.desc, len(lens), n))
    cfg = rope_config(span, n_rot, layout, magnitude=1.125)
    for _ in range(2):                                  # storing the same rows again changes nothing
        B.spec_qcache_write(c.desc, cfg, c.d["table"], c.max_pages, c.d["lens"], len(lens), n, k, H * D, v, H * D,
                            ws, ws.numel())
        assert B.spec_read_device_status(ws, ws.numel()) == 0
        c.same()


def test_write_strided_rows_without_rotation():
    """Keys and values as slices of fused rows; extreme magnitudes; a block of zeros."""
    H, D, n = 2, 128, 40
    c = Cache(3, [7, 90], n, H, D, 32)
    c.fill()
    fused = torch.randn(2 * n, 3 * H * D, device="cuda").to(torch.bfloat16)
    fused[:10] *= 2.0 ** -120
    fused[10:20] *= 2.0 ** 110
    fused[n:] = 0
    fused[20:24, ::3] *= 2.0 ** -20
    k, v = fused[:, H * D:2 * H * D], fused[:, 2 * H * D:]
    for b, L in enumerate(c.lens):
        Q.append(c.k, c.ks, 32, c.table[b], L, k[b * n:(b + 1) * n].reshape(n, H, D).double().cpu().numpy())
        Q.append(c.v, c.vs, 32, c.table[b], L, v[b * n:(b + 1) * n].reshape(n, H, D).double().cpu().numpy())
    ws = workspace(4096)
    B.spec_qcache_write(c.desc, None, c.d["table"], c.max_pages, c.d["lens"], 2, n, k, k.stride(0), v, v.stride(0),
                        ws, 4096)
    c.same()


def test_write_flags_what_it_cannot_store():
    """Bad lengths and pages leave the pools alone; infinities and NaN are flagged and kept out of the scale."""
    H, D, n, block = 1, 128, 4, 16
    c = Cache(4, [3, -1, 120, 20], n, H, D, block)
    c.max_pages = 2
    table = np.ascontiguousarray(c.table[:, :2])
    table[3, 0] = 10 ** 6
    c.d["table"] = torch.from_numpy(table).cuda()
    c.lens[2] = 125                                     # 125 + 4 > 2 pages
    c.d["lens"] = torch.from_numpy(c.lens).cuda()
    k, v = c.rows(n, H), c.rows(n, H)
    v[0, 1, 0, 5], v[0, 2, 0, 6], v[0, 3, 0, 7] = math.inf, -math.inf, math.nan
    Q.append(c.k, c.ks, block, table[0], 3, k[0].double().cpu().numpy())
    rows = v[0].double().cpu().numpy()
    Q.append(c.v, c.vs, block, table[0], 3, rows)
    ws = workspace(4096)
    B.spec_qcache_write(c.desc, None, c.d["table"], 2, c.d["lens"], 4, n, k, D, v, D, ws, 4096)
    assert B.spec_read_device_status(ws, 4096) == B.SPEC_DEV_BAD_LENGTH | B.SPEC_DEV_BAD_PAGE | B.SPEC_DEV_NONFINITE
    c.same()


@pytest.mark.parametrize("ties", [1.0, 0.02])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_write_of_keys_next_to_rounding_borders(ties, layout):
    """Angles of 10^-9: keys that lie half way between two codes turn just off the border, and
    the side decides.  All of them, and a few."""
    H, D, n, block = 2, 256, 70, 64
    c = Cache(5, [64, 3], n, H, D, block)
    c.fill()
    shape = (2, n, H, D)
    border = (1 + (2 * c.rng.integers(0, 8, shape) + 1) / 16) * 2.0 ** c.rng.integers(-2, 3, shape)
    x = np.where(c.rng.random(shape) < ties, border * c.rng.choice([-1.0, 1.0], shape), c.rng.normal(size=shape))
    k, v = torch.from_numpy(x).to(torch.bfloat16).cuda(), c.rows(n, H)
    kw = dict(scaling="linear", factor=1e12)
    freq = Q.rope_frequencies(256, 128, 10000.0, **kw)
    for b, L in enumerate(c.lens):
        Q.append(c.k, c.ks, block, c.table[b], L, turned(k[b], L, freq, layout, 256))
        Q.append(c.v, c.vs, block, c.table[b], L, v[b].double().cpu().numpy())
    ws = workspace(B.spec_qcache_write_workspace_bytes(c.desc, 2, n))
    B.spec_qcache_write(c.desc, rope_config(256, 128, layout, **kw), c.d["table"], c.max_pages, c.d["lens"], 2, n, k,
                        H * D, v, H * D, ws, ws.numel())
    c.same()


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("side", [-1, 0, 1])
def test_write_of_blocks_whose_scale_turns_on_one_entry(layout, side):
    """The largest key within 10^-7 of 448 x a power of two: just below (the smaller scale), on it
    (a dim that passes through), or just above (the larger one)."""
    H, D, n, block, n_rot = 3, 128, 40, 16, 32
    c = Cache(6, [20, 0], n, H, D, block)
    c.fill()
    freq = Q.rope_frequencies(128, n_rot)
    x = torch.from_numpy(c.rng.normal(size=(2, n, H, D)) * 0.2).clamp(-0.8, 0.8).to(torch.bfloat16)
    if side == 0:
        x[..., 60] = 1.75                               # neither turned half nor pair
    else:
        # the pair of bf16 numbers that turns closest to 1.75 from that side, at each position and pair
        one = (1 + np.arange(128) / 128)
        v = np.concatenate([one / 2, one])
        for b, L in enumerate(c.lens):
            for i in range(0, n, 3):
                j = int(c.rng.integers(0, n_rot))
                angle = (L + i) * freq[j]
                y = v[:, None] * math.cos(angle) - np.concatenate([-v, v])[None] * math.sin(angle)
                off = (np.abs(y) - 1.75) * side
                other = v[:, None] * math.sin(angle) + np.concatenate([-v, v])[None] * math.cos(angle)
                off[(off <= 0) | (np.abs(other) > 1.7)] = np.inf
                a, w = np.unravel_index(np.argmin(off), off.shape)
                d0, d1 = (j, j + 64) if layout == "half" else (2 * j, 2 * j + 1)
                x[b, i, i % H, d0], x[b, i, i % H, d1] = float(v[a]), float(np.concatenate([-v, v])[w])
    k, v = x.cuda(), c.rows(n, H)
    for b, L in enumerate(c.lens):
        Q.append(c.k, c.ks, block, c.table[b], L, turned(k[b], L, freq, layout, 128))
        Q.append(c.v, c.vs, block, c.table[b], L, v[b].double().cpu().numpy())
    ws = workspace(B.spec_qcache_write_workspace_bytes(c.desc, 2, n))
    B.spec_qcache_write(c.desc, rope_config(128, n_rot, layout), c.d["table"], c.max_pages, c.d["lens"], 2, n, k, H * D,
                        v, H * D, ws, ws.numel())
    c.same()


# ----------------------------------------------------------------- attention

def attention_bound(out, spread, mass, tail, rows=1):
    """Half a bf16 step of the result; the queries' two codes keep each to 2^-8 of
    itself, which moves score j by at most 2^-8 e_j and so its weight by that
    share (spread); each weight's two codes are off by 2^-8 of it (mass) and, the
    smallest, by 2^-19 of the largest weight (prompt chunks of more than 64 rows a KV
    head: 2^-15), each key's values up to the block's largest (tail); sums and
    exponentials in binary32 cost 2^-16 of the mass.

    2^-19: a weight w (1 for the row's reference, which the largest weight is not
    below) is coded as 32 w = w0 + w1 / 16.  The least step of e4m3 is 2^-9, so w1
    is off by up to 2^-10, 32 w by 2^-14 and w by 2^-19.  2^-15: there 32 w = w0 + w1,
    so 32 w is off by 2^-10.  2^-8: 32 w in binary16 is
    off by 2^-11 of itself, w0 leaves at most 2^-4 of the power of two below 32 w,
    and w1 half a step of the 2^-5 below that, 2^-9: 2^-9 + 2^-11 < 2^-8."""
    return (HALF_BF16 * np.abs(out) + 1.1 * 2.0 ** -8 * spread + (2.0 ** -8 + 2.0 ** -16) * mass
            + (2.0 ** -15 if rows > 64 else 2.0 ** -19) * tail + 1e-30)


def check_attention(c, q, got, cfg_args, q_offset, extra, window, scale=None, table=None):
    freq, layout, span, magnitude = cfg_args
    table = c.table if table is None else table
    worst = 0.0
    n, heads = q.shape[1:3]
    rows = n * heads // c.H if n > B.SPEC_MAX_K + 1 else 1
    for b, L in enumerate(c.lens):
        x = turned(q[b], L, freq, layout, span, magnitude, q_offset)
        want, spread, mass, tail = Q.attention(x, c.k, c.ks, c.v, c.vs, c.block, table[b], L, q_offset, extra,
                                               window, scale)
        bound = attention_bound(want, spread, mass, tail, rows)
        err = np.abs(got[b].double().cpu().numpy() - want)
        assert np.all(err <= bound), (b, float((err / bound).max()))
        # the typical error is far smaller than the worst case: the result's own rounding and little more
        norm = np.linalg.norm(want)
        assert np.linalg.norm(err) <= 2.0 ** -8 * norm + 1e-30
        worst = max(worst, float((err / bound).max()))
    return worst


ATTNS = [
    # lens, n, Hq, H, D, block, split, window, layout, span, n_rot
    ([0], 1, 1, 1, 128, 64, 128, 0, "half", 128, 64),
    ([256], 5, 8, 1, 128, 64, 256, 0, "half", 128, 64),
    ([0, 1, 63, 64, 65, 127, 128, 129], 1, 4, 2, 128, 16, 128, 0, "half", 128, 16),
    ([300, 7, 1025], 5, 16, 8, 256, 64, 256, 0, "half", 256, 32),
    ([900, 130, 2500], 5, 32, 4, 256, 32, 1024, 0, "interleaved", 256, 128),
    ([700], 9, 8, 2, 256, 64, 128, 0, "half", 64, 32),
    ([500, 3, 64, 1000], 4, 4, 2, 256, 16, 256, 100, "half", 256, 128),
    ([500, 90], 6, 6, 2, 128, 32, 128, 1, "half", 128, 64),
    ([400, 77], 17, 16, 1, 128, 64, 256, 0, "half", 128, 64),
    ([200, 1], 17, 14, 2, 256, 64, 128, 70, "interleaved", 128, 64),
    ([0, 130], 100, 4, 2, 128, 64, 128, 0, "half", 128, 64),
    ([64], 256, 8, 2, 256, 16, 1024, 0, "half", 256, 32),
    ([200], 150, 3, 1, 256, 64, 128, 50, "half", 256, 128),
    ([5000], 3, 10, 2, 128, 64, 4096, 0, "half", 128, 64)]


@pytest.mark.parametrize("case", range(len(ATTNS)))
def test_attention(case):
    lens, n, Hq, H, D, block, split, window, layout, span, n_rot = ATTNS[case]
    c = Cache(case, lens, n, H, D, block, split)
    c.fill()
    k, v, q = c.rows(n, H, 3.0), c.rows(n, H), c.rows(n, Hq, 1.5)
    freq = Q.rope_frequencies(span, n_rot)
    cfg = rope_config(span, n_rot, layout, magnitude=1.125)
    ws = workspace(B.spec_qcache_attn_workspace_bytes(c.desc, Hq, len(lens), n, c.max_pages, window))
    out = torch.full((len(lens) + 1, n, Hq, D), 3.0, dtype=torch.bfloat16, device="cuda")
    B.spec_qcache_verify_attn(c.desc, cfg, q, Hq * D, Hq, k, H * D, v, H * D, c.d["table"], c.max_pages, c.d["lens"],
                              len(lens), n, window, 0.0, out, ws, ws.numel())
    assert B.spec_read_device_status(ws, ws.numel()) == 0
    for b, L in enumerate(lens):
        Q.append(c.k, c.ks, block, c.table[b], L, turned(k[b], L, freq, layout, span, 1.125))
        Q.append(c.v, c.vs, block, c.table[b], L, v[b].double().cpu().numpy())
    c.same()
    assert torch.all(out[-1] == 3.0)                    # behind the last sequence
    check_attention(c, q, out, (freq, layout, span, 1.125), 0, n, window)
    # the two calls it stands for, on a workspace that holds something else, give the same bits
    two = torch.empty_like(out)
    ws.random_(0, 256)
    B.spec_workspace_init(ws, 4096)
    B.spec_qcache_attn(c.desc, cfg, q, Hq * D, Hq, c.d["table"], c.max_pages, c.d["lens"], len(lens), n, 0, n, window,
                       0.0, two, ws, ws.numel())
    assert torch.equal(out[:-1], two[:-1])


@pytest.mark.parametrize("q_offset,window", [(0, 0), (3, 0), (3, 4), (7, 5), (0, 3)])
def test_attention_of_a_drafter(q_offset, window):
    """Rows past the committed cache; a short window may leave them without a key: zeros."""
    c = Cache(11, [40, 0, 70, 1], 1, 2, 128, 16, 128)
    c.fill()
    q = c.rows(3, 4)
    ws = workspace(B.spec_qcache_attn_workspace_bytes(c.desc, 4, 4, 3, c.max_pages, window))
    out = torch.full((4, 3, 4, 128), 3.0, dtype=torch.bfloat16, device="cuda")
    freq = Q.rope_frequencies(128, 64)
    B.spec_qcache_attn(c.desc, rope_config(128, 64), q, 512, 4, c.d["table"], c.max_pages, c.d["lens"], 4, 3,
                       q_offset, 0, window, 0.11, out, ws, ws.numel())
    check_attention(c, q, out, (freq, "half", 128, 1.0), q_offset, 0, window, float(np.float32(0.11)))
    assert torch.all(out[1] == 0)
    if window and q_offset >= window:
        assert torch.all(out == 0)


def test_attention_long_tail_beside_a_dominant_key():
    """One key far above thousands that together weigh as much: small weights must not be lost."""
    D, L = 128, 4000
    c = Cache(12, [L], 1, 1, D, 64, 4096)
    k = np.zeros((L, 1, D))
    k[0, 0, 0] = 8.0
    v = np.full((L, 1, D), 1.0)
    v[0] = -1.0
    for rows, pool, s in ((k, c.k, c.ks), (v, c.v, c.vs)):
        Q.append(pool, s, 64, c.table[0], 0, rows)
    c.upload()
    q = torch.zeros(1, 1, 1, D, dtype=torch.bfloat16, device="cuda")
    ws = workspace(B.spec_qcache_attn_workspace_bytes(c.desc, 1, 1, 1, c.max_pages, 0))
    out = torch.empty_like(q)
    for lead in (2.0, 8.3, 11.0):                       # exp(8.3) = 4000
        q[..., 0] = 1.0
        B.spec_qcache_attn(c.desc, None, q, D, 1, c.d["table"], c.max_pages, c.d["lens"], 1, 1, 0, 0, 0, lead / 8.0,
                           out, ws, ws.numel())
        w = math.exp(8.0 * float(np.float32(lead / 8.0)))
        want = ((L - 1) - w) / ((L - 1) + w)
        # weights at 2^-16 of the largest are still 2^5 times the smallest step: half a step each is 2^-6 of them
        bound = HALF_BF16 * abs(want) + 2.0 ** -8 + (2.0 ** -6 if lead > 9 else 0.0)
        assert abs(float(out[0, 0, 0, 3]) - want) <= bound


def test_attention_blocks_of_very_different_scales():
    """Values of one block 2^40 times another's: the weight decides, not the scale."""
    D, L, H = 128, 256, 2
    c = Cache(13, [L], 1, H, D, 64, 128)
    k, v = c.rng.normal(size=(L, H, D)), c.rng.normal(size=(L, H, D))
    v[:64] *= 2.0 ** 40
    v[192:] = 0.0
    k[:64, 0] = 0.0
    k[:64, 0, 0] = -300.0                               # head 0: the large values carry no weight
    k[64:, 0, 0] = 3.0
    for rows, pool, s in ((k, c.k, c.ks), (v, c.v, c.vs)):
        Q.append(pool, s, 64, c.table[0], 0, rows)
    c.upload()
    q = c.rows(1, H)
    q[..., 0] = 8.0
    ws = workspace(B.spec_qcache_attn_workspace_bytes(c.desc, H, 1, 1, c.max_pages, 0))
    out = torch.empty_like(q)
    B.spec_qcache_attn(c.desc, None, q, H * D, H, c.d["table"], c.max_pages, c.d["lens"], 1, 1, 0, 0, 0, 0.0, out, ws,
                       ws.numel())
    check_attention(c, q, out, (Q.rope_frequencies(2, 0), "half", 2, 1.0), 0, 0, 0)


def test_attention_flags_and_contains_bad_rows():
    """A NaN query row is NaN and no other; a page id outside the pool is left out; bad lengths give zeros."""
    c = Cache(14, [200, 150, 100, 90], 2, 2, 128, 16, 128)
    c.fill()
    q = c.rows(2, 4)
    q[0, 1, 2, 9], q[1, 0, 0, 3] = math.nan, math.inf
    table = c.table.copy()
    table[1, 1] = c.k.shape[0]                          # keys 64..127 of sequence 1
    table[0, 0] = -5
    c.d["table"] = torch.from_numpy(table).cuda()
    c.lens[2], c.lens[3] = -3, 10 ** 8
    c.d["lens"] = torch.from_numpy(c.lens).cuda()
    ws = workspace(B.spec_qcache_attn_workspace_bytes(c.desc, 4, 4, 2, c.max_pages, 0))
    out = torch.full((4, 2, 4, 128), 3.0, dtype=torch.bfloat16, device="cuda")
    B.spec_qcache_attn(c.desc, None, q, 512, 4, c.d["table"], c.max_pages, c.d["lens"], 4, 2, 0, 0, 0, 0.0, out, ws,
                       ws.numel())
    assert B.spec_read_device_status(ws, ws.numel()) == B.SPEC_DEV_BAD_LENGTH | B.SPEC_DEV_BAD_PAGE
    assert torch.all(torch.isnan(out[0, 1, 2])) and torch.all(torch.isnan(out[1, 0, 0]))
    assert torch.isnan(out).sum() == 2 * 128 and torch.all(out[2:] == 0)
    q[0, 1, 2], q[1, 0, 0] = 0.0, 0.0
    out2 = torch.empty_like(out)
    B.spec_qcache_attn(c.desc, None, q, 512, 4, c.d["table"], c.max_pages, c.d["lens"], 4, 2, 0, 0, 0, 0.0, out2, ws,
                       ws.numel())
    c.lens[2:] = 0
    check_attention(c, q, out2, (Q.rope_frequencies(2, 0), "half", 2, 1.0), 0, 0, 0, table=table)


def test_rows_do_not_depend_on_the_rows_beside_them():
    """One step of 17 rows and 17 steps of one row, alone and in a batch, give the same bits."""
    for window in (0, 33):
        c = Cache(15, [300, 77], 17, 2, 256, 64, 128)
        c.fill()
        k, v, q = c.rows(17, 2), c.rows(17, 2), c.rows(17, 8)
        ws = workspace(B.spec_qcache_attn_workspace_bytes(c.desc, 8, 2, 17, c.max_pages, window))
        cfg = rope_config(256, 32)
        out = torch.empty_like(q)
        B.spec_qcache_verify_attn(c.desc, cfg, q, 2048, 8, k, 512, v, 512, c.d["table"], c.max_pages, c.d["lens"], 2,
                                  17, window, 0.0, out, ws, ws.numel())
        for i in (0, 4, 16):
            one = torch.empty(2, 1, 8, 256, dtype=torch.bfloat16, device="cuda")
            at, table, row = c.d["lens"] + i, c.d["table"], q[:, i].contiguous()
            B.spec_qcache_attn(c.desc, cfg, row, 2048, 8, table, c.max_pages, at, 2, 1, 0, 1, window, 0.0, one, ws,
                               ws.numel())
            assert torch.equal(one[:, 0], out[:, i]), (window, i)
            B.spec_qcache_attn(c.desc, cfg, row[1:], 2048, 8, table[1:], c.max_pages, at[1:], 1, 1, 0, 1, window, 0.0,
                               one, ws, ws.numel())
            assert torch.equal(one[0, 0], out[1, i]), (window, i)


def attend(c, cfg, q, Hq, n, window=0, stream=None, extra=None, table=None, ws=None, lens=None):
    """spec_qcache_attn of n cached tokens on a workspace of its own; the result."""
    table, lens = c.d["table"] if table is None else table, c.d["lens"] if lens is None else lens
    batch, max_pages = table.shape
    if ws is None:
        ws = workspace(B.spec_qcache_attn_workspace_bytes(c.desc, Hq, batch, n, max_pages, window))
    out = torch.empty_like(q)
    B.spec_qcache_attn(c.desc, cfg, q, Hq * c.D, Hq, table, max_pages, lens, batch, n, 0, n if extra is None else extra,
                       window, 0.0, out, ws, ws.numel(), stream)
    return out


@pytest.mark.parametrize("window", [0, 60])
def test_attention_of_many_ragged_sequences(window):
    """More sequences than a warp has lanes, most of them short, some empty."""
    lens = [int(x) for x in np.random.default_rng(17).integers(0, 150, 75)]
    lens[3], lens[40], lens[70], lens[74] = 0, 700, 0, 128
    c = Cache(17, lens, 1, 2, 128, 32, 128)
    c.fill()
    q = c.rows(2, 6)
    out = attend(c, None, q, 6, 2, window, extra=0)
    check_attention(c, q, out, (Q.rope_frequencies(2, 0), "half", 2, 1.0), 0, 0, window)


def test_results_depend_neither_on_the_table_s_width_nor_on_who_shares_a_page():
    """One split and its join: the same bits from a wider table; a prefix shared by two sequences."""
    c = Cache(18, [100, 100], 4, 2, 256, 16, 128)
    c.fill()
    c.d["lens"] -= 4                                    # the rows are the cache's last four
    cfg, q = rope_config(256, 128), c.rows(4, 8)
    narrow = attend(c, cfg, q, 8, 4)
    wide = torch.full((2, 64), -1, dtype=torch.int32, device="cuda")
    wide[:, :c.max_pages] = c.d["table"]
    assert torch.equal(attend(c, cfg, q, 8, 4, table=wide), narrow)
    shared = c.d["table"].clone()
    shared[1] = shared[0]
    q[1] = q[0]
    both = attend(c, cfg, q, 8, 4, table=shared)
    assert torch.equal(both[0], narrow[0]) and torch.equal(both[1], narrow[0])


def test_pools_past_four_gigabytes():
    """Pages whose offsets in bytes pass 32 bits: append and attention."""
    lens, n, Hq, H, D, block = [200, 61], 5, 16, 8, 256, 32
    c = Cache(19, lens, n, H, D, block, 128)
    c.fill()
    P = c.k.shape[0]
    N = 2 ** 32 // (H * 64 * D) + 500
    big = {m: torch.zeros((N, H, 64, D), dtype=torch.uint8, device="cuda") for m in ("k", "v")}
    big.update({m: torch.zeros((N, H, 64 // block), dtype=torch.float32, device="cuda") for m in ("ks", "vs")})
    for m, t in big.items():
        t[N - P:] = c.d[m]
        c.d[m] = t[N - P:]
    c.d["table"] += N - P
    c.desc = B.SpecQCache(D, H, N, 64, block, 128, *(big[m].data_ptr() for m in ("k", "v", "ks", "vs")))
    k, v, q = c.rows(n, H), c.rows(n, H), c.rows(n, Hq)
    freq, cfg = Q.rope_frequencies(256, 64), rope_config(256, 64)
    ws = workspace(B.spec_qcache_attn_workspace_bytes(c.desc, Hq, 2, n, c.max_pages, 0))
    out = torch.empty_like(q)
    B.spec_qcache_verify_attn(c.desc, cfg, q, Hq * D, Hq, k, H * D, v, H * D, c.d["table"], c.max_pages, c.d["lens"], 2,
                              n, 0, 0.0, out, ws, ws.numel())
    assert B.spec_read_device_status(ws, ws.numel()) == 0
    for b, L in enumerate(lens):
        Q.append(c.k, c.ks, block, c.table[b], L, turned(k[b], L, freq, "half", 256))
        Q.append(c.v, c.vs, block, c.table[b], L, v[b].double().cpu().numpy())
    c.same()
    check_attention(c, q, out, (freq, "half", 256, 1.0), 0, n, 0)
    assert not big["k"][:N - P].any() and not big["v"][:N - P].any()


def test_two_calls_at_once_and_a_workspace_used_again():
    """Calls on two streams with workspaces of their own; then different shapes in turn on one."""
    c = Cache(20, [700, 300, 40], 20, 2, 128, 16, 128)
    c.fill()
    c.d["lens"] -= 20
    cfg = rope_config(128, 64)
    qs = [c.rows(n, 8) for n in (1, 5, 17, 20)]
    want = [attend(c, cfg, q, 8, q.shape[1]) for q in qs]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    spaces = [workspace(B.spec_qcache_attn_workspace_bytes(c.desc, 8, 3, 20, c.max_pages, 0)) for _ in streams]
    torch.cuda.synchronize()
    got = []
    for i in range(12):
        with torch.cuda.stream(streams[i % 2]):
            got.append(attend(c, cfg, qs[i % 4], 8, qs[i % 4].shape[1], stream=streams[i % 2], ws=spaces[i % 2]))
    torch.cuda.synchronize()
    assert all(torch.equal(g, want[i % 4]) for i, g in enumerate(got))
    for i in (3, 0, 2, 1, 3):
        assert torch.equal(attend(c, cfg, qs[i], 8, qs[i].shape[1], ws=spaces[0]), want[i])
    assert all(B.spec_read_device_status(ws, ws.numel()) == 0 for ws in spaces)


def test_few_and_many_rows_give_the_same_bits():
    """Steps of one and of five rows take row blocks of different heights: 500,000 results, to the bit."""
    B_, Hq, H, D = 16, 32, 4, 256
    c = Cache(21, list(range(1200, 1200 + B_)), 5, H, D, 64, 512)
    c.fill()
    q = c.rows(5, Hq)
    five = attend(c, None, q, Hq, 5, extra=0)
    for i in range(5):
        # (q_offset i and no new key: the row sees what it saw among the five)
        out = torch.empty(B_, 1, Hq, D, dtype=torch.bfloat16, device="cuda")
        row = q[:, i].contiguous()
        ws = workspace(B.spec_qcache_attn_workspace_bytes(c.desc, Hq, B_, 1, c.max_pages, 0))
        B.spec_qcache_attn(c.desc, None, row, Hq * D, Hq, c.d["table"], c.max_pages, c.d["lens"], B_, 1, i, 0, 0, 0.0,
                           out, ws, ws.numel())
        assert torch.equal(out[:, 0], five[:, i]), i


# ------------------------------------------------------------------ together

def test_a_decode_loop_on_another_stream_and_in_a_graph():
    """Prompt chunk, verify steps with drafts rolled back, on a stream of their own; then one
    step captured into a graph and replayed with new rows: each as the definition has it."""
    H, Hq, D, block = 2, 4, 128, 16
    c = Cache(16, [0, 0], 200, H, D, block, 128)
    freq = Q.rope_frequencies(128, 64, scaling="parts", factor=4.0, original=64)
    cfg = rope_config(128, 64, scaling="parts", factor=4.0, original=64)
    ws = workspace(B.spec_qcache_attn_workspace_bytes(c.desc, Hq, 2, 100, c.max_pages, 0))
    torch.cuda.synchronize()
    side = torch.cuda.Stream()

    def step(n, q, k, v, out, stream):
        B.spec_qcache_verify_attn(c.desc, cfg, q, Hq * D, Hq, k, H * D, v, H * D, c.d["table"], c.max_pages,
                                  c.d["lens"], 2, n, 0, 0.0, out, ws, ws.numel(), stream)

    def expect(n, q, k, v, out):
        for b, L in enumerate(c.lens):
            Q.append(c.k, c.ks, block, c.table[b], L, turned(k[b], L, freq, "half", 128))
            Q.append(c.v, c.vs, block, c.table[b], L, v[b].double().cpu().numpy())
        c.same()
        check_attention(c, q, out, (freq, "half", 128, 1.0), 0, n, 0)

    for n, kept in ((90, [90, 50]), (5, [1, 5]), (5, [3, 2]), (1, [1, 1]), (9, [2, 9])):
        q, k, v = c.rows(n, Hq), c.rows(n, H, 2.0), c.rows(n, H, 2.0)
        out = torch.empty_like(q)
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            step(n, q, k, v, out, side)
        side.synchronize()
        expect(n, q, k, v, out)
        c.lens += np.array(kept, dtype=np.int32)
        c.d["lens"] += torch.tensor(kept, dtype=torch.int32, device="cuda")
    q, k, v = c.rows(3, Hq), c.rows(3, H), c.rows(3, H)
    out = torch.empty_like(q)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        step(3, q, k, v, out, torch.cuda.current_stream())
    for _ in range(2):
        for t, heads in ((q, Hq), (k, H), (v, H)):
            t.copy_(c.rows(3, heads, 1.5))
        graph.replay()
        torch.cuda.synchronize()
        expect(3, q, k, v, out)
        c.lens += 2
        c.d["lens"] += 2
    assert B.spec_read_device_status(ws, ws.numel()) == 0

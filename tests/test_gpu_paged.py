"""The paged 8-bit cache on the GPU against the fp64 oracle: append (bit for bit) and attention.

Tolerance of an attention output, for weights p and values v: one rounding of the result (half a step of its type);
one of the weights for bf16 (2^-11 each; two f16 parts, 2^-21, for fp16); the logits' errors e, absolute, twice (in the
weight and in the sum): 32-bit sums of d products and a few scalings, e <= (d + 16) 2^-24 sum |q| |k| scale, and the
fast exponential's 2^-22; sums of the weights and of the outputs in 32 bits, random in sign, 2^-20:
|o - ref| <= half |ref| + (w + 2 e + 2^-19) sum p |v| + floors.  The floors are absolute: an fp16 result below 2^-14 is
rounded to multiples of 2^-24 (half a step: 2^-25; a bf16 result's smallest step is 2^-133); a weight is stored as f16
2^15 times itself, in units of the largest value scale (a power of two below twice it), so one below 2^-29 of them is
rounded to multiples of 2^-39 (half a step: 2^-40): 2^-39 max(vs) sum |c| over the visible tokens.
"""

import math

import numpy as np
import pytest

from oracle import paged as OP

pytestmark = pytest.mark.gpu

HALF = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11}
FLOOR = {"bf16": 2.0 ** -134, "fp16": 2.0 ** -25}
WEIGHT = {"bf16": 2.0 ** -11, "fp16": 2.0 ** -21}


def f64(t):
    return t.double().cpu().numpy()


class Paged:
    """A cache of shuffled pages with random histories; unused codes are e4m3's NaN (int8: -128) and unused scales NaN."""

    def __init__(self, lens, page=16, Hkv=2, d=64, kind="e4m3", dtype="bf16", seed=0, spare=3, spread=1.0):
        import torch
        import hybrid_sparse_linear_decode_b200 as H
        rng = np.random.default_rng(seed)
        self.rng, self.lens, self.page, self.Hkv, self.d, self.kind, self.dtype = rng, list(lens), page, Hkv, d, kind, dtype
        need = [max(1, -(-n // page)) for n in lens]
        n = sum(need) + spare
        order = rng.permutation(n)
        self.table = np.full((len(lens), max(need) + 1), -1, np.int32)
        at = 0
        for b, m in enumerate(need):
            self.table[b, :m] = order[at:at + m]
            at += m
        junk = 0x7f if kind == "e4m3" else 0x80
        self.codes = {x: np.full((n, Hkv, page, d), junk, np.uint8) for x in "kv"}
        self.scales = {x: np.full((n, Hkv), np.nan, np.float32) for x in "kv"}
        for b, m in enumerate(lens):
            for lo in range(0, m, page):
                p, c = self.table[b, lo // page], min(page, m - lo)
                for x in "kv":
                    s = np.exp2(np.round(rng.uniform(-6 * spread, 2 * spread, Hkv))) if kind == "e4m3" else \
                        np.exp(rng.uniform(-5 * spread, -2 * spread, Hkv))
                    self.scales[x][p] = s.astype(np.float32)
                    y = rng.standard_normal((Hkv, c, d)) * (100 if kind == "e4m3" else 40)
                    self.codes[x][p, :, :c] = OP.encode(y, kind)
        self.torch, self.dev = torch, torch.device("cuda")
        tt = {"e4m3": torch.float8_e4m3fn, "int8": torch.int8}[kind]
        self.t = {x: torch.from_numpy(self.codes[x].view(np.int8).copy()).to(self.dev).view(tt) for x in "kv"}
        self.ts = {x: torch.from_numpy(self.scales[x].copy()).to(self.dev) for x in "kv"}
        self.h = H.PagedKVCache.from_tensors(self.t["k"], self.t["v"], self.ts["k"], self.ts["v"])

    def ints(self, x):
        return self.torch.tensor(np.asarray(x, np.int32), device=self.dev)

    def rows(self, n, heads, size=1.0, wide=0):
        """Random rows in the cache's 16-bit type; with `wide` as a slice of wider rows."""
        dt = {"bf16": self.torch.bfloat16, "fp16": self.torch.float16}[self.dtype]
        x = self.torch.from_numpy(self.rng.standard_normal((n, heads + wide, self.d)) * size).to(self.dev).to(dt)
        return x[:, wide // 2:wide // 2 + heads]

    def values(self, b, n, x):
        """Sequence b's first n values [n, Hkv, d] in fp64, from the host copies."""
        out = np.zeros((n, self.Hkv, self.d))
        for lo in range(0, n, self.page):
            p, c = self.table[b, lo // self.page], min(self.page, n - lo)
            out[lo:lo + c] = (OP.values(self.codes[x][p, :, :c], self.kind) * self.scales[x][p].astype(np.float64)[:, None, None]).transpose(1, 0, 2)
        return out

    def check_attend(self, new, Hq, window=0, n_sink=0, scale=0.0, wide=0, size=1.0, tail=0, gone=None, **kw):
        cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        n = int(cu[-1]) + tail
        q = self.rows(n, Hq, size, wide)
        out = self.torch.full((n, Hq, self.d), 7.0, dtype=q.dtype, device=self.dev)
        args = dict(max_new=max(max(new), 1), max_len=max(self.lens), window=window, n_sink=n_sink, scale=scale)
        args.update(kw)
        got, lse = self.h.attend(q, self.ints(cu), self.ints(self.lens), self.ints(self.table), out=out, return_lse=True, **args)
        again, lse2 = self.h.attend(q, self.ints(cu), self.ints(self.lens), self.ints(self.table), return_lse=True, **args)
        m = int(cu[-1])
        assert self.torch.equal(got[:m], again[:m]) and self.torch.equal(lse[:m], lse2[:m])   # no order of atomics in it
        assert (got[m:] == 7).all()
        self.compare(q, got, lse, new, cu, window, n_sink, scale, gone)
        return q, got, lse

    def compare(self, q, got, lse, new, cu, window, n_sink, scale, gone=None):
        sc = scale or 1 / math.sqrt(self.d)
        o, l, qq = f64(got), f64(lse), f64(q)
        for b, m in enumerate(new):
            L, rows = self.lens[b], slice(cu[b], cu[b] + m)
            ref, rl, mag, most = OP.attend(qq[rows], self.values(b, L, "k"), self.values(b, L, "v"), m, L, sc, window, n_sink,
                                           None if gone is None else gone[b])
            e = (self.d + 16) * 2.0 ** -24 * most[..., None]
            tol = HALF[self.dtype] * np.abs(ref) + (WEIGHT[self.dtype] + 2 * e + 2.0 ** -19) * mag + FLOOR[self.dtype]
            pages = self.table[b, :-(-L // self.page)]
            pages = pages[(pages >= 0) & (pages < len(self.codes["v"]))]
            if len(pages):
                # [Hkv, d]: the largest scale, and the sum of the codes' magnitudes
                top = self.scales["v"][pages].max(0)[:, None]
                c = (np.abs(self.values(b, L, "v")).sum(0) / self.scales["v"][pages].min(0)[:, None])
                tol = tol + 2.0 ** -39 * np.repeat(top * c, q.shape[1] // self.Hkv, 0)
            assert (np.abs(o[rows] - ref) <= tol).all(), (b, float(np.max(np.abs(o[rows] - ref) / np.maximum(tol, 1e-30))))
            seen = np.isfinite(rl)
            assert np.array_equal(np.isneginf(l[rows]), ~seen)
            tl = e[..., 0] + 2.0 ** -20 + 2.0 ** -22 * np.abs(np.where(seen, rl, 0))
            assert (np.abs(np.where(seen, l[rows], 0) - np.where(seen, rl, 0)) <= tl).all()


# ---- append ------------------------------------------------------------------------------------------
def angles(n, rot):
    import torch
    a = np.arange(n)[:, None] * 10000.0 ** (-np.arange(rot // 2) / (rot // 2))
    return torch.from_numpy(np.concatenate([np.cos(a), np.sin(a)], 1).astype(np.float32)).cuda()


def check_append(c, start, new, rot=0, interleaved=False, Hq=0, wide=0, k=None, v=None, max_new=None, inplace=False, n_pos=None):
    """Appends `new` tokens at `start` and compares the whole cache, junk included, bit for bit."""
    torch = c.torch
    c.lens = [s + n for s, n in zip(start, new)]
    cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    n = int(cu[-1])
    k = c.rows(n, c.Hkv, 3.0, wide) if k is None else k
    v = c.rows(n, c.Hkv, 0.3, wide) if v is None else v
    rope = angles(n_pos or max(c.lens) + 1, rot) if rot else None
    q = c.rows(n, Hq, 1.0, wide) if Hq else None
    qh = f64(q) if Hq else None
    got = c.h.append(k, v, c.ints(cu), c.ints(c.lens), c.ints(c.table), max_new=max_new or max(new), rope=rope,
                     interleaved=interleaved, q=q, q_out=q if inplace else None)
    table = f64(rope).astype(np.float32) if rot else np.zeros((max(c.lens) + 1, 0), np.float32)
    for b, m in enumerate(new):
        at = np.arange(start[b], start[b] + m)
        kk = f64(k[cu[b]:cu[b + 1]])
        kk = (OP.rotate(kk, table, at, interleaved) if rot else kk).astype(np.float32)
        OP.append(c.codes["k"], c.scales["k"], kk, start[b], c.table[b], c.kind, c.page)
        OP.append(c.codes["v"], c.scales["v"], f64(v[cu[b]:cu[b + 1]]).astype(np.float32), start[b], c.table[b], c.kind, c.page)
        if Hq:
            ref = OP.rotate(qh[cu[b]:cu[b + 1]], table, at, interleaved) if rot else qh[cu[b]:cu[b + 1]]
            # a rounding of the result, and products rounded once in 32 bits before it
            tol = HALF[c.dtype] * np.abs(ref) + 2.0 ** -22 * np.abs(qh[cu[b]:cu[b + 1]]).max(-1, keepdims=True)
            assert (np.abs(f64(got[cu[b]:cu[b + 1]]) - ref) <= tol).all()
    for x in "kv":
        assert np.array_equal(c.t[x].view(torch.uint8).cpu().numpy(), c.codes[x]), x
        assert np.array_equal(c.ts[x].cpu().numpy(), c.scales[x], equal_nan=True), x
    return k, v, rope, q, cu


@pytest.mark.parametrize("kind", ["e4m3", "int8"])
@pytest.mark.parametrize("dtype,page,Hkv,d,rot,interleaved,Hq,wide", [
    ("bf16", 16, 2, 64, 64, False, 4, 0), ("fp16", 32, 1, 128, 128, True, 3, 2), ("bf16", 48, 3, 128, 64, False, 0, 4),
    ("fp16", 256, 2, 128, 16, True, 2, 0), ("bf16", 64, 8, 64, 0, False, 8, 0), ("bf16", 240, 1, 64, 48, True, 5, 6)])
def test_append(kind, dtype, page, Hkv, d, rot, interleaved, Hq, wide):
    """Lengths that end inside pages, pages begun and continued in one call, an empty sequence, sequences from nothing."""
    start, new = [0, 5, page - 1, page, 3 * page + 7, 2], [1, page, 2, 3 * page + 1, 1, 0]
    c = Paged([s + n for s, n in zip(start, new)], page, Hkv, d, kind, dtype, seed=page + d)
    check_append(c, start, new, rot, interleaved, Hq, wide)
    assert c.h.status() == 0


@pytest.mark.parametrize("kind", ["e4m3", "int8"])
def test_append_token_by_token_grows_scales(kind):
    """A page filled one token at a time with growing values: its scale grows and its codes are rewritten each time."""
    c = Paged([40, 33], 16, 2, 64, kind, "bf16", seed=1)
    for x in "kv":
        c.scales[x][:] = 1e-4
        c.ts[x].fill_(1e-4)
    start = [20, 33]
    for i in range(20):
        size = 1.7 ** i * 1e-3
        k, v = c.rows(2, 2, size), c.rows(2, 2, 1 / size)
        check_append(c, start, [1, 1], rot=32, Hq=2, k=k, v=v)
        start = list(c.lens)
        if max(start) >= 48:
            break


def test_append_int8_ties():
    """Codes halfway between two, and scales where a division by 127 and a product with 1 / 127 differ."""
    import torch
    c = Paged([0] * 3, 16, 2, 64, "int8", "bf16", seed=21)
    x = (torch.arange(128, 256).double() / 128).float()      # all significands of bf16
    turn = x[x / torch.full_like(x, 127.0) != x * (torch.ones(1) / torch.full((1,), 127.0))]
    assert len(turn) >= 3
    n = 3 * 16
    v = torch.zeros(n, 2, 64)
    for page in range(3):
        for h in range(2):
            top = turn[(2 * page + h) % len(turn)]
            v[16 * page:16 * page + 16, h] = torch.cat([top / 2 ** torch.arange(8.0), -top / 2 ** torch.arange(8.0)]).repeat(64).view(16, 64)
    rows = v.cuda().bfloat16()
    assert torch.equal(rows.float().cpu(), v)
    check_append(c, [0, 0, 0], [16, 16, 16], k=rows, v=rows)


def test_append_again_is_the_same():
    import torch
    c = Paged([50], 16, 2, 128, "e4m3", "bf16", seed=2)
    k, v, rope, q, cu = check_append(c, [21], [29], rot=128, Hq=4)
    before = [c.t[x].view(torch.uint8).clone() for x in "kv"] + [c.ts[x].clone() for x in "kv"]
    c.h.append(k, v, c.ints(cu), c.ints(c.lens), c.ints(c.table), max_new=29, rope=rope)
    after = [c.t[x].view(torch.uint8) for x in "kv"] + [c.ts[x] for x in "kv"]
    assert all(torch.equal(a, b) or torch.equal(a.isnan(), b.isnan()) for a, b in zip(before, after))


def test_append_queries_in_place_and_strided():
    c = Paged([9, 30], 16, 2, 64, "int8", "fp16", seed=3)
    check_append(c, [1, 25], [8, 5], rot=64, interleaved=True, Hq=7, wide=3, inplace=True)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("new", [1, 5, 60])
def test_rotation_in_place_then_attention(new, dtype):
    """Steps one behind the other on the stream, nothing between them, whose queries are rotated where they lie, in a buffer
    that the next step uses again: the same as step by step with waits and buffers of their own."""
    import torch
    import hybrid_sparse_linear_decode_b200 as H
    steps = 12
    c, e = (Paged([0, 0], 16, 2, 128, "e4m3", dtype, seed=28) for _ in "ab")
    table = c.ints(c.rng.permutation(2 * 64).reshape(2, 64))
    for x in (c, e):
        x.h = H.PagedKVCache(128, 16, 2, 128)
    rope = angles(1024, 128)
    cu = c.ints([0, new, 2 * new])
    rows = [[c.rows(2 * new, h) for h in (8, 2, 2)] for _ in range(steps)]
    lens = [c.ints([new * (i + 1)] * 2) for i in range(steps)]
    want = []
    for (q, k, v), n in zip(rows, lens):
        turned = e.h.append(k, v, cu, n, table, max_new=new, rope=rope, q=q)
        torch.cuda.synchronize()
        want.append(e.h.attend(turned, cu, n, table, new, 1024).clone())
        torch.cuda.synchronize()
    got = [torch.empty_like(w) for w in want]
    bq, bk, bv = (torch.empty_like(x) for x in rows[0])
    for (q, k, v), n, out in zip(rows, lens, got):
        bq.copy_(q), bk.copy_(k), bv.copy_(v)
        c.h.append(bk, bv, cu, n, table, max_new=new, rope=rope, q=bq, q_out=bq)
        c.h.attend(bq, cu, n, table, new, 1024, out=out)
    torch.cuda.synchronize()
    assert c.h.status() == 0 and e.h.status() == 0
    for i in range(steps):
        assert torch.equal(got[i], want[i]), i
    assert torch.equal(c.h.k_pages.view(torch.uint8), e.h.k_pages.view(torch.uint8)) and torch.equal(c.h.v_scales, e.h.v_scales)


def test_append_extremes():
    """Zeros, values far below and above a code's range, infinities and NaN: stored as the header says."""
    import torch
    import hybrid_sparse_linear_decode_b200 as H
    for kind in ("e4m3", "int8"):
        c = Paged([48], 16, 1, 64, kind, "bf16", seed=4)
        k = c.rows(48, 1)
        v = c.rows(48, 1)
        k[:16] = 0
        k[16:32] *= 1e-38
        k[32:] *= 1e37
        v[:16, :, 0] = float("inf")
        v[16:32, :, 1] = float("-inf")
        v[20, :, 2] = float("nan")
        v[32:] = float("nan")
        check_append(c, [0], [48], k=k, v=v)
        assert c.h.status(clear=True) == H.HYB_STATUS_NONFINITE and c.h.status() == 0
        assert torch.isfinite(c.t["v"].float()[c.table[0, :3].tolist()]).all()


def test_append_bad_pages_lengths_and_positions():
    """A page outside the cache is not written; lengths past the table and positions past the angles are held."""
    import hybrid_sparse_linear_decode_b200 as H
    c = Paged([40, 40, 40], 16, 2, 64, seed=5)
    keep = c.table.copy()
    c.table[0, 1], c.table[1, 2], c.table[2, 0] = -1, 1 << 30, c.codes["k"].shape[0]
    check_append(c, [10, 30, 0], [30, 10, 40])
    assert c.h.status(clear=True) == H.HYB_STATUS_BAD_PAGE
    c.table = keep[:1]
    check_append(c, [39], [1], rot=32, n_pos=40)
    c.table = keep
    assert c.h.status(clear=True) == 0
    # a length past the table: nothing but a status (the rows' positions are the last that fit)
    k, v = c.rows(1, 2), c.rows(1, 2)
    c.h.append(k, v, c.ints([0, 1]), c.ints([1 << 20]), c.ints(c.table[:1, :3]), max_new=1)
    assert c.h.status(clear=True) & H.HYB_STATUS_BAD_LENGTH
    # ranges that fall or pass the rows
    c.h.append(k, v, c.ints([0, 5, 3, -2]), c.ints([40, 40, 40]), c.ints(c.table), max_new=1)
    assert c.h.status(clear=True) & H.HYB_STATUS_BAD_LENGTH
    # more new tokens than tokens
    c.h.append(c.rows(4, 2), c.rows(4, 2), c.ints([0, 4]), c.ints([2]), c.ints(c.table[:1]), max_new=4)
    assert c.h.status(clear=True) & H.HYB_STATUS_BAD_LENGTH
    # a position past the angles
    c.h.append(k, v, c.ints([0, 1]), c.ints([30]), c.ints(c.table[:1]), max_new=1, rope=angles(29, 32))
    assert c.h.status(clear=True) & H.HYB_STATUS_BAD_LENGTH


def test_append_leaves_rows_behind_the_last_sequence():
    c = Paged([20], 16, 1, 64, seed=6)
    q = c.rows(6, 2)
    out = c.torch.full_like(q, 5.0)
    c.h.append(c.rows(6, 1), c.rows(6, 1), c.ints([0, 4]), c.ints([20]), c.ints(c.table), max_new=4, rope=angles(32, 64), q=q, q_out=out)
    assert (out[4:] == 5).all() and not (out[:4] == 5).all() and c.h.status() == 0


# Sequences that contradict what the call was told: cu, kv_lens, max_new, and the position of each row that counts.  Tables of
# four pages of 16 have room for 64 tokens.
CONTRADICTIONS = [
    ([0, 1], [65], 1, 1, {}),                          # one token past the table
    ([0, 4], [66], 4, 4, {0: 62, 1: 63}),              # a run that passes the table's end
    ([0, 3], [1 << 30], 3, 3, {}),
    ([0, 3], [(1 << 31) - 1], 3, 3, {}),
    ([0, 5], [30], 5, 2, {0: 25, 1: 26}),              # more rows than max_new
    ([0, 20], [41], 20, 17, {i: 21 + i for i in range(17)}),
    ([0, 4], [2], 4, 4, {2: 0, 3: 1}),                 # more new tokens than tokens
    ([0, 4], [0], 4, 4, {}),
    ([0, 4], [-5], 4, 4, {}),
    ([-2, 3], [10], 5, 5, {0: 7, 1: 8, 2: 9}),         # rows before the first
    ([0, 9], [20], 4, 4, {i: 11 + i for i in range(4)}),   # and behind the last
    ([3, 1], [20], 4, 4, {}),                          # a range that falls
    ([-(1 << 31), (1 << 31) - 1], [20], 4, 4, {}),
]


@pytest.mark.parametrize("cu,lens,rows,max_new,pos", CONTRADICTIONS)
def test_append_contradictions_move_no_token(cu, lens, rows, max_new, pos):
    """Rows without a place are skipped; the others keep their positions, and older tokens their codes."""
    import hybrid_sparse_linear_decode_b200 as H
    c = Paged([64], 16, 2, 64, seed=23)
    k, v, q = c.rows(rows, 2), c.rows(rows, 2), c.rows(rows, 4)
    rope = angles(80, 64)
    out = c.torch.full_like(q, 3.0)
    c.h.append(k, v, c.ints(cu), c.ints(lens), c.ints(c.table[:, :4]), max_new=max_new, rope=rope, q=q, q_out=out)
    assert c.h.status() == H.HYB_STATUS_BAD_LENGTH
    if pos:
        first, n = min(pos), len(pos)
        at = np.arange(pos[first], pos[first] + n)
        table = f64(rope).astype(np.float32)
        kk = OP.rotate(f64(k[first:first + n]), table, at, False).astype(np.float32)
        OP.append(c.codes["k"], c.scales["k"], kk, int(at[0]), c.table[0], c.kind, c.page)
        OP.append(c.codes["v"], c.scales["v"], f64(v[first:first + n]).astype(np.float32), int(at[0]), c.table[0], c.kind, c.page)
        ref = OP.rotate(f64(q[first:first + n]), table, at, False)
        tol = HALF[c.dtype] * np.abs(ref) + 2.0 ** -22 * np.abs(f64(q[first:first + n])).max(-1, keepdims=True)
        assert (np.abs(f64(out[first:first + n]) - ref) <= tol).all()
    for x in "kv":
        assert np.array_equal(c.t[x].view(c.torch.uint8).cpu().numpy(), c.codes[x]), x
        assert np.array_equal(c.ts[x].cpu().numpy(), c.scales[x], equal_nan=True), x


def test_append_contradictions_of_one_sequence_leave_the_others():
    import hybrid_sparse_linear_decode_b200 as H
    c = Paged([64, 64, 64], 16, 1, 64, seed=24)
    k = c.rows(6, 1)
    c.h.append(k, k, c.ints([0, 2, 4, 6]), c.ints([30, 99, 64]), c.ints(c.table[:, :4]), max_new=2)
    assert c.h.status() == H.HYB_STATUS_BAD_LENGTH
    for b, start in ((0, 28), (2, 62)):
        for x in "kv":
            OP.append(c.codes[x], c.scales[x], f64(k[2 * b:2 * b + 2]).astype(np.float32), start, c.table[b], c.kind, c.page)
    for x in "kv":
        assert np.array_equal(c.t[x].view(c.torch.uint8).cpu().numpy(), c.codes[x]), x
        assert np.array_equal(c.ts[x].cpu().numpy(), c.scales[x], equal_nan=True), x


# ---- attention -----------------------------------------------------------------------------------------
@pytest.mark.parametrize("kind,dtype", [("e4m3", "bf16"), ("int8", "bf16"), ("e4m3", "fp16"), ("int8", "fp16")])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("lens,new,Hkv,G,page", [
    ([1, 2, 31, 32, 33, 700], [1, 1, 1, 1, 1, 1], 2, 4, 16),      # one row tile of 8
    ([5, 0, 640], [1, 0, 1], 1, 8, 48),                            # an empty sequence
    ([100, 17], [3, 3], 2, 5, 32),                                 # 16 rows
    ([300, 40], [8, 2], 1, 4, 64),                                 # 32 rows
    ([257, 9], [9, 4], 2, 7, 256),                                 # 64 rows
    ([130, 200, 77], [70, 1, 33], 1, 3, 16),                       # the wide form, ragged
    ([90], [90], 2, 2, 32),                                        # a whole prompt
    ([600], [21], 1, 16, 16)])                                     # the wide form, split
def test_attend(kind, dtype, d, lens, new, Hkv, G, page):
    c = Paged(lens, page, Hkv, d, kind, dtype, seed=d + page)
    c.check_attend(new, Hkv * G, tail=2)
    assert c.h.status() == 0


@pytest.mark.parametrize("window,n_sink", [(1, 0), (1, 1), (7, 4), (33, 0), (64, 40), (500, 17), (5000, 3)])
@pytest.mark.parametrize("new", [[1, 1, 1], [3, 1, 2], [40, 3, 5]])
def test_attend_window_and_sinks(window, n_sink, new):
    c = Paged([600, 3, 95], 32, 1, 64, "int8", "bf16", seed=window)
    c.check_attend(new, 4, window, n_sink)


def test_attend_rows_that_see_nothing():
    """More new tokens than tokens: the first rows lie before the sequence's begin."""
    import hybrid_sparse_linear_decode_b200 as H
    for new in ([4, 3], [60, 50]):
        c = Paged([2, 0], 16, 2, 64, seed=7)
        c.check_attend(new, 4)
        c.check_attend(new, 4, window=1)


@pytest.mark.parametrize("new", [1, 30, 80])
def test_attend_bad_pages(new):
    """Tokens on pages outside the cache are not seen; every other one is."""
    import hybrid_sparse_linear_decode_b200 as H
    c = Paged([200, 90], 16, 1, 64, "e4m3", seed=8)
    gone = [np.zeros(200, bool), np.zeros(90, bool)]
    vals = {x: [c.values(b, n, x) for b, n in enumerate(c.lens)] for x in "kv"}
    for b, i, bad in ((0, 3, -1), (0, 12, 10 ** 6), (1, 0, c.codes["k"].shape[0])):
        c.table[b, i] = bad
        gone[b][i * 16:i * 16 + 16] = True
    c.values = lambda b, n, x: vals[x][b]
    c.check_attend([new, min(new, 70)], 2, gone=gone)
    assert c.h.status(clear=True) == H.HYB_STATUS_BAD_PAGE


def test_attend_bad_lengths():
    """A length past the table and ranges that fall or pass the rows are held to what is there."""
    import hybrid_sparse_linear_decode_b200 as H
    c = Paged([64, 64], 16, 1, 64, seed=9)
    t = c.ints(c.table[:, :4])
    for rows in (2, 50):
        q = c.rows(rows, 4)
        full = c.h.attend(q[:1], c.ints([0, 1]), c.ints([64]), t[:1], max_new=1, max_len=64)
        got = c.h.attend(q[:1], c.ints([0, 1]), c.ints([1 << 29]), t[:1], max_new=1, max_len=64)
        assert c.torch.equal(full, got) and c.h.status(clear=True) == H.HYB_STATUS_BAD_LENGTH
        c.h.attend(q, c.ints([0, rows + 9, 1]), c.ints([64, -5]), t, max_new=rows, max_len=64)
        assert c.h.status(clear=True) & H.HYB_STATUS_BAD_LENGTH


def check_positions(c, q, out, lse, pos, cap, window, n_sink, step=2.0 ** -31):
    """Each row against the oracle at the position it has; the others as they were.  The floor of the weights is the
    row's own: `step` times the largest value scale that it sees, for each code that it sees.  A weight is stored as f16
    2^15 times itself (tcgen05: 2^7 at least), in units of a power of two below twice that scale, so one below 2^-14 there is
    rounded to multiples of 2^-24: half a step is 2^-40 (2^-32) of these units."""
    sc = 1 / math.sqrt(c.d)
    K, V = c.values(0, cap, "k"), c.values(0, cap, "v")
    scale = c.scales["v"][c.table[0, :cap // c.page]].astype(np.float64).repeat(c.page, 0)[..., None]   # of each token
    for i in range(q.shape[0]):
        if i not in pos:
            assert (out[i] == 7).all()
            continue
        t = pos[i]
        gone = np.zeros(cap, bool)
        if t < 0:
            gone[:] = True
        else:
            gone |= np.arange(cap) > t
            if window:
                gone |= (np.arange(cap) <= t - window) & (np.arange(cap) >= n_sink)
        ref, rl, mag, most = OP.attend(f64(q[i:i + 1]), K, V, 1, cap, sc, gone=gone)
        e = (c.d + 16) * 2.0 ** -24 * most[..., None]
        low = step * (scale[~gone].max(0) * np.abs(V[~gone] / scale[~gone]).sum(0)) if (~gone).any() else np.zeros(V.shape[1:])
        tol = HALF[c.dtype] * np.abs(ref) + (WEIGHT[c.dtype] + 2 * e + 2.0 ** -19) * mag + FLOOR[c.dtype] + np.repeat(low, q.shape[1] // c.Hkv, 0)
        assert (np.abs(f64(out[i:i + 1]) - ref) <= tol).all(), i
        assert np.array_equal(np.isneginf(f64(lse[i])), np.isneginf(rl[0]))
        fin = np.isfinite(rl[0])
        assert (np.abs(f64(lse[i])[fin] - rl[0][fin]) <= (e[0, :, 0] + 2.0 ** -20 + 2.0 ** -22 * np.abs(rl[0]))[fin]).all()


@pytest.mark.parametrize("window,n_sink", [(0, 0), (5, 2), (20, 40), ((1 << 31) - 1, 0)])
@pytest.mark.parametrize("G,dtype", [(1, "bf16"), (4, "bf16"), (16, "bf16"), (64, "bf16"), (16, "fp16"), (64, "fp16")])
def test_attend_contradictions_move_no_row(window, n_sink, G, dtype):
    """Rows past max_new are left as they were, rows before a sequence's begin see nothing, rows past the table see what is
    in it, and the status is set, for every number of rows a KV head (and so every form)."""
    import hybrid_sparse_linear_decode_b200 as H
    c = Paged([64], 16, 1, 64, dtype=dtype, seed=25)
    table = c.ints(c.table[:, :4])
    for cu, lens, rows, max_new, _ in CONTRADICTIONS:
        first = max(cu[0], 0)
        n = max(0, min(cu[1], rows) - first, 0)
        pos = {first + i: lens[0] - cu[1] + first + i for i in range(min(n, max_new))}
        q = c.rows(rows, G)
        out = c.torch.full_like(q, 7.0)
        got, lse = c.h.attend(q, c.ints(cu), c.ints(lens), table, max_new, 64, window=window, n_sink=n_sink, out=out, return_lse=True)
        assert c.h.status(clear=True) == H.HYB_STATUS_BAD_LENGTH, (cu, lens)
        check_positions(c, q, out, lse, pos, 64, window, n_sink)


@pytest.mark.parametrize("new,length", [(1, 9000), (9, 9000), (2, 9000), (40, 9000)])
def test_attend_status_of_sequences_without_work(new, length):
    """A contradiction is told where its sequence has nothing to do, too: beside long sequences, which go by the line."""
    import hybrid_sparse_linear_decode_b200 as H
    for B in (2, 40):
        lens = [length] + [16] * (B - 1)
        c = Paged(lens, 64, 1, 64, "int8", seed=26)
        cu = np.full(B + 1, new, np.int32)
        cu[0] = 0
        for bad in (1, B - 1):
            worse = list(lens)
            worse[bad] = -1
            for ls, want in ((lens, 0), (worse, H.HYB_STATUS_BAD_LENGTH)):
                c.h.attend(c.rows(new, 4), c.ints(cu), c.ints(ls), c.ints(c.table), new, length)
                assert c.h.status(clear=True) == want


@pytest.mark.parametrize("kind", ["e4m3", "int8"])
@pytest.mark.parametrize("dtype,G,new,step", [("bf16", 1, 4, 2.0 ** -39), ("bf16", 4, 4, 2.0 ** -39), ("fp16", 2, 15, 2.0 ** -39),
                                              ("bf16", 4, 20, 2.0 ** -31), ("bf16", 16, 20, 2.0 ** -31), ("fp16", 16, 20, 2.0 ** -39)])
@pytest.mark.parametrize("times", [2.0 ** 24, 2.0 ** 30, 2.0 ** 36, 2.0 ** 60, np.inf, np.nan])
def test_attend_scales_of_pages_a_row_does_not_see(kind, dtype, G, new, step, times):
    """Value scales far larger on a page that only later rows see, or only earlier ones (behind the others' window): each
    row's weights keep their bits whatever it does not see."""
    import hybrid_sparse_linear_decode_b200 as H
    for page, length, window in ((3, 48 + new // 2, 0), (0, 31 + new // 2, 16)):
        c = Paged([length], 16, 2, 64, kind, dtype, seed=27)
        pid = c.table[0, page]
        for x in "kv":
            c.scales[x][c.table[0, :4]] = 2.0 ** -7       # all alike but for that page
        c.scales["v"][pid] *= np.float32(times)
        if not np.isfinite(times):
            c.scales["k"][pid] = times
        for x in "kv":
            c.ts[x].copy_(c.torch.from_numpy(c.scales[x]))
        sees = (lambda t: t >= 48) if page else (lambda t: t - window < 15)
        first = length - new
        assert 0 < sum(sees(first + i) for i in range(new)) < new
        q = c.rows(new, 2 * G)
        out, lse = c.h.attend(q, c.ints([0, new]), c.ints([length]), c.ints(c.table), new, length, window=window, return_lse=True)
        rows = [i for i in range(new) if np.isfinite(times) or not sees(first + i)]
        if not np.isfinite(times):
            c.scales["k"][pid] = c.scales["v"][pid] = 1.0    # for the oracle, whose rows do not see it either
        if dtype == "fp16":     # whose results end at 65504
            rows = [i for i in rows if not sees(first + i)]
        check_positions(c, q[rows], out[rows], lse[rows], {j: first + i for j, i in enumerate(rows)}, 16 * -(-length // 16), window, 0, step)


@pytest.mark.parametrize("dtype,G,new,step", [("bf16", 1, 1, 2.0 ** -39), ("bf16", 4, 4, 2.0 ** -39), ("bf16", 4, 20, 2.0 ** -31),
                                              ("fp16", 2, 3, 2.0 ** -39), ("fp16", 16, 20, 2.0 ** -39)])
@pytest.mark.parametrize("length,window,n_sink", [(200, 70, 0), (200, 70, 5), (200, 33, "between"), (200, 33, 16), (90, 1, 3), (5000, 4090, 7)])
def test_attend_nothing_outside_the_window_is_used(dtype, G, new, step, length, window, n_sink):
    """NaN codes wherever no row looks (in pages that hold visible tokens too), NaN scales of pages that hold none."""
    c = Paged([length], 64, 1, 128, "e4m3", dtype, seed=31)
    first = length - new
    if n_sink == "between":     # sinks that end inside the 16 tokens in which the window begins
        n_sink = ((first - window + 1) & ~15) + 2
    unseen = [j for j in range(length) if j <= first - window and j >= n_sink]
    assert unseen
    for j in unseen:
        for x in "kv":
            c.codes[x][c.table[0, j // 64], :, j % 64] = 0x7f
    for i in range(-(-length // 64)):
        if all(j in set(unseen) for j in range(64 * i, min(64 * i + 64, length))):
            for x in "kv":
                c.scales[x][c.table[0, i]] = np.nan
    for x in "kv":
        c.t[x].view(c.torch.uint8).copy_(c.torch.from_numpy(c.codes[x]))
        c.ts[x].copy_(c.torch.from_numpy(c.scales[x]))
    q = c.rows(new, G)
    out, lse = c.h.attend(q, c.ints([0, new]), c.ints([length]), c.ints(c.table), new, length, window=window, n_sink=n_sink, return_lse=True)
    check_positions(c, q, out, lse, {i: first + i for i in range(new)}, 64 * -(-length // 64), window, n_sink, step)
    assert c.h.status() == 0


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_attend_large_and_tiny_values(dtype):
    """Queries of very different sizes, scales of pages 2^40 apart, logits far apart."""
    for seed, spread in ((1, 3.0), (2, 5.0)):
        c = Paged([300, 120], 16, 2, 64, "e4m3", dtype, seed=seed, spread=spread)
        c.check_attend([2, 1], 4, size=1e-3)
        c.check_attend([1, 1], 4, size=30.0)
    big = Paged([200], 16, 1, 128, "int8", "bf16", seed=3)
    q = big.rows(1, 2)
    q[:, 0] *= 1e30
    q[:, 1] *= 1e-30
    cu = np.array([0, 1], np.int32)
    out, lse = big.h.attend(q, big.ints(cu), big.ints([200]), big.ints(big.table), 1, 200, scale=1e-30, return_lse=True)
    big.compare(q, out, lse, [1], cu, 0, 0, 1e-30)


def test_attend_non_finite_queries_stay_in_their_rows():
    c = Paged([70], 16, 1, 64, seed=10)
    for n in (3, 50):
        q = c.rows(n, 2)
        q[1, 0, 3], q[2, 1, 5] = float("nan"), float("inf")
        out = f64(c.h.attend(q, c.ints([0, n]), c.ints([70]), c.ints(c.table), n, 70))
        bad = np.isnan(out).any(-1)
        assert bad[1, 0] and bad[2, 1] and bad.sum() == 2


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("length,new,G", [(70, 3, 2), (70, 50, 2), (5000, 3, 2), (5000, 12, 4), (5000, 150, 2)])
def test_attend_sums_of_rows_that_are_not_finite(dtype, length, new, G):
    """A NaN output has a NaN logarithm of its sum: -inf would pass for a row that sees nothing where rows are merged."""
    c = Paged([length], 64, 1, 64, dtype=dtype, seed=32)
    q = c.rows(new, G)
    q[1, 0, 3], q[2, 1, 5] = float("nan"), float("inf")
    out, lse = c.h.attend(q, c.ints([0, new]), c.ints([length]), c.ints(c.table), new, length, return_lse=True)
    bad = np.isnan(f64(out)).any(-1)
    assert bad[1, 0] and bad[2, 1] and bad.sum() == 2
    assert np.array_equal(np.isnan(f64(lse)), bad)


def test_attend_strided_rows_and_scale():
    c = Paged([50, 120], 32, 2, 128, "e4m3", "fp16", seed=11)
    c.check_attend([2, 3], 6, wide=5, scale=0.3)


def test_attend_many_sequences():
    """More sequences than a warp has lanes, most of them short, and CTAs that take several units."""
    rng = np.random.default_rng(12)
    lens = rng.integers(0, 90, 75).tolist()
    c = Paged(lens, 16, 2, 64, "int8", seed=12)
    c.check_attend([1 if n else 0 for n in lens], 4)


def needs_workspace(c, new, Hq, window=0, n_sink=0):
    """Whether the call's parts go through the workspace (a line of all units' stages that CTAs share, or split row tiles):
    without one it is refused before anything is launched."""
    import hybrid_sparse_linear_decode_b200 as H
    q = c.rows(sum(new), Hq)
    keep = [c.ints(np.concatenate([[0], np.cumsum(new)])), c.ints(c.lens), c.ints(c.table), q]
    b = H.hyb_attn_paged_batch(keep[2].data_ptr(), keep[0].data_ptr(), keep[1].data_ptr(), len(new), c.table.shape[1], sum(new), max(new), max(c.lens), 0)
    try:
        H.hyb_attn_paged_attend(c.h._c, b, {"bf16": H.HYB_TYPE_BF16, "fp16": H.HYB_TYPE_FP16}[c.dtype], q.data_ptr(), Hq * c.d,
                                c.torch.empty_like(q).data_ptr(), Hq * c.d, None, Hq, window, n_sink, 0.0, None, 0,
                                c.torch.cuda.current_stream().cuda_stream)
    except H.HybAttnError as e:
        return e.code == -6
    return False


RAGGED = np.random.default_rng(33).integers(0, 5000, 45).tolist()
RAGGED[3], RAGGED[40], RAGGED[44] = 0, 4999, 5000


@pytest.mark.parametrize("kind,dtype,d", [("e4m3", "bf16", 128), ("int8", "fp16", 128), ("int8", "bf16", 64), ("e4m3", "fp16", 64)])
@pytest.mark.parametrize("lens,new,Hkv,G,page,window,n_sink", [
    ([4096], [1], 2, 4, 64, 0, 0),                       # one sequence
    ([4097, 9000], [1, 1], 1, 8, 16, 0, 0),
    ([5001, 0, 4100], [3, 0, 8], 2, 4, 48, 0, 0),        # drafts, and an empty sequence between
    ([5000, 7, 6100], [2, 2, 1], 1, 5, 64, 0, 0),        # a short one between long ones
    ([6000, 4999], [8, 5], 1, 2, 128, 2500, 5),          # a window that begins inside a page
    ([4500, 33], [1, 1], 1, 4, 32, 4000, 0),
    ([5000, 4096], [8, 7], 1, 8, 64, 0, 0),              # 64 rows: fp16 on the line, bf16 on tcgen05's
    ([7000, 4100], [16, 3], 1, 8, 32, 3000, 40),         # 128 rows
    (RAGGED, [1 if n else 0 for n in RAGGED], 1, 4, 64, 0, 0),         # more sequences than a warp has lanes
    (RAGGED, [min(3, n) for n in RAGGED], 1, 4, 16, 1700, 3),
    (RAGGED, [min(9 + i % 3, n) for i, n in enumerate(RAGGED)], 1, 4, 64, 0, 0)])
def test_attend_line(kind, dtype, d, lens, new, Hkv, G, page, window, n_sink):
    """Long sequences, whose units' stages lie on one line that the CTAs cut into equal parts, and their joins."""
    c = Paged(lens, page, Hkv, d, kind, dtype, seed=d + len(lens))
    rows = max(new) * G
    if dtype == "bf16" or rows <= 64:      # beyond, fp16 goes in row tiles
        assert needs_workspace(c, new, Hkv * G, window, n_sink)
    c.check_attend(new, Hkv * G, window, n_sink, tail=1)
    assert c.h.status() == 0


@pytest.mark.parametrize("lens,new,Hkv,G,window", [
    ([2300], [330], 8, 8, 0),               # 168 row tiles: fewer than the SMs hold, in parts
    ([2100, 90], [640, 90], 4, 8, 0),       # 320, many of them without rows; the last ones in parts
    ([2200], [620], 8, 8, 0),               # 312, whole but for the last 16
    ([2500], [330], 8, 8, 700),             # as the first, behind a window
    ([9000], [17], 1, 8, 0)])               # 2, in many parts
def test_attend_row_tiles_in_parts(lens, new, Hkv, G, window):
    c = Paged(lens, 64, Hkv, 64, "e4m3", "bf16", seed=13)
    c.check_attend(new, Hkv * G, window, 5, tail=1)
    assert c.h.status() == 0


def test_attend_long_cache_and_far_pages():
    """A cache whose codes lie past 2^31 bytes, and a sequence whose tokens do."""
    import torch
    import hybrid_sparse_linear_decode_b200 as H
    free, _ = torch.cuda.mem_get_info()
    if free < 16 << 30:
        pytest.skip("needs 16 GB")
    n, page, Hkv, d = 17000, 128, 8, 128    # 2.2 GB each
    shape = (n, Hkv, page, d)
    k, v = (torch.zeros(shape, dtype=torch.int8, device="cuda") for _ in "kv")
    s = torch.full((n, Hkv), 0.01, device="cuda")
    cache = H.PagedKVCache.from_tensors(k, v, s, s.clone())
    g = torch.Generator("cuda").manual_seed(0)
    lens = [300, 129]
    ids = torch.tensor([[n - 1, n - 2, n - 3], [n - 4, n - 5, -1]], dtype=torch.int32, device="cuda")
    for p in range(n - 5, n):
        k[p] = torch.randint(-127, 128, shape[1:], generator=g, device="cuda", dtype=torch.int8)
        v[p] = torch.randint(-127, 128, shape[1:], generator=g, device="cuda", dtype=torch.int8)
    small = H.PagedKVCache.from_tensors(k[n - 5:].clone(), v[n - 5:].clone(), s[:5].clone(), s[:5].clone())
    tens = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    for new in (1, 60):
        q = torch.randn(2 * new, 32, d, generator=g, device="cuda").bfloat16()
        kk, vv = (torch.randn(2 * new, Hkv, d, generator=g, device="cuda").bfloat16() for _ in "kv")
        outs = []
        for c, t in ((cache, ids), (small, torch.where(ids >= 0, ids - (n - 5), ids))):
            c.append(kk, vv, tens([0, new, 2 * new]), tens(lens), t, max_new=new)
            outs.append(c.attend(q, tens([0, new, 2 * new]), tens(lens), t, max_new=new, max_len=300))
            assert c.status() == 0
        assert torch.equal(outs[0], outs[1])
    assert torch.equal(k[n - 5:], small.k_pages) and not k[:n - 5].any()


def test_attend_pages_past_64_gigabytes():
    """Codes past 2^32 pieces of 16 bytes, for every form (one buffer as keys and values; only its last pages are written)."""
    import torch
    import hybrid_sparse_linear_decode_b200 as H
    page, Hkv, d = 128, 8, 128
    n = (1 << 36) // (page * Hkv * d) + 4
    free, _ = torch.cuda.mem_get_info()
    if free < 80 << 30:
        pytest.skip("needs 80 GB")
    codes = torch.empty((n, Hkv, page, d), dtype=torch.int8, device="cuda")
    g = torch.Generator("cuda").manual_seed(0)
    codes[n - 4:] = torch.randint(-127, 128, (4, Hkv, page, d), generator=g, device="cuda", dtype=torch.int8)
    s = torch.full((n, Hkv), 0.01, device="cuda")
    far = H.PagedKVCache.from_tensors(codes, codes, s, s)
    near = H.PagedKVCache.from_tensors(codes[n - 4:].clone(), codes[n - 4:].clone(), s[:4].clone(), s[:4].clone())
    ints = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    at = ints([[2, 0, 3, 1]])
    for new in (1, 8, 12, 60):
        for dtype in (torch.bfloat16, torch.float16):
            q = torch.randn(new, 32, d, generator=g, device="cuda").to(dtype)
            outs = [c.attend(q, ints([0, new]), ints([500]), t, max_new=new, max_len=500) for c, t in ((far, at + (n - 4)), (near, at))]
            assert torch.equal(*outs) and far.status() == near.status() == 0
    del far, codes
    torch.cuda.empty_cache()


# ---- streams, graphs, refusals -----------------------------------------------------------------------
def test_calls_on_another_stream():
    import torch
    c = Paged([80, 40], 16, 2, 64, seed=13)
    cu, lens, table = c.ints([0, 1, 2]), c.ints([80, 40]), c.ints(c.table)
    q = c.rows(2, 8)
    ref = c.h.attend(q, cu, lens, table, 1, 80)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    a = c.h.attend(q, cu, lens, table, 1, 80, stream=s)
    b = c.h.attend(q, cu, lens, table, 1, 80, stream=s.cuda_stream)
    s.synchronize()
    assert torch.equal(a, ref) and torch.equal(b, ref)
    with pytest.raises(ValueError):
        c.h.attend(q.cpu(), cu, lens, table, 1, 80)


def test_two_captured_graphs_share_a_cache():
    """Steps captured once and replayed with new lengths and rows; two graphs of the same handle at once on two
    streams do not disturb each other (each owns its outputs and workspace)."""
    import torch
    c = Paged([200, 90], 16, 2, 128, seed=14)
    table = c.ints(c.table)
    lens, cu = c.ints([150, 60]), c.ints([0, 1, 2])
    graphs = []
    for i in range(2):
        q = c.rows(2, 8)
        c.h.attend(q, cu, lens, table, 1, 200)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = c.h.attend(q, cu, lens, table, 1, 200)
        graphs.append((g, q, out))
    for n0, n1 in ((150, 60), (200, 90), (1, 0)):
        lens.copy_(c.ints([n0, n1]))
        torch.cuda.synchronize()
        streams = [torch.cuda.Stream() for _ in graphs]
        for _ in range(20):
            for (g, q, out), s in zip(graphs, streams):
                with torch.cuda.stream(s):
                    g.replay()
        torch.cuda.synchronize()
        for g, q, out in graphs:
            assert torch.equal(out, c.h.attend(q, cu, lens, table, 1, 200))


@pytest.mark.parametrize("new", [1, 20])
def test_two_captured_graphs_on_the_line(new):
    """As above with sequences whose parts go through workspaces, replayed at once on two streams with other lengths."""
    import torch
    c = Paged([5000, 4200], 64, 1, 128, seed=29)
    assert needs_workspace(c, [new, new], 4)
    table, lens, cu = c.ints(c.table), c.ints([5000, 4200]), c.ints([0, new, 2 * new])
    graphs = []
    for i in range(2):
        q = c.rows(2 * new, 4)
        c.h.attend(q, cu, lens, table, new, 5000)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = c.h.attend(q, cu, lens, table, new, 5000)
        graphs.append((g, q, out))
    for n0, n1 in ((5000, 4200), (3000, 64), (64, 4199)):
        lens.copy_(c.ints([n0, n1]))
        torch.cuda.synchronize()
        streams = [torch.cuda.Stream() for _ in graphs]
        for _ in range(20):
            for (g, q, out), s in zip(graphs, streams):
                with torch.cuda.stream(s):
                    g.replay()
        torch.cuda.synchronize()
        for g, q, out in graphs:
            assert torch.equal(out, c.h.attend(q, cu, lens, table, new, 5000))
    assert c.h.status() == 0


def test_status_waits_for_calls_on_other_streams():
    """What a call raises on a busy stream of the caller's is there when the status is read from another one."""
    import torch
    import hybrid_sparse_linear_decode_b200 as H
    c = Paged([64], 16, 2, 64, seed=30)
    d = H.GatedDeltaState(1, 1, 1, 64, 64)
    cu, bad, table, q, k = c.ints([0, 1]), c.ints([65]), c.ints(c.table[:, :4]), c.rows(1, 2), c.rows(1, 2)
    row, gate, slot = c.rows(1, 1), torch.zeros(1, 1, device="cuda"), c.ints([5])
    s = torch.cuda.Stream()
    calls = [(c.h, H.HYB_STATUS_BAD_LENGTH, lambda: c.h.append(k, k, cu, bad, table, max_new=1, stream=s)),
             (c.h, H.HYB_STATUS_BAD_LENGTH, lambda: c.h.attend(q, cu, bad, table, 1, 64, stream=s)),
             (d, H.HYB_STATUS_BAD_SLOT, lambda: d.run(row, row, row, gate, gate, cu, max_new=1, slots=slot, stream=s))]
    for h, flag, call in calls:
        call()      # loads the kernel, which waits
        torch.cuda.synchronize()
        h.status(clear=True)
        with torch.cuda.stream(s):
            torch.cuda._sleep(50_000_000)
        call()
        assert h.status(clear=True) == flag
        assert h.status() == 0


def test_calls_refuse_what_they_do_not_take():
    c = Paged([40], 16, 2, 64, seed=15)
    t, cu, lens, table = c.torch, c.ints([0, 1]), c.ints([40]), c.ints(c.table)
    q, k = c.rows(1, 4), c.rows(1, 2)
    ok = dict(max_new=1, max_len=40)
    with pytest.raises(ValueError):
        c.h.attend(q.float(), cu, lens, table, **ok)
    with pytest.raises(ValueError):
        c.h.attend(q, cu.long(), lens, table, **ok)
    with pytest.raises(ValueError):
        c.h.attend(q, cu, lens[:0], table, **ok)
    with pytest.raises(ValueError):
        c.h.attend(q, cu, lens, table[0], **ok)
    with pytest.raises(ValueError):
        c.h.attend(q.transpose(1, 2).contiguous().transpose(1, 2), cu, lens, table, **ok)
    with pytest.raises(ValueError):
        c.h.attend(q, cu, lens, table, max_new=0, max_len=40)
    with pytest.raises(ValueError):
        c.h.attend(q, cu, lens, table, out=t.empty(2, 4, 64, dtype=q.dtype, device="cuda"), **ok)
    import hybrid_sparse_linear_decode_b200 as H
    for bad in (dict(window=-1), dict(n_sink=-2), dict(scale=-1.0)):
        with pytest.raises(H.HybAttnError):
            c.h.attend(q, cu, lens, table, **ok, **bad)
    with pytest.raises(H.HybAttnError):
        c.h.attend(c.rows(1, 3), cu, lens, table, **ok)
    with pytest.raises(ValueError):
        c.h.append(k, k.half(), cu, lens, table, max_new=1)
    with pytest.raises(ValueError):
        c.h.append(k, k, cu, lens, table, max_new=1, q_out=q)
    with pytest.raises(ValueError):
        c.h.append(k, k, cu, lens, table, max_new=1, rope=angles(50, 32).double())
    with pytest.raises(H.HybAttnError):
        c.h.append(k, k, cu, lens, table, max_new=1, rope=angles(50, 24))
    assert c.h.status() == 0

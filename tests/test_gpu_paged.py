"""The paged cache and the rotary embedding on the GPU, against plain implementations in 64
bits (attention, rotation) and a plain model of the page table (reserve, release, fork,
compact).

Tolerances. A rounding moves a value by at most half a step, u = finfo.eps / 2 of its type
(bf16 2^-8, fp32 2^-24, E4M3 2^-4 and half of 2^-9 below its normals).
Rotation: with |angle| left <= an eighth of a turn, its fp32 rounding moves the sine by at
most pi/4 2^-24, the function by 2^-24 more; two products and a sum add 2^-24 (|a| + |b|)
each: below 4 * 2^-24 (|a| + |b|) in all, then the output's own rounding.
Attention: p is rounded to the pages' matrix type (u_p: bf16 2^-8, for E4M3 pages f16 2^-11)
in numerator and denominator alike, so o moves by at most 2 u_p A with A = sum p |v| / den,
and by 2 dz A for logits that are dz off; fp32 sums of 512 products give dz <= 512 * 2^-24 *
scale * sum |q||k|, in practice far less; with E4M3 pages two E4M3 parts of the query leave
2^-22 of a head's largest |q| besides; ex2.approx adds 2^-22. The output's rounding comes on top. Over many values the roundings are independent: each contributes at most u / sqrt(3)
in the mean square, so the relative error in the 2-norm stays below
sqrt(2) * 2^-8 / sqrt(3) = 3.2e-3; 4e-3 is asked for."""
import math

import numpy as np
import pytest
import torch

from csa2_compressed_sparse_02_gb300 import api

pytestmark = pytest.mark.gpu
DEV = "cuda"
D = 512
U = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device=DEV)


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def randn(*shape, seed, dtype=torch.float32):
    return torch.randn(*shape, generator=gen(seed), device=DEV).to(dtype)


# ------------------------------------------------------------------------------ rotation
def rotate64(x, pos, p, layout, first=None, inverse=False):
    """(rotated x in 64 bits, |a| + |b| of each channel's pair), x [N, H, C]."""
    dim = p.rope_dim
    first = x.shape[-1] - dim if first is None else first
    i = np.arange(dim // 2, dtype=np.float64)
    f = float(p.rope_theta) ** (-2 * i / dim)
    turns = p.rope_orig_len * f / (2 * math.pi)
    keep = np.clip((turns - p.rope_beta_slow) / (p.rope_beta_fast - p.rope_beta_slow), 0, 1)
    f = f * keep + f / p.rope_factor * (1 - keep)
    ang = np.asarray(pos, np.float64)[:, None, None] * f * (-1 if inverse else 1)
    x = x.double().cpu().numpy()
    y, m = x.copy(), np.zeros_like(x)
    ch = np.arange(dim)
    a, b = (ch[0::2], ch[1::2]) if layout == api.ROPE_PAIRS else (ch[:dim // 2], ch[dim // 2:])
    u, v = x[..., first + a], x[..., first + b]
    y[..., first + a] = u * np.cos(ang) - v * np.sin(ang)
    y[..., first + b] = u * np.sin(ang) + v * np.cos(ang)
    m[..., first + a] = m[..., first + b] = np.abs(u) + np.abs(v)
    return y, m


def assert_rotated(got, ref, mag, u):
    err = np.abs(got.double().cpu().numpy() - ref)
    tol = 4 * 2.0 ** -24 * mag * (1 + u) + u * np.abs(ref) * (mag > 0) * (u > 2.0 ** -20)
    over = err - tol
    assert over.max(initial=0) <= 0, over.max()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("layout", [api.ROPE_PAIRS, api.ROPE_HALF])
@pytest.mark.parametrize("N,H,C,dim,first", [
    (1, 1, 2, 2, -1), (5, 3, 64, 64, -1), (64, 64, 512, 64, -1), (33, 7, 80, 20, -1),
    (129, 2, 192, 64, 0), (7, 5, 96, 32, 40), (3, 1, 512, 512, -1), (2, 70, 513, 126, 3),
    (700, 1, 66, 6, 1), (1, 4096, 8, 4, -1), (2, 3, 4096, 512, -1)])
def test_rope_matches_the_definition(dtype, layout, N, H, C, dim, first):
    p = api.default_params(rope_dim=dim)
    x = randn(N, H, C, seed=N + H, dtype=dtype)
    rng = np.random.default_rng(N * H + C)
    pos = rng.integers(0, 1 << 20, N)
    pos[0] = 0
    for inverse in (False, True):
        y = api.rope(p, x, i32(pos), layout=layout, first=first, inverse=inverse)
        ref, mag = rotate64(x, pos, p, layout, None if first < 0 else first, inverse)
        assert_rotated(y, ref, mag, U[dtype])
        z = x.clone()
        assert api.rope(p, z, i32(pos), out=z, layout=layout, first=first, inverse=inverse) is z
        assert torch.equal(z, y)


@pytest.mark.parametrize("layout", [api.ROPE_PAIRS, api.ROPE_HALF])
@pytest.mark.parametrize("off", [0, 1, 3, 8])
def test_rope_strided_views_padding_and_settings(layout, off):
    """Heads of a wider projection (row and head strides, odd offsets), padding rows left
    alone, plain and linearly scaled positions."""
    for over in (dict(), dict(rope_factor=1.0, rope_theta=10000.0),
                 dict(rope_beta_slow=1e29, rope_beta_fast=2e29, rope_factor=8.0)):
        p = api.default_params(rope_dim=32, **over)
        wide = randn(21, 9, 160, seed=3, dtype=torch.bfloat16)
        dst = torch.full((21, 6, 100), 7.0, device=DEV, dtype=torch.bfloat16)
        x, out = wide[:, 2:7, off:off + 96], dst[:, :5, 4:100]
        pos = np.arange(21) * 1777
        pos[[4, 20]] = -1
        before = wide.clone()
        api.rope(p, x, i32(pos), out=out, layout=layout)
        ref, mag = rotate64(x, pos, p, layout)
        live = pos >= 0
        assert_rotated(out[torch.from_numpy(live).to(DEV)], ref[live], mag[live], U[torch.bfloat16])
        assert torch.all(dst[4] == 7) and torch.all(dst[20] == 7)
        assert torch.all(dst[:, 5] == 7) and torch.all(dst[:, :, :4] == 7) and torch.equal(wide, before)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("layout", [api.ROPE_PAIRS, api.ROPE_HALF])
@pytest.mark.parametrize("C,dim,first", [(128, 64, -1), (50, 20, 3), (64, 64, 0)])
def test_rope_padding_of_a_new_tensor_is_zero(dtype, layout, C, dim, first):
    """Not whatever its memory held: here NaN, which a block of the same size had before. Padded rows
    of x may be NaN themselves."""
    p = api.default_params(rope_dim=dim)
    x, pos = randn(300, 5, C, seed=C, dtype=dtype), np.arange(300) * 7
    pos[[0, 7, 8, 250, 299]] = -1
    pad = torch.from_numpy(pos < 0).to(DEV)
    x[7] = float("nan")
    where, ref = i32(pos), torch.full_like(x, 5)
    api.rope(p, x, where, out=ref, layout=layout, first=first)
    assert torch.all(ref[pad] == 5)
    for inverse in (False, True):
        torch.cuda.synchronize()
        torch.cuda.empty_cache()
        block = torch.full_like(x, float("nan"))
        del block
        y = api.rope(p, x, where, layout=layout, first=first, inverse=inverse)
        assert torch.all(y[pad] == 0)
        if not inverse:
            assert torch.equal(y[~pad], ref[~pad])


@pytest.mark.parametrize("layout", [api.ROPE_PAIRS, api.ROPE_HALF])
def test_rope_inverse_is_the_gradient(layout):
    """<dy, J x'> = <J^T dy, x'> with J^T the inverse call, and differences of the call."""
    p = api.default_params(rope_dim=16)
    x, dy, d = (randn(40, 3, 24, seed=s) for s in (1, 2, 3))
    pos = i32(np.arange(40) * 4099)
    turned, back = api.rope(p, d, pos, layout=layout), api.rope(p, dy, pos, layout=layout, inverse=True)
    lhs, rhs = (dy.double() * turned.double()).sum(), (back.double() * d.double()).sum()
    # each of the 2,880 products is off by at most 4 2^-24 (|a| + |b|) |d|
    bound = 2 * 4 * 2.0 ** -24 * 2 * (dy.double().norm() * d.double().norm())
    assert abs(lhs - rhs) <= bound, (lhs, rhs)
    diff = (api.rope(p, x + d, pos, layout=layout).double() - api.rope(p, x, pos, layout=layout).double())
    lhs = (dy.double() * diff).sum()
    # x + d is rounded too: one more 2^-24 of |x + d|
    assert abs(lhs - (back.double() * d.double()).sum()) <= 2 * bound + 2.0 ** -23 * dy.double().norm() * (x + d).double().norm()


def test_rope_nothing_to_do():
    p = api.default_params(rope_dim=16)
    for shape in ((0, 3, 16), (3, 0, 16)):
        x = torch.zeros(shape, device=DEV)
        assert api.rope(p, x, i32(np.zeros(shape[0]))).shape == shape


# ------------------------------------------------------------------------------ rows into pages
def dtype_of(kv):
    return torch.bfloat16 if kv == api.BF16 else torch.float8_e4m3fn


def raw(t):
    return t.view(torch.int16 if t.dtype == torch.bfloat16 else torch.uint8)


def bits(t):
    return t.contiguous().view(torch.uint8)


@pytest.mark.parametrize("kv", [api.BF16, api.E4M3], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("rope", [0, 4, 64, 512])
@pytest.mark.parametrize("xt", [torch.float32, torch.bfloat16])
def test_page_write(kv, rope, xt):
    p = api.default_params(kv_format=kv, rope_dim=rope)
    c = api.PagedCache(p, 12, 24, 3, 4, layers=2, device=DEV)
    raw(c.pool).fill_(0x41)
    c.table.copy_(i32([[3, 0, 11, -1], [7, 12, 1, 2], [-1, -1, -1, -1]]))
    seq = np.array([0, 0, 1, 0, -1, 1, 1, 2, 0, 5, 0, 0, 1, 1], np.int32)
    pos = np.array([0, 71, 95, 24, 3, 0, 30, 0, 72, 1, -2, 96, 96, 49], np.int32)
    N = len(seq)
    x = randn(N, 520, seed=9, dtype=xt)[:, :512] * 3
    x[0, 100:104] = torch.tensor([500.0, -500.0, 1e-4, -0.0], dtype=xt, device=DEV)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    before = bits(c.pool).clone()
    api.page_write(p, c, 1, x, i32(seq), i32(pos), st)
    # row 6 names a page past the pool, 7 and 8 entries without one, 9 a sequence out of
    # range; 10, 11, 12 positions outside the table's row
    assert st.item() == 1 | 2
    table = c.table.cpu().numpy()
    want = before.view(c.pool.shape[:3] + (-1,)).clone()
    good = [0, 1, 2, 3, 5, 13]
    ref, mag = rotate64(x[:, None], np.maximum(pos, 0), p, api.ROPE_PAIRS) if rope else (
        x[:, None].double().cpu().numpy(), np.zeros((N, 1, 512)))
    ref, mag = ref[:, 0], mag[:, 0]
    got = bits(c.pool).view(want.shape)
    for i in good:
        page, r = table[seq[i], pos[i] // 24], pos[i] % 24
        row = c.pool[1, page, r].float().cpu().numpy().astype(np.float64)
        flat = 512 - rope
        exact = x[i].float().clamp(-448, 448).to(dtype_of(kv)) if kv == api.E4M3 else x[i].bfloat16()
        assert torch.equal(bits(exact[:flat]), bits(c.pool[1, page, r, :flat])), i
        lim = np.clip(ref[i], -448, 448) if kv == api.E4M3 else ref[i]
        half = np.maximum(2.0 ** -4 * np.abs(lim), 2.0 ** -10) if kv == api.E4M3 else 2.0 ** -8 * np.abs(lim)
        assert np.all(np.abs(row - lim)[flat:] <= (half + 4 * 2.0 ** -24 * mag[i] * 2)[flat:]), i
        want[1, page, r] = got[1, page, r]
    assert torch.equal(got, want)  # no other row, page or layer was touched


# ------------------------------------------------------------------------------ the page table
class Model:
    """The table and the counts as the calls' descriptions have them, and each row's owner
    mark, in plain Python."""

    def __init__(self, c, params):
        self.ps = c.pool.shape[2]
        self.table, self.ref = c.table.cpu().numpy().copy(), c.ref.cpu().numpy().copy()
        self.pool = bits(c.pool).cpu().numpy().reshape(c.pool.shape[:3] + (-1,)).copy()
        self.status = 0

    def take(self):
        free = np.flatnonzero(self.ref <= 0)
        if not len(free):
            self.status |= 16
            return -1
        self.ref[free[0]] = 1
        return free[0]

    def reserve(self, seq, a, e):
        seen = set()
        for s, x, y in zip(seq, a, e):
            if s < 0:
                continue
            if s >= len(self.table) or s in seen:
                self.status |= 1
                continue
            seen.add(s)
            if x < 0 or y > self.table.shape[1] * self.ps:
                self.status |= 2
                continue
            for k in range(x // self.ps, -(-y // self.ps) if y > x else 0):
                if self.table[s, k] < 0:
                    self.table[s, k] = self.take()

    def release(self, seq, T=None, window=0, first=0):
        for i, s in enumerate(seq):
            if s < 0:
                continue
            if s >= len(self.table):
                self.status |= 1
                continue
            if T is not None and not 0 <= T[i] <= self.table.shape[1] * self.ps:
                self.status |= 2
                continue
            for k in range(self.table.shape[1]):
                if T is not None and not (window > 0 and k * self.ps >= first
                                          and (k + 1) * self.ps <= T[i] - window):
                    continue
                if self.table[s, k] >= 0:
                    self.ref[self.table[s, k]] -= 1
                    self.table[s, k] = -1

    def fork(self, parent, child, T):
        seen, todo = set(), []
        for p, ch, t in zip(parent, child, T):
            if ch < 0:
                continue
            dup = ch in seen
            seen.add(ch)
            if ch >= len(self.table) or not 0 <= p < len(self.table) or dup or ch in [
                    q for q, d in zip(parent, child) if d >= 0]:
                self.status |= 1
            elif not 0 <= t <= self.table.shape[1] * self.ps:
                self.status |= 2
            else:
                fresh = -1
                if t % self.ps:
                    src = self.table[p, t // self.ps]
                    if src < 0:
                        self.status |= 1
                    else:
                        fresh = self.take()
                        if fresh >= 0:
                            self.pool[:, fresh, :t % self.ps] = self.pool[:, src, :t % self.ps]
                todo.append((p, ch, t, fresh))
        for p, ch, t, fresh in todo:
            old = self.table[ch].copy()
            for k in range(self.table.shape[1]):
                g = self.table[p, k] if k < t // self.ps else -1
                if g >= 0:
                    self.ref[g] += 1
                self.table[ch, k] = fresh if k == t // self.ps else g
            for g in old[old >= 0]:
                self.ref[g] -= 1

    def compact(self):
        used = self.ref > 0
        n = int(used.sum())
        src = [g for g in range(n, len(self.ref)) if used[g]]
        dst = [g for g in range(n) if not used[g]]
        for a, b in zip(src, dst):
            self.pool[:, b] = self.pool[:, a]
            self.table[self.table == a] = b
            self.ref[b], self.ref[a] = self.ref[a], 0
        return n

    def check(self, c, st):
        assert np.array_equal(c.table.cpu().numpy(), self.table)
        assert np.array_equal(c.ref.cpu().numpy(), self.ref)
        assert np.array_equal(bits(c.pool).cpu().numpy().reshape(self.pool.shape), self.pool)
        assert st.item() == self.status


def cache_of(kv, n_pages, ps, seqs, wide, layers=1, seed=0):
    p = api.default_params(kv_format=kv)
    c = api.PagedCache(p, n_pages, ps, seqs, wide, layers=layers, device=DEV)
    raw(c.pool).random_(0, 100, generator=gen(seed))
    return p, c


@pytest.mark.parametrize("kv,n_pages,ps,seqs,wide,layers", [
    (api.BF16, 40, 8, 6, 9, 2), (api.E4M3, 5000, 16, 40, 300, 1), (api.E4M3, 4099, 8, 70, 120, 3),
    (api.BF16, 1, 64, 1, 1, 1), (api.BF16, 9, 48, 1100, 3, 1),
    # more sequences, entries to fill and pages than the planning kernels keep on chip
    (api.E4M3, 9001, 8, 5000, 2, 1), (api.E4M3, 33_333, 8, 300, 400, 1)])
def test_page_table_calls_follow_the_model(kv, n_pages, ps, seqs, wide, layers):
    """A random run of reserve, fork, release (whole and behind a window) and compact,
    shared and exhausted pools included, compared after each call."""
    p, c = cache_of(kv, n_pages, ps, seqs, wide, layers)
    m, rng = Model(c, p), np.random.default_rng(n_pages)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    T = np.zeros(seqs, np.int64)
    for step in range(14):
        some = rng.permutation(seqs)[:int(rng.integers(1, seqs + 1))]
        kind = ["reserve", "reserve", "fork", "window", "release", "compact"][step % 6]
        if kind == "reserve":
            more = wide * ps // 2 if wide == 400 else 2 * ps
            to = np.minimum(T[some] + rng.integers(0, more + 1, len(some)), wide * ps)
            api.page_reserve(p, c, i32(some), i32(T[some]), i32(to), st)
            m.reserve(some, T[some], to)
            T[some] = to
        elif kind == "fork" and seqs > 1:
            half = max(1, len(some) // 2)
            child, parent = some[:half], rng.choice(np.setdiff1d(np.arange(seqs), some[:half]), half) \
                if half < seqs else some[:half]
            api.page_fork(p, c, i32(parent), i32(child), i32(T[parent]), st)
            m.fork(parent, child, T[parent])
            T[child] = T[parent]
        elif kind == "window":
            w, f = int(rng.integers(1, 3 * ps)), int(rng.integers(0, ps + 1))
            api.page_release(p, c, i32(some), i32(T[some]), w, f, st)
            m.release(some, T[some], w, f)
        elif kind == "release":
            some = some[:max(1, len(some) // 3)]
            api.page_release(p, c, i32(some), dev_status=st)
            m.release(some)
            T[some] = 0
        elif kind == "compact":
            n = torch.zeros(1, dtype=torch.int32, device=DEV)
            api.page_compact(p, c, n, st)
            assert n.item() == m.compact()
        m.check(c, st)


def test_page_table_calls_flag_and_skip_what_they_refuse():
    p, c = cache_of(api.BF16, 10, 16, 4, 3)
    m, st = Model(c, p), torch.zeros(1, dtype=torch.int32, device=DEV)
    # twice the same sequence, one out of range, padding, lengths below 0 and past the row
    for seq, a, e in (([0, 0, 4, -1, 1], [0] * 5, [20, 40, 8, 8, 17]), ([1, 2], [-1, 0], [30, 49]),
                      ([1], [17], [5]), ([3], [0], [48])):
        api.page_reserve(p, c, i32(seq), i32(a), i32(e), st)
        m.reserve(seq, a, e)
        m.check(c, st)
    # a child that is a parent, one listed twice, sequences and lengths out of range
    for par, ch, T in (([0, 0, 1], [1, 2, 2], [20, 20, 5]), ([0, 9], [7, 2], [5, 5]), ([-1], [2], [4]),
                       ([0], [2], [49]), ([0], [2], [-3]), ([0, 0], [-1, 2], [3, 0]), ([2], [1], [7])):
        api.page_fork(p, c, i32(par), i32(ch), i32(T), st)
        m.fork(par, ch, T)
        m.check(c, st)
    for seq, T in (([0, 0, 5], None), ([3, 3], [48, 49]), ([1], [-1])):
        api.page_release(p, c, i32(seq), None if T is None else i32(T), 8, 0, st)
        m.release(seq, T, 8)
        m.check(c, st)


def test_fork_and_reserve_without_a_free_page():
    p, c = cache_of(api.E4M3, 2, 8, 4, 2)
    m, st = Model(c, p), torch.zeros(1, dtype=torch.int32, device=DEV)
    api.page_reserve(p, c, i32([0, 1]), i32([0, 0]), i32([12, 3]), st)
    m.reserve([0, 1], [0, 0], [12, 3])
    m.check(c, st)
    assert st.item() == 16
    api.page_fork(p, c, i32([0, 0]), i32([2, 3]), i32([12, 8]), st)
    m.fork([0, 0], [2, 3], [12, 8])
    m.check(c, st)


# ------------------------------------------------------------------------------ attention
def attn64(p, c, layer, q, sink, rows, T, window, first):
    """(o, A, dz, F): the definition in 64 bits, A = sum p |v| / den [B, H, 512], the bound of
    the logits' error, and F = sum |v| + n |o|: the share a step that every weight may be off by
    has in the output."""
    ps, B, H = c.pool.shape[2], q.shape[0], q.shape[1]
    pool, table = c.pool[layer].float().double().cpu().numpy(), c.table.cpu().numpy()
    o, A, F = np.zeros((B, H, D)), np.zeros((B, H, D)), np.zeros((B, H, D))
    dz = 0.0
    for b in range(B):
        t = np.arange(min(max(int(T[b]), 0), table.shape[1] * ps))
        if window > 0:
            t = t[(t >= T[b] - window) | (t < first)]
        if rows[b] < 0 or rows[b] >= len(table):
            continue
        g = table[rows[b], t // ps]
        ok = (g >= 0) & (g < pool.shape[0])
        k = pool[g[ok], t[ok] % ps]
        if not len(k):
            continue
        qb = q[b].double().cpu().numpy()
        z = qb @ k.T * float(p.softmax_scale)
        dq = 2.0 ** -22 * np.abs(qb).max(1, keepdims=True) if p.kv_format == api.E4M3 else 0.0
        dz = max(dz, float(((np.abs(qb) * 512 * 2.0 ** -24 + dq) @ np.abs(k).T).max()) * float(p.softmax_scale))
        s = np.full((H, 1), -np.inf) if sink is None else sink.double().cpu().numpy()[:, None]
        mx = np.maximum(z.max(1, keepdims=True), s)
        e = np.exp(z - mx)
        den = e.sum(1, keepdims=True) + np.exp(s - mx)
        o[b], A[b] = e @ k / den, e @ np.abs(k) / den
        F[b] = np.abs(k).sum(0) + len(k) * np.abs(o[b])
    return o, A, dz, F


def assert_attn(got, ref, kv):
    o, A, dz, F = ref
    g = got.double().cpu().numpy()
    u_p = 2.0 ** -8 if kv == api.BF16 else 2.0 ** -11
    # weights below fp32's normals (2^-126 of the largest) count as 0: at most 2,100
    # positions of |v| < 2^5 here, so 2^-109 in all. The three E5M2 parts of an f16 weight hold
    # it exactly, but for multiples of 2^-16, half a step off at most, when the largest weight
    # is 2^9 or more: 2^-26 of the sum of weights each, in the numerator (times |v|).
    step = 0.0 if kv == api.BF16 else 2.0 ** -26
    over = np.abs(g - o) - (2.0 ** -8 * np.abs(o) + (2 * u_p + 2 * dz + 2.0 ** -20) * A + step * F + 2.0 ** -109)
    assert over.max(initial=0) <= 0, over.max()
    n = np.linalg.norm(o)
    assert np.linalg.norm(g - o) <= 4e-3 * n, np.linalg.norm(g - o) / n


def filled(kv, heads, T, ps, seed, layers=1, spare=2, wide=0, window=0, first=0, scale=1.0):
    """A cache holding sequences of T positions on random pages; everything a query must not
    use (rows past the end, pages no one holds, pages behind the window) is NaN."""
    rng = np.random.default_rng(seed)
    T = np.asarray(T)
    need = -(-T // ps)
    wide = max(wide, int(need.max()), 1)
    n_pages = int(need.sum()) + spare
    p = api.default_params(kv_format=kv, heads=heads)
    c = api.PagedCache(p, n_pages, ps, len(T), wide, layers=layers, device=DEV)
    perm = rng.permutation(n_pages)
    table = np.full((len(T), wide), -1, np.int64)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = perm[at:at + n]
        at += n
    vals = (randn(layers, n_pages, ps, D, seed=seed) * scale)
    keep = np.zeros((n_pages, ps), bool)
    for b in range(len(T)):
        t = np.arange(T[b])
        if window > 0:
            t = t[(t >= T[b] - window) | (t < first)]
        keep[table[b, t // ps], t % ps] = True
    vals[:, ~torch.from_numpy(keep).to(DEV)] = float("nan")
    c.pool.copy_(vals.to(dtype_of(kv)))
    if window > 0:  # pages wholly behind the window are gone
        for b in range(len(T)):
            for k in range(need[b]):
                if k * ps >= first and (k + 1) * ps <= T[b] - window:
                    table[b, k] = -1
    c.table.copy_(i32(table))
    q = randn(len(T), heads, D, seed=seed + 1, dtype=torch.bfloat16) * 2
    return p, c, q.bfloat16(), randn(heads, seed=seed + 2)


def attend(p, c, q, sink, rows, T, window=0, first=0, layer=0, st=None, ws=None):
    out = torch.full(q.shape, 9.0, dtype=torch.bfloat16, device=DEV)
    ws = api.paged_attn_workspace(p, c, q.shape[0]) if ws is None else ws
    api.paged_attn(p, c, layer, q, sink, None if rows is None else i32(rows), i32(T), out, ws,
                   window=window, n_first=first, dev_status=st)
    return out


LENGTHS = [1, 2, 7, 8, 9, 63, 64, 65, 127, 128, 129, 255, 256, 257, 640, 1000, 0, 2049]


@pytest.mark.parametrize("kv", [api.BF16, api.E4M3], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("heads,ps,ctas", [(64, 64, 0), (64, 16, 1), (33, 8, 3), (32, 128, 0), (17, 24, 0),
                                           (16, 64, 5), (8, 1024, 0), (3, 32, 0), (1, 16, 2)])
def test_attention_ragged(kv, heads, ps, ctas):
    p, c, q, sink = filled(kv, heads, LENGTHS, ps, seed=heads + ps, layers=2)
    p.max_ctas = ctas
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    rows = np.arange(len(LENGTHS))
    for layer in (0, 1):
        out = attend(p, c, q, sink, None, LENGTHS, layer=layer, st=st)
        assert_attn(out, attn64(p, c, layer, q, sink, rows, LENGTHS, 0, 0), kv)
        assert torch.all(out[LENGTHS.index(0)] == 0)
    assert st.item() == 0


@pytest.mark.parametrize("kv", [api.BF16, api.E4M3], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("heads", [64, 20])
@pytest.mark.parametrize("window,first", [(1, 0), (1, 1), (100, 0), (128, 4), (129, 200), (1000, 128),
                                          (300, 129), (5000, 10), (256, 3000)])
def test_attention_window_and_first_tokens(kv, heads, window, first):
    T = [1, 2, 100, 101, 128, 129, 130, 257, 385, 1024, 1025, 3001, 5001]
    p, c, q, sink = filled(kv, heads, T, 16, seed=window + first, window=window, first=first)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    out = attend(p, c, q, sink, None, T, window, first, st=st)
    assert st.item() == 0
    assert_attn(out, attn64(p, c, 0, q, sink, np.arange(len(T)), T, window, first), kv)


@pytest.mark.parametrize("seed", range(24))
def test_attention_random_batches(seed):
    """Batches of both schedules (at most as many sequences as CTAs, and more), any page size,
    head count, window and grid, empty sequences and padding among them."""
    rng = np.random.default_rng(1000 + seed)
    kv = [api.BF16, api.E4M3][seed % 2]
    B = int(rng.choice([1, 2, 3, 9, 40, 153, 300]))
    top = int(min(4000, 30000 // B))
    T = rng.integers(0, top + 1, B) * (rng.random(B) < 0.9)
    T[0] = top
    heads, ps = int(rng.integers(1, 65)), 8 * int(rng.choice([1, 2, 3, 4, 7, 8, 16, 20, 32, 128]))
    window = int(rng.choice([0, 1, rng.integers(1, top + 200), 128, 256]))
    first = int(rng.choice([0, 1, 100, 128, 300])) if window else 0
    p, c, q, sink = filled(kv, heads, T, ps, seed=seed, window=window, first=first)
    p.max_ctas = int(rng.choice([0, 0, 1, 2, 7, 41, 150]))
    rows = rng.permutation(B)
    rows[rng.random(B) < 0.1] = -1
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    lens = np.where(rows >= 0, T[np.maximum(rows, 0)], 17)
    out = attend(p, c, q, sink, rows, lens, window, first, st=st)
    assert st.item() == 0
    live = rows >= 0
    assert torch.all(out[torch.from_numpy(~live).to(DEV)] == 9)
    if live.any():
        o, A, dz, F = attn64(p, c, 0, q, sink, rows, lens, window, first)
        if np.linalg.norm(o[live]) > 0:
            assert_attn(out[torch.from_numpy(live).to(DEV)], (o[live], A[live], dz, F[live]), kv)


@pytest.mark.parametrize("kv", [api.BF16, api.E4M3], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("ctas,B", [(1, 1), (2, 2), (3, 3), (4, 3), (3, 4), (152, 151), (0, 160)])
def test_attention_one_piece_or_ranges_at_the_border(kv, ctas, B):
    T = [700 + 37 * (b % 5) for b in range(B)]
    p, c, q, sink = filled(kv, 40, T, 32, seed=ctas + B)
    p.max_ctas = ctas
    out = attend(p, c, q, sink, None, T)
    assert_attn(out, attn64(p, c, 0, q, sink, np.arange(B), T, 0, 0), kv)


@pytest.mark.parametrize("kv", [api.BF16, api.E4M3], ids=["bf16", "e4m3"])
def test_attention_long_and_split(kv):
    """One sequence over every CTA, and a few that share them unevenly; the same bytes in
    every run."""
    for T in ([40000], [1, 30011, 5, 12800]):
        p, c, q, sink = filled(kv, 64, T, 64, seed=len(T))
        out = attend(p, c, q, sink, None, T)
        assert_attn(out, attn64(p, c, 0, q, sink, np.arange(len(T)), T, 0, 0), kv)
        for _ in range(3):
            assert torch.equal(attend(p, c, q, sink, None, T), out)


@pytest.mark.parametrize("kv", [api.BF16, api.E4M3], ids=["bf16", "e4m3"])
def test_attention_of_more_sequences_than_threads(kv):
    rng = np.random.default_rng(4)
    T = rng.integers(0, 40, 1500)
    p, c, q, sink = filled(kv, 2, T, 8, seed=5)
    out = attend(p, c, q, sink, None, T)
    assert_attn(out, attn64(p, c, 0, q, sink, np.arange(len(T)), T, 0, 0), kv)


@pytest.mark.parametrize("kv", [api.BF16, api.E4M3], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("heads", [64, 16])
def test_attention_sees_exactly_its_positions(kv, heads):
    """A key along the query outweighs all others: the output is its row if it is seen, and
    not if it lies just outside."""
    T, window, first = [1300], 500, 130
    for at, seen in ((0, True), (129, True), (130, False), (799, False), (800, True), (1299, True),
                     (1023, True), (1024, True)):
        p, c, q, _ = filled(kv, heads, T, 16, seed=7)
        c.pool.copy_(randn(*c.pool.shape, seed=8).to(c.pool.dtype))  # nothing is NaN here
        page = c.table[0, at // 16].item()
        # all heads alike; z = 8 * 512 / sqrt(512) = 181 against |z| < 8 * 6 of the others
        sign = torch.sign(randn(D, seed=9))
        c.pool[0, page, at % 16] = sign.to(c.pool.dtype)
        q = (8 * sign).bfloat16().expand(1, heads, D).contiguous()
        out = attend(p, c, q, None, None, T, window, first).float()
        near = (out - sign).abs().max().item()
        assert (near < 1e-2) == seen, (at, near)


@pytest.mark.parametrize("kv", [api.BF16, api.E4M3], ids=["bf16", "e4m3"])
def test_attention_sinks_and_large_logits(kv):
    T = [5, 300, 0, 1200]
    p, c, q, _ = filled(kv, 64, T, 32, seed=11)
    q = (q.float() * 20).bfloat16()  # logits to +-200: the running maximum moves
    rows = np.arange(4)
    lowest = torch.finfo(torch.float32).min
    base = attend(p, c, q, None, None, T)
    assert_attn(base, attn64(p, c, 0, q, None, rows, T, 0, 0), kv)
    for s in (-math.inf, lowest):
        sink = torch.full((64,), s, device=DEV)
        assert torch.equal(attend(p, c, q, sink, None, T), base), s
    sink = torch.linspace(-300, 300, 64, device=DEV)
    assert_attn(attend(p, c, q, sink, None, T), attn64(p, c, 0, q, sink, rows, T, 0, 0), kv)
    big = torch.full((64,), 1e30, device=DEV)  # the sink takes everything
    assert torch.all(attend(p, c, q, big, None, T) == 0)


@pytest.mark.parametrize("kv", [api.BF16, api.E4M3], ids=["bf16", "e4m3"])
def test_attention_rising_logits_rescale(kv):
    """Later tiles outweigh earlier ones by more each time, so every tile moves the maximum."""
    T = [1100]
    p, c, q, sink = filled(kv, 64, T, 64, seed=12)
    p.max_ctas = 1
    sign = torch.sign(randn(D, seed=13))
    ramp = torch.arange(T[0], device=DEV).float() / 400
    rows = (sign[None] * ramp[:, None] * 0.5 + randn(T[0], D, seed=14) * 0.25)
    g = c.table[0].long().repeat_interleave(64)[:T[0]]
    c.pool[0, g, torch.arange(T[0], device=DEV) % 64] = rows.to(c.pool.dtype)
    q = (4 * sign[None, None] + randn(1, 64, D, seed=15) * 0.1).bfloat16()
    assert_attn(attend(p, c, q, sink, None, T), attn64(p, c, 0, q, sink, [0], T, 0, 0), kv)


@pytest.mark.parametrize("kv", [api.BF16, api.E4M3], ids=["bf16", "e4m3"])
def test_attention_rows_padding_strides_and_flags(kv):
    T0 = [300, 20, 700, 129]
    p, c, q0, sink = filled(kv, 24, T0, 16, seed=21)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    wide = randn(7, 30, 600, seed=22, dtype=torch.bfloat16)
    q = wide[:, 3:27, 40:552]  # heads of a wider projection
    rows = np.array([2, -1, 0, 2, 3, -1, 1])
    T = np.array([700, 50, 300, 650, 100, 9, 20])
    out = attend(p, c, q, sink, rows, T, st=st)
    assert st.item() == 0
    ref = attn64(p, c, 0, q, sink, rows, T, 0, 0)
    live = rows >= 0
    assert_attn(out[torch.from_numpy(live).to(DEV)], (ref[0][live], ref[1][live], ref[2], ref[3][live]), kv)
    assert torch.all(out[1] == 9) and torch.all(out[5] == 9)  # padding is left as it was
    # a length below 0 sees nothing, one past the table is cut
    wide_T = c.table.shape[1] * 16
    c.pool.copy_(randn(*c.pool.shape, seed=23).to(c.pool.dtype))
    out = attend(p, c, q[:2], sink, [2, 0], [wide_T + 5, -1], st=st)
    assert st.item() == 2
    assert torch.all(out[1] == 0)
    assert_attn(out, attn64(p, c, 0, q[:2], sink, [2, 0], [wide_T, 0], 0, 0), kv)
    # a sequence out of range, pages missing or outside the pool: not seen, and flagged
    st.zero_()
    out = attend(p, c, q[:1], sink, [4], [10], st=st)
    assert st.item() == 1 and torch.all(out == 0)
    st.zero_()
    c.table[0, 3], c.table[0, 5], c.table[0, 18] = -1, c.pool.shape[1], 1 << 30
    out = attend(p, c, q[:1], sink, [0], [300], st=st)
    assert st.item() == 1
    assert_attn(out, attn64(p, c, 0, q[:1], sink, [0], [300], 0, 0), kv)
    c.table[0] = -1
    assert torch.all(attend(p, c, q[:1], sink, [0], [300], st=st) == 0)


def test_attention_nan_that_is_seen_reaches_the_output():
    p, c, q, sink = filled(api.BF16, 8, [200, 200], 16, seed=31)
    c.pool[0, c.table[1, 3].item(), 5, 100] = float("nan")
    out = attend(p, c, q, sink, None, [200, 200])
    assert torch.isfinite(out[0]).all() and torch.isnan(out[1]).all()


@pytest.mark.parametrize("heads", [5, 16, 64])
def test_attention_e4m3_queries_of_a_wide_range(heads):
    """The query's two E4M3 parts: channels down to 2^-18 of a head's largest, heads from 2^-40 on."""
    p, c, q, sink = filled(api.E4M3, heads, [700, 129], 16, seed=35)
    g = torch.Generator(device=DEV).manual_seed(36)
    q = q.float() * torch.exp2(-torch.randint(0, 19, q.shape, generator=g, device=DEV).float())
    q = (q * torch.exp2(torch.randint(-40, 4, q.shape[:2], generator=g, device=DEV).float())[..., None]).bfloat16()
    assert_attn(attend(p, c, q, sink, None, [700, 129]), attn64(p, c, 0, q, sink, [0, 1], [700, 129], 0, 0), api.E4M3)


@pytest.mark.parametrize("heads", [16, 64])
@pytest.mark.parametrize("low,high", [(-16.0, 0.0), (-11.0, -10.0), (-6.0, -5.0)])
def test_attention_e4m3_long_tails(low, high, heads):
    """One position far above the others, whose weights reach below the smallest part of P:
    sums of 16-bit weights in 8-bit parts. The peak comes late, so the maximum moves."""
    T = 2049
    p, c, q, sink = filled(api.E4M3, heads, [T], 64, seed=37)
    g = torch.Generator(device=DEV).manual_seed(38)
    k0 = torch.rand(T, generator=g, device=DEV) * (high - low) + low
    k0[T - 300] = 0
    t = torch.arange(T, device=DEV)
    pool = c.pool[0].float()
    pool[c.table[0, t // 64].long(), t % 64, 0] = k0
    c.pool[0].copy_(pool.to(dtype_of(api.E4M3)))
    q = torch.zeros_like(q)
    q[..., 0] = 32
    sink = torch.full_like(sink, -100.0)
    assert_attn(attend(p, c, q, sink, None, [T]), attn64(p, c, 0, q, sink, [0], [T], 0, 0), api.E4M3)


def one_peak(kv, T, drop, heads, at, ctas=1):
    """(params, cache, q, ref) of a sequence in which position `at` weighs 1 and every other one
    2^-drop, for `ctas` CTAs. ref: the output in 64 bits, sum w |v| / den, that of the others alone,
    and max |v| [512], then the others' share of the weight. Channel 0 sets the logits, channel 1 is
    one everywhere, 2 and 3 are +-1 but zero at the peak, the rest random."""
    ps = 64
    n = -(-T // ps)
    p = api.default_params(kv_format=kv, heads=heads)
    p.max_ctas, p.softmax_scale = ctas, drop * math.log(2) / 512
    rows = randn(64, D, seed=T % 1000).to(dtype_of(kv)).bfloat16().repeat(n, 1)
    rows[:, 0], rows[:, 1], rows[:, 2], rows[:, 3] = -16, 1, 1, -1
    rows[at] = 0
    rows[at, 1] = 1
    c = api.PagedCache(p, pool=rows.to(dtype_of(kv)).view(1, n, ps, D), device=DEV,
                       table=i32(np.arange(n)[None]), ref=i32(np.ones(n)))
    total, size = torch.zeros(2, D, dtype=torch.float64, device=DEV)
    for i in range(0, T, 1 << 16):
        part = rows[i:min(T, i + (1 << 16))].double()
        total += part.sum(0)
        size += part.abs().sum(0)
    w, peak = 2.0 ** -drop, rows[at].double()
    q = torch.zeros(1, heads, D, dtype=torch.bfloat16, device=DEV)
    q[..., 0] = 32
    den, others = 1 + w * (T - 1), w * (size - peak.abs())
    return p, c, q, ((peak + w * (total - peak)) / den, (peak.abs() + others) / den, others / den,
                     rows.abs().amax(0).double(), 1 - 1 / den)


@pytest.mark.parametrize("heads", [16, 64])
@pytest.mark.parametrize("T", [300_000, 1_000_000])
def test_attention_e4m3_weights_below_the_parts_add_up_to_one(heads, T):
    """What the three parts of a weight leave out is left out of the sum too: a channel that is one
    everywhere comes out as one (whatever is off by less than 2^-9 rounds to it), although 0.4 and
    1.4 % of the weight lie below the last part's steps at these lengths."""
    p, c, q, _ = one_peak(api.E4M3, T, 26.1, heads, at=5)
    out = attend(p, c, q, None, None, [T])
    assert torch.all(out[..., 1] == 1), out[..., 1].min()


def assert_one_peak(got, ref, drop, u_p, lost):
    """A bound that does not grow with the length. The peak's weight is a power of two; the others
    are off by their rounding u_p, that of their logits (four fp32 roundings of `drop` in log2, times
    ln 2) and ex2's 2^-22, in numerator and denominator. For the 16,384 positions that meet in one
    accumulator a product's alignment to it, 2^-25 for each of at most three parts, and 2^-23 for
    each sum of at least 16 products: below 2^-23 a position, 2^-9 of the whole. `lost` of the
    largest weight for each of them, which the parts leave out, in numerator (times |v|) and
    denominator. Then the output's rounding."""
    o, A, others, V, share = ref
    tol = (u_p + 4 * drop * 2.0 ** -24 + 2.0 ** -22) * (others + share * o.abs())
    tol = tol + 2.0 ** -9 * A + 2.0 ** 14 * lost * (V + o.abs())
    over = (got.double() - o).abs() - (tol + 2.0 ** -8 * (o.abs() + tol))
    assert over.max().item() <= 0, (over.max().item(), over.argmax().item() % D)


@pytest.mark.parametrize("heads", [16, 64])
@pytest.mark.parametrize("T,ctas,at", [(300_000, 1, 5), (300_000, 2, 299_000), (1_000_000, 1, 9), (1_000_000, 3, 700_000)])
@pytest.mark.parametrize("drop", [24.4, 25.4, 26.1, 28.0])
def test_attention_e4m3_tails_of_long_contexts(drop, T, ctas, at, heads):
    """Weights about the steps of a weight's last part and below, whose share grows with the length:
    one position above a million others, many of them to a CTA."""
    p, c, q, ref = one_peak(api.E4M3, T, drop, heads, at, ctas)
    assert_one_peak(attend(p, c, q, None, None, [T]), ref, drop, 2.0 ** -11, 2.0 ** -26)


@pytest.mark.parametrize("heads", [16, 64])
@pytest.mark.parametrize("ctas,at", [(1, 9), (1, 999_990), (3, 700_000)])
@pytest.mark.parametrize("drop", [24.5, 25.4, 26.1, 28.0])
def test_attention_bf16_tails_of_long_contexts(drop, ctas, at, heads):
    """bf16 weights have no steps to fall below, but the tensor cores align each product to the
    accumulator: of 2^-25.4 beside one nothing is left, so a CTA that added a million of them to
    one accumulator lost their 2.2 %."""
    p, c, q, ref = one_peak(api.BF16, 1_000_000, drop, heads, at, ctas)
    out = attend(p, c, q, None, None, [1_000_000])
    assert_one_peak(out, ref, drop, 2.0 ** -8, 0.0)


@pytest.mark.parametrize("kv", [api.BF16, api.E4M3], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("ctas,T,window,first", [
    (1, [40_000], 0, 0), (1, [16_384, 16_385, 32_768, 100, 32_897], 0, 0), (2, [60_000, 5, 34_000, 0, 17_000], 0, 0),
    (3, [90_000, 21_000], 0, 0), (2, [70_000], 40_000, 9000), (2, [17_500] * 4, 17_000, 3)])
@pytest.mark.parametrize("heads", [3, 33, 64])
def test_attention_long_pieces(kv, heads, ctas, T, window, first):
    """More tiles to a CTA than meet in one accumulator, in sequences that are cut and in whole
    ones, first, in the middle and last of a CTA's range; the same bytes in every run."""
    p, c, q, sink = filled(kv, heads, T, 64, seed=heads + ctas, window=window, first=first)
    p.max_ctas = ctas
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    ws = torch.full_like(api.paged_attn_workspace(p, c, len(T)), 0xFF)  # NaN, wherever it is read unwritten
    out = attend(p, c, q, sink, None, T, window, first, st=st, ws=ws)
    assert st.item() == 0
    assert_attn(out, attn64(p, c, 0, q, sink, np.arange(len(T)), T, window, first), kv)
    assert torch.equal(attend(p, c, q, sink, None, T, window, first, st=st, ws=ws), out)


@pytest.mark.parametrize("heads", [16, 64])
def test_attention_e4m3_nan_and_infinity(heads):
    """A NaN that is seen reaches every head of its sequence; an infinite query its head only."""
    p, c, q, sink = filled(api.E4M3, heads, [300, 200], 16, seed=39)
    ref = attend(p, c, q, sink, None, [300, 200])
    q2 = q.clone()
    q2[1, 3, 100] = float("inf")
    out = attend(p, c, q2, sink, None, [300, 200])
    assert out[1, 3].isnan().all()
    out[1, 3] = ref[1, 3]
    assert torch.equal(out, ref)
    pool = c.pool[0].view(torch.uint8)
    pool[c.table[0, 150 // 16].long(), 150 % 16, 7] = 0x7F
    out = attend(p, c, q, sink, None, [300, 200])
    assert out[0].isnan().all() and torch.equal(out[1], ref[1])


def test_attention_wide_values_of_bf16():
    """Latents beyond fp16's range stay exact in bf16 pages."""
    p, c, q, sink = filled(api.BF16, 64, [333], 16, seed=33, scale=1e6)
    p.softmax_scale = 1e-7
    assert_attn(attend(p, c, q, sink, None, [333]), attn64(p, c, 0, q, sink, [0], [333], 0, 0), api.BF16)


# ------------------------------------------------------------------------------ together
@pytest.mark.parametrize("kv", [api.BF16, api.E4M3], ids=["bf16", "e4m3"])
def test_a_dense_layer_decodes_forks_and_compacts(kv):
    """A server's steps in one: prompts reserved, turned and written; each step appends one
    token per sequence, attends over window and first tokens and turns the outputs back;
    pages behind the window go; a sequence forks, both continue; the pool is compacted. The
    outputs follow the definition over the written rows throughout, and the captured step
    replays to the same bytes."""
    ps, W, F, H, S = 16, 96, 20, 12, 5
    p = api.default_params(kv_format=kv, rope_dim=64, heads=H)
    c = api.PagedCache(p, 64, ps, S, 40, device=DEV)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    ws = api.paged_attn_workspace(p, c, S)
    T = np.array([37, 150, 1, 0, 0])
    seqs, sink = np.array([0, 1, 2]), randn(H, seed=1)
    api.page_reserve(p, c, i32(seqs), i32(T[seqs] * 0), i32(T[seqs]), st)
    sq = np.repeat(seqs, T[seqs])
    ps_ = np.concatenate([np.arange(T[s]) for s in seqs])
    api.page_write(p, c, 0, randn(len(sq), D, seed=2), i32(sq), i32(ps_), st)
    for step in range(12):
        if step == 4:  # sequence 1 goes on as 3 too
            api.page_fork(p, c, i32([1]), i32([3]), i32([T[1]]), st)
            T[3] = T[1]
            seqs = np.array([0, 1, 2, 3])
        if step == 8:
            n = torch.zeros(1, dtype=torch.int32, device=DEV)
            api.page_release(p, c, i32([0]), dev_status=st)
            api.page_compact(p, c, n, st)
            seqs = np.array([1, 2, 3])
            held = c.table[c.table >= 0].unique()
            assert n.item() == held.numel() and held.max().item() == n.item() - 1
            assert torch.equal(c.ref > 0, torch.arange(64, device=DEV) < n.item())
        B = len(seqs)
        x, q = randn(B, D, seed=100 + step), randn(B, H, D, seed=200 + step, dtype=torch.bfloat16) * 2
        sq, t0, t1 = i32(seqs), i32(T[seqs]), i32(T[seqs] + 1)
        out = torch.empty_like(q)

        def one():
            api.page_reserve(p, c, sq, t0, t1, st)
            api.page_write(p, c, 0, x, sq, t0, st)
            qr = api.rope(p, q, t0)
            api.paged_attn(p, c, 0, qr, sink, sq, t1, out, ws, window=W, n_first=F, dev_status=st)
            api.page_release(p, c, sq, t1, W, F, st)
            return qr, api.rope(p, out, t0, inverse=True)

        qr, back = one()
        T[seqs] += 1
        first = out.clone()
        assert_attn(out, attn64(p, c, 0, qr, sink, seqs, T[seqs], W, F), kv)
        ref, mag = rotate64(out, T[seqs] - 1, p, api.ROPE_PAIRS, inverse=True)
        assert_rotated(back, ref, mag, U[torch.bfloat16])
        if step in (3, 9):  # the same step as a graph, on a side stream
            side = torch.cuda.Stream()
            side.wait_stream(torch.cuda.current_stream())
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=side):
                one()
            for _ in range(2):
                out.zero_()
                graph.replay()
                torch.cuda.synchronize()
                assert torch.equal(out, first)
    assert st.item() == 0
    used = c.table[c.table >= 0]
    counts = torch.bincount(used.long(), minlength=64)
    assert torch.equal(counts.int(), c.ref)


@pytest.mark.parametrize("kv", [api.BF16, api.E4M3], ids=["bf16", "e4m3"])
def test_offsets_past_32_bits_and_positions_past_a_million(kv):
    """Pages beyond 4 GB of a pool and beyond a layer's 4 GB, held at the far end of a long
    table: written, forked, attended through a window, compacted to the front."""
    n_pages = 70_001 if kv == api.BF16 else 140_001
    ps, T, W, F = 64, 1_000_003, 300, 5
    p = api.default_params(kv_format=kv, heads=16)
    c = api.PagedCache(p, n_pages, ps, 3, 16_000, layers=2, device=DEV)
    assert c.pool[0].numel() * c.pool.element_size() > 1 << 32
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    c.ref[:n_pages - 9] = 1  # taken by others: the lowest free page is far out
    at = np.concatenate([np.arange(F), np.arange(T - W, T)])
    api.page_reserve(p, c, i32([1]), i32([0]), i32([F]), st)
    api.page_reserve(p, c, i32([1]), i32([T - W]), i32([T]), st)
    held = c.table[1][c.table[1] >= 0]
    assert st.item() == 0 and held.min().item() == n_pages - 9
    assert held.numel() == 1 + 6  # page 0, and 15,620 (from 999,703) to 15,625 (to 1,000,002)
    x = randn(len(at), D, seed=3)
    for layer in (0, 1):
        api.page_write(p, c, layer, x * (layer + 1), i32(np.ones(len(at))), i32(at), st)
    api.page_fork(p, c, i32([1]), i32([2]), i32([T]), st)
    q, sink = randn(1, 16, D, seed=4, dtype=torch.bfloat16), randn(16, seed=5)
    k64 = {}
    for layer in (0, 1):
        rows = (x * (layer + 1)).to(dtype_of(kv)).double().cpu().numpy()
        z = q[0].double().cpu().numpy() @ rows.T * float(p.softmax_scale)
        sk = sink.double().cpu().numpy()[:, None]
        e, es = np.exp(z - z.max()), np.exp(sk - z.max())
        den = e.sum(1, keepdims=True) + es
        o = e @ rows / den
        k64[layer] = (o[None], (e @ np.abs(rows) / den)[None], 512 * 2.0 ** -24 * 40, np.abs(rows).sum(0)[None] + len(at) * np.abs(o)[None])
    for row in (1, 2):
        for layer in (0, 1):
            assert_attn(attend(p, c, q, sink, [row], [T], W, F, layer=layer, st=st), k64[layer], kv)
    c.ref[:n_pages - 9] = 0
    n = torch.zeros(1, dtype=torch.int32, device=DEV)
    api.page_compact(p, c, n, st)
    # those 7, and the fork's copy of the last, which holds 3 rows
    assert n.item() == 8 and c.table.max().item() == 7 and st.item() == 0
    for row in (1, 2):
        for layer in (0, 1):
            assert_attn(attend(p, c, q, sink, [row], [T], W, F, layer=layer, st=st), k64[layer], kv)


def test_two_streams_with_workspaces_of_their_own():
    p, c, q, sink = filled(api.BF16, 64, [3000, 500], 64, seed=41)
    alone = attend(p, c, q, sink, None, [3000, 500])
    streams = [torch.cuda.Stream() for _ in range(2)]
    spaces = [api.paged_attn_workspace(p, c, 2) for _ in range(2)]
    outs = [torch.empty_like(q) for _ in range(2)]
    T = i32([3000, 500])
    torch.cuda.synchronize()
    for _ in range(10):
        for s, w, o in zip(streams, spaces, outs):
            api.paged_attn(p, c, 0, q, sink, None, T, o, w, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(outs[0], alone) and torch.equal(outs[1], alone)


def test_strides_of_single_rows_and_heads_do_not_count():
    """A single sequence, head or row cut out of tensors with odd strides, and a side stream."""
    p, c, q, sink = filled(api.BF16, 1, [300], 16, seed=61)
    odd = torch.zeros(1, 1, 512, dtype=torch.bfloat16, device=DEV).as_strided((1, 1, 512), (513, 517, 1))
    odd.copy_(q)
    assert torch.equal(attend(p, c, odd, sink, None, [300]), attend(p, c, q, sink, None, [300]))
    x = randn(1, D, seed=62)
    p2, c2 = api.default_params(kv_format=api.BF16), api.PagedCache(p, 2, 16, 1, 2, device=DEV)
    api.page_reserve(p2, c2, i32([0]), i32([0]), i32([1]))
    api.page_write(p2, c2, 0, x.as_strided((1, D), (D + 1, 1)), i32([0]), i32([0]))
    assert torch.equal(c2.pool[0, c2.table[0, 0].item(), 0], x[0].bfloat16())
    p3 = api.default_params(rope_dim=64)
    side, y = torch.cuda.Stream(), randn(1, 1, D, seed=63)
    ref = api.rope(p3, y, i32([7]))
    pos = i32([7])
    side.wait_stream(torch.cuda.current_stream())
    got = api.rope(p3, y.as_strided((1, 1, D), (D + 3, D + 1, 1)), pos, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got, ref)


def test_a_new_tensor_on_a_side_stream_is_not_in_use_elsewhere():
    """The current stream lets go of a block that work queued there has still to write; a call on a
    side stream that waits for none of it must not get that block for its output."""
    p, side = api.default_params(rope_dim=64), torch.cuda.Stream()
    with torch.cuda.stream(side):
        x = torch.randn(4096, 8, 128, device=DEV)
        pos = torch.arange(4096, dtype=torch.int32, device=DEV)
        ref = api.rope(p, x, pos)
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    block = torch.empty_like(x)
    torch.cuda._sleep(1)
    block.fill_(1)  # (the kernels are loaded: nothing below waits for the device)
    torch.cuda.synchronize()
    torch.cuda._sleep(200_000_000)  # about a tenth of a second
    block.fill_(7)
    del block
    got = api.rope(p, x, pos, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(got, ref)


def test_calls_name_what_they_refuse():
    p, c, q, sink = filled(api.BF16, 8, [20], 16, seed=51)
    small = torch.empty(256, dtype=torch.uint8, device=DEV)
    T, out = i32([20]), torch.empty_like(q)
    with pytest.raises(api.Csa2Error, match="workspace smaller"):
        api.paged_attn(p, c, 0, q, sink, None, T, out, small)
    ws = api.paged_attn_workspace(p, c, 1)
    with pytest.raises(api.Csa2Error, match="layer out of range"):
        api.paged_attn(p, c, 1, q, sink, None, T, out, ws)
    with pytest.raises(api.Csa2Error, match="int32"):
        api.paged_attn(p, c, 0, q, sink, None, T.long(), out, ws)
    with pytest.raises(api.Csa2Error, match="is on cpu"):
        api.paged_attn(p, c, 0, q, sink, None, T.cpu(), out, ws)
    with pytest.raises(api.Csa2Error, match="max_seqs"):
        api.page_reserve(p, c, *[i32(np.zeros(1025))] * 3)

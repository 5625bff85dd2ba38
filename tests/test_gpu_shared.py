"""Slot maps, prefix groups and the attention behind shared prefixes on the GPU: the first two against
plain models, exactly; the attention against its definition in 64 bits, within the bounds that
test_gpu_paged.py derives (weights rounded to the pages' matrix type in numerator and denominator
alike, fp32 sums, the output's rounding). A query on E4M3 pages is two E4M3 parts that hold it down to
2^-17 of its head's largest value."""
import math

import numpy as np
import pytest
import torch

from csa2_compressed_sparse_02_gb300 import api
from test_gpu_paged import D, DEV, assert_attn, assert_rotated, dtype_of, i32, randn, rotate64

pytestmark = pytest.mark.gpu
BOTH = pytest.mark.parametrize("kv", [api.BF16, api.E4M3], ids=["bf16", "e4m3"])


def status():
    return torch.zeros(1, dtype=torch.int32, device=DEV)


# ------------------------------------------------------------------------------ slot maps
def model_slots(table, ref, ps, seq, held, new, N):
    """(table, ref, n_after, start, row_seq, row_pos, row_slot, status) of csa2_page_slots."""
    table, ref, bits = table.copy(), ref.copy(), 0
    seqs, wide = table.shape
    after, start = held.astype(np.int64).copy(), [0]
    rows, taken, full = [], set(), False
    for i, (s, T, n) in enumerate(zip(seq.tolist(), held.tolist(), new.tolist())):
        good = s >= 0
        if s >= seqs or (s >= 0 and s in taken):
            bits, good = bits | 1, False
        elif s >= 0 and (T < 0 or n < 0 or T + n > wide * ps):
            bits, good = bits | 2, False
        taken.add(s)
        n = n if good else 0
        if n and (full or len(rows) + n > N):
            bits, full, n = bits | 2, True, 0
        if n:
            for k in range(T // ps, -(-(T + n) // ps)):
                if table[s, k] < 0:
                    free = np.flatnonzero(ref <= 0)
                    if len(free):
                        table[s, k] = free[0]
                        ref[free[0]] = 1
                    else:
                        bits |= 16
        after[i] = T + n
        rows += [(s, T + r) for r in range(n)]
        start.append(len(rows))
    rseq, rpos, slot = np.full(N, -1), np.full(N, -1), np.full(N, -1, np.int64)
    for r, (s, t) in enumerate(rows):
        rseq[r], rpos[r] = s, t
        if table[s, t // ps] >= 0:
            slot[r] = table[s, t // ps] * ps + t % ps
    return table, ref, after, np.asarray(start), rseq, rpos, slot, bits


def slots_of(kv, table, ref, ps, seq, held, new, N, alias=False):
    p = api.default_params(kv_format=kv)
    pool = torch.zeros(1, len(ref), ps, D, dtype=torch.int8, device=DEV).view(dtype_of(api.E4M3))
    c = api.PagedCache(p, pool=pool, table=i32(table), ref=i32(ref))
    out, st = api.SlotMap(len(seq), N, device=DEV), status()
    for t in (out.n_tokens, out.start, out.seq, out.pos, out.slot):
        t.fill_(77)
    T = i32(held)
    if alias:
        out.n_tokens = T
    api.page_slots(p, c, i32(seq), T, i32(new), out, st)
    return [t.cpu().numpy() for t in (c.table, c.ref, out.n_tokens, out.start, out.seq, out.pos, out.slot)] + [st.item()]


def random_table(rng, seqs, wide, ps, used, spare):
    """Rows that hold the pages of `used` positions each, on random pages."""
    n = -(-used // ps)
    pages = int(n.sum()) + spare
    perm, table, ref = rng.permutation(pages), np.full((seqs, wide), -1, np.int64), np.zeros(pages, np.int64)
    at = 0
    for s in range(seqs):
        table[s, :n[s]] = perm[at:at + n[s]]
        at += n[s]
    ref[perm[:at]] = 1
    return table, ref


@pytest.mark.parametrize("seed", range(16))
def test_slots_follow_the_model(seed):
    rng = np.random.default_rng(seed)
    seqs, ps = int(rng.choice([1, 5, 40, 300])), int(rng.choice([8, 16, 24, 64, 1024]))
    wide = int(rng.integers(2, 12))
    B = min(int(rng.integers(1, 2 * seqs + 3)), max(seqs, 1024))
    seq = rng.permutation(np.concatenate([np.arange(seqs), np.full(B, -1)]))[:B]
    held = rng.integers(0, wide * ps, seqs)
    table, ref = random_table(rng, seqs, wide, ps, held, int(rng.integers(0, 3 * seqs)))
    T = np.where(seq >= 0, held[np.maximum(seq, 0)], rng.integers(-5, 5, B))
    new = np.minimum(rng.choice([0, 1, 1, 3, ps, 5 * ps], B), wide * ps - np.maximum(T, 0))
    if seed % 4 == 1:  # what is refused
        seq[rng.integers(0, B)] = seqs + 3
        seq[rng.integers(0, B)] = seq[0]
        new[rng.integers(0, B)] = -1
        T[rng.integers(0, B)] = -2
        new[rng.integers(0, B)] = wide * ps + 1
    total = int(np.maximum(new, 0)[seq >= 0].sum())
    N = [total, total + 37, max(0, total - 1), total // 2, 0][seed % 5]
    for alias in (False, True):
        got = slots_of(api.E4M3, table, ref, ps, seq, T, new, N, alias)
        want = model_slots(table, ref, ps, seq, T, new, N)
        for name, g, w in zip(("table", "ref", "n_tokens", "start", "seq", "pos", "slot", "status"), got, want):
            assert np.array_equal(g, w), (name, alias)


@pytest.mark.parametrize("N", [4096, 4097, 60_000])
def test_slots_of_many_requests_and_rows(N):
    """More requests than the planning kernel has threads, rows for the second kernel, long lists of
    new pages."""
    rng = np.random.default_rng(N)
    seqs, ps, wide = 2500, 16, 20
    held = rng.integers(0, 200, seqs)
    table, ref = random_table(rng, seqs, wide, ps, held, 6000)
    seq = rng.permutation(seqs)
    new = rng.integers(0, 45, seqs)
    got = slots_of(api.E4M3, table, ref, ps, seq, held[seq], new, N)
    for g, w in zip(got, model_slots(table, ref, ps, seq, held[seq], new, N)):
        assert np.array_equal(g, w)


@pytest.mark.parametrize("spare", [40_000, 9_000, 3_000])
def test_slots_of_prompts(spare):
    """A thousand requests of several pages each, free pages here and there in a large pool, or too few of them."""
    rng = np.random.default_rng(spare)
    seqs, ps, wide = 1000, 8, 30
    held = rng.integers(0, 100, seqs)
    table, ref = random_table(rng, seqs, wide, ps, held, spare)
    seq = rng.permutation(seqs)
    new = rng.integers(0, 130, seqs)
    total = int(new.sum())
    for N in (total + 5, total - 300):
        got = slots_of(api.E4M3, table, ref, ps, seq, held[seq], new, N)
        for g, w in zip(got, model_slots(table, ref, ps, seq, held[seq], new, N)):
            assert np.array_equal(g, w)


def test_slots_of_lengths_that_reach_31_bits():
    """A table whose rows hold more positions than 31 bits: a request up to the last of those is served, one
    that passes it is refused, and the ones around it stand."""
    most, ps, wide = 2 ** 31 - 1, 1024, 2_100_000
    p = api.default_params(kv_format=api.E4M3)
    pool = torch.zeros(1, 8, ps, D, dtype=torch.int8, device=DEV).view(dtype_of(api.E4M3))
    for held, new, bits in (([most - 3, 5, 70], [3, 2, 1], 0), ([most - 3, 5, 70], [4, 2, 1], 2),
                            ([most - 47, 5, 70], [100, 2, 1], 2), ([most, 5, 70], [1, 2, 1], 2),
                            ([most, 5, 70], [0, 2, 1], 0), ([7, 5, 70], [most, 2, 1], 2)):
        c = api.PagedCache(p, pool=pool, table=torch.full((3, wide), -1, dtype=torch.int32, device=DEV),
                           ref=torch.zeros(8, dtype=torch.int32, device=DEV))
        out, st, taken = api.SlotMap(3, 8, device=DEV), status(), new[0] if not bits else 0
        api.page_slots(p, c, i32([1, 0, 2]), i32(held), i32(new), out, st)
        assert st.item() == bits
        assert out.n_tokens.tolist() == [held[0] + taken, 7, 71] and out.start.tolist() == [0, taken, taken + 2, taken + 3]
        rest = 8 - taken - 3
        assert out.seq.tolist() == [1] * taken + [0, 0, 2] + [-1] * rest
        assert out.pos.tolist() == [held[0] + r for r in range(taken)] + [5, 6, 70] + [-1] * rest
        page = 1 if taken else 0  # the lowest free pages, in the order of the call
        first = [(held[0] + r) % ps for r in range(taken)]
        assert out.slot.tolist() == first + [page * ps + 5, page * ps + 6, (page + 1) * ps + 70] + [-1] * rest
        assert int((c.table >= 0).sum()) == page + 2 == int(c.ref.sum())
        if taken:
            assert c.table[1, (most - 3) // ps].item() == 0


def test_slots_without_requests_or_pages():
    table, ref = np.full((3, 4), -1), np.zeros(5, np.int64)
    none = np.zeros(0, np.int64)
    got = slots_of(api.E4M3, table, ref, 16, none, none, none, 6)
    assert got[3].tolist() == [0] and all((got[k] == -1).all() for k in (4, 5, 6)) and got[7] == 0
    seq = np.array([2, 0, 1])
    args = (table, ref, 16, seq, np.zeros(3, np.int64), np.array([40, 33, 17]))  # 3 + 3 + 2 pages of 5
    got = slots_of(api.E4M3, *args, 90)
    want = model_slots(*args, 90)
    assert want[7] == 16
    for g, w in zip(got, want):
        assert np.array_equal(g, w)


# ------------------------------------------------------------------------------ prefix groups
def model_groups(table, pages, ps, seq, T, least):
    B, (seqs, wide) = len(seq), table.shape
    row = np.where((seq >= 0) & (seq < seqs), seq, -1)
    n = np.where(row < 0, 0, np.clip(T, 0, wide * ps))
    key = {}
    lead, common = np.arange(B), np.zeros(B, np.int64)
    for b in range(B):
        if n[b] < least or (least - 1) // ps >= wide:
            continue
        g = table[row[b], (least - 1) // ps]
        if not 0 <= g < pages:
            continue
        l = key.setdefault(int(g), b)
        if l == b:
            continue
        k, most = 0, min(n[b], n[l])
        while k * ps < most and table[row[b], k] == table[row[l], k] and 0 <= table[row[b], k] < pages:
            k += 1
        common[b] = min(most, k * ps)
        if common[b] >= least:
            lead[b] = l
    order, first, shared = [], [], []
    for l in range(B):
        m = [b for b in range(B) if lead[b] == l and seq[b] >= 0]
        least_of = min((int(common[b]) for b in m if b != l), default=0)
        first += [len(order)] * len(m)
        order += m
        shared += [least_of] * len(m)
    for b in range(B):
        if seq[b] < 0:
            first.append(len(order))
            order.append(b)
            shared.append(0)
    return np.asarray(order), np.asarray(first), np.asarray(shared)


def groups_of(table, pages, ps, seq, T, least, st=None):
    p = api.default_params(kv_format=api.E4M3)
    pool = torch.zeros(1, pages, ps, D, dtype=torch.int8, device=DEV).view(dtype_of(api.E4M3))
    c = api.PagedCache(p, pool=pool, table=i32(table), ref=i32(np.ones(pages)))
    g = api.PrefixGroups(len(T), device=DEV)
    g.workspace.fill_(0xA5)
    api.prefix_groups(p, c, None if seq is None else i32(seq), i32(T), g, least=least, dev_status=st)
    return [t.cpu().numpy() for t in (g.order, g.first, g.shared)]


def forest(rng, seqs, wide, ps):
    """Rows of a table as forks of forks leave them: each continues some earlier row's first pages."""
    table, n, page = np.full((seqs, wide), -1, np.int64), np.zeros(seqs, np.int64), 0
    for s in range(seqs):
        n[s] = rng.integers(0, wide * ps + 1)
        k = 0
        if s and rng.random() < 0.8:
            o = int(rng.integers(0, s))
            k = int(rng.integers(0, min(n[s], n[o]) // ps + 1))
            table[s, :k] = table[o, :k]
        for j in range(k, -(-int(n[s]) // ps)):
            table[s, j] = page
            page += 1
    perm = rng.permutation(page + 3)
    return np.where(table >= 0, perm[np.maximum(table, 0)], -1), n, page + 3


@pytest.mark.parametrize("seed", range(20))
def test_groups_follow_the_model(seed):
    rng = np.random.default_rng(seed)
    seqs, ps, wide = int(rng.choice([1, 2, 7, 60])), int(rng.choice([8, 24, 64])), int(rng.choice([1, 5, 40, 300]))
    table, n, pages = forest(rng, seqs, wide, ps)
    B = int(rng.integers(1, 3 * seqs + 2))
    seq = rng.integers(0, seqs, B)  # the same one often
    T = np.maximum(0, n[seq] - rng.integers(0, 3, B))
    seq = np.where(rng.random(B) < 0.1, -1, seq)
    if seed % 3 == 2:  # entries without a page, or outside the pool
        table[rng.integers(0, seqs), rng.integers(0, wide)] = -1
        table[rng.integers(0, seqs), rng.integers(0, wide)] = pages + 7
    for least in (1, ps, ps + 1, 4 * ps, 200, 10 ** 9):
        st = status()
        got = groups_of(table, pages, ps, seq, T, least, st)
        assert st.item() == 0
        for g, w in zip(got, model_groups(table, pages, ps, seq, T, least)):
            assert np.array_equal(g, w), least


@pytest.mark.parametrize("B", [1023, 1024, 1025, 3000, 5000])
def test_groups_of_large_batches(B):
    rng = np.random.default_rng(B)
    table, n, pages = forest(rng, 400, 6, 16)
    seq = rng.integers(-1, 400, B)
    T = np.where(seq >= 0, n[np.maximum(seq, 0)], 5)
    for least in (1, 40):
        for g, w in zip(groups_of(table, pages, 16, seq, T, least), model_groups(table, pages, 16, seq, T, least)):
            assert np.array_equal(g, w)


def test_groups_flag_what_is_out_of_range():
    table = np.array([[0, 1], [0, 2], [0, 3]])
    for seq, T, bit in (([0, 3, 1], [20, 20, 20], 1), ([0, 2, 1], [20, -1, 20], 2), ([0, 2, 1], [20, 33, 20], 2)):
        st = status()
        got = groups_of(table, 5, 16, np.array(seq), np.array(T), 1, st)
        assert st.item() == bit
        for g, w in zip(got, model_groups(table, 5, 16, np.array(seq), np.array(T), 1)):
            assert np.array_equal(g, w)
    assert [x.tolist() for x in groups_of(table, 5, 16, None, np.array([20, 17, 9]), 1)] == [[0, 1, 2], [0] * 3, [9] * 3]


# ------------------------------------------------------------------------------ attention
def shared64(p, c, layer, q, sink, seq, T, order, first, shared):
    """(o, A, dz, F) of every sequence of the call, as test_gpu_paged.attn64 gives them: positions below
    the group's shared ones through its first sequence's row, the others through its own."""
    ps, (B, H, _) = c.pool.shape[2], q.shape
    pool, table = c.pool[layer].float().double().cpu().numpy(), c.table.cpu().numpy()
    o, A, F, dz = np.zeros((B, H, D)), np.zeros((B, H, D)), np.zeros((B, H, D)), 0.0
    for i, b in enumerate(order):
        if not 0 <= b < B or not 0 <= seq[b] < len(table):
            continue
        lead, sh = order[first[i]], shared[first[i]]
        if not 0 <= seq[lead] < len(table):
            sh = 0
        t = np.arange(min(max(int(T[b]), 0), table.shape[1] * ps))
        row = np.where(t < sh, seq[lead], seq[b])
        g = np.where((row >= 0) & (row < len(table)), table[np.clip(row, 0, len(table) - 1), t // ps], -1)
        ok = (g >= 0) & (g < pool.shape[0])
        k = pool[g[ok], t[ok] % ps]
        if not len(k):
            continue
        qb = q[b].double().cpu().numpy()
        z = qb @ k.T * float(p.softmax_scale)
        dq = 2.0 ** -17 * np.abs(qb).max(1, keepdims=True) if p.kv_format == api.E4M3 else 0.0
        dz = max(dz, float(((np.abs(qb) * 512 * 2.0 ** -24 + dq * (np.abs(qb) < 2.0 ** -10 * np.abs(qb).max(1, keepdims=True)))
                            @ np.abs(k).T).max()) * float(p.softmax_scale))
        s = np.full((H, 1), -np.inf) if sink is None else sink.double().cpu().numpy()[:, None]
        mx = np.maximum(z.max(1, keepdims=True), s)
        e = np.exp(z - mx)
        den = e.sum(1, keepdims=True) + np.exp(s - mx)
        o[b], A[b] = e @ k / den, e @ np.abs(k) / den
        F[b] = np.abs(k).sum(0) + len(k) * np.abs(o[b])
    return o, A, dz, F


class Batch:
    """Families [(shared positions, lengths)] on random pages, in a mixed order. What no query may use is
    NaN: rows behind a sequence's end, pages no one holds, a family's shared rows but its first member's
    (whose entries the others lack), and everything else of the pool."""

    def __init__(self, kv, heads, families, ps, seed, layers=1, scale=1.0, mix=True):
        rng = np.random.default_rng(seed)
        self.kv, self.p = kv, api.default_params(kv_format=kv, heads=heads)
        lead, shared, T = [], [], []
        for sh, lens in families:
            lead += [len(T)] * len(lens)
            shared += [sh] * len(lens)
            T += lens
        B = len(T)
        lead, shared, T = np.asarray(lead), np.asarray(shared), np.asarray(T)
        wide = max(1, int(-(-max(T.max(), shared.max()) // ps)))
        table, used, keep = np.full((B, wide), -1, np.int64), 0, []
        for b in range(B):
            lo = 0 if lead[b] == b else min(shared[b], T[b])
            hi = max(T[b], shared[b]) if lead[b] == b else T[b]
            for k in range(lo // ps, -(-int(hi) // ps)):
                if hi > lo:
                    table[b, k] = used
                    keep += [(used, t - k * ps) for t in range(max(lo, k * ps), min(int(hi), (k + 1) * ps))]
                    used += 1
        pages = used + 2
        perm = rng.permutation(pages)
        vals = randn(layers, pages, ps, D, seed=seed) * scale
        hold = np.zeros((pages, ps), bool)
        if keep:
            at = np.asarray(keep)
            hold[perm[at[:, 0]], at[:, 1]] = True
        vals[:, ~torch.from_numpy(hold).to(DEV)] = float("nan")
        self.c = api.PagedCache(self.p, pages, ps, B, wide, layers=layers, device=DEV)
        self.c.pool.copy_(vals.to(dtype_of(kv)))
        self.c.table.copy_(i32(np.where(table >= 0, perm[np.maximum(table, 0)], -1)))
        place = rng.permutation(B) if mix else np.arange(B)  # of member m in the call
        self.seq, self.T = np.empty(B, np.int64), np.empty(B, np.int64)
        self.seq[place], self.T[place] = np.arange(B), T
        self.order, self.first, self.shared = place, lead, shared
        self.q = (randn(B, heads, D, seed=seed + 1) * 2).bfloat16()
        self.sink = randn(heads, seed=seed + 2)

    def groups(self):
        return api.PrefixGroups(order=i32(self.order), first=i32(self.first), shared=i32(self.shared))

    def run(self, st=None, layer=0, sink=True, ws=None, q=None):
        q = self.q if q is None else q
        out = torch.full(q.shape, 9.0, dtype=torch.bfloat16, device=DEV)
        ws = api.paged_attn_shared_workspace(self.p, self.c, len(self.T)) if ws is None else ws
        api.paged_attn_shared(self.p, self.c, layer, q, self.sink if sink else None, i32(self.seq), i32(self.T),
                              self.groups(), out, ws, dev_status=st)
        return out

    def ref(self, layer=0, sink=True, q=None):
        return shared64(self.p, self.c, layer, self.q if q is None else q, self.sink if sink else None, self.seq,
                        self.T, self.order, self.first, self.shared)

    def check(self, **k):
        st = status()
        out = self.run(st=st, **k)
        assert st.item() == 0
        assert_attn(out, self.ref(**{n: v for n, v in k.items() if n != "ws"}), self.kv)
        return out


FAMILIES = [
    [(0, [1])], [(1, [1])], [(1, [2])], [(0, [0])], [(0, [5, 0, 300])], [(128, [128, 129, 128])],
    [(127, [127, 128, 255, 256]), (129, [200, 129]), (0, [1, 2, 3])],
    [(300, [340, 301, 300, 333]), (64, [700, 65]), (0, [129, 640])],
    [(1000, [1000 + 7 * i for i in range(9)])],
    [(200, [50, 199, 0, 200, 201, 1])],  # shorter than what the group shares
    [(640, [650] * 5), (513, [514 + i for i in range(3)]), (0, [257] * 4), (8, [9, 300])],
]


@BOTH
@pytest.mark.parametrize("heads,ps,ctas", [(64, 64, 0), (64, 16, 2), (48, 8, 6), (33, 24, 3), (32, 128, 0), (16, 64, 5),
                                           (12, 1024, 0), (5, 32, 4), (1, 16, 0)])
def test_attention_of_families(kv, heads, ps, ctas):
    for n, families in enumerate(FAMILIES):
        b = Batch(kv, heads, families, ps, seed=heads + ps + n, layers=2)
        b.p.max_ctas = ctas
        out = b.check(layer=n & 1)
        for i, T in enumerate(b.T):
            assert T or torch.all(out[i] == 0)


@BOTH
@pytest.mark.parametrize("seed", range(12))
def test_attention_of_random_batches(kv, seed):
    rng = np.random.default_rng(seed)
    families = []
    for _ in range(int(rng.integers(1, 9))):
        sh = int(rng.choice([0, 1, 100, 128, 500, 1500]))
        families.append((sh, [int(sh + rng.choice([0, 1, 30, 200, 600]) - (rng.random() < 0.1) * rng.integers(0, sh + 1))
                              for _ in range(int(rng.integers(1, 14)))]))
    heads, ps = int(rng.choice([1, 3, 8, 20, 40, 63, 64])), int(rng.choice([8, 16, 40, 64, 256]))
    b = Batch(kv, heads, families, ps, seed=100 + seed)
    b.p.max_ctas = int(rng.choice([0, 0, 1, 4, 9, 30]))
    b.check(sink=bool(seed & 1))


@BOTH
@pytest.mark.parametrize("heads", [64, 3])
@pytest.mark.parametrize("ctas,families", [
    (2, [(30_000, [30_100, 30_001])]), (2, [(24_577, [24_577] * 3), (0, [40_000, 5])]),
    (4, [(60_000, [60_001, 60_300, 60_000]), (100, [30_000])]), (6, [(16_384, [16_384] * 7), (16_385, [16_385])])])
def test_attention_of_long_pieces(kv, heads, ctas, families):
    """More tiles to a pair of CTAs than meet in one accumulator, in units that are cut and in whole
    ones, first, in the middle and last of a range; the same bytes in every run, whatever the
    workspace holds."""
    b = Batch(kv, heads, families, 64, seed=heads + ctas)
    b.p.max_ctas = ctas
    ws = torch.full_like(api.paged_attn_shared_workspace(b.p, b.c, len(b.T)), 0xFF)
    out = b.check(ws=ws)
    assert torch.equal(b.run(ws=ws), out)


@BOTH
@pytest.mark.parametrize("ctas,n", [(2, 1), (4, 3), (152, 75), (152, 76), (152, 77), (0, 600)])
def test_attention_of_as_many_units_as_pairs(kv, ctas, n):
    """Both schedules, at their border, and more sequences than a CTA has threads."""
    rng = np.random.default_rng(n)
    b = Batch(kv, 64, [(int(rng.integers(1, 400)),) * 2 for _ in range(0)] + [(130, [131 + i % 200, 135]) for i in range(n)], 16, seed=n)
    b.p.max_ctas = ctas
    b.check()


@BOTH
@pytest.mark.parametrize("heads", [64, 7])
def test_attention_of_many_units_of_one_tile(kv, heads):
    """Units that are done before the ones behind them are staged, a hundred to a pair, with rows and
    positions around each that no other may notice."""
    rng = np.random.default_rng(heads)
    b = Batch(kv, heads, [(0, [int(rng.integers(1, 129)) for _ in range(int(rng.integers(1, 128 // heads + 1)))])
                          for _ in range(400)], 32, seed=heads)
    b.p.max_ctas = 8
    out = b.check()
    for _ in range(3):
        assert torch.equal(b.run(), out)


@BOTH
def test_attention_of_single_sequences_agrees_with_paged_attn(kv):
    T = [1, 700, 129, 0, 64, 3000]
    b = Batch(kv, 32, [(0, [t]) for t in T], 32, seed=7)
    out, one = b.check(), torch.empty_like(b.q)
    api.paged_attn(b.p, b.c, 0, b.q, b.sink, i32(b.seq), i32(b.T), one, api.paged_attn_workspace(b.p, b.c, len(T)))
    n = one.double().norm()
    # each is within 4e-3 of the definition
    assert (out.double() - one.double()).norm() <= 8e-3 * n


@BOTH
@pytest.mark.parametrize("heads,B", [(1, 65535), (5, 6000)])
def test_attention_of_large_batches_agrees_with_paged_attn(kv, heads, B):
    """Groups as prefix_groups finds them among forks of many short prompts. Each call is off by its rounding of
    the output (2^-8 of it) and of the weights, in numerator and denominator (2^-8 or 2^-11 of the largest value)."""
    g = torch.Generator(device=DEV).manual_seed(heads)
    p, S, ps = api.default_params(kv_format=kv, heads=heads), 2048, 8
    c = api.PagedCache(p, n_pages=6 * S, page_size=ps, max_seqs=S, max_pages=6, device=DEV)
    c.pool.copy_(torch.randn(c.pool.shape, generator=g, device=DEV).to(c.pool.dtype))
    table = torch.randperm(6 * S, generator=g, device=DEV).view(S, 6).to(torch.int32)
    table[:, :2] = table[torch.arange(S, device=DEV) // 8 * 8][:, :2]
    c.table.copy_(table)
    seq = torch.randint(-1, S, (B,), generator=g, device=DEV).to(torch.int32)
    T = torch.randint(0, 6 * ps + 1, (B,), generator=g, device=DEV).to(torch.int32)
    st, groups = status(), api.PrefixGroups(B, device=DEV)
    api.prefix_groups(p, c, seq, T, groups, least=9, dev_status=st)
    q = torch.randn(B, heads, D, generator=g, device=DEV).bfloat16()
    sink = torch.randn(heads, generator=g, device=DEV)
    one, two = torch.full_like(q, 9), torch.full_like(q, 9)
    api.paged_attn_shared(p, c, 0, q, sink, seq, T, groups, one, api.paged_attn_shared_workspace(p, c, B), dev_status=st)
    api.paged_attn(p, c, 0, q, sink, seq, T, two, api.paged_attn_workspace(p, c, B), dev_status=st)
    u_p = 2.0 ** -8 if kv == api.BF16 else 2.0 ** -11
    tol = 2 * (2.0 ** -8 + 2 * u_p + 2.0 ** -15) * c.pool.float().abs().max()
    assert st.item() == 0 and (one.float() - two.float()).abs().max() <= tol
    assert torch.all(one[seq < 0] == 9) and torch.all(one[(seq >= 0) & (T == 0)] == 0)


@BOTH
def test_attention_sinks_and_large_logits(kv):
    b = Batch(kv, 64, [(300, [301, 400, 1200]), (0, [5, 0])], 32, seed=11)
    b.q = (b.q.float() * 20).bfloat16()  # logits to +-200: the running maximum moves
    base = b.check(sink=False)
    for s in (-math.inf, torch.finfo(torch.float32).min):
        b.sink = torch.full((64,), s, device=DEV)
        assert torch.equal(b.run(), base), s
    b.sink = torch.linspace(-300, 300, 64, device=DEV)
    b.check()
    b.sink = torch.full((64,), 1e30, device=DEV)  # the sink takes everything
    assert torch.all(b.run() == 0)


@BOTH
@pytest.mark.parametrize("ctas,families", [
    (2, [(300, [301, 420])]), (0, [(300, [301, 420])]), (0, [(1500, [1500, 1600, 1501])] * 2 + [(0, [700])]),
    (8, [(1500, [1500, 1600, 1501])] * 2 + [(0, [700])])])
@pytest.mark.parametrize("sink", [False, True])
def test_attention_of_logits_far_from_zero(kv, ctas, families, sink):
    """Maxima from 0 to +-1e5 and beyond, heads of every size in one unit, in whole and in cut units. Products of
    whole numbers, so that the logits are exact but for their rounding to 32 bits: 2^-24 of the largest, twice in the
    ratio of two weights (of a weight and the sink's: as much again)."""
    b = Batch(kv, 64, families, 64, seed=61)
    b.p.max_ctas = ctas
    hold = ~torch.isnan(b.c.pool.float()[0, :, :, 0])
    g = torch.Generator(device=DEV).manual_seed(62)
    whole = lambda lo, hi, *shape: torch.randint(lo, hi + 1, shape, generator=g, device=DEV).float()
    rows = b.c.pool[0].float()
    n = int(hold.sum())
    some = torch.where(torch.rand(n, generator=g, device=DEV) < 0.1, 64.0, 60.0)  # the maximum moves to these
    rows[hold] = torch.cat([some[:, None], whole(-4, 4, n, 4), rows[hold][:, 5:]], 1)
    b.c.pool[0] = rows.to(b.c.pool.dtype)
    b.p.softmax_scale = 0.125
    size = torch.tensor([0, 1, 7, 33, 128, 182, 200, 256, 320, 480, 500, 800, 1000, 1600, 2944, 4000, 5120, 8128, 8256 - 64,
                         10240, 12800, 11392 // 2, 64 * 177 // 2, 13056, 6016, 9984, 15104, 16128, 3008, 2000, 240, 60], device=DEV)
    q = torch.zeros_like(b.q, dtype=torch.float32)
    q[..., 0] = torch.cat([size, -size]).bfloat16().float()
    q[..., 1:5] = whole(-1, 1, *q.shape[:2], 4)
    b.q = q.bfloat16()
    if sink:
        top = torch.where(q[0, :, 0] > 0, 64 * q[0, :, 0], 60 * q[0, :, 0]) / 8
        b.sink = top + randn(64, seed=63)
    else:
        b.sink = None
    st = status()
    out = torch.full(b.q.shape, 9.0, dtype=torch.bfloat16, device=DEV)
    api.paged_attn_shared(b.p, b.c, 0, b.q, b.sink, i32(b.seq), i32(b.T), b.groups(), out,
                          api.paged_attn_shared_workspace(b.p, b.c, len(b.T)), dev_status=st)
    assert st.item() == 0
    o, A, _, F = shared64(b.p, b.c, 0, b.q, b.sink, b.seq, b.T, b.order, b.first, b.shared)
    z = (b.q[0, :, 0].double().abs() * 64 + 16).cpu().numpy()[:, None] / 8  # no logit of the head is larger
    u = 2.0 ** -8 if kv == api.BF16 else 2.0 ** -11
    # as assert_attn has it, with each head's own logits; those in the log2 domain are 1.45 times as large, and what
    # is rounded there weighs 0.7 of it here: 1.01 x 2^-24 z, for a weight and for the largest
    tol = 2.0 ** -8 * np.abs(o) + (2 * u + 4.1 * 2.0 ** -24 * z + 2.0 ** -20) * A + 2.0 ** -26 * F + 2.0 ** -109
    over = np.abs(out.double().cpu().numpy() - o) - tol
    assert over.max() <= 0, (over.max(), np.argwhere(over.max((0, 2)) > 0).ravel())


@BOTH
@pytest.mark.parametrize("ctas", [2, 0])
def test_attention_of_the_largest_logits(kv, ctas):
    """Logits up to 32 bits' end, of either sign, and halves of them: the outputs are the means of the rows whose
    logit is the largest, each with the same weight."""
    b = Batch(kv, 20, [(700, [700, 760, 701]), (0, [300])], 16, seed=65)
    b.p.max_ctas, b.p.softmax_scale = ctas, math.log(2)
    hold = ~torch.isnan(b.c.pool.float()[0, :, :, 0])
    rows = b.c.pool[0].float()
    rows[..., 0] = torch.where(torch.rand(hold.shape, generator=torch.Generator(device=DEV).manual_seed(66), device=DEV) < 0.5, 1.0, 0.5)
    rows[~hold] = float("nan")
    b.c.pool[0] = rows.to(b.c.pool.dtype)
    size = torch.tensor([torch.finfo(torch.bfloat16).max, 1e38, 1e37, 1e30, 1e20, 1e10, 1e7, 1e6, 2.0 ** 17, 2.0 ** 14], device=DEV)
    b.q = torch.zeros_like(b.q)
    b.q[..., 0] = torch.cat([size, -size]).bfloat16()
    out = b.run(sink=False).double().cpu().numpy()
    pool, table = b.c.pool[0].double().cpu().numpy(), b.c.table.cpu().numpy()
    u = 2.0 ** -8 if kv == api.BF16 else 2.0 ** -11
    for i, s in enumerate(b.order):
        lead = b.order[b.first[i]]
        t = np.arange(b.T[s])
        k = pool[table[np.where(t < b.shared[i], b.seq[lead], b.seq[s]), t // 16], t % 16]
        for sign, heads in ((1, slice(0, 10)), (-1, slice(10, 20))):
            v = k[k[:, 0] == (1.0 if sign > 0 else 0.5)]
            o, A = v.mean(0), np.abs(v).mean(0)
            assert (np.abs(out[s, heads] - o) <= 2.0 ** -8 * np.abs(o) + (2 * u + 2.0 ** -20) * A).all()


@BOTH
@pytest.mark.parametrize("scale", [1.0, -1.0])
def test_attention_rising_logits_rescale(kv, scale):
    """Later tiles outweigh earlier ones by more each time, so every tile moves the maximum, in some
    rows of a unit and not in others; a negative scale turns the order around."""
    b = Batch(kv, 64, [(1000, [1100, 1090])], 64, seed=12, mix=False)
    b.p.max_ctas, b.p.softmax_scale = 2, scale * b.p.softmax_scale
    sign = torch.sign(randn(D, seed=13))
    for s, (lo, hi) in enumerate(((0, 1100), (1000, 1090))):
        t = torch.arange(lo, hi, device=DEV)
        rows = sign[None] * (t.float() / 400)[:, None] * 0.5 + randn(hi - lo, D, seed=14 + s) * 0.25
        b.c.pool[0, b.c.table[s].long()[t // 64], t % 64] = rows.to(b.c.pool.dtype)
    b.q = (4 * sign[None, None] * torch.linspace(-1, 1, 128, device=DEV).view(2, 64, 1) + randn(2, 64, D, seed=15) * 0.1).bfloat16()
    b.check()


@BOTH
@pytest.mark.parametrize("heads,members", [(64, 2), (64, 5), (20, 6), (1, 130)])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_attention_keeps_what_a_sequence_does_not_see_from_it(kv, heads, members, bad):
    """A position that is not finite reaches the sequences that see it, and no other one of their unit:
    in a sequence's own positions only that sequence, in the shared ones every one. (E4M3 has no
    infinity: it is written as NaN.)"""
    b = Batch(kv, heads, [(200, [210 + 3 * i for i in range(members)])], 16, seed=heads + members, mix=False)
    clean = b.check()
    who, at = members // 2, 205  # a position of its own, in a tile that the shared ones begin
    page = b.c.table[who, at // 16].item()
    row = b.c.pool[0, page, at % 16].clone()
    bits = b.c.pool[0, page, at % 16].view(torch.int16 if kv == api.BF16 else torch.uint8)
    bits[300] = torch.tensor(bad).bfloat16().view(torch.int16).item() if kv == api.BF16 else 0x7F
    out = b.run()
    seen = out[who].float()
    if math.isnan(bad) or kv == api.E4M3:
        assert seen.isnan().all()
    else:  # a logit of +infinity is NaN everywhere, one of -infinity takes the position out
        up = (b.q[who, :, 300].float() * bad) > 0
        assert seen[up].isnan().all() and seen[~up].isfinite().all()
    others = [i for i in range(members) if i != who]
    assert torch.equal(out[others], clean[others])
    b.c.pool[0, page, at % 16] = row
    assert torch.equal(b.run(), clean)
    page = b.c.table[0, 2].item()
    bits = b.c.pool[0, page, 7].view(torch.int16 if kv == api.BF16 else torch.uint8)
    bits[5] = torch.tensor(float("nan")).bfloat16().view(torch.int16).item() if kv == api.BF16 else 0x7F
    assert b.run().isnan().all()


@BOTH
@pytest.mark.parametrize("heads,ctas", [(64, 2), (64, 0), (20, 2), (20, 6), (3, 4)])
def test_attention_of_many_tiles_that_are_not_finite(kv, heads, ctas):
    """Positions that are not finite in every tile of one sequence's own positions, first and last ones among them,
    whichever CTA of the pair has its rows; then in every sequence's."""
    T = [1700, 300, 900, 1290, 333, 257]
    b = Batch(kv, heads, [(200, T)], 16, seed=81, mix=False)
    b.p.max_ctas = ctas
    clean, good = b.check(), b.c.pool.clone()
    bits = b.c.pool.view(torch.int16 if kv == api.BF16 else torch.uint8)
    def spoil(who):
        at = torch.tensor(sorted({200, T[who] - 1, *range(230, T[who], 60)}), device=DEV)
        bits[0, b.c.table[who].long()[at // 16], at % 16, 7 * who] = 0x7FC0 if kv == api.BF16 else 0x7F
    for who in range(6):
        spoil(who)
        for _ in range(2):
            out = b.run()
            assert out[who].isnan().all()
            others = [i for i in range(6) if i != who]
            assert torch.equal(out[others], clean[others])
        b.c.pool.copy_(good)
    for who in range(6):
        spoil(who)
    assert b.run().isnan().all()
    b.c.pool.copy_(good)
    assert torch.equal(b.run(), clean)


@BOTH
@pytest.mark.parametrize("families", [1, 5])
@pytest.mark.parametrize("ctas", [2, 4, 6, 30, 0])
def test_attention_of_a_piece_without_a_finite_logit(kv, families, ctas):
    """A sequence's only own position is NaN, in a tile by itself, which may be a piece by itself: its output is
    NaN wherever the unit is cut, and the others' are what they were."""
    b = Batch(kv, 64, [(640, [641, 700, 640])] * families, 64, seed=71, mix=False)
    b.p.max_ctas = ctas
    clean = b.check()
    for who in range(0, 3 * families, 3):
        page = b.c.table[who, 10].item()
        b.c.pool[0, page, 0].view(torch.int16 if kv == api.BF16 else torch.uint8)[3] = 0x7FC0 if kv == api.BF16 else 0x7F
    out = b.run()
    bad = torch.arange(3 * families, device=DEV) % 3 == 0
    assert out[bad].isnan().all() and torch.equal(out[~bad], clean[~bad])


@pytest.mark.parametrize("ctas", [2, 0])
@pytest.mark.parametrize("heads", [64, 20, 1])
@pytest.mark.parametrize("bad", [float("inf"), -float("inf")])
@pytest.mark.parametrize("at", [40, 255, 300])
def test_attention_of_an_infinity_that_all_rows_see(heads, ctas, bad, at):
    """An infinity in a tile that every row of the unit sees (a shared one, or a sequence's by itself): a logit
    of -infinity takes the position out, as in the other tiles, any other is NaN."""
    for families in ([(384, [390, 400, 384])], [(0, [700])]):
        b = Batch(api.BF16, heads, families, 16, seed=heads + at, mix=False)
        b.p.max_ctas = ctas
        clean, ref = b.check(), b.ref()
        row = b.c.pool[0, b.c.table[0, at // 16].item(), at % 16]
        was = row[300].item()
        row[300] = bad
        out = b.run().float()
        down = (b.q[:, :, 300].float() * bad) < 0
        assert out[~down].isnan().all()
        row[300] = 1e30 if bad > 0 else -1e30  # weights of the heads with `down`: 0, so finite, and taken out in the definition
        o, A, _, F = b.ref()
        keep = down.cpu().numpy()
        assert out[down].isfinite().all()
        assert_attn(out[down], (o[keep], A[keep], ref[2], 0.0), api.BF16)
        row[300] = was
        assert torch.equal(b.run(), clean)


@BOTH
def test_attention_of_a_query_that_is_not_finite(kv):
    b = Batch(kv, 24, [(200, [210, 260, 200, 333, 201])], 16, seed=17, mix=False)
    clean = b.check()
    for bad in (float("nan"), float("inf")):
        q = b.q.clone()
        q[1, 3, 100] = bad
        out = b.run(q=q)
        assert out[1, 3].isnan().all()
        out[1, 3] = clean[1, 3]
        assert torch.equal(out, clean)


@BOTH
def test_attention_padding_strides_and_rows_of_the_table(kv):
    """Padding is left as it was, in a group and by itself; heads of a wider projection; sequences that
    appear often, with lengths of their own; no seq."""
    b = Batch(kv, 24, [(100, [130, 101, 128])], 16, seed=21, mix=False)
    wide = randn(7, 30, 600, seed=22, dtype=torch.bfloat16)
    b.q = wide[:, 3:27, 40:552]
    b.seq, b.T = np.array([0, -1, 2, 0, 1, -1, 0]), np.array([130, 50, 128, 129, 101, 9, 100])
    b.order, b.first, b.shared = np.array([0, 1, 2, 3, 4, 6, 5]), np.array([0] * 6 + [6]), np.array([100] * 6 + [50])
    st = status()
    out = b.run(st=st)
    assert st.item() == 0 and torch.all(out[1] == 9) and torch.all(out[5] == 9)
    live = b.seq >= 0
    o, A, dz, F = b.ref()
    assert_attn(out[torch.from_numpy(live).to(DEV)], (o[live], A[live], dz, F[live]), kv)
    c = Batch(kv, 24, [(100, [130, 101, 128])], 16, seed=21, mix=False)
    out2 = torch.empty_like(c.q)
    api.paged_attn_shared(c.p, c.c, 0, c.q, c.sink, None, i32(c.T), c.groups(), out2,
                          api.paged_attn_shared_workspace(c.p, c.c, 3))
    assert torch.equal(out2, c.run())


@BOTH
def test_attention_of_an_output_at_any_16_bytes(kv):
    b = Batch(kv, 40, [(100, [130, 101, 128]), (0, [60])], 16, seed=31)
    base = b.check()
    flat = torch.full((b.q.numel() + 16,), 9.0, dtype=torch.bfloat16, device=DEV)
    out = flat[8:-8].view(b.q.shape)
    assert out.data_ptr() % 32 == 16
    api.paged_attn_shared(b.p, b.c, 0, b.q, b.sink, i32(b.seq), i32(b.T), b.groups(), out,
                          api.paged_attn_shared_workspace(b.p, b.c, len(b.T)))
    assert torch.equal(out, base) and torch.all(flat[:8] == 9) and torch.all(flat[-8:] == 9)


@BOTH
def test_attention_flags_and_skips_what_is_out_of_range(kv):
    """Lengths, sequences, pages and groups outside their ranges: the call ends, flags them and leaves
    what they name unseen; the other sequences are what they were."""
    def fresh():
        b = Batch(kv, 40, [(150, [160, 170, 200]), (0, [90, 20])], 16, seed=23, mix=False)
        raw = torch.isnan(b.c.pool.float())
        b.c.pool.copy_(torch.where(raw, torch.zeros((), device=DEV), b.c.pool.float()).to(b.c.pool.dtype))
        return b
    b = fresh()
    base, ref = b.check(), b.ref()
    most = b.c.table.shape[1] * 16
    for T, bit in ((most + 5, 2), (-3, 2)):  # cut, or nothing seen
        b = fresh()
        b.T[4] = T
        b.c.table[4] = b.c.table[0]
        st = status()
        out = b.run(st=st)
        b.T[4] = min(max(T, 0), most)
        assert_attn(out, b.ref(), kv)
        assert st.item() & bit
    b = fresh()
    b.seq[1] = 5  # out of range: nothing seen
    st = status()
    out = b.run(st=st)
    assert st.item() == 1 and torch.all(out[1] == 0)
    assert_attn(out, b.ref(), kv)
    b = fresh()
    b.c.table[0, 3], b.c.table[2, 12], b.c.table[3, 1] = -1, b.c.pool.shape[1], 1 << 30
    st = status()
    out = b.run(st=st)
    assert st.item() == 1
    assert_attn(out, b.ref(), kv)
    for name, at, v, lost in (("first", 4, 5, []), ("first", 4, -1, []), ("order", 4, 9, [4]), ("order", 4, -1, [4])):
        b = fresh()
        getattr(b, name)[at] = v
        st = status()
        out = b.run(st=st)
        assert st.item() == 1, (name, v)
        assert all(torch.all(out[i] == 9) for i in lost)
        keep = [i for i in range(5) if i not in lost]
        o, A, dz, F = ref
        assert_attn(out[keep], (o[keep], A[keep], dz, F[keep]), kv)
    for v in (-1, most + 1):
        b = fresh()
        b.shared[3] = v
        st = status()
        out = b.run(st=st)
        b.shared[3] = max(0, min(v, most))
        assert_attn(out, b.ref(), kv)
        assert st.item() & 2
    # groups that contradict themselves: whatever comes out, the call ends and the others stand
    b = fresh()
    b.first, b.shared = np.array([0, 0, 1, 3, 3]), np.array([150, 3, 7, 0, 10 ** 6])
    b.run(st=status())
    torch.cuda.synchronize()
    assert torch.equal(fresh().run(), base)


def groups_that_hold(first, members):
    """What csa2_paged_attn_shared makes of any `first`: the slot where each slot's group begins."""
    out = []
    for i, f in enumerate(first):
        good = 0 <= f <= i and first[f] == f and all(first[j] == f for j in range(i - (i - f) % members, i))
        out.append(f if good else i)
    return out


@BOTH
@pytest.mark.parametrize("heads,B,ctas", [(64, 20, 0), (1, 32, 0), (1, 33, 4), (16, 90, 0), (5, 200, 6), (40, 600, 0)])
def test_attention_of_groups_that_contradict_themselves(kv, heads, B, ctas):
    """Any `first` at all: a slot whose group does not hold together is one of its own, and the others stand."""
    rng = np.random.default_rng(B)
    ps, wide = 16, 20
    p = api.default_params(kv_format=kv, heads=heads)
    p.max_ctas = ctas
    c = api.PagedCache(p, 60, ps, 12, wide, device=DEV)
    c.pool.copy_(randn(*c.pool.shape, seed=B).to(c.pool.dtype))
    c.table.copy_(i32(rng.integers(0, 60, (12, wide))))
    q, sink = randn(B, heads, D, seed=B + 1, dtype=torch.bfloat16), randn(heads, seed=B + 2)
    slot = np.arange(B)
    families = np.sort(rng.integers(0, B, B))
    families = np.searchsorted(families, families)
    two = slot % 2
    wrong = families.copy()
    wrong[rng.integers(0, B, 3)] = rng.integers(0, B, 3)
    for n, first in enumerate([rng.integers(-1, slot + 2), np.append(slot[:-1], 0), families, two, wrong,
                               np.where(slot < 2, slot, rng.integers(0, 2, B)), np.maximum(slot - 1, 0)]):
        seq, T, order = rng.integers(0, 12, B), rng.integers(0, wide * ps + 1, B), rng.permutation(B)
        shared, st = rng.integers(0, wide * ps + 1, B), status()
        out = torch.empty_like(q)
        api.paged_attn_shared(p, c, 0, q, sink, i32(seq), i32(T),
                              api.PrefixGroups(order=i32(order), first=i32(first), shared=i32(shared)), out,
                              api.paged_attn_shared_workspace(p, c, B), dev_status=st)
        held = groups_that_hold(first.tolist(), 128 // heads)
        assert st.item() == (held != first.tolist()), n
        assert_attn(out, shared64(p, c, 0, q, sink, seq, T, order, held, shared), kv)


@BOTH
@pytest.mark.parametrize("ctas", [0, 6])
def test_attention_whatever_the_workspace_holds(kv, ctas):
    """Words that look like outputs, sums or ends of ranges; what lies around the output stays."""
    b = Batch(kv, 20, [(1500, [1600, 1501, 1500]), (200, [0, 333]), (0, [700, 1])], 16, seed=91)
    b.p.max_ctas = ctas
    base, n = b.check(), b.q.numel()
    flat = torch.full((3 * n,), 9.0, dtype=torch.bfloat16, device=DEV)
    out, ws = flat[n:2 * n].view(b.q.shape), api.paged_attn_shared_workspace(b.p, b.c, len(b.T))
    words = ws[:ws.numel() // 4 * 4].view(torch.int32)
    g = torch.Generator(device=DEV).manual_seed(92)
    for lo, hi in ((-5, 200), (0, 8), (-2 ** 31, 2 ** 31 - 1), (0x7F800000, 0x7FC00001)):
        words.random_(lo, hi, generator=g)
        api.paged_attn_shared(b.p, b.c, 0, b.q, b.sink, i32(b.seq), i32(b.T), b.groups(), out, ws)
        assert torch.equal(out, base) and torch.all(flat[:n] == 9) and torch.all(flat[2 * n:] == 9)


@pytest.mark.parametrize("heads", [5, 64])
def test_attention_e4m3_queries_of_a_wide_range(heads):
    """The query's two E4M3 parts: channels down to 2^-18 of a head's largest, heads from 2^-40 on."""
    b = Batch(api.E4M3, heads, [(500, [700, 513, 500])], 16, seed=35)
    g = torch.Generator(device=DEV).manual_seed(36)
    q = b.q.float() * torch.exp2(-torch.randint(0, 19, b.q.shape, generator=g, device=DEV).float())
    b.q = (q * torch.exp2(torch.randint(-40, 4, q.shape[:2], generator=g, device=DEV).float())[..., None]).bfloat16()
    b.check()


def test_attention_wide_values_of_bf16():
    """Latents beyond fp16's range stay exact in bf16 pages."""
    b = Batch(api.BF16, 64, [(300, [333, 301])], 16, seed=33, scale=1e6)
    b.p.softmax_scale = 1e-7
    b.check()


@BOTH
@pytest.mark.parametrize("drop", [24.5, 26.1])
def test_attention_long_tails(kv, drop):
    """One position above a million others of 2^-drop each, all of them to one pair of CTAs: of what lies
    about the last steps of the weights and of the accumulator less than 2^-9 of the whole is lost,
    and a channel that is one everywhere comes out as one."""
    T, heads, ps = 1_000_000, 64, 64
    n = -(-T // ps)
    p = api.default_params(kv_format=kv, heads=heads)
    p.max_ctas, p.softmax_scale = 2, drop * math.log(2) / 512
    rows = randn(64, D, seed=3).to(dtype_of(kv)).bfloat16().repeat(n, 1)
    rows[:, 0], rows[:, 1], rows[:, 2], rows[:, 3] = -16, 1, 1, -1
    rows[9] = 0
    rows[9, 1] = 1
    table = i32(np.stack([np.arange(n)] * 2))
    c = api.PagedCache(p, pool=rows.to(dtype_of(kv)).view(1, n, ps, D), device=DEV, table=table, ref=i32(np.full(n, 2)))
    q = torch.zeros(2, heads, D, dtype=torch.bfloat16, device=DEV)
    q[..., 0] = 32
    out = torch.empty_like(q)
    groups = api.PrefixGroups(order=i32([1, 0]), first=i32([0, 0]), shared=i32([T, T]))
    api.paged_attn_shared(p, c, 0, q, None, None, i32([T, T]), groups, out, api.paged_attn_shared_workspace(p, c, 2))
    assert torch.all(out[..., 1] == 1)
    total = sum(rows[i:min(T, i + (1 << 16))].double().sum(0) for i in range(0, T, 1 << 16))
    w, peak = 2.0 ** -drop, rows[9].double()
    den = 1 + w * (T - 1)
    o, share = (peak + w * (total - peak)) / den, 1 - 1 / den
    # every weight is off by its rounding and by that of its logit, in numerator and denominator
    u = (2.0 ** -8 if kv == api.BF16 else 2.0 ** -11) + 4 * drop * 2.0 ** -24 + 2.0 ** -22
    V = rows.abs().amax(0).double()
    tol = 2 * u * (share * V + share * o.abs()) + 2.0 ** -9 * V + 2.0 ** 14 * 2.0 ** -26 * (V + o.abs())
    assert ((out.double() - o).abs() <= tol + 2.0 ** -8 * (o.abs() + tol)).all()


@BOTH
def test_attention_of_the_longest_sequence(kv):
    """2^31 - 1 positions, all but the last 1,023 of them the same page, whose weights are 2^-64 of the others' (2^-33 in
    all): the outputs are the mean of those, up to the last box of rows."""
    T, ps, heads = 2 ** 31 - 1, 1024, 8
    p = api.default_params(kv_format=kv, heads=heads)
    p.softmax_scale = math.log(2) / 64
    table = torch.zeros(1, -(-T // ps), dtype=torch.int32, device=DEV)
    table[0, -1] = 1
    rows = randn(2, ps, D, seed=97)
    rows[0, :, 0], rows[1, :, 0] = -16, 0
    rows[1, :, 5] = 0
    rows[1, 960:, 5] = 16
    rows[1, 1023] = float("nan")
    c = api.PagedCache(p, pool=rows.to(dtype_of(kv))[None].contiguous(), table=table, ref=i32([T // ps, 1]))
    q = torch.zeros(1, heads, D, dtype=torch.bfloat16, device=DEV)
    q[..., 0] = 256
    out, st, groups = torch.empty_like(q), status(), api.PrefixGroups(1, device=DEV)
    api.prefix_groups(p, c, None, i32([T]), groups, dev_status=st)
    assert groups.shared.tolist() == [0]
    api.paged_attn_shared(p, c, 0, q, None, None, i32([T]), groups, out, api.paged_attn_shared_workspace(p, c, 1), dev_status=st)
    assert st.item() == 0
    v = c.pool[0, 1, :1023].double()
    # the largest weights are alike, and added up in 64 steps that lose 2^-24 each at most; the others' share is 2^31 x
    # 2^-64 / 1,023, of values of 16 at most
    o, A = v.mean(0), v.abs().mean(0)
    assert ((out.double() - o).abs() <= 2.0 ** -8 * o.abs() + 2.0 ** -17 * A + 2.0 ** -38).all()


def test_offsets_past_32_bits():
    """Shared pages beyond 4 GB of a pool, in its second layer."""
    n_pages, ps = 70_001, 64
    p = api.default_params(kv_format=api.BF16, heads=16)
    c = api.PagedCache(p, n_pages, ps, 3, 8, layers=2, device=DEV)
    far = n_pages - 1 - np.arange(8)
    c.table.copy_(i32(np.stack([far, np.concatenate([far[:5], far[5:] - 10, ])] + [far - 20])))
    x = randn(n_pages - 40_000, ps, D, seed=3, dtype=torch.bfloat16)
    c.pool[1, 40_000:] = x
    q, sink = randn(3, 16, D, seed=4, dtype=torch.bfloat16), randn(16, seed=5)
    T, st, out = [400, 350, 512], status(), torch.empty_like(q)
    groups = api.PrefixGroups(3, device=DEV)
    api.prefix_groups(p, c, None, i32(T), groups, dev_status=st)
    assert groups.shared.tolist() == [320, 320, 0] and groups.order.tolist() == [0, 1, 2]
    api.paged_attn_shared(p, c, 1, q, sink, None, i32(T), groups, out, api.paged_attn_shared_workspace(p, c, 3), dev_status=st)
    assert st.item() == 0
    c2 = type("C", (), dict(pool=torch.cat([x[None]]), table=c.table - 40_000))
    assert_attn(out, shared64(p, c2, 0, q, sink, np.arange(3), T, [0, 1, 2], [0, 0, 2], [320, 320, 0]), api.BF16)


def test_two_streams_with_workspaces_of_their_own():
    b = Batch(api.BF16, 64, [(2000, [2100, 2001, 2300]), (0, [500])], 64, seed=41)
    alone, g = b.run(), b.groups()
    streams = [torch.cuda.Stream() for _ in range(2)]
    spaces = [api.paged_attn_shared_workspace(b.p, b.c, 4) for _ in range(2)]
    outs, seq, T = [torch.empty_like(b.q) for _ in range(2)], i32(b.seq), i32(b.T)
    torch.cuda.synchronize()
    for _ in range(10):
        for s, w, o in zip(streams, spaces, outs):
            api.paged_attn_shared(b.p, b.c, 0, b.q, b.sink, seq, T, g, o, w, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(outs[0], alone) and torch.equal(outs[1], alone)


@BOTH
def test_a_batch_forks_shares_and_decodes(kv):
    """A server's steps in one: a prompt's chunk and other requests in one step of fixed size (slot maps,
    rows turned and written), the prompt forked, then steps of one token or a few: slot maps, rows,
    groups, attention behind the shared pages; the captured step replays to the same bytes, with other
    lengths too."""
    ps, H, S, N = 16, 12, 8, 64
    p = api.default_params(kv_format=kv, rope_dim=64, heads=H)
    c = api.PagedCache(p, 120, ps, S, 30, device=DEV)
    st = status()
    ws = api.paged_attn_shared_workspace(p, c, N)
    slots, groups, sink = api.SlotMap(S, N, device=DEV), api.PrefixGroups(N, device=DEV), randn(H, seed=1)
    seq, T, new = i32(np.full(S, -1)), i32(np.zeros(S)), i32(np.zeros(S))
    x, q, out = torch.empty(N, D, device=DEV), torch.empty(N, H, D, dtype=torch.bfloat16, device=DEV), \
        torch.zeros(N, H, D, dtype=torch.bfloat16, device=DEV)

    def step():
        api.page_slots(p, c, seq, T, new, slots, st)
        api.page_write(p, c, 0, x, slots.seq, slots.pos, st)
        turned = api.rope(p, q, slots.pos)
        # each new row sees the positions up to its own
        seen = slots.pos + 1
        api.prefix_groups(p, c, slots.seq, seen, groups, least=ps, dev_status=st)
        api.paged_attn_shared(p, c, 0, turned, sink, slots.seq, seen, groups, out, ws, dev_status=st)
        T.copy_(slots.n_tokens)
        return turned

    def check(turned):
        rows, pos = slots.seq.cpu().numpy(), slots.pos.cpu().numpy()
        o = shared64(p, c, 0, turned, sink, rows, pos + 1, np.arange(N), np.arange(N), np.zeros(N, int))
        live = rows >= 0
        assert_attn(out[torch.from_numpy(live).to(DEV)], (o[0][live], o[1][live], o[2], o[3][live]), kv)
        assert torch.all(out[torch.from_numpy(~live).to(DEV)] == 0)

    def feed(k, seqs, counts):
        seq.fill_(-1)
        new.zero_()
        seq[:len(seqs)] = i32(seqs)
        new[:len(counts)] = i32(counts)
        held = lengths[np.asarray(seqs)]
        T.zero_()
        T[:len(seqs)] = i32(held)
        lengths[np.asarray(seqs)] += counts
        x.copy_(randn(N, D, seed=100 + k))
        q.copy_((randn(N, H, D, seed=200 + k) * 2).bfloat16())
        out.zero_()  # (the calls leave rows of padding as they were)

    lengths = np.zeros(S, np.int64)
    for k, (seqs, counts) in enumerate([([0, 1], [50, 9]), ([0, 1, 2], [31, 1, 20])]):
        feed(k, seqs, counts)
        check(step())
    api.page_fork(p, c, i32([0, 0, 0, 1]), i32([3, 4, 5, 6]), i32([lengths[0]] * 3 + [lengths[1]]), st)
    lengths[[3, 4, 5]], lengths[6] = lengths[0], lengths[1]
    feed(2, [5, 0, 3, 1, 4, 6], [1, 1, 4, 1, 2, 1])
    check(step())
    assert groups.shared.max().item() == 80  # the prompt's five full pages
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    feed(3, [5, 0, 3, 1, 4, 6], [1] * 6)
    with torch.cuda.graph(graph, stream=side):
        turned = step()
    for k, (seqs, counts) in enumerate([(None, None), ([3, 2, 4], [20, 1, 3]), ([0, 5], [1, 1])]):
        if seqs is not None:
            feed(10 + k, seqs, counts)
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        check(turned)
        first, held = out.clone(), T.clone()
        T.copy_(held - new)  # the same step again: its pages are there already
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, first)
    assert st.item() == 0
    used = c.table[c.table >= 0]
    assert torch.equal(torch.bincount(used.long(), minlength=120).int(), c.ref)


def test_calls_name_what_they_refuse():
    b = Batch(api.BF16, 8, [(16, [20, 30])], 16, seed=51)
    small = torch.empty(256, dtype=torch.uint8, device=DEV)
    T, out, seq = i32(b.T), torch.empty_like(b.q), i32(b.seq)
    with pytest.raises(api.Csa2Error, match="workspace smaller"):
        api.paged_attn_shared(b.p, b.c, 0, b.q, b.sink, seq, T, b.groups(), out, small)
    ws = api.paged_attn_shared_workspace(b.p, b.c, 2)
    with pytest.raises(api.Csa2Error, match="layer out of range"):
        api.paged_attn_shared(b.p, b.c, 1, b.q, b.sink, seq, T, b.groups(), out, ws)
    with pytest.raises(api.Csa2Error, match="is on cpu"):
        api.paged_attn_shared(b.p, b.c, 0, b.q, b.sink, seq, T, api.PrefixGroups(2, device="cpu"), out, ws)
    with pytest.raises(api.Csa2Error, match="is on cpu"):
        api.prefix_groups(b.p, b.c, seq, T.cpu(), b.groups())
    with pytest.raises(api.Csa2Error, match="least"):
        api.prefix_groups(b.p, b.c, seq, T, b.groups(), least=0)
    with pytest.raises(api.Csa2Error, match="is on cpu"):
        api.page_slots(b.p, b.c, seq, T, T, api.SlotMap(2, 8, device="cpu"))


@BOTH
def test_a_workspace_is_for_batches_of_up_to_its_size(kv):
    """A workspace for fewer sequences is refused where it is smaller (E4M3 pages: the queries' parts lie there), one for
    more is not."""
    b = Batch(kv, 64, [(100, [130, 101, 128]), (0, [60])], 16, seed=95)
    out = b.check(ws=api.paged_attn_shared_workspace(b.p, b.c, 40))
    small = api.paged_attn_shared_workspace(b.p, b.c, 3)
    if kv == api.E4M3:
        with pytest.raises(api.Csa2Error, match="workspace smaller"):
            b.run(ws=small)
    else:
        assert torch.equal(b.run(ws=small), out)

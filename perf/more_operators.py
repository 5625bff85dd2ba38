"""A ragged batch on the paged cache: the cases its operators are measured on, their plain
forms and their 64-bit definitions.

``slots``   block tables and slot maps of a step from the requests' lengths,
``groups``  which sequences of a batch hold the same leading pages, and how many positions,
``attn``    attention of a batch in which groups of sequences share a long prefix.

``own`` False: ``run`` computes a case with elementary torch operations in 32 bits; True: with
the calls a user of the framework makes. The sizes are those of the framework's default
configuration (64 heads sharing one 512-wide latent) and its tensor-parallel shards.
"""
import math

import numpy as np
import torch

own = False

D = 512
DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn}


# ------------------------------------------------------------------------------- cases
def listed():
    return [
        # one new token of each of 64 sequences
        dict(name="slots decode", op="slots", seqs=64, chunks=0, chunk=0, idle=0, rows=64, page=64,
             longest=32768),
        # decoding sequences with eight prefill chunks among them, in a step of fixed size with
        # idle requests and rows behind the last token
        dict(name="slots mixed", op="slots", seqs=240, chunks=8, chunk=1000, idle=16, rows=8192,
             page=64, longest=16384),
        # a step of prompts only: many rows, many small pages
        dict(name="slots prompts", op="slots", seqs=1001, chunks=1001, chunk=120, idle=0, rows=131072,
             page=16, longest=4096),
        # 40 continuations of one prompt among other requests
        dict(name="groups one prompt", op="groups", families="40 1*8", prefix=8192, even=True, tail=700, page=64,
             least=1),
        # large batch, families of many sizes, of which only long prefixes count
        dict(name="groups 2000", op="groups", families="16*100 2*150 1*100", prefix=65536,
             even=False, tail=2000, page=32, least=1024),
        # four samples of a short question: latency
        dict(name="attn four short", op="attn", families="4", heads=64, prefix=300, even=True, tail=40,
             page=16, kv="bf16"),
        # 32 requests behind one system prompt
        dict(name="attn 32 behind 8192", op="attn", families="32", heads=64, prefix=8192, even=True, tail=1024,
             page=64, kv="bf16"),
        # documents that several requests ask about, and requests of their own
        dict(name="attn families e4m3", op="attn", families="31 17 9 5 3 2 1*12", heads=64,
             prefix=16384, even=False, tail=2000, page=64, kv="e4m3"),
        # a shard of 16 heads, large batch
        dict(name="attn 16 heads", op="attn", families="128", heads=16, prefix=32768, even=True, tail=500,
             page=64, kv="bf16"),
        # five drafted tokens of each of 16 sequences, checked in one step by a shard of 32 heads
        dict(name="attn drafts", op="attn", families="5*16", heads=32, prefix=16384, even=False, tail=0,
             page=64, kv="bf16"),
        # many samples of a long document, 8-bit
        dict(name="attn long e4m3", op="attn", families="64", heads=64, prefix=131072, even=True, tail=512,
             page=64, kv="e4m3"),
        # fewer of them, unquantised
        dict(name="attn long bf16", op="attn", families="24", heads=64, prefix=131072, even=True, tail=2000,
             page=128, kv="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _families(rng, seqs):
    """seqs sequences in families of mixed sizes."""
    left, out = seqs, []
    most = _log(rng, 1, seqs)
    while left:
        n = min(left, _log(rng, 1, most)) if len(out) < 40 else left
        out.append(n)
        left -= n
    return " ".join(map(str, out))


def _sizes(case):
    """The families' sizes: "5*16 3" is sixteen of five sequences and one of three."""
    out = []
    for part in case["families"].split():
        n, _, times = part.partition("*")
        out += [int(n)] * int(times or 1)
    return out


def draw(rng):
    op = rng.choice(["slots", "slots", "groups", "attn", "attn", "attn", "attn"])
    page = rng.choice([8, 16, 24, 32, 64, 128])
    if op == "slots":
        seqs = _log(rng, 1, 1001)
        chunks = rng.choice([0, rng.randint(0, seqs), seqs])
        chunk = _log(rng, 1, min(8192, max(1, 120120 // max(chunks, 1))))
        idle = rng.choice([0, rng.randint(0, 20)])
        return dict(op=op, seqs=seqs, chunks=chunks, chunk=chunk, idle=idle, page=page,
                    rows=seqs + chunks * chunk + rng.choice([0, rng.randint(0, 500)]),
                    longest=_log(rng, 16, 32768 if seqs < 200 else 4096))
    if op == "groups":
        prefix, page = _log(rng, 256, 32768), max(page, 16)
        return dict(op=op, families="3 %s 1 1" % _families(rng, _log(rng, 4, 1995)), prefix=prefix, even=rng.random() < 0.5,
                    tail=_log(rng, 1, 2000), page=page, least=_log(rng, 1, prefix // 2))
    seqs, heads = _log(rng, 1, 192), rng.choice([1, 8, 12, 16, 32, 48, 64])
    drafts = rng.random() < 0.2
    return dict(op=op, families=_families(rng, seqs), heads=heads, kv=rng.choice(["bf16", "e4m3"]),
                prefix=_log(rng, 1, min(131072, (1 << 28) // (seqs * heads), 2500000 // seqs)),
                even=rng.random() < 0.4, tail=0 if drafts else _log(rng, 1, min(4096, 400000 // seqs)), page=page)


# ------------------------------------------------------------------------------- inputs
def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _i32(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).to(DEV)


def _spread(r, n, top, even):
    """n lengths: all the longest, or from an eighth of it up; the first is the longest."""
    t = np.full(n, top, np.int64)
    if not even:
        t[1:] = np.maximum(1, np.floor(top * (0.125 + 0.875 * r.random(n - 1))))
    return t


def _batch(case, seed):
    """Sequences of families as forks of their prompts leave them: the prompt's full pages are
    shared, the rows behind them everyone's own. A family of one shares nothing. tail = 0: the
    members are drafted tokens of one sequence, each of which sees one position more."""
    r = np.random.default_rng([seed, 1])
    ps, sizes = case["page"], np.asarray(_sizes(case))
    F, B = len(sizes), int(sizes.sum())
    P = _spread(r, F, case["prefix"], case["even"])
    fam = np.repeat(np.arange(F), sizes)
    rank = np.arange(B) - np.repeat(np.cumsum(sizes) - sizes, sizes)
    if case["tail"]:
        T = P[fam] + r.integers(1, case["tail"] + 1, B)
        seq, rows, row_len, row_fam = np.arange(B), B, T, fam
        shared = np.where(sizes > 1, P // ps * ps, 0)
    else:
        T = P[fam] + rank
        seq, rows, row_len, row_fam = fam, F, P + sizes - 1, np.arange(F)
        shared = np.where(sizes > 1, P, 0)
    # pages: the families' shared ones, then the rows' own, in random places of the pool
    n = -(-row_len // ps)
    kept = P // ps if case["tail"] else np.zeros(F, np.int64)
    own_n = n - kept[row_fam]
    pages = int(kept.sum() + own_n.sum()) + 3
    place = np.random.default_rng([seed, 2]).permutation(pages)
    table = np.full((rows, int(n.max())), -1, np.int64)
    k = np.arange(table.shape[1])[None]
    head, body = k < kept[row_fam][:, None], (k >= kept[row_fam][:, None]) & (k < n[:, None])
    f0 = np.cumsum(kept) - kept
    o0 = kept.sum() + np.cumsum(own_n) - own_n
    table[head] = place[(f0[row_fam][:, None] + k)[head]]
    table[body] = place[(o0[:, None] + k - kept[row_fam][:, None])[body]]
    # the batch comes in no order
    mix = np.random.default_rng([seed, 3]).permutation(B)
    return dict(T=T[mix], seq=seq[mix], fam=fam[mix], table=table, pages=pages, shared=shared)


def _grouped(fam, shared):
    """order, first, shared of the batch: families by their first member, members ascending."""
    B = len(fam)
    lead = np.full(fam.max() + 1, B)
    np.minimum.at(lead, fam, np.arange(B))
    order = np.lexsort((np.arange(B), lead[fam]))
    slot = np.empty(B, np.int64)
    slot[order] = np.arange(B)
    return order, slot[lead[fam[order]]], shared[fam[order]]


def prepare(case, seed):
    g, s = _gen(seed), {"case": case}
    if case["op"] == "slots":
        r = np.random.default_rng([seed, 1])
        S, ps, idle = case["seqs"], case["page"], case["idle"]
        new = np.ones(S, np.int64)
        new[r.permutation(S)[:case["chunks"]]] += r.integers(0, case["chunk"] + 1, case["chunks"])
        T = r.integers(0, case["longest"] + 1, S)
        wide = -(-(case["longest"] + 1 + case["chunk"]) // ps)
        held = -(-T // ps)
        k = np.arange(wide)[None]
        mine = k < held[:, None]
        n_held = int(mine.sum())
        pages = S * (case["longest"] // ps + 2) + case["chunks"] * (case["chunk"] // ps + 1) + 17  # some are left over
        place = np.random.default_rng([seed, 2]).permutation(pages)
        table = np.full((S, wide), -1, np.int64)
        table[mine] = place[:n_held]
        ref = np.zeros(pages, np.int64)
        ref[place[:n_held]] = 1
        seq = np.full(S + idle, -1, np.int64)
        at = np.sort(r.permutation(S + idle)[:S])
        seq[at] = r.permutation(S)
        live = seq >= 0
        s["table"], s["ref"] = _i32(table), _i32(ref)
        s["which"] = _i32(seq)
        s["held"] = _i32(np.where(live, T[seq], 0))
        s["new"] = _i32(np.where(live, new[seq], 0))
        s["pool"] = torch.empty(1, pages, ps, D, dtype=torch.int8, device=DEV).view(TYPES["e4m3"])
        return s
    b = _batch(case, seed)
    s["table"], s["T"], s["seq"] = _i32(b["table"]), _i32(b["T"]), _i32(b["seq"])
    s["ref"] = torch.ones(b["pages"], dtype=torch.int32, device=DEV)
    if case["op"] == "groups":
        s["pool"] = torch.empty(1, b["pages"], case["page"], D, dtype=torch.int8, device=DEV).view(TYPES["e4m3"])
        return s
    pool = torch.empty(1, b["pages"], case["page"], D, dtype=torch.bfloat16, device=DEV).normal_(generator=g)
    s["pool"] = pool if case["kv"] == "bf16" else pool.to(TYPES["e4m3"])
    # logits of standard deviation 2: some positions matter more than others
    s["q"] = (2 * torch.randn(len(b["T"]), case["heads"], D, generator=g, device=DEV)).bfloat16()
    s["sink"] = torch.randn(case["heads"], generator=g, device=DEV)
    s["out"] = torch.empty_like(s["q"])
    order, first, shared = _grouped(b["fam"], b["shared"])
    s["order"], s["first"], s["shared"] = _i32(order), _i32(first), _i32(shared)
    # the scheduler's own lists: members and shared positions of each family
    alone = [i for i in range(len(b["fam"])) if b["shared"][b["fam"][i]] == 0]
    s["lists"] = [(torch.tensor(alone, device=DEV), 0, int(b["T"][alone].max()))] if alone else []
    for f in np.flatnonzero(b["shared"]):
        m = np.flatnonzero(b["fam"] == f)
        s["lists"].append((torch.from_numpy(m).to(DEV), int(b["shared"][f]), int((b["T"][m] - b["shared"][f]).max())))
    return s


# ------------------------------------------------------------------------------- plain forms
def _plain_slots(s, case):
    table, ref, ps = s["table"], s["ref"], case["page"]
    seq, t0 = s["which"].long(), s["held"].long()
    new = torch.where(seq >= 0, s["new"].long(), 0)
    t1 = t0 + new
    row = seq.clamp(min=0)
    k = torch.arange(table.shape[1], device=DEV)
    need = (k >= (t0 // ps)[:, None]) & (k < ((t1 + ps - 1) // ps)[:, None]) & (new > 0)[:, None] & (table[row] < 0)
    rank = need.flatten().cumsum(0).view(need.shape) - 1
    free = torch.argsort((ref > 0).to(torch.int8), stable=True)
    i, j = need.nonzero(as_tuple=True)
    taken = free[rank[i, j]]
    table[row[i], j] = taken.int()
    ref[taken] = 1
    start = torch.cat([new.new_zeros(1), new.cumsum(0)])
    at = torch.arange(case["rows"], device=DEV)
    which = torch.searchsorted(start[1:], at, right=True)
    live = which < len(seq)
    which = which.clamp(max=len(seq) - 1)
    rseq = torch.where(live, seq[which], -1)
    rpos = torch.where(live, t0[which] + at - start[which], -1)
    page = table[rseq.clamp(min=0), rpos.clamp(min=0) // ps].long()
    slot = torch.where(live, page * ps + rpos % ps, -1)
    return table, ref, t1.int(), start.int(), rseq.int(), rpos.int(), slot


def _plain_groups(s, case):
    table, T, ps, least = s["table"], s["T"].long(), case["page"], case["least"]
    seq, B = s["seq"].long(), len(s["T"])
    b = torch.arange(B, device=DEV)
    deep = T >= least
    key = table[seq, (least - 1) // ps].long() if (least - 1) // ps < table.shape[1] else torch.full_like(seq, -1)
    deep &= key >= 0
    lead = torch.full((len(s["ref"]),), B, device=DEV).scatter_reduce(0, key[deep], b[deep], "amin")
    lead = torch.where(deep, lead[key.clamp(min=0)], b)
    mine, other = table[seq], table[seq[lead]]
    same = ((mine == other) & (mine >= 0)).int().cumprod(1).sum(1) * ps
    common = torch.minimum(torch.minimum(same, T), T[lead])
    lead = torch.where(deep & (common >= least), lead, b)
    order = torch.argsort(lead, stable=True)
    slot = torch.empty_like(order).scatter_(0, order, b)
    top = torch.full((B,), 1 << 40, device=DEV)
    top = top.scatter_reduce(0, lead, torch.where(lead == b, 1 << 40, common), "amin")
    shared = torch.where(top[lead] == 1 << 40, 0, top[lead])
    return order.int(), slot[lead[order]].int(), shared[order].int()


def _rows(s, case, page, row):
    raw = torch.int16 if case["kv"] == "bf16" else torch.uint8
    return s["pool"][0].view(raw)[page, row].view(TYPES[case["kv"]]).float()


def _plain_attn(s, case):
    ps, H, sink = case["page"], case["heads"], s["sink"]
    for m, shared, tail in s["lists"]:
        n = len(m)
        q = s["q"][m].float() * D ** -0.5
        rows, T = s["table"][s["seq"][m].long()].long(), s["T"][m].long()
        top, zp, zt = sink.expand(n, H), None, None
        if shared:
            pos = torch.arange(shared, device=DEV)
            kp = _rows(s, case, rows[0][pos // ps], pos % ps)
            zp = torch.matmul(q.view(n * H, D), kp.T).view(n, H, shared)
            top = torch.maximum(top, zp.amax(-1))
        if tail:
            pos = shared + torch.arange(tail, device=DEV)
            there = pos < T[:, None]
            pos = torch.where(there, pos, 0)
            kt = _rows(s, case, rows.gather(1, pos // ps).clamp(min=0), pos % ps)
            zt = torch.matmul(q, kt.transpose(1, 2)).masked_fill(~there[:, None], -math.inf)
            top = torch.maximum(top, zt.amax(-1))
        den, o = torch.exp(sink - top), 0
        if shared:
            e = torch.exp(zp - top[..., None])
            den = den + e.sum(-1)
            o = o + torch.matmul(e.view(n * H, shared), kp).view(n, H, D)
        if tail:
            e = torch.exp(zt - top[..., None])
            den = den + e.sum(-1)
            o = o + torch.matmul(e, kt)
        s["out"][m] = (o / den[..., None]).bfloat16()
    return s["out"]


# ------------------------------------------------------------------------------- the framework's calls
def _handle(s, case):
    """What a user's program keeps between calls: parameters, the cache, buffers, a workspace."""
    if "handle" not in s:
        from csa2_compressed_sparse_02_gb300 import api
        p = api.default_params(kv_format=api.BF16 if case.get("kv") == "bf16" else api.E4M3)
        if case["op"] == "attn":
            p.heads = case["heads"]
        cache = api.PagedCache(p, pool=s["pool"], ref=s["ref"], table=s["table"])
        if case["op"] == "slots":
            kept = api.SlotMap(len(s["which"]), case["rows"], device=DEV)
        elif case["op"] == "groups":
            kept = api.PrefixGroups(len(s["seq"]), device=DEV)
        else:
            kept = (api.PrefixGroups(order=s["order"], first=s["first"], shared=s["shared"]),
                    api.paged_attn_shared_workspace(p, cache, len(s["seq"])))
        s["handle"] = api, p, cache, kept
    return s["handle"]


def _own(s, case):
    api, p, cache, kept = _handle(s, case)
    if case["op"] == "slots":
        api.page_slots(p, cache, s["which"], s["held"], s["new"], kept)
        return s["table"], s["ref"], kept.n_tokens, kept.start, kept.seq, kept.pos, kept.slot
    if case["op"] == "groups":
        api.prefix_groups(p, cache, s["seq"], s["T"], kept, least=case["least"])
        return kept.order, kept.first, kept.shared
    groups, ws = kept
    api.paged_attn_shared(p, cache, 0, s["q"], s["sink"], s["seq"], s["T"], groups, s["out"], ws)
    return s["out"]


def run(state):
    case = state["case"]
    if own:
        return _own(state, case)
    return {"slots": _plain_slots, "groups": _plain_groups, "attn": _plain_attn}[case["op"]](state, case)


# ------------------------------------------------------------------------------- work
def work(case):
    """Each shared position is read once a family, each other one once; means of what is drawn."""
    if case["op"] == "slots":
        rows = case["seqs"] + case["chunks"] * case["chunk"] / 2
        pages = rows / case["page"] + 1
        return {"bytes": 16.0 * case["rows"] + 20.0 * (case["seqs"] + case["idle"]) + 12.0 * pages, "flops": 0.0}
    sizes, P = _sizes(case), case["prefix"]
    P = [P] + [P if case["even"] else P * 9.0 / 16] * (len(sizes) - 1)
    B = sum(sizes)
    if case["op"] == "groups":  # entries that two sequences have in common are compared
        entries = sum(n * p / case["page"] for n, p in zip(sizes, P) if n > 1)
        return {"bytes": 4.0 * entries + 20.0 * B, "flops": 0.0}
    tail = (case["tail"] + 1) / 2 if case["tail"] else 0
    seen = sum(n * (p + tail) for n, p in zip(sizes, P))
    if case["tail"]:
        read = sum(p + n * tail for n, p in zip(sizes, P))
    else:
        read = sum(p + n - 1 for n, p in zip(sizes, P))
    row = 2 * D if case["kv"] == "bf16" else D
    return {"bytes": read * row + 4.0 * B * case["heads"] * D, "flops": 4.0 * D * case["heads"] * seen}


# ------------------------------------------------------------------------------- 64-bit definitions
def exact(case, seed):
    """Every sequence by itself, through its own row of the table."""
    if case["op"] != "attn":
        return None
    s, ps = prepare(case, seed), case["page"]
    flat = s["pool"][0].view(-1, D)
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    for b, (T, row) in enumerate(zip(s["T"].tolist(), s["seq"].tolist())):
        pos = torch.arange(T, device=DEV)
        kv = flat[s["table"][row].long()[pos // ps] * ps + pos % ps].double()
        z = s["q"][b].double() @ kv.T / math.sqrt(D)
        w = torch.softmax(torch.cat([z, s["sink"].double()[:, None]], 1), 1)
        out[b] = w[:, :-1] @ kv
    return out

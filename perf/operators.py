"""The paged-cache operators and the rotary embedding: the cases they are measured on,
their plain forms and their 64-bit definitions.

``own`` False: ``run`` computes a case with elementary torch operations in 32 bits (angles
in 64); True: with the calls a user of the framework makes. A case's ``op`` names the
operator; the sizes are those of the framework's default configuration (64 heads sharing
one 512-wide latent, of which the last 64 channels are rotated, base 160000, YaRN factor
16 over 65,536) and its tensor-parallel shards.
"""
import math

import numpy as np
import torch

own = False

D = 512
THETA, FACTOR, ORIG_LEN, BETA_FAST, BETA_SLOW = 160000.0, 16.0, 65536.0, 32.0, 1.0
DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32, "e4m3": torch.float8_e4m3fn}


# ------------------------------------------------------------------------------- cases
def listed():
    return [
        # the queries of a decode step: 64 sequences, 64 heads, the last 64 of 512 channels
        dict(name="rope decode", op="rope", rows=64, heads=64, dim=512, rope=64, layout="pairs",
             type="bf16", inverse=False, far=1048576),
        # the outputs of a prefill chunk turned back (the inverse, which is also the gradient)
        dict(name="rope chunk inverse", op="rope", rows=8192, heads=64, dim=512, rope=64,
             layout="pairs", type="bf16", inverse=True, far=262144),
        # a whole head in the half layout, unquantised, an odd number of rows
        dict(name="rope half f32", op="rope", rows=1023, heads=8, dim=128, rope=128,
             layout="half", type="f32", inverse=False, far=65536),
        # one new token of each of 64 sequences: pages reserved, rows rotated and written
        dict(name="write decode", op="write", seqs=64, new=1, page=64, kv="bf16", rope=64,
             longest=32768),
        # a prefill chunk of 4 sequences into 8-bit pages, ending inside a page
        dict(name="write chunk e4m3", op="write", seqs=4, new=4001, page=64, kv="e4m3", rope=64,
             longest=65536),
        # a single short conversation: latency
        dict(name="attn one short", op="attn", seqs=1, heads=64, longest=200, even=True, page=16,
             kv="bf16", window=0, first=0),
        # ordinary ragged batch on 8-bit pages
        dict(name="attn ragged e4m3", op="attn", seqs=32, heads=64, longest=8192, even=False,
             page=64, kv="e4m3", window=0, first=0),
        # a shard of 16 heads, window of 4096 and 64 first tokens, pages behind it released
        dict(name="attn window 16 heads", op="attn", seqs=48, heads=16, longest=1000000,
             even=False, page=64, kv="bf16", window=4096, first=64),
        # long contexts, all heads
        dict(name="attn long bf16", op="attn", seqs=16, heads=64, longest=131072, even=True,
             page=64, kv="bf16", window=0, first=0),
        # 8 prompts forked into 32 continuations over 4 layers, the former ones released
        dict(name="fork 8 to 32", op="fork", parents=8, children=32, longest=4096, page=64,
             layers=4, pages=4096, kv="bf16"),
        # many continuations of long prompts, large pages, 8-bit
        dict(name="fork 64 to 256", op="fork", parents=64, children=256, longest=32768, page=128,
             layers=8, pages=24576, kv="e4m3"),
        # a pool after its sequences came and went, half of it in use
        dict(name="compact half", op="compact", pages=16384, used=8192, page=64, layers=2,
             seqs=64, kv="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "rope", "write", "attn", "attn", "attn", "fork", "compact"])
    if op == "rope":
        dim = rng.choice([64, 80, 128, 192, 512])
        heads = rng.choice([1, 2, 8, 16, 31, 64])
        return dict(op=op, rows=min(_log(rng, 1, 8192), max(1, (1 << 28) // (heads * dim))),
                    heads=heads, dim=dim,
                    rope=rng.choice([r for r in (32, 64, dim // 2, dim) if r <= dim]),
                    layout=rng.choice(["pairs", "half"]), type=rng.choice(["bf16", "f32"]),
                    inverse=rng.random() < 0.5, far=_log(rng, 1000, 1 << 20))
    if op == "write":
        seqs = _log(rng, 1, 200)
        return dict(op=op, seqs=seqs, new=rng.choice([1, _log(rng, 1, max(1, 16000 // seqs))]),
                    page=rng.choice([16, 32, 64, 128]), kv=rng.choice(["bf16", "e4m3"]),
                    rope=rng.choice([0, 64, 128]), longest=_log(rng, 64, 65536))
    if op == "attn":
        seqs = _log(rng, 1, 128)
        window = rng.choice([0, 0, _log(rng, 1, 8192)])
        longest = _log(rng, 1, 1000000 if window else min(131072, 2000000 // seqs))
        return dict(op=op, seqs=seqs, heads=rng.choice([1, 8, 12, 16, 32, 64]), longest=longest,
                    even=rng.random() < 0.3, page=rng.choice([8, 16, 32, 64, 128]),
                    kv=rng.choice(["bf16", "e4m3"]), window=window,
                    first=rng.choice([0, 4, 128]) if window else 0)
    if op == "fork":
        parents = _log(rng, 1, 64)
        longest, page = _log(rng, 10, 16384), rng.choice([16, 64, 128])
        children = parents * rng.choice([1, 2, 4])
        return dict(op=op, parents=parents, children=children, longest=longest, page=page,
                    layers=rng.choice([1, 2, 4]), kv=rng.choice(["bf16", "e4m3"]),
                    pages=parents * -(-longest // page) + children + rng.randrange(1, 1000))
    pages = _log(rng, 100, 16384)
    return dict(op=op, pages=pages, used=max(1, int(pages * rng.uniform(0.05, 0.95))),
                page=rng.choice([16, 64]), layers=rng.choice([1, 2]), seqs=_log(rng, 1, 100),
                kv=rng.choice(["bf16", "e4m3"]))


# ------------------------------------------------------------------------------- inputs
def _lengths(case, seed):
    """Tokens each sequence holds: all the longest, or from an eighth of it up, spread evenly."""
    n, top = case.get("seqs", case.get("parents")), case["longest"]
    if case.get("even"):
        return np.full(n, top, np.int64)
    r = np.random.default_rng([seed, 1])
    t = np.maximum(1, np.floor(top * (0.125 + 0.875 * r.random(n))).astype(np.int64))
    t[0] = top
    return t


def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _pool(shape, kv, gen):
    """Latents of unit variance: a pool of pages."""
    pool = torch.empty(shape, dtype=torch.bfloat16, device=DEV).normal_(generator=gen)
    return pool if kv == "bf16" else pool.to(TYPES["e4m3"])


def _i32(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).to(DEV)


def _visible(T, window, first):
    """Lowest position of the window and how many first tokens lie before it."""
    lo = max(0, T - window) if window else 0
    return lo, min(first, lo)


def _tables(case, T, seed, spare):
    """Pages of each sequence in random order; those that no later token can see are absent."""
    ps, w, f = case["page"], case.get("window", 0), case.get("first", 0)
    n = -(-T // ps)
    table = np.full((len(T), int(n.max())), -1, np.int64)
    k = np.arange(table.shape[1])
    held = k[None, :] < n[:, None]
    if w:
        held &= (k[None, :] * ps < f) | ((k[None, :] + 1) * ps > (T - w)[:, None])
    pages = int(held.sum()) + spare
    table[held] = np.random.default_rng([seed, 2]).permutation(pages)[:int(held.sum())]
    return table, pages


def prepare(case, seed):
    g, s = _gen(seed), {"case": case}
    if case["op"] == "rope":
        s["x"] = torch.randn(case["rows"], case["heads"], case["dim"], generator=g,
                             device=DEV).to(TYPES[case["type"]])
        s["pos"] = torch.randint(0, case["far"], (case["rows"],), generator=g, device=DEV,
                                 dtype=torch.int32)
        s["out"] = torch.empty_like(s["x"])
    elif case["op"] == "write":
        S, ps, new = case["seqs"], case["page"], case["new"]
        T = _lengths(case, seed)
        table, have = _tables(case, T, seed, 0)
        wide = int((-(-(T + new) // ps)).max())
        table = np.concatenate([table, np.full((S, wide - table.shape[1]), -1, np.int64)], 1)
        # of the sequences' earlier rows only the pages' places matter here, so the pool holds
        # those the new rows touch, in random order among pages of other owners
        touched = (np.arange(wide)[None] >= (T // ps)[:, None]) & (np.arange(wide)[None] < (-(-(T + new) // ps))[:, None])
        own_ = touched & (table >= 0)
        n_own, n_new = int(own_.sum()), int((touched & (table < 0)).sum())
        pages = 2 * S * (new // ps + 2) + 64
        perm = np.random.default_rng([seed, 3]).permutation(pages)
        table = np.full_like(table, -1)
        table[own_] = perm[:n_own]
        ref = np.zeros(pages, np.int64)
        ref[perm[:n_own + (pages - n_own - n_new) // 2]] = 1
        s["table"], s["ref"] = _i32(table), _i32(ref)
        s["pool"] = torch.zeros(1, pages, ps, D, dtype=torch.bfloat16, device=DEV).to(TYPES[case["kv"]])
        s["x"] = torch.randn(S * new, D, generator=g, device=DEV)
        s["seq"] = _i32(np.repeat(np.arange(S), new))
        s["pos"] = _i32((T[:, None] + np.arange(new)[None]).reshape(-1))
        s["which"], s["t0"], s["t1"] = _i32(np.arange(S)), _i32(T), _i32(T + new)
    elif case["op"] == "attn":
        T = _lengths(case, seed)
        table, pages = _tables(case, T, seed, 3)
        s["table"], s["T"] = _i32(table), _i32(T)
        s["ref"] = torch.ones(pages, dtype=torch.int32, device=DEV)
        s["pool"] = _pool((1, pages, case["page"], D), case["kv"], g)
        # logits of standard deviation 2: some positions matter more than others
        s["q"] = (2 * torch.randn(len(T), case["heads"], D, generator=g, device=DEV)).bfloat16()
        s["sink"] = torch.randn(case["heads"], generator=g, device=DEV)
        s["seq"] = _i32(np.arange(len(T)))
        s["out"] = torch.empty_like(s["q"])
    elif case["op"] == "fork":
        T, ps = _lengths(case, seed), case["page"]
        table, held = _tables(case, T, seed, 0)
        P, C = case["parents"], case["children"]
        place = np.random.default_rng([seed, 4]).permutation(case["pages"])[:held]
        rows = np.full((P + C, table.shape[1] + 1), -1, np.int64)
        rows[:P, :-1] = np.where(table >= 0, place[np.maximum(table, 0)], -1)
        ref = np.zeros(case["pages"], np.int64)
        ref[place] = 1
        parent = np.arange(C) % P
        s["table"], s["ref"] = _i32(rows), _i32(ref)
        s["pool"] = _pool((case["layers"], case["pages"], ps, D), case["kv"], g)
        s["parent"], s["child"], s["T"] = _i32(parent), _i32(P + np.arange(C)), _i32(T[parent])
    else:
        P, n = case["pages"], case["used"]
        r = np.random.default_rng([seed, 5])
        held = r.permutation(P)[:n]
        S = case["seqs"]
        wide = -(-n // S) + 2
        table = np.full((S, wide), -1, np.int64)
        at = np.arange(n)
        table[at % S, at // S] = held
        ref = np.zeros(P, np.int64)
        ref[held] = 1
        if S > 1:  # a shared page: the first sequence's first is also the last one's last
            table[S - 1, wide - 1] = table[0, 0]
            ref[table[0, 0]] += 1
        s["table0"], s["ref0"] = _i32(table), _i32(ref)
        s["table"], s["ref"] = s["table0"].clone(), s["ref0"].clone()
        s["pool"] = _pool((case["layers"], P, case["page"], D), case["kv"], g)
        s["n_used"] = torch.zeros(1, dtype=torch.int32, device=DEV)
    return s


# ------------------------------------------------------------------------------- plain forms
def _frequencies(dim):
    """YaRN's angles a position (Peng et al. 2023, NTK-by-parts), in 64 bits."""
    f = torch.tensor(THETA, dtype=torch.float64, device=DEV) ** (
        -torch.arange(0, dim, 2, dtype=torch.float64, device=DEV) / dim)
    keep = ((ORIG_LEN * f / (2 * math.pi) - BETA_SLOW) / (BETA_FAST - BETA_SLOW)).clamp(0, 1)
    return f * keep + f / FACTOR * (1 - keep)


def _rotate(x, pos, dim, layout, inverse):
    """The last `dim` channels of x [..., channels] (32 bits) turned by the angles of pos [...]."""
    a = pos.double()[..., None] * _frequencies(dim)
    c, s = a.cos().float(), a.sin().float()
    if inverse:
        s = -s
    t = x[..., x.shape[-1] - dim:]
    if layout == "pairs":
        u, v = t[..., 0::2], t[..., 1::2]
        y = torch.stack([u * c - v * s, u * s + v * c], -1).flatten(-2)
    else:
        u, v = t[..., :dim // 2], t[..., dim // 2:]
        y = torch.cat([u * c - v * s, u * s + v * c], -1)
    return torch.cat([x[..., :x.shape[-1] - dim], y], -1)


def _e4m3(x):
    return x.clamp(-448, 448).to(TYPES["e4m3"])


def _plain_rope(s, case):
    y = _rotate(s["x"].float(), s["pos"][:, None], case["rope"], case["layout"], case["inverse"])
    s["out"].copy_(y)
    return s["out"]


def _lowest_free(ref):
    return torch.argsort((ref > 0).to(torch.int8), stable=True)


def _plain_write(s, case):
    table, ref, pool, ps = s["table"], s["ref"], s["pool"], case["page"]
    k = torch.arange(table.shape[1], device=DEV)
    need = (k >= (s["t0"] // ps)[:, None]) & (k < ((s["t1"] + ps - 1) // ps)[:, None]) & (table < 0)
    rank = need.flatten().cumsum(0).view(need.shape) - 1
    taken = _lowest_free(ref)[rank.clamp(min=0)].int()
    table.copy_(torch.where(need, taken, table))
    ref.scatter_add_(0, torch.where(need, taken, 0).flatten().long(), need.flatten().int())
    y = s["x"]
    if case["rope"]:
        y = _rotate(y, s["pos"], case["rope"], "pairs", False)
    y = y.bfloat16() if case["kv"] == "bf16" else _e4m3(y)
    page = table[s["seq"].long(), (s["pos"] // ps).long()].long()
    raw = torch.int16 if case["kv"] == "bf16" else torch.uint8
    pool[0].view(raw)[page, (s["pos"] % ps).long()] = y.view(raw)
    return pool, table, ref


def _plain_attn(s, case):
    ps, w, f = case["page"], case["window"], case["first"]
    T = s["T"].long()[:, None]
    lo = (T - w).clamp(min=0) if w else torch.zeros_like(T)
    most = min(case["longest"], w + f) if w else case["longest"]
    j = torch.arange(most, device=DEV)[None]
    head = lo.clamp(max=f)
    pos = torch.where(j < head, j, lo + j - head)
    there = pos < T
    pos = torch.where(there, pos, 0)
    page = s["table"].long().gather(1, pos // ps).clamp(min=0)
    raw = torch.int16 if case["kv"] == "bf16" else torch.uint8
    k = s["pool"][0].view(raw)[page, pos % ps].view(TYPES[case["kv"]]).float()
    z = torch.matmul(s["q"].float(), k.transpose(1, 2)) * D ** -0.5
    z = z.masked_fill(~there[:, None], -math.inf)
    sink = s["sink"][None, :, None]
    m = torch.maximum(z.amax(-1, keepdim=True), sink)
    e = torch.exp(z - m)
    o = torch.matmul(e, k) / (e.sum(-1, keepdim=True) + torch.exp(sink - m))
    s["out"].copy_(o)
    return s["out"]


def _plain_fork(s, case):
    table, ref, pool, ps = s["table"], s["ref"], s["pool"], case["page"]
    parent, child, T = s["parent"].long(), s["child"].long(), s["T"].long()
    old = table[child]  # the former continuations go
    ref.scatter_add_(0, old.clamp(min=0).flatten().long(), -(old >= 0).flatten().int())
    rows = table[parent]
    k = torch.arange(table.shape[1], device=DEV)[None]
    full = (T // ps)[:, None]
    shared = (k < full) & (rows >= 0)
    ref.scatter_add_(0, rows.clamp(min=0).flatten().long(), shared.flatten().int())
    part = T % ps > 0
    taken = _lowest_free(ref)[(part.cumsum(0) - 1).clamp(min=0)].int()
    table[child] = torch.where(shared, rows, torch.where((k == full) & part[:, None], taken[:, None], -1))
    ref.scatter_add_(0, torch.where(part, taken, 0).long(), part.int())
    raw = torch.int16 if case["kv"] == "bf16" else torch.uint8
    rowsof = pool.view(raw)
    src = rows.gather(1, full).clamp(min=0).flatten().long()
    kept = torch.arange(ps, device=DEV)[None] < (T % ps)[:, None]
    i, r = kept.nonzero(as_tuple=True)
    rowsof[:, taken.long()[i], r] = rowsof[:, src[i], r]
    return pool, table, ref


def _plain_compact(s, case):
    s["table"].copy_(s["table0"])  # the next batch's tables
    s["ref"].copy_(s["ref0"])
    table, ref, pool = s["table"], s["ref"], s["pool"]
    at = torch.arange(ref.numel(), device=DEV)
    used = ref > 0
    n = used.sum()
    src = (used & (at >= n)).nonzero().flatten()
    dst = (~used & (at < n)).nonzero().flatten()
    to = at.int()
    to[src] = dst.int()
    pool[:, dst] = pool[:, src]
    table.copy_(torch.where(table >= 0, to[table.clamp(min=0).long()], table))
    ref[dst] = ref[src]
    ref[src] = 0
    s["n_used"].copy_(n)
    return pool, table, ref, s["n_used"]


# ------------------------------------------------------------------------------- the framework's calls
def _handle(s, case):
    """What a user's program keeps between calls: parameters, the cache, a workspace."""
    if "handle" not in s:
        from csa2_compressed_sparse_02_gb300 import api
        kv = {"bf16": api.BF16, "e4m3": api.E4M3}.get(case.get("kv"), api.BF16)
        p = api.default_params(kv_format=kv, rope_dim=case.get("rope", 0))
        if case["op"] == "attn":
            p.heads = case["heads"]
        cache = ws = None
        if case["op"] != "rope":
            cache = api.PagedCache(p, pool=s["pool"], ref=s["ref"], table=s["table"])
        if case["op"] == "attn":
            ws = api.paged_attn_workspace(p, cache, case["seqs"])
        s["handle"] = api, p, cache, ws
    return s["handle"]


def _own(s, case):
    api, p, cache, ws = _handle(s, case)
    op = case["op"]
    if op == "rope":
        layout = api.ROPE_PAIRS if case["layout"] == "pairs" else api.ROPE_HALF
        api.rope(p, s["x"], s["pos"], s["out"], layout=layout, inverse=case["inverse"])
        return s["out"]
    if op == "write":
        api.page_reserve(p, cache, s["which"], s["t0"], s["t1"])
        api.page_write(p, cache, 0, s["x"], s["seq"], s["pos"])
        return s["pool"], s["table"], s["ref"]
    if op == "attn":
        api.paged_attn(p, cache, 0, s["q"], s["sink"], s["seq"], s["T"], s["out"], ws,
                       window=case["window"], n_first=case["first"])
        return s["out"]
    if op == "fork":
        api.page_release(p, cache, s["child"])
        api.page_fork(p, cache, s["parent"], s["child"], s["T"])
        return s["pool"], s["table"], s["ref"]
    s["table"].copy_(s["table0"])
    s["ref"].copy_(s["ref0"])
    api.page_compact(p, cache, s["n_used"])
    return s["pool"], s["table"], s["ref"], s["n_used"]


def run(state):
    case = state["case"]
    if own:
        return _own(state, case)
    plain = {"rope": _plain_rope, "write": _plain_write, "attn": _plain_attn, "fork": _plain_fork,
             "compact": _plain_compact}
    return plain[case["op"]](state, case)


# ------------------------------------------------------------------------------- work
def work(case):
    op = case["op"]
    row = {"bf16": 2 * D, "e4m3": D}.get(case.get("kv"), 0)
    if op == "rope":
        n = case["rows"] * case["heads"]
        es = 2 if case["type"] == "bf16" else 4
        return {"bytes": 2.0 * n * case["dim"] * es + 4.0 * case["rows"], "flops": 3.0 * n * case["rope"]}
    if op == "write":
        n = case["seqs"] * case["new"]
        return {"bytes": n * (4.0 * D + row + 8), "flops": 3.0 * n * case["rope"]}
    if op == "attn":  # mean length of _lengths: 9/16 of the longest where they differ
        T = case["longest"] * (1.0 if case["even"] else 9.0 / 16)
        T = max(1.0, min(T, case["window"] + case["first"]) if case["window"] else T)
        q = 2 * 2 * case["heads"] * D
        return {"bytes": case["seqs"] * (T * row + q), "flops": case["seqs"] * T * case["heads"] * D * 4.0}
    if op == "fork":  # half a page of rows in the mean, and the shared entries of table and counts
        entries = case["children"] * (0.5625 * case["longest"] / case["page"] + 1)
        rows = case["children"] * case["layers"] * case["page"] / 2
        return {"bytes": 2.0 * rows * row + 16.0 * entries, "flops": 0.0}
    moved = case["used"] * (1 - case["used"] / case["pages"])
    return {"bytes": 2.0 * moved * case["layers"] * case["page"] * row + 8.0 * (case["used"] + case["pages"]),
            "flops": 0.0}


# ------------------------------------------------------------------------------- 64-bit definitions
def _angles64(pos, dim):
    i = np.arange(dim // 2, dtype=np.float64)
    f = THETA ** (-2 * i / dim)
    turns = ORIG_LEN * f / (2 * np.pi)
    keep = np.where(turns > BETA_FAST, 1.0,
                    np.where(turns < BETA_SLOW, 0.0, (turns - BETA_SLOW) / (BETA_FAST - BETA_SLOW)))
    f = f * keep + f / FACTOR * (1 - keep)
    return torch.from_numpy(pos.cpu().numpy().astype(np.float64)[:, None] * f[None]).to(DEV)


def _turned64(x, pos, dim, layout, inverse):
    """x [rows, heads, channels] in 64 bits as complex numbers times e^(i angle)."""
    ang = _angles64(pos, dim)
    turn = torch.polar(torch.ones_like(ang), -ang if inverse else ang)[:, None]
    y = x.double().clone()
    n = y.shape[-1]
    if layout == "pairs":
        z = torch.view_as_complex(y[..., n - dim:].reshape(*y.shape[:2], dim // 2, 2).contiguous()) * turn
        y[..., n - dim:] = torch.view_as_real(z).reshape(*y.shape[:2], dim)
    else:
        z = torch.complex(y[..., n - dim:n - dim // 2], y[..., n - dim // 2:]) * turn
        y[..., n - dim:n - dim // 2], y[..., n - dim // 2:] = z.real, z.imag
    return y


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rope":
        return _turned64(s["x"], s["pos"], case["rope"], case["layout"], case["inverse"])
    if case["op"] == "write":
        table, ps = s["table"].cpu().numpy(), case["page"]
        free = list(np.flatnonzero(s["ref"].cpu().numpy() == 0))
        for b, (a, e) in enumerate(zip(s["t0"].tolist(), s["t1"].tolist())):
            for k in range(a // ps, -(-e // ps)):
                if table[b, k] < 0:
                    table[b, k] = free.pop(0)
        y = s["x"].double()
        if case["rope"]:
            y = _turned64(s["x"][:, None], s["pos"], case["rope"], "pairs", False)[:, 0]
        pool = s["pool"].double()
        seq, pos = s["seq"].cpu().numpy(), s["pos"].cpu().numpy()
        page = torch.from_numpy(table[seq, pos // ps].astype(np.int64)).to(DEV)
        pool[0, page, torch.from_numpy((pos % ps).astype(np.int64)).to(DEV)] = y
        return pool, None, None
    if case["op"] == "attn":
        ps, out = case["page"], torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
        for b, T in enumerate(s["T"].tolist()):
            lo, head = _visible(T, case["window"], case["first"])
            pos = torch.cat([torch.arange(head, device=DEV), torch.arange(lo, T, device=DEV)])
            page = s["table"][b].long()[pos // ps]
            kv = s["pool"][0].view(-1, D)[page * ps + pos % ps].double()
            z = s["q"][b].double() @ kv.T / math.sqrt(D)
            both = torch.cat([z, s["sink"].double()[:, None]], 1)
            out[b] = torch.softmax(both, 1)[:, :-1] @ kv
        return out
    return None

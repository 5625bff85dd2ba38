"""Host-side checks of the slot maps, the prefix groups and the attention behind shared prefixes (no
GPU): what they refuse before anything is enqueued. The buffers are host memory, never
dereferenced."""
import ctypes
import os
import re

import pytest
import torch

from csa2_compressed_sparse_02_gb300 import _lib, api

INVALID, SHAPE, ALIGN, UNSUPPORTED = 1, 2, 3, 4
ROOM = 1 << 30


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(_lib.LIB_PATH):
        import __graft_entry__
        __graft_entry__.build()
    return _lib.lib()


_buf = (ctypes.c_uint8 * 1024)()
A = (ctypes.addressof(_buf) + 255) & ~255  # aligned, host


def params(**over):
    return api.default_params(**dict(dict(kv_format=api.BF16), **over))


def pages(**over):
    f = dict(pool=A, layer_bytes=1 << 20, table=A, ref=A, layers=2, n_pages=16, page_size=64,
             max_seqs=4, max_pages=8)
    f.update(over)
    return _lib.Pages(**f)


def slots(L, p, c, B=2, N=8, seq=A, held=A, new=A, after=A, start=A, rows=A, pos=A, slot=A, ws=A, n=ROOM):
    return L.csa2_page_slots(p, c, B, seq, held, new, N, after, start, rows, pos, slot, ws, n, None, None)


def groups(L, p, c, B=2, seq=A, held=A, least=1, order=A, first=A, shared=A, ws=A, n=ROOM):
    return L.csa2_prefix_groups(p, c, B, seq, held, least, order, first, shared, ws, n, None, None)


def attn(L, p, c, layer=0, B=2, q=A, qs=32768, qh=512, seq=A, held=A, order=A, first=A, shared=A, out=A, ws=A,
         n=ROOM):
    return L.csa2_paged_attn_shared(p, c, layer, B, q, qs, qh, None, seq, held, order, first, shared, out, ws, n,
                                    None, None)


CALLS = dict(slots=slots, groups=groups, attn=attn)


@pytest.mark.parametrize("call", CALLS.values(), ids=CALLS)
@pytest.mark.parametrize("over,code", [
    (dict(pool=None), INVALID), (dict(table=None), INVALID), (dict(ref=None), INVALID), (dict(layers=0), INVALID),
    (dict(n_pages=0), INVALID), (dict(max_seqs=0), INVALID), (dict(page_size=12), UNSUPPORTED),
    (dict(page_size=1032), UNSUPPORTED), (dict(layer_bytes=16 * 64 * 1024 - 16), SHAPE), (dict(pool=A + 8), ALIGN),
    (dict(table=A + 2), ALIGN)])
def test_a_malformed_cache_is_refused(L, call, over, code):
    assert call(L, params(), pages(**over)) == code
    assert L.csa2_last_error()


@pytest.mark.parametrize("call", CALLS.values(), ids=CALLS)
def test_what_all_three_refuse(L, call):
    for over in (dict(head_dim=256), dict(kv_format=api.NVFP4), dict(kv_format=api.F32)):
        assert call(L, params(**over), pages()) == UNSUPPORTED, over
    p, c = params(), pages()
    assert call(L, None, c) == INVALID and call(L, p, None) == INVALID
    assert call(L, p, c, B=-1) == INVALID
    assert call(L, p, c, ws=None) == INVALID and call(L, p, c, ws=A + 64) == ALIGN
    assert call(L, p, c, held=None) == INVALID


def test_slots_refusals(L):
    p, c = params(), pages()
    assert slots(L, p, c, B=1025) == INVALID  # beyond max_seqs and 1,024
    assert slots(L, p, c, N=-1) == INVALID and slots(L, p, c, N=2 ** 31 - 1) == INVALID
    for name in ("seq", "new", "after", "start", "rows", "pos", "slot"):
        assert slots(L, p, c, **{name: None}) == INVALID, name
    assert slots(L, p, c, slot=A + 4) == ALIGN
    assert slots(L, p, c, n=L.csa2_page_workspace_size(ctypes.byref(c)) - 256) == SHAPE


def test_groups_refusals(L):
    p, c = params(), pages()
    assert groups(L, p, c, least=0) == INVALID and groups(L, p, c, B=65536) == UNSUPPORTED
    assert groups(L, p, c, B=5, seq=None) == INVALID  # rows 0 .. 4 of a table of 4
    for name in ("order", "first", "shared"):
        assert groups(L, p, c, **{name: None}) == INVALID, name
    assert groups(L, p, c, B=100, n=L.csa2_prefix_groups_workspace_size(100) - 256) == SHAPE
    assert groups(L, p, c, B=0, held=None, order=None, ws=None) == 0


def test_attention_refusals(L):
    p, c = params(), pages()
    assert attn(L, p, c, layer=2) == INVALID and attn(L, p, c, layer=-1) == INVALID
    assert attn(L, p, c, B=65536) == UNSUPPORTED and attn(L, p, c, B=5, seq=None) == INVALID
    for over in (dict(heads=0), dict(heads=65), dict(q_format=api.F32)):
        assert attn(L, params(**over), c) == UNSUPPORTED, over
    for name in ("q", "order", "first", "shared", "out"):
        assert attn(L, p, c, **{name: None}) == INVALID, name
    assert attn(L, p, c, q=A + 8) == ALIGN and attn(L, p, c, out=A + 2) == ALIGN
    assert attn(L, p, c, qs=516) == ALIGN and attn(L, p, c, qh=514) == ALIGN
    assert attn(L, p, c, B=0, q=None, out=None, ws=None) == 0


def test_workspace_sizes(L):
    p, c = ctypes.byref(params()), ctypes.byref(pages())
    assert L.csa2_prefix_groups_workspace_size(0) == 0 and L.csa2_prefix_groups_workspace_size(-1) == 0
    assert L.csa2_prefix_groups_workspace_size(65535) >= 2 * 4 * 65535
    assert L.csa2_paged_attn_shared_workspace_size(p, c, 0) == 0
    assert L.csa2_paged_attn_shared_workspace_size(None, c, 4) == 0
    assert L.csa2_paged_attn_shared_workspace_size(ctypes.byref(params(heads=65)), c, 4) == 0


def test_binding_refuses_tensors_the_pointers_would_not_stand_for():
    p = params()
    pool = torch.zeros(1, 4, 16, 512, dtype=torch.bfloat16)
    table, ref = torch.full((2, 3), -1, dtype=torch.int32), torch.zeros(4, dtype=torch.int32)
    c = api.PagedCache(p, pool=pool, table=table, ref=ref)
    i, g = torch.zeros(2, dtype=torch.int32), api.PrefixGroups(2, device="cpu")
    s = api.SlotMap(2, 8, device="cpu")
    assert [t.shape[0] for t in (s.n_tokens, s.start, s.seq, s.pos, s.slot)] == [2, 3, 8, 8, 8]
    for bad in (dict(order=i, first=i), dict(order=i.long(), first=i, shared=i), dict(order=i, first=i[:1], shared=i),
                dict(order=torch.zeros(4, dtype=torch.int32)[::2], first=i, shared=i)):
        with pytest.raises(api.Csa2Error):
            api.PrefixGroups(**bad)
    q = torch.zeros(2, 64, 512, dtype=torch.bfloat16)
    for k in (dict(q=q.float()), dict(q=q[:, :, :256]), dict(q=q[:, :32]), dict(out=q.float()), dict(out=q[:, :32]),
              dict(sink=torch.zeros(63)), dict(sink=torch.zeros(64).double()), dict(g=api.PrefixGroups(3, device="cpu"))):
        a = dict(dict(q=q, sink=None, out=torch.empty_like(q), g=g), **k)
        with pytest.raises(api.Csa2Error):
            api.paged_attn_shared(p, c, 0, a["q"], a["sink"], i, i, a["g"], a["out"], i)
    with pytest.raises(api.Csa2Error, match="another format"):
        api.paged_attn_shared(params(kv_format=api.E4M3), c, 0, q, None, i, i, g, torch.empty_like(q), i)
    with pytest.raises(api.Csa2Error, match="requests"):
        api.page_slots(p, c, torch.zeros(3, dtype=torch.int32), i, i, s)
    with pytest.raises(api.Csa2Error, match="int32"):
        api.page_slots(p, c, i, i.long(), i, s)
    with pytest.raises(api.Csa2Error, match="int32"):
        api.prefix_groups(p, c, i, i, api.PrefixGroups(3, device="cpu"))
    for call in (lambda: api.page_slots(p, c, i, i, i, s), lambda: api.prefix_groups(p, c, i, i, g),
                 lambda: api.prefix_groups(p, c, None, i, g),
                 lambda: api.paged_attn_shared(p, c, 0, q, None, i, i, g, torch.empty_like(q), i)):
        with pytest.raises(api.Csa2Error, match="CUDA"):  # nothing is enqueued for host tensors
            call()


def test_waits_of_the_kernel_are_decided_by_the_warp():
    """A bounded wait can give up lane by lane; the roles go on with shuffles, votes and TMEM accesses of
    the whole warp. By the source: every wait of a role votes, and none of a lane's own is left."""
    path = os.path.join(os.path.dirname(_lib.LIB_PATH), "csrc", "paged_shared.cu")
    code = re.sub(r"//[^\n]*", "", open(path).read())
    assert set(re.findall(r"\bmbar_(?:try_)?(?:wait|test)\w*(?=\()", code)) == {"mbar_try_wait_at", "mbar_wait_drain"}
    tries = [line for line in code.split("\n") if "mbar_try_wait_at(" in line]
    assert len(tries) == 2 and all("__all_sync(0xffffffffu, mbar_try_wait_at(" in line for line in tries)
    loop = code.split("bool wait_on(", 1)[1].split("\n}\n", 1)[0]
    returns = [line for line in loop.split("\n") if "*abort" in line and "return" in line]
    assert returns and all("__any_sync(0xffffffffu" in line for line in returns)


def test_outputs_of_the_join_lie_in_the_batch():
    """Rows of a partial result name their outputs in the workspace, which holds anything where a wait gave up before
    they were stored. By the source: they are read in one place, which bounds them by the batch's rows."""
    path = os.path.join(os.path.dirname(_lib.LIB_PATH), "csrc", "paged_shared.cu")
    code = re.sub(r"//[^\n]*", "", open(path).read())
    reads = [line for line in code.split("\n") if "kD + 2" in line and "__ldcg" in line]
    place_of = code.split("int place_of(", 1)[1].split("\n}\n", 1)[0]
    assert len(reads) == 1 and reads[0] in place_of
    assert "(uint32_t)place < (uint32_t)(a.B * a.heads) ? place : -1" in place_of

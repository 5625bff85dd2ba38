"""Host-side checks of the paged-cache calls and the rotary embedding (no GPU): what they
refuse before anything is enqueued. The buffers are host memory, never dereferenced."""
import ctypes
import os
import re
import subprocess
import sys

import pytest
import torch

from csa2_compressed_sparse_02_gb300 import _lib, api

INVALID, SHAPE, ALIGN, UNSUPPORTED = 1, 2, 3, 4


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


def rope(L, p, layout=0, N=2, heads=4, dim=128, first=-1, fmt=api.BF16, x=A, xr=512, xh=128, out=A + 512,
         orow=512, oh=128, pos=A):
    return L.csa2_rope(ctypes.byref(p), layout, 0, N, heads, dim, first, fmt, x, xr, xh, out, orow, oh,
                       pos, None)


def test_rope_refusals(L):
    p = params(rope_dim=64)
    assert rope(L, p, N=-1) == INVALID and rope(L, p, heads=-1) == INVALID
    assert rope(L, p, layout=2) == UNSUPPORTED and rope(L, p, fmt=api.E4M3) == UNSUPPORTED
    for dim in (0, 1, 63, -2, 514):
        assert rope(L, params(rope_dim=dim), dim=1024) == UNSUPPORTED, dim
    assert rope(L, p, dim=62) == UNSUPPORTED and rope(L, p, dim=4100) == UNSUPPORTED
    assert rope(L, p, first=65) == INVALID and rope(L, p, first=-2) == INVALID
    for over in (dict(rope_theta=0.0), dict(rope_factor=-1.0), dict(rope_beta_fast=1.0),
                 dict(rope_theta=float("inf")), dict(rope_factor=float("nan")),
                 dict(rope_beta_slow=-float("inf"))):
        assert rope(L, params(rope_dim=64, **over)) == INVALID, over
    assert rope(L, p, x=None) == INVALID and rope(L, p, pos=None) == INVALID
    assert rope(L, p, x=A + 1) == ALIGN and rope(L, p, fmt=api.F32, out=A + 2) == ALIGN
    assert rope(L, p, out=A, orow=1024) == INVALID  # in place with other strides
    assert rope(L, p, orow=0) == INVALID and rope(L, p, oh=0) == INVALID  # out over itself
    assert rope(L, p, N=0, x=None, out=None, pos=None) == 0 and rope(L, p, heads=0) == 0
    assert L.csa2_rope(None, 0, 0, 1, 1, 64, -1, api.BF16, A, 64, 64, A, 64, 64, A, None) == INVALID


def test_rope_in_place_keeps_its_padding(L):
    assert rope(L, params(rope_dim=64), layout=16, out=A) == INVALID
    for layout in (18, 32, 3, -1):
        assert rope(L, params(rope_dim=64), layout=layout) == UNSUPPORTED, layout


def calls(L, p, c, ws=A, n=1 << 30):
    """Every call on a cache, with sound arguments of its own."""
    p, c = ctypes.byref(p), ctypes.byref(c) if c is not None else None
    return dict(
        reserve=lambda N=2, a=A: L.csa2_page_reserve(p, c, N, a, A, A, ws, n, None, None),
        release=lambda N=2, a=A: L.csa2_page_release(p, c, N, a, None, 0, 0, None, None),
        fork=lambda N=2, a=A: L.csa2_page_fork(p, c, N, a, A, A, ws, n, None, None),
        compact=lambda: L.csa2_page_compact(p, c, None, ws, n, None, None),
        write=lambda N=2, a=A, layer=0, fmt=api.F32, x=A, row=512:
            L.csa2_page_write(p, c, layer, N, x, fmt, row, a, A, None, None),
        attn=lambda N=2, a=A, layer=0, q=A, qs=512, qh=512, out=A, seq=A:
            L.csa2_paged_attn(p, c, layer, N, q, qs, qh, None, seq, a, 0, 0, out, ws, n, None, None))


@pytest.mark.parametrize("over,code", [
    (dict(pool=None), INVALID), (dict(table=None), INVALID), (dict(ref=None), INVALID),
    (dict(layers=0), INVALID), (dict(n_pages=0), INVALID), (dict(max_seqs=0), INVALID),
    (dict(max_pages=0), INVALID), (dict(page_size=4), UNSUPPORTED), (dict(page_size=12), UNSUPPORTED),
    (dict(page_size=1032), UNSUPPORTED), (dict(n_pages=1 << 26, layer_bytes=1 << 42), UNSUPPORTED),
    (dict(max_pages=1 << 30), UNSUPPORTED), (dict(layer_bytes=16 * 64 * 1024 - 16), SHAPE),
    (dict(pool=A + 8), ALIGN), (dict(ref=A + 4), ALIGN), (dict(table=A + 2), ALIGN),
    (dict(layer_bytes=(1 << 20) + 8), ALIGN)])
def test_every_call_refuses_a_malformed_cache(L, over, code):
    for name, call in calls(L, params(), pages(**over)).items():
        assert call() == code, name
    assert L.csa2_last_error()


def test_calls_refuse_bad_parameters(L):
    for over in (dict(head_dim=256), dict(kv_format=api.NVFP4), dict(kv_format=api.F32)):
        for name, call in calls(L, params(**over), pages()).items():
            assert call() == UNSUPPORTED, (name, over)
    for name, call in calls(L, params(), None).items():
        assert call() == INVALID, name
    p, c = params(), pages()
    f = calls(L, p, c)
    for name in ("reserve", "release", "fork", "write", "attn"):
        assert f[name](N=-1) == INVALID, name
        assert f[name](N=0, a=None) == 0, name
        assert f[name](a=None) == INVALID, name
    assert f["reserve"](N=1025) == INVALID and f["fork"](N=1025) == INVALID  # beyond max_seqs and 1,024
    for name in ("reserve", "fork", "compact"):
        assert calls(L, p, c, ws=None)[name]() == INVALID
        assert calls(L, p, c, ws=A + 16)[name]() == ALIGN
        assert calls(L, p, c, n=L.csa2_page_workspace_size(ctypes.byref(c)) - 256)[name]() == SHAPE
    assert f["write"](layer=2) == INVALID and f["write"](layer=-1) == INVALID
    assert f["write"](fmt=api.E4M3) == UNSUPPORTED and f["write"](x=None) == INVALID
    assert f["write"](x=A + 8) == ALIGN and f["write"](row=514) == ALIGN
    for dim, code in ((62, UNSUPPORTED), (516, UNSUPPORTED), (-4, UNSUPPORTED)):
        assert calls(L, params(rope_dim=dim), c)["write"]() == code
    assert calls(L, params(rope_dim=64, rope_theta=0.0), c)["write"]() == INVALID
    assert f["attn"](layer=2) == INVALID and f["attn"](q=None) == INVALID and f["attn"](out=None) == INVALID
    assert f["attn"](N=5, seq=None) == INVALID and f["attn"](N=65536) == UNSUPPORTED
    assert f["attn"](q=A + 8) == ALIGN and f["attn"](qs=516) == ALIGN and f["attn"](out=A + 2) == ALIGN
    for over in (dict(heads=0), dict(heads=65), dict(q_format=api.F32)):
        assert calls(L, params(**over), c)["attn"]() == UNSUPPORTED, over
    assert calls(L, p, c, ws=None)["attn"]() == INVALID and calls(L, p, c, ws=A + 64)["attn"]() == ALIGN


def test_workspace_sizes(L):
    c = pages()
    n = L.csa2_page_workspace_size(ctypes.byref(c))
    assert n % 256 == 0 and n >= 8 * (c.max_seqs + 1) + 4 * (3 * c.max_seqs + 3 * c.n_pages + 1)
    assert L.csa2_page_workspace_size(None) == 0
    assert L.csa2_paged_attn_workspace_size(ctypes.byref(params()), ctypes.byref(c), 0) == 0
    assert L.csa2_paged_attn_workspace_size(None, ctypes.byref(c), 4) == 0


def test_binding_refuses_tensors_the_pointers_would_not_stand_for():
    p = params(rope_dim=64)
    x, pos = torch.zeros(3, 2, 128, dtype=torch.bfloat16), torch.zeros(3, dtype=torch.int32)
    for bad in (x[0], x.half(), x.double()):
        with pytest.raises(api.Csa2Error, match="rope: x"):
            api.rope(p, bad, pos)
    with pytest.raises(api.Csa2Error, match="shape and type"):
        api.rope(p, x, pos, out=x.float())
    with pytest.raises(api.Csa2Error, match="contiguous"):
        api.rope(p, x.transpose(1, 2), pos)
    with pytest.raises(api.Csa2Error, match="CUDA"):
        api.rope(p, x, pos)
    pool = torch.zeros(1, 4, 16, 512, dtype=torch.bfloat16)
    table, ref = torch.full((2, 3), -1, dtype=torch.int32), torch.zeros(4, dtype=torch.int32)
    for k in (dict(pool=pool.float()), dict(pool=pool[0]), dict(pool=pool.transpose(1, 2)),
              dict(table=table.long()), dict(table=table.t()), dict(ref=ref.long()), dict(ref=ref[:3])):
        with pytest.raises(api.Csa2Error):
            api.PagedCache(p, **dict(dict(pool=pool, table=table, ref=ref), **k))
    with pytest.raises(api.Csa2Error, match="BF16 or E4M3"):
        api.PagedCache(api.default_params(), pool=pool, table=table, ref=ref)
    c = api.PagedCache(p, pool=pool, table=table, ref=ref)
    e4m3, j = params(kv_format=api.E4M3), torch.zeros(1, dtype=torch.int32)
    for call in (lambda: api.page_fork(e4m3, c, j, j, j), lambda: api.page_compact(e4m3, c),
                 lambda: api.page_write(e4m3, c, 0, torch.zeros(1, 512), j, j),
                 lambda: api.paged_attn(e4m3, c, 0, torch.zeros(1, 64, 512, dtype=torch.bfloat16), None, j, j,
                                        torch.zeros(1, 64, 512, dtype=torch.bfloat16), j)):
        with pytest.raises(api.Csa2Error, match="another format"):
            call()
    i = torch.zeros(2, dtype=torch.int32)
    q = torch.zeros(2, 64, 512, dtype=torch.bfloat16)
    for k in (dict(q=q.float()), dict(q=q[:, :, :256]), dict(q=q[:, :32]), dict(out=q.float()),
              dict(out=q[:, :32]), dict(sink=torch.zeros(63)), dict(sink=torch.zeros(64).double())):
        a = dict(dict(q=q, sink=None, out=torch.empty_like(q)), **k)
        with pytest.raises(api.Csa2Error):
            api.paged_attn(p, c, 0, a["q"], a["sink"], i, i, a["out"], i)
    for x in (torch.zeros(2, 512, dtype=torch.float16), torch.zeros(2, 256), torch.zeros(512, 2).t()):
        with pytest.raises(api.Csa2Error, match="page_write"):
            api.page_write(p, c, 0, x, i, i)
    for call in (lambda j: api.page_reserve(p, c, i, j, i), lambda j: api.page_release(p, c, i, j),
                 lambda j: api.page_fork(p, c, j, i, i), lambda j: api.page_write(p, c, 0, torch.zeros(2, 512), j, i),
                 lambda j: api.paged_attn(p, c, 0, q, None, j, i, torch.empty_like(q), i)):
        with pytest.raises(api.Csa2Error, match="CUDA"):  # nothing is enqueued for host tensors
            call(i)


def test_waits_of_the_attention_kernel_are_decided_by_the_warp():
    """A bounded wait can give up lane by lane. The roles go on with shuffles, votes and TMEM
    accesses of the whole warp, so a lane that left alone would leave the others waiting without a
    bound. By the source: every wait of a role votes, and none of a lane's own is left."""
    csrc = os.path.join(os.path.dirname(_lib.LIB_PATH), "csrc")
    code = {n: re.sub(r"//[^\n]*", "", open(os.path.join(csrc, n)).read()) for n in ("paged_attn.cu", "sm100.cuh")}
    waits = re.findall(r"\bmbar_(?:try_)?(?:wait|test)\w*(?=\()", code["paged_attn.cu"])
    # (a drain is the last thing a role does)
    assert set(waits) == {"mbar_wait_warp", "mbar_wait_either_warp", "mbar_wait_drain"}
    for name in ("mbar_wait_warp", "mbar_wait_either_warp"):
        body = code["sm100.cuh"].split(name + "(", 1)[1].split("\n}\n", 1)[0]
        tries = [line for line in body.split("\n") if "mbar_t" in line or "mbar_wait" in line]
        assert tries and all(re.search(r"__(all|ballot)_sync\(0xffffffffu", line) for line in tries), name
        returns = [line for line in body.split("\n") if "*abort" in line and "return" in line]
        assert returns and all("__any_sync(0xffffffffu" in line for line in returns), name


def test_import_with_a_torch_built_without_cuda(L):
    """Such a torch lacks the private calls of the fast path; the module imports, and what needs no
    device works."""
    code = """
import torch
for name in ("_cuda_getCurrentRawStream", "_cuda_getDevice"):
    if hasattr(torch._C, name):
        delattr(torch._C, name)
from csa2_compressed_sparse_02_gb300 import api
p = api.default_params(rope_dim=16)
try:
    api.rope(p, torch.zeros(2, 1, 16), torch.zeros(2, dtype=torch.int32))
except api.Csa2Error as e:
    assert "CUDA tensor" in str(e)
else:
    raise SystemExit("a host tensor was taken")
"""
    root = os.path.dirname(os.path.dirname(_lib.LIB_PATH))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr

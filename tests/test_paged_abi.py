"""Host-side checks of the paged K+V cache calls (no GPU): every refusal comes before any launch."""
import ctypes
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

from oracle import paged_oracle as P

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def S():
    from only_cache_exact_b200 import build
    build.build()
    from only_cache_exact_b200 import slim
    return slim


F = 1 << 20  # never dereferenced: the checks fail first


def cache(S, **kw):
    a = dict(kpages=F, vpages=F, kscale=F, vscale=F, table=F, num_pages=100, dtype=S.SLIM_E4M3, B=4, Hkv=8, dh=128,
             page=64, max_pages=20)
    a.update(kw)
    return ctypes.byref(S._PagedCacheC(*[a[f] for f, _ in S._PagedCacheC._fields_]))


BAD_CACHES = [
    (dict(kpages=None), "EINVAL"), (dict(vpages=None), "EINVAL"), (dict(table=None), "EINVAL"),
    (dict(kpages=F + 8), "EINVAL"), (dict(kscale=None), "EINVAL"), (dict(vscale=None), "EINVAL"),
    (dict(dtype=7), "EINVAL"), (dict(B=0), "EINVAL"), (dict(Hkv=0), "EINVAL"), (dict(Hkv=1025), "EINVAL"),
    (dict(page=0), "EINVAL"), (dict(max_pages=0), "EINVAL"), (dict(num_pages=0), "EINVAL"),
    (dict(num_pages=1 << 22), "EINVAL"), (dict(max_pages=1 << 25), "EINVAL"), (dict(num_pages=1 << 62), "EINVAL"),
    (dict(page=16, max_pages=(1 << 26) + 1, B=1), "EINVAL"), (dict(max_pages=1 << 21, B=300), "EINVAL"),
    (dict(dtype=0), "EUNSUPPORTED"), (dict(dh=96), "EUNSUPPORTED"), (dict(page=48), "EUNSUPPORTED"),
    (dict(page=256), "EUNSUPPORTED"), (dict(B=4097), "EUNSUPPORTED"),
]


def append(S, c=None, **kw):
    a = dict(q=F, qs=4096, k=F, ks=1024, v=F, vs=1024, cos=F, sin=F, rot=128, inter=0, n_pos=10, starts=F, lens=F,
             rows=7, max_new=0, Hq=32, q_out=F, status=F)
    a.update(kw)
    return S.raw_lib().slim_mha_paged_append(
        cache(S) if c is None else c, a["q"], a["qs"], a["k"], a["ks"], a["v"], a["vs"], a["cos"], a["sin"], a["rot"],
        a["inter"], a["n_pos"], a["starts"], a["lens"], a["rows"], a["max_new"], a["Hq"], a["q_out"], a["status"], None)


def gather(S, c=None, **kw):
    a = dict(starts=F, first=F, rows=7, max_new=0, k=F, v=F, status=F)
    a.update(kw)
    return S.raw_lib().slim_mha_paged_gather(cache(S) if c is None else c, a["starts"], a["first"], a["rows"],
                                             a["max_new"], a["k"], a["v"], a["status"], None)


def decode(S, c=None, **kw):
    a = dict(q=F, qs=4096, lens=F, extra=1, Hq=32, hint=0, out=F, ws=F, wsb=1 << 40, status=F)
    a.update(kw)
    return S.raw_lib().slim_mha_paged_decode(cache(S) if c is None else c, a["q"], a["qs"], a["lens"], a["extra"],
                                             a["Hq"], a["hint"], a["out"], a["ws"], a["wsb"], a["status"], None)


def prefill(S, c=None, **kw):
    a = dict(q=F, qs=4096, starts=F, lens=F, rows=7, max_new=0, Hq=32, hint=0, out=F, ws=F, wsb=1 << 40, status=F)
    a.update(kw)
    return S.raw_lib().slim_mha_paged_prefill(cache(S) if c is None else c, a["q"], a["qs"], a["starts"], a["lens"],
                                              a["rows"], a["max_new"], a["Hq"], a["hint"], a["out"], a["ws"], a["wsb"],
                                              a["status"], None)


@pytest.mark.parametrize("kw,code", BAD_CACHES)
@pytest.mark.parametrize("call", [append, gather, decode, prefill])
def test_cache_refusals(S, call, kw, code):
    assert call(S, cache(S, **kw)) == getattr(S, "SLIM_" + code)
    assert S.raw_lib().slim_mha_paged_decode_workspace_bytes(cache(S, **kw), 32) == 0


def test_null_cache(S):
    null = ctypes.POINTER(S._PagedCacheC)()
    for call in (append, gather, decode, prefill):
        assert call(S, null) == S.SLIM_EINVAL


@pytest.mark.parametrize("kw", [
    dict(k=None), dict(v=None), dict(starts=None), dict(lens=None), dict(status=None), dict(q_out=None),
    dict(q=None), dict(k=F + 2), dict(q_out=F + 4), dict(ks=1016), dict(vs=1028), dict(qs=4088), dict(rot=-16),
    dict(rot=8), dict(rot=144), dict(rot=0), dict(cos=None), dict(sin=None), dict(cos=None, sin=None),
    dict(cos=F + 4), dict(n_pos=0), dict(inter=2), dict(rows=-1), dict(max_new=-1), dict(Hq=0), dict(Hq=33),
    dict(rows=1 << 31), dict(starts=F + 2), dict(Hq=8200, qs=1 << 21), dict(qs=8192, q_out=F),
])
def test_append_refusals(S, kw):
    assert append(S, **kw) == S.SLIM_EINVAL


@pytest.mark.parametrize("kw", [dict(k=None), dict(v=None), dict(starts=None), dict(first=None), dict(status=None),
                                dict(k=F + 8), dict(v=F + 4), dict(rows=-5), dict(max_new=-1)])
def test_gather_refusals(S, kw):
    assert gather(S, **kw) == S.SLIM_EINVAL


@pytest.mark.parametrize("kw,code", [
    (dict(q=None), "EINVAL"), (dict(lens=None), "EINVAL"), (dict(out=None), "EINVAL"), (dict(status=None), "EINVAL"),
    (dict(q=F + 8), "EINVAL"), (dict(out=F + 2), "EINVAL"), (dict(qs=4000), "EINVAL"), (dict(qs=4100), "EINVAL"),
    (dict(extra=2), "EINVAL"), (dict(extra=-1), "EINVAL"), (dict(Hq=0), "EINVAL"), (dict(Hq=12), "EINVAL"),
    (dict(ws=None), "EWORKSPACE"), (dict(ws=F + 16), "EWORKSPACE"), (dict(wsb=100), "EWORKSPACE"),
])
def test_decode_refusals(S, kw, code):
    assert decode(S, **kw) == getattr(S, "SLIM_" + code)


@pytest.mark.parametrize("kw,code", [
    (dict(q=None), "EINVAL"), (dict(lens=None), "EINVAL"), (dict(starts=None), "EINVAL"), (dict(out=None), "EINVAL"),
    (dict(status=None), "EINVAL"), (dict(q=F + 8), "EINVAL"), (dict(out=F + 2), "EINVAL"), (dict(qs=4000), "EINVAL"),
    (dict(rows=-1), "EINVAL"), (dict(max_new=-2), "EINVAL"), (dict(Hq=12), "EINVAL"), (dict(rows=1 << 31), "EINVAL"),
    (dict(Hq=8 * 129, qs=1 << 20), "EUNSUPPORTED"), (dict(ws=None), "EWORKSPACE"), (dict(ws=F + 16), "EWORKSPACE"),
    (dict(wsb=100), "EWORKSPACE"),
])
def test_prefill_refusals(S, kw, code):
    # both ways to run it need scratch: 4 rows of 4 heads take the few-row kernel, and 20 rows of 4 sequences over a
    # capacity of 1280 rows have too few CTAs, so that keys are split
    for rows in (4, 20):
        assert S.raw_lib().slim_mha_paged_prefill_workspace_bytes(cache(S), 32, rows, 0, 0) > 100
    assert prefill(S, **kw) == getattr(S, "SLIM_" + code)


def test_prefill_workspace(S):
    size = S.raw_lib().slim_mha_paged_prefill_workspace_bytes
    assert size(cache(S), 32, 20, 0, 128) == 0      # short: one CTA walks all keys
    assert size(cache(S), 32, 8000, 0, 0) == 0      # many rows: CTAs enough
    assert size(cache(S), 32, 20, 0, 0) > 0         # long cache, few CTAs
    decode = S.raw_lib().slim_mha_paged_decode_workspace_bytes
    assert size(cache(S), 8, 7, 1, 0) == decode(cache(S), 8)  # one row of a key head: the same kernel
    assert size(cache(S), 31, 7, 0, 0) == 0 and size(cache(S), 32, 0, 0, 0) == 0
    assert size(cache(S, Hkv=1024), 9 * 1024, 20, 0, 0) == 0  # as the call refuses them
    assert prefill(S, cache(S, Hkv=1024), Hq=9 * 1024, qs=1 << 21) == S.SLIM_EINVAL
    assert size(cache(S), 32, 20, 0, 1 << 40) == size(cache(S), 32, 20, 0, 0)  # a hint past the capacity is the capacity


def test_nothing_to_do(S):
    assert append(S, rows=0, k=None, v=None, q=None, q_out=None) == S.SLIM_OK
    assert gather(S, rows=0, k=None, v=None) == S.SLIM_OK
    assert prefill(S, rows=0, q=None, out=None, ws=None) == S.SLIM_OK
    assert S.slim_last_launch_count() == 0


def test_workspace_sizes(S):
    L = S.raw_lib()
    one = L.slim_mha_paged_decode_workspace_bytes(cache(S), 32)
    assert one > 0
    assert L.slim_mha_paged_decode_workspace_bytes(cache(S), 128) >= one  # 16 heads a group: partials of 16
    assert L.slim_mha_paged_decode_workspace_bytes(cache(S), 31) == 0
    assert L.slim_mha_paged_decode_workspace_bytes(cache(S, B=4096), 32) >= one


def test_binding_refusals(S):
    """The binding names what is wrong before the library is called."""
    kp = torch.zeros(4, 2, 16, 64, dtype=torch.bfloat16)
    table = torch.zeros(2, 3, dtype=torch.int32)
    with pytest.raises(ValueError, match="kpages"):
        S.PagedKV(kp.float(), kp.float(), table)
    with pytest.raises(ValueError, match="kpages and vpages"):
        S.PagedKV(kp, kp[:2], table)
    with pytest.raises(ValueError, match="table"):
        S.PagedKV(kp, kp, table.long())
    with pytest.raises(ValueError, match="kscale"):
        S.PagedKV(kp, kp, table, torch.ones(4, 2), torch.ones(4, 2))
    with pytest.raises(ValueError, match="CUDA"):
        S.PagedKV(kp, kp, table)
    assert "page" in S.slim_strerror(S.SLIM_DEV_BADPAGE)


def test_oracle_grid():
    """The oracle's e4m3 rounding against the code table, and its scale rule at the borders."""
    t = P.e4m3_table()
    fin = np.unique(t[np.isfinite(t)])
    assert fin.max() == 448 and np.abs(fin[fin != 0]).min() == 2.0 ** -9
    x = np.concatenate([fin, (fin[1:] + fin[:-1]) / 2, np.linspace(-448, 448, 4001)])
    near = np.abs(fin[None] - x[:, None]).min(axis=1)
    y = P.round_e4m3(x)
    assert np.isin(y, fin).all() and np.allclose(np.abs(y - x), near, rtol=0, atol=1e-15)
    torch_y = torch.from_numpy(x).to(torch.float32).to(torch.float8_e4m3fn).to(torch.float64).numpy()
    assert np.array_equal(P.round_e4m3(x.astype(np.float32)), torch_y)
    assert P.needed_scale(448.0) == 1 and P.needed_scale(448.0001) == 2 and P.needed_scale(224.0) == 0.5
    assert P.needed_scale(0.0) == 2.0 ** -100 and P.needed_scale(3e38) == 2.0 ** 120


def test_import_without_private_torch_names():
    """The module loads where torch lacks the private names that the paged calls take their stream and device from (a
    build without CUDA, a later release), and then asks torch's public functions."""
    code = ("import torch\n"
            "for name in ('_cuda_getCurrentRawStream', '_cuda_getDevice'):\n"
            "    if hasattr(torch._C, name): delattr(torch._C, name)\n"
            "from only_cache_exact_b200 import slim\n"
            "class Stream: cuda_stream = 77\n"
            "torch.cuda.current_stream = lambda dev: Stream() if dev == 3 else None\n"
            "torch.cuda.current_device = lambda: 3\n"
            "got = []\n"
            "slim._paged_call(lambda *a: got.append(a) or 0, 'call', 3, None, 1, 2)\n"
            "assert got == [(1, 2, 77)], got\n")
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr

"""slim_mha_paged_decode against the float64 oracle.

Tolerance, element by element, with o the output, A = Σ p|V| and D the largest Σ_c |q_c K_tc|/sqrt(dh):
  output rounded to bf16           2^-8 |o|
  scores: dh products summed in fp32, then 3 roundings of factors and the base-2 exponential (2^-22):
          |δs| <= (dh + 8)·2^-24·D, and p, also through the sum in the denominator, moves by 2 δs
  probabilities: f16 halves (2^-11) for e4m3, two bf16 parts (2^-16) for bf16
  sums of p and p·V in fp32 and the joins of partials: 2^-16 A covers 2^8 of them
  f16 underflow of p and of the scaled query: 2^-24 of the largest term, in 2^-16 A as well
"""
import numpy as np
import pytest
import torch

from oracle import paged_oracle as P
from tests.paged_cases import PagedState, angles, f64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def S():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from only_cache_exact_b200 import slim
    return slim


def bound(kind, dh, o, A, D):
    ds = (dh + 8) * 2.0 ** -24 * D + 2.0 ** -22
    return 2.0 ** -8 * np.abs(o) + A * (2 * ds + (2.0 ** -11 if kind == "e4m3" else 2.0 ** -16) + 2.0 ** -16)


def check(st, q, out, lens, extra):
    for b, L in enumerate(lens):
        n = L + extra
        if n == 0:
            assert (out[b] == 0).all()
            continue
        K, V = (st.oracle[w].read(st.table_h[b], n) for w in (0, 1))
        o, A, D = P.attend(f64(q[b:b + 1]), K, V, [n - 1])
        err = np.abs(f64(out[b:b + 1]) - o)
        assert (err <= bound(st.kind, st.dh, o, A, D)).all(), (b, L, err.max())


HEADS = [(4, 4, 64), (20, 20, 64), (8, 1, 128), (14, 2, 64), (12, 4, 128), (9, 1, 64), (16, 1, 128), (34, 2, 64),
         (40, 8, 128), (33, 1, 128), (70, 1, 64)]


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("Hq,Hkv,dh", HEADS)
@pytest.mark.parametrize("page", [16, 64])
@pytest.mark.parametrize("t_hint", [1, 0])
def test_ragged(S, kind, Hq, Hkv, dh, page, t_hint):
    """Lengths of nothing, one, around tile and page borders and long ones; both ways to split the work (t_hint = 1
    takes one CTA per sequence and head group, 0 takes shares of the line for the larger ones)."""
    lens = [0, 1, 15, 16, 17, 63, 64, 65, 500, 1031]
    st = PagedState(S, kind, Hkv, dh, page, lens, lens, seed=11)
    q = st.rows([1] * st.B, Hq, 2.0)
    out = torch.full((st.B, Hq, dh), float("nan"), dtype=torch.bfloat16, device="cuda")
    ws = S.alloc_paged_decode_workspace(st.cache, Hq)
    ws.fill_(0xFF)
    S.slim_mha_paged_decode(st.cache, q, st.lens, out, ws, st.status, rows_extra=0, t_hint=t_hint)
    torch.cuda.synchronize()
    assert int(st.status.item()) == 0
    check(st, q, out, lens, 0)
    if min(lens) < max(lens):  # the same with one row that lens does not count
        lens1 = [max(0, x - 1) for x in lens]
        lens1[0] = 0
        st2 = torch.tensor(lens1[1:], dtype=torch.int32, device="cuda")
        cache = S.PagedKV(st.pages[0], st.pages[1], st.table[1:].contiguous(), st.scales[0], st.scales[1])
        out2 = torch.empty_like(out[1:])
        S.slim_mha_paged_decode(cache, q[1:], st2, out2, ws, st.status, rows_extra=1, t_hint=t_hint)
        torch.cuda.synchronize()
        assert torch.equal(out2, out[1:])


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("B,Hq,Hkv,dh,page,lo,hi", [(1, 4, 4, 64, 16, 9000, 9000), (1, 8, 1, 128, 128, 20000, 20000),
                                                    (300, 4, 2, 64, 16, 0, 90), (37, 8, 8, 128, 32, 100, 700),
                                                    (3, 64, 4, 128, 64, 2000, 4000), (4096, 2, 1, 64, 16, 0, 20),
                                                    (2, 8192, 1024, 64, 16, 30, 40), (1, 8192, 1, 128, 16, 100, 100)])
def test_split_shapes(S, kind, B, Hq, Hkv, dh, page, lo, hi):
    """One long sequence over all CTAs, many short ones in one CTA, and mixtures."""
    rng = np.random.default_rng(5)
    lens = rng.integers(lo, hi + 1, size=B)
    st = PagedState(S, kind, Hkv, dh, page, lens, lens, seed=12)
    q = st.rows([1] * B, Hq, 2.0)
    out = torch.full((B, Hq, dh), float("nan"), dtype=torch.bfloat16, device="cuda")
    ws = S.alloc_paged_decode_workspace(st.cache, Hq)
    ws.fill_(0xFF)
    S.slim_mha_paged_decode(st.cache, q, st.lens, out, ws, st.status, rows_extra=0)
    torch.cuda.synchronize()
    assert int(st.status.item()) == 0
    check(st, q, out, [int(x) for x in lens], 0)
    again = torch.empty_like(out)
    S.slim_mha_paged_decode(st.cache, q, st.lens, again, ws, st.status, rows_extra=0)
    assert torch.equal(out, again)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("t_hint", [1, 0])
def test_skipped_sequences(S, kind, t_hint):
    """Bad lengths and bad pages give zero rows and status bits; the others are right."""
    lens = [20, 40, 40, 40, 700, 33]
    st = PagedState(S, kind, 2, 64, 16, lens, lens, seed=13)
    cap = st.cache.cap
    table = st.table.clone()
    table[3, 1] = -7
    table[4, 30] = st.cache.num_pages
    dl = torch.tensor([-2, cap, cap + 5, 40, 700, 33], dtype=torch.int32, device="cuda")
    cache = S.PagedKV(st.pages[0], st.pages[1], table, st.scales[0], st.scales[1])
    q = st.rows([1] * 6, 6)
    ws = S.alloc_paged_decode_workspace(cache, 6)
    out = torch.full_like(q, 9.0)
    dl1 = dl.clone()
    dl1[3:] -= 1
    S.slim_mha_paged_decode(cache, q, dl1, out, ws, st.status, rows_extra=1, t_hint=t_hint)
    torch.cuda.synchronize()
    assert int(st.status.item()) == S.SLIM_DEV_BADLEN | S.SLIM_DEV_OVERFLOW | S.SLIM_DEV_BADPAGE
    assert (out[:5] == 0).all()
    K, V = (st.oracle[w].read(st.table_h[5], 33) for w in (0, 1))
    o, A, D = P.attend(f64(q[5:6]), K, V, [32])
    assert (np.abs(f64(out[5:6]) - o) <= bound(kind, 64, o, A, D)).all()


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("t_hint", [1, 0])
def test_large_scores_and_scales(S, kind, t_hint):
    """Scores far beyond the exponential's range, pages whose scales lie 2^40 apart, and one dominating key."""
    lens = [200, 64]
    st = PagedState(S, kind, 1, 64, 16, lens, lens, seed=14)
    pid = [int(x) for x in st.table_h[0, :13]]
    f = torch.ones(13)
    f[3], f[7] = 2.0 ** 20, 2.0 ** -20
    for i, p in enumerate(pid):
        if kind == "e4m3":
            st.scales[1][p] *= f[i].item()
            st.scales[0][p] *= 4.0
            st.oracle[1].scale[p] *= f[i].item()
        else:
            st.pages[1][p] *= f[i].item()
            st.pages[0][p] *= 4.0
        st.oracle[1].values[p] *= f[i].item()
        st.oracle[0].values[p] *= 4.0
    q = st.rows([1, 1], 3, 30.0)
    q[1, 1] = 0
    out = torch.empty_like(q)
    ws = S.alloc_paged_decode_workspace(st.cache, 3)
    S.slim_mha_paged_decode(st.cache, q, st.lens, out, ws, st.status, rows_extra=0, t_hint=t_hint)
    torch.cuda.synchronize()
    check(st, q, out, lens, 0)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_strided_query_shared_pages_capture(S, kind):
    """Queries as a slice of a projection's output, two sequences that read the same pages, a call on another stream
    and a captured one."""
    lens = [100, 90]
    st = PagedState(S, kind, 2, 128, 32, lens, [128, 128], seed=15)
    st.table[1] = st.table[0]
    st.table_h[1] = st.table_h[0]
    big = st.rows([1, 1], 12)
    q = big[:, 4:8]
    out = torch.empty(2, 4, 128, dtype=torch.bfloat16, device="cuda")
    ws = S.alloc_paged_decode_workspace(st.cache, 4)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    S.slim_mha_paged_decode(st.cache, q, st.lens, out, ws, st.status, rows_extra=0, stream=s)
    s.synchronize()
    check(st, q, out, lens, 0)
    want = out.clone()
    out.zero_()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        S.slim_mha_paged_decode(st.cache, q, st.lens, out, ws, st.status, rows_extra=0)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_steps_through_the_cache(S, kind):
    """Prompt rows appended, then steps of append and decode, as a server runs them: every step against the oracle."""
    Hq, Hkv, dh, page = 8, 2, 64, 16
    st = PagedState(S, kind, Hkv, dh, page, [0, 0, 0], [70, 40, 24], seed=16)
    prompts = [50, 0, 15]
    cos, sin = angles(st.cache.cap, dh)
    ws = S.alloc_paged_decode_workspace(st.cache, Hq)
    lens = [0, 0, 0]
    for step in range(9):
        n = prompts if step == 0 else [1, 1, 1]
        k, v, q = st.rows(n, Hkv), st.rows(n, Hkv), st.rows(n, Hq, 2.0)
        q_rot = torch.empty_like(q)
        S.slim_mha_paged_append(st.cache, k, v, st.starts(n), st.lens, st.status, q=q, q_out=q_rot, cos=cos, sin=sin,
                                max_new=max(n))
        if step:
            out = torch.empty_like(q)
            S.slim_mha_paged_decode(st.cache, q_rot, st.lens, out, ws, st.status, rows_extra=1)
        torch.cuda.synchronize()
        for w in (0, 1):  # the oracle attends over what the device stores
            st.oracle[w].values = np.nan_to_num(st.values(w), nan=0.0)
        if step:
            check(st, q_rot, out, lens, 1)
        lens = [a + b for a, b in zip(lens, n)]
        st.lens += torch.tensor(n, dtype=torch.int32, device="cuda")
    assert int(st.status.item()) == 0 and st.lens.tolist() == lens


@pytest.mark.parametrize("which", [0, 1])
@pytest.mark.parametrize("dh,Hq,Hkv,page", [(64, 4, 4, 16), (128, 8, 1, 16), (64, 20, 1, 64), (128, 64, 16, 128)])
@pytest.mark.parametrize("at", [0, 2560, 4992])
def test_poisoned_page_in_parts(S, which, dh, Hq, Hkv, page, at):
    """A page whose scale is NaN, in the first, a middle or (alone, for small pages) the last warp's share of a split
    sequence: NaN where it is attended, and the other sequence as it was."""
    lens = [at + 5 if at == 4992 else 4992, 300]
    st = PagedState(S, "e4m3", Hkv, dh, page, lens, [5000, 300], seed=17)
    q = st.rows([1, 1], Hq)
    ws = S.alloc_paged_decode_workspace(st.cache, Hq)
    x, ok = st.rows([1], Hkv), st.rows([1], Hkv)
    x[0, :, 5] = float("-inf")
    starts = torch.tensor([0, 1, 1], dtype=torch.int32, device="cuda")
    S.slim_mha_paged_append(st.cache, *((x, ok) if which == 0 else (ok, x)), starts,
                            torch.tensor([at, 300], dtype=torch.int32, device="cuda"), st.status)
    out = torch.full_like(q, 7.0)
    S.slim_mha_paged_decode(st.cache, q, st.lens, out, ws, st.status, rows_extra=0)
    assert S.slim_last_launch_count() == 2
    torch.cuda.synchronize()
    assert int(st.status.item()) == 0
    assert torch.isnan(out[0]).all() and torch.isfinite(out[1]).all()
    K, V = (st.oracle[w].read(st.table_h[1], 300) for w in (0, 1))
    o, A, D = P.attend(f64(q[1:]), K, V, [299])
    assert (np.abs(f64(out[1:]) - o) <= bound("e4m3", dh, o, A, D)).all()
    if at:
        lens2 = torch.tensor([at, 300], dtype=torch.int32, device="cuda")
        S.slim_mha_paged_decode(st.cache, q, lens2, out, ws, st.status, rows_extra=0)
        torch.cuda.synchronize()
        check(st, q, out, [at, 300], 0)

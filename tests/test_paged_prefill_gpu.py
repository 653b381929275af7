"""slim_mha_paged_prefill against the float64 oracle.

Tolerance, element by element, with o the output, A = Σ p|V| and D the largest Σ_c |q_c K_tc|/sqrt(dh):
  output rounded to bf16           2^-8 |o|
  scores: dh products summed in fp32, then roundings of the factors and the base-2 exponential (2^-22):
          |δs| <= (dh + 8)·2^-24·D, and p, also through the sum in the denominator, moves by 2 δs
  probabilities rounded for the MMA: 2^-8 for bf16 values, 2^-11 (f16) for e4m3
  sums in fp32, joins of splits, f16 underflow: 2^-16 A
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
    return 2.0 ** -8 * np.abs(o) + A * (2 * ds + (2.0 ** -11 if kind == "e4m3" else 2.0 ** -8) + 2.0 ** -16)


def run(S, st, q, n, cached, max_new=0, t_hint=0, first=0, out=None, lens=None):
    Hq = q.shape[1]
    out = torch.full(q.shape, 7.0, dtype=torch.bfloat16, device="cuda") if out is None else out
    ws = S.alloc_paged_prefill_workspace(st.cache, Hq, q.shape[0], max_new, t_hint)
    ws.fill_(0xFF)
    S.slim_mha_paged_prefill(st.cache, q, st.starts(n, first), st.lens if lens is None else lens, out, ws, st.status,
                             max_new=max_new, t_hint=t_hint)
    torch.cuda.synchronize()
    return out


def check(st, q, out, n, cached, first=0):
    r = first
    for b, (a, k) in enumerate(zip(cached, n)):
        if k:
            K, V = (st.oracle[w].read(st.table_h[b], a + k) for w in (0, 1))
            o, A, D = P.attend(f64(q[r:r + k]), K, V, [a + j for j in range(k)])
            err = np.abs(f64(out[r:r + k]) - o)
            lim = bound(st.kind, st.dh, o, A, D)
            assert (err <= lim).all(), (b, a, k, (err / lim).max(), np.argwhere(err > lim)[0].tolist())
        r += k


CASES = [
    # Hq, Hkv, dh, page, cached, new
    (4, 4, 64, 16, [0], [1]),
    (4, 4, 64, 16, [0, 0, 0], [16, 130, 1]),
    (2, 2, 128, 64, [0, 63, 64], [129, 65, 64]),
    (6, 2, 64, 32, [100, 0, 31, 5], [3, 85, 0, 200]),       # 42 queries a tile, rows left over
    (7, 1, 128, 128, [300, 1], [40, 128]),
    (16, 1, 128, 16, [0, 511, 512], [9, 1, 17]),
    (64, 1, 64, 64, [700], [5]),                            # 2 queries a tile
    (128, 1, 128, 32, [33, 0], [2, 3]),                     # 1 query a tile
    (5, 5, 64, 128, [127, 128, 129], [1, 1, 1]),
    (3, 1, 128, 16, [0], [700]),
]


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("Hq,Hkv,dh,page,cached,new", CASES)
@pytest.mark.parametrize("t_hint", [1, 0])
def test_ragged(S, kind, Hq, Hkv, dh, page, cached, new, t_hint):
    """Odd sizes, grouped heads and chunks; t_hint = 1 keeps each tile's keys in one CTA, 0 may split them."""
    st = PagedState(S, kind, Hkv, dh, page, [a + n for a, n in zip(cached, new)], [a + n for a, n in zip(cached, new)],
                    seed=21)
    st.lens = torch.tensor(cached, dtype=torch.int32, device="cuda")
    big = st.rows(new, Hq + 2, 2.0)  # queries as a slice: rows lie apart
    pad = torch.zeros(3, Hq + 2, dh, dtype=torch.bfloat16, device="cuda")
    q = torch.cat([pad[:1], big, pad])[:, 1:1 + Hq]
    out = run(S, st, q, new, cached, max_new=max(new) if t_hint else 0, t_hint=t_hint, first=1)
    assert int(st.status.item()) == 0
    total = sum(new)
    assert (out[0] == 7).all() and (out[1 + total:] == 7).all()  # rows of no sequence stay as they were
    check(st, q, out, new, cached, first=1)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("dh,page,G", [(64, 16, 1), (128, 64, 4), (128, 128, 8)])
def test_long_cache_few_rows(S, kind, dh, page, G):
    """Keys split over many CTAs and joined, among them splits that a short sequence has nothing in."""
    cached, new = [5000, 3, 2047], [3, 2, 1]
    st = PagedState(S, kind, 1, dh, page, [a + n for a, n in zip(cached, new)], [a + n for a, n in zip(cached, new)],
                    seed=22)
    st.lens = torch.tensor(cached, dtype=torch.int32, device="cuda")
    q = st.rows(new, G, 2.0)
    out = run(S, st, q, new, cached, max_new=3)
    assert S.slim_last_launch_count() == 2 and int(st.status.item()) == 0
    check(st, q, out, new, cached)
    assert torch.equal(out, run(S, st, q, new, cached, max_new=3))
    one = run(S, st, q, new, cached, max_new=3, t_hint=1)  # unsplit
    assert S.slim_last_launch_count() == 1
    check(st, q, one, new, cached)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("dh,page,G", [(64, 16, 2), (128, 64, 4), (128, 128, 8)])
def test_long_cache_short_chunks(S, kind, dh, page, G):
    """More rows than the few-row kernel takes, keys split over CTAs and joined, among them splits that a short
    sequence has nothing in."""
    cached, new = [5000, 3, 2047], [21, 33, 1]
    total = [a + n for a, n in zip(cached, new)]
    st = PagedState(S, kind, 1, dh, page, total, total, seed=30)
    st.lens = torch.tensor(cached, dtype=torch.int32, device="cuda")
    q = st.rows(new, G, 2.0)
    out = run(S, st, q, new, cached, max_new=33)
    assert S.slim_last_launch_count() == 2 and int(st.status.item()) == 0
    check(st, q, out, new, cached)
    assert torch.equal(out, run(S, st, q, new, cached, max_new=33))
    one = run(S, st, q, new, cached, max_new=33, t_hint=1)  # unsplit
    assert S.slim_last_launch_count() == 1
    check(st, q, one, new, cached)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("dh,page,G", [(64, 16, 4), (128, 64, 4), (128, 128, 8), (128, 32, 1), (64, 64, 128)])
@pytest.mark.parametrize("t_hint", [0, 900, 300])
def test_one_row_tile(S, kind, dh, page, G, t_hint):
    """No sequence has more queries than one row tile holds: over e4m3 two parts of its keys run side by side in a
    CTA, with and without a split over CTAs, among them parts and splits that have no key tile."""
    q_tile = 128 // G
    cached = [5000, 3, 2047, 0, 640, 255, 60]
    new = [q_tile, min(5, q_tile), 1, q_tile, (q_tile + 1) // 2, 1, min(6, q_tile)]
    total = [a + n for a, n in zip(cached, new)]
    st = PagedState(S, kind, 2, dh, page, total, total, seed=34)
    st.lens = torch.tensor(cached, dtype=torch.int32, device="cuda")
    q = st.rows(new, 2 * G, 2.0)
    out = run(S, st, q, new, cached, max_new=q_tile, t_hint=t_hint)
    assert S.slim_last_launch_count() == (1 if t_hint == 300 else 2) and int(st.status.item()) == 0
    check(st, q, out, new, cached)
    assert torch.equal(out, run(S, st, q, new, cached, max_new=q_tile, t_hint=t_hint))


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("t_hint", [0, 900])
def test_one_row_tile_skipped(S, kind, t_hint):
    """The same with bad lengths and with pages outside the pool, in a key tile of either part."""
    cached, new = [3, 9, 600, 700, 640], [10, 10, 16, 10, 7]
    total = [a + n for a, n in zip(cached, new)]
    st = PagedState(S, kind, 2, 128, 16, total, total, seed=35)
    cap = st.cache.cap
    st.table[2, 38] = -1       # positions 608..623
    st.table[3, 7] = 1 << 30   # positions 112..127, in the first key tile
    st.table[4, 10] = -5       # positions 160..175, in the second
    lens = torch.tensor([-1, cap - 2, 600, 700, 640], dtype=torch.int32, device="cuda")
    q = st.rows(new, 8)
    out = run(S, st, q, new, cached, max_new=16, t_hint=t_hint, lens=lens)
    assert int(st.status.item()) == S.SLIM_DEV_BADLEN | S.SLIM_DEV_OVERFLOW | S.SLIM_DEV_BADPAGE
    assert (out[:20] == 0).all() and (out[28:] == 0).all()
    K, V = (st.oracle[w].read(st.table_h[2], 608) for w in (0, 1))
    o, A, D = P.attend(f64(q[20:28]), K, V, [600 + j for j in range(8)])
    assert (np.abs(f64(out[20:28]) - o) <= bound(kind, 128, o, A, D)).all()


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("Hq,Hkv,dh,page,new", [
    (3, 3, 64, 16, [5, 0, 8, 1, 2]), (6, 3, 128, 32, [4, 1, 0, 3, 2]), (4, 2, 64, 64, [8, 7, 1, 5, 0]),
    (4, 1, 128, 128, [4, 4, 4, 3, 1]), (8, 1, 64, 32, [1, 4, 3, 2, 4]), (32, 1, 128, 16, [1, 1, 0, 1, 1]),
    (5, 1, 128, 64, [6, 1, 2, 0, 5]), (2, 2, 64, 128, [32, 17, 16, 1, 0])])
@pytest.mark.parametrize("t_hint", [1, 0])
def test_few_rows(S, kind, Hq, Hkv, dh, page, new, t_hint):
    """Up to 32 rows (queries and heads) of a key head: each row has its own last key, among others inside a 16-key
    tile and on either side of its border."""
    cached = [0, 14, 700, 1500, 31]
    total = [a + n for a, n in zip(cached, new)]
    st = PagedState(S, kind, Hkv, dh, page, total, total, seed=31)
    st.lens = torch.tensor(cached, dtype=torch.int32, device="cuda")
    q = st.rows(new, Hq, 2.0)
    out = run(S, st, q, new, cached, max_new=max(new), t_hint=t_hint)
    assert int(st.status.item()) == 0
    check(st, q, out, new, cached)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("t_hint", [1, 0])
def test_few_rows_skipped(S, kind, t_hint):
    """Bad lengths and pages with few rows: zeros for the sequence, or for the rows that reach the page."""
    cached, new = [3, 9, 45, 700], [4, 4, 5, 2]
    total = [a + n for a, n in zip(cached, new)]
    st = PagedState(S, kind, 2, 64, 16, total, total, seed=32)
    cap = st.cache.cap
    st.table[2, 3] = -1      # positions 48..63
    st.table[3, 7] = 1 << 30
    lens = torch.tensor([-1, cap - 2, 45, 700], dtype=torch.int32, device="cuda")
    q = st.rows(new, 4)
    out = run(S, st, q, new, cached, max_new=5, t_hint=t_hint, lens=lens)
    assert int(st.status.item()) == S.SLIM_DEV_BADLEN | S.SLIM_DEV_OVERFLOW | S.SLIM_DEV_BADPAGE
    assert (out[:8] == 0).all() and (out[11:] == 0).all()
    K, V = (st.oracle[w].read(st.table_h[2], 48) for w in (0, 1))
    o, A, D = P.attend(f64(q[8:11]), K, V, [45, 46, 47])
    assert (np.abs(f64(out[8:11]) - o) <= bound(kind, 64, o, A, D)).all()


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_agrees_with_decode(S, kind):
    """One new row per sequence: the two forms of the attention agree within their tolerances."""
    cached = [0, 100, 1500]
    st = PagedState(S, kind, 4, 128, 32, [c + 1 for c in cached], [c + 1 for c in cached], seed=23)
    st.lens = torch.tensor(cached, dtype=torch.int32, device="cuda")
    q = st.rows([1, 1, 1], 8, 2.0)
    a = run(S, st, q, [1, 1, 1], cached, max_new=1)
    b = torch.empty_like(a)
    S.slim_mha_paged_decode(st.cache, q, st.lens, b, S.alloc_paged_decode_workspace(st.cache, 8), st.status)
    torch.cuda.synchronize()
    check(st, q, a, [1, 1, 1], cached)
    check(st, q, b, [1, 1, 1], cached)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("t_hint", [1, 0])
def test_skipped_sequences(S, kind, t_hint):
    """Bad lengths give zero rows; a page outside the pool gives zeros to the rows that reach it and only to them."""
    cached, new = [3, 9, 40, 700], [4, 4, 30, 6]
    st = PagedState(S, kind, 2, 64, 16, [a + n for a, n in zip(cached, new)], [a + n for a, n in zip(cached, new)],
                    seed=24)
    cap = st.cache.cap
    st.table[2, 3] = -1      # positions 48..63
    st.table[3, 7] = 1 << 30
    lens = torch.tensor([-1, cap - 2, 40, 700], dtype=torch.int32, device="cuda")
    q = st.rows(new, 4)
    out = run(S, st, q, new, cached, max_new=30, t_hint=t_hint, lens=lens)
    assert int(st.status.item()) == S.SLIM_DEV_BADLEN | S.SLIM_DEV_OVERFLOW | S.SLIM_DEV_BADPAGE
    assert (out[:8] == 0).all() and (out[16:] == 0).all()
    K, V = (st.oracle[w].read(st.table_h[2], 48) for w in (0, 1))
    o, A, D = P.attend(f64(q[8:16]), K, V, list(range(40, 48)))
    assert (np.abs(f64(out[8:16]) - o) <= bound(kind, 64, o, A, D)).all()
    st.status.zero_()
    bad = torch.tensor([0, 4, 2, 38, 50], dtype=torch.int32, device="cuda")  # descending, then past the rows
    ws = S.alloc_paged_prefill_workspace(st.cache, 4, q.shape[0], 44, t_hint)
    S.slim_mha_paged_prefill(st.cache, q, bad, st.lens, out, ws, st.status, max_new=44, t_hint=t_hint)
    torch.cuda.synchronize()
    assert int(st.status.item()) & S.SLIM_DEV_BADLEN


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("t_hint", [1, 0])
def test_large_scores_and_scales(S, kind, t_hint):
    """Scores far beyond the exponential's range, growing maxima (late keys dominate), pages whose value scales lie
    2^40 apart, zero queries."""
    st = PagedState(S, kind, 1, 64, 16, [600], [600], seed=25)
    pid = [int(x) for x in st.table_h[0, :38]]
    for i, p in enumerate(pid):
        fk = 2.0 ** (i // 6)
        fv = 2.0 ** 20 if i == 9 else 2.0 ** -20 if i == 20 else 1.0
        for w, f in ((0, fk), (1, fv)):
            if kind == "e4m3":
                st.scales[w][p] *= f
                st.oracle[w].scale[p] *= f
            else:
                st.pages[w][p] *= f
            st.oracle[w].values[p] *= f
    n, cached = [300], [300]
    st.lens = torch.tensor(cached, dtype=torch.int32, device="cuda")
    q = st.rows(n, 3, 10.0)
    q[5, 1] = 0
    out = run(S, st, q, n, cached, max_new=300, t_hint=t_hint)
    check(st, q, out, n, cached)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("new", [5, 200])
@pytest.mark.parametrize("t_hint", [1, 0])
def test_zero_queries_small_keys(S, kind, new, t_hint):
    """Padding rows of zeros beside ordinary ones, over keys so small that the factor of a zero row's scores leaves
    fp32's range: equal weights, also where the causal mask ends inside a tile."""
    st = PagedState(S, kind, 1, 64, 16, [600], [600], seed=30)
    for w in (st.scales if kind == "e4m3" else st.pages)[:1]:
        w *= 2.0 ** -60
    st.oracle[0].values = st.oracle[0].values * 2.0 ** -60
    n, cached = [new], [600 - new]
    st.lens = torch.tensor(cached, dtype=torch.int32, device="cuda")
    q = st.rows(n, 3)
    q[: new // 2] = 0
    out = run(S, st, q, n, cached, max_new=new, t_hint=t_hint)
    check(st, q, out, n, cached)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_chunks_then_tokens(S, kind):
    """A prompt in chunks, each appended and attended, then single tokens: a model layer's use of the cache, captured
    per chunk size and on a stream of its own."""
    Hq, Hkv, dh, page = 8, 2, 64, 16
    st = PagedState(S, kind, Hkv, dh, page, [0, 0], [160, 120], seed=26)
    cos, sin = angles(st.cache.cap, dh)
    cached = [0, 0]
    ws1 = S.alloc_paged_decode_workspace(st.cache, Hq)
    s = torch.cuda.Stream()
    for n in ([100, 37], [20, 60], [1, 1], [3, 0], [1, 1]):
        k, v, q = st.rows(n, Hkv), st.rows(n, Hkv), st.rows(n, Hq, 2.0)
        qr, out = torch.empty_like(q), torch.empty_like(q)
        starts = st.starts(n)
        ws = S.alloc_paged_prefill_workspace(st.cache, Hq, sum(n), max(n))
        s.wait_stream(torch.cuda.current_stream())
        S.slim_mha_paged_append(st.cache, k, v, starts, st.lens, st.status, q=q, q_out=qr, cos=cos, sin=sin,
                                max_new=max(n), stream=s)
        if n == [1, 1]:
            S.slim_mha_paged_decode(st.cache, qr, st.lens, out, ws1, st.status, stream=s)
        else:
            S.slim_mha_paged_prefill(st.cache, qr, starts, st.lens, out, ws, st.status, max_new=max(n), stream=s)
        s.synchronize()
        for w in (0, 1):
            st.oracle[w].values = np.nan_to_num(st.values(w), nan=0.0)
        check(st, qr, out, n, cached)
        cached = [a + b for a, b in zip(cached, n)]
        st.lens += torch.tensor(n, dtype=torch.int32, device="cuda")
    assert int(st.status.item()) == 0


@pytest.mark.parametrize("which", [0, 1])
@pytest.mark.parametrize("t_hint", [1, 0])
def test_poisoned_page(S, which, t_hint):
    """A page whose scale is NaN makes the outputs that attend a row of it NaN, in both forms, and no other."""
    st = PagedState(S, "e4m3", 1, 64, 16, [700], [700], seed=29)
    st.lens = torch.tensor([600], dtype=torch.int32, device="cuda")
    x = st.rows([20], 1)
    x[16] = float("inf")  # row 656
    ok = st.rows([20], 1)
    k, v = (x, ok) if which == 0 else (ok, x)
    S.slim_mha_paged_append(st.cache, k, v, st.starts([20]), st.lens + 40, st.status)
    torch.cuda.synchronize()
    for w in (0, 1):
        st.oracle[w].values = np.nan_to_num(st.values(w), nan=0.0)
    q = st.rows([100], 4)
    out = run(S, st, q, [100], [600], max_new=100, t_hint=t_hint)
    # row 656 begins a page: rows 656..671 share its scale
    assert torch.isnan(out[56:]).all() and torch.isfinite(out[:56]).all()
    check(st, q[:56], out[:56], [56], [600])
    for n, bad in ((655, False), (656, True)):
        lens = torch.tensor([n], dtype=torch.int32, device="cuda")
        o = torch.zeros(1, 4, 64, dtype=torch.bfloat16, device="cuda")
        S.slim_mha_paged_decode(st.cache, q[:1], lens, o, S.alloc_paged_decode_workspace(st.cache, 4), st.status,
                                t_hint=t_hint)
        assert torch.isnan(o).all().item() == bad and torch.isfinite(o).all().item() != bad
    assert int(st.status.item()) == 0


def test_capture(S):
    st = PagedState(S, "e4m3", 2, 128, 32, [400, 150], [400, 150], seed=27)
    n, cached = [100, 1], [300, 149]
    st.lens = torch.tensor(cached, dtype=torch.int32, device="cuda")
    q = st.rows(n, 4, 2.0)
    want = run(S, st, q, n, cached, max_new=100)
    out = torch.zeros_like(want)
    ws = S.alloc_paged_prefill_workspace(st.cache, 4, 101, 100)
    starts = st.starts(n)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        S.slim_mha_paged_prefill(st.cache, q, starts, st.lens, out, ws, st.status, max_new=100)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)


def test_no_rows(S):
    st = PagedState(S, "bf16", 2, 64, 16, [9, 0], [40, 40], seed=28)
    e = torch.empty(0, 4, 64, dtype=torch.bfloat16, device="cuda")
    S.slim_mha_paged_prefill(st.cache, e, st.starts([0, 0]), st.lens, e,
                             torch.empty(0, dtype=torch.uint8, device="cuda"), st.status)
    assert S.slim_last_launch_count() == 0


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_offsets_past_32_bits(S, kind):
    """Both attentions over pools of more than 2^32 bytes whose used pages lie at the far end: as over a copy of those
    pages in small pools, bit by bit."""
    Hkv, Hq, dh, page = 64, 128, 128, 128
    per = Hkv * dh * page * (2 if kind == "bf16" else 1)
    num = (1 << 32) // per + 4
    dt = torch.bfloat16 if kind == "bf16" else torch.float8_e4m3fn
    gen = torch.Generator(device="cuda").manual_seed(3)
    far = [num - 1, num - 3, num - 2, num - 4]
    big = [torch.empty(num, Hkv, page, dh, dtype=dt, device="cuda") for _ in range(2)]
    small = [torch.randn(4, Hkv, page, dh, device="cuda", generator=gen).to(dt) for _ in range(2)]
    for w in (0, 1):
        for i, p in enumerate(far):
            big[w][p] = small[w][i]
    sc = [[None, None], [None, None]]
    if kind == "e4m3":
        sc = [[torch.ones(n, Hkv, device="cuda") for _ in range(2)] for n in (num, 4)]
    tables = [torch.tensor([f[:3], f[3:] * 3], dtype=torch.int32, device="cuda") for f in (far, [0, 1, 2, 3])]
    caches = [S.PagedKV(p[0], p[1], t, s[0], s[1]) for p, t, s in zip((big, small), tables, sc)]
    lens = torch.tensor([330, 100], dtype=torch.int32, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    n = [40, 25]
    q = torch.randn(sum(n), Hq, dh, device="cuda", generator=gen).bfloat16()
    starts = torch.tensor([0, 40, 65], dtype=torch.int32, device="cuda")
    got = []
    for c in caches:
        o, d = torch.zeros_like(q), torch.zeros_like(q[:2])
        S.slim_mha_paged_prefill(c, q, starts, lens, o, S.alloc_paged_prefill_workspace(c, Hq, 65, 40), status, max_new=40)
        S.slim_mha_paged_decode(c, q[:2], lens, d, S.alloc_paged_decode_workspace(c, Hq), status, rows_extra=0)
        got.append((o, d))
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    for a, b in zip(*got):
        assert torch.equal(a, b) and torch.isfinite(a).all() and (a != 0).any()


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("B,Hq,Hkv", [(4096, 2, 1), (4096, 40, 1), (2, 8192, 1024), (3, 8192, 64)])
def test_most_sequences_and_heads(S, kind, B, Hq, Hkv):
    """The largest batch and the most heads, in the few-row form and on row tiles."""
    rng = np.random.default_rng(6)
    cached, new = [int(x) for x in rng.integers(0, 24, size=B)], [int(x) for x in rng.integers(0, 4, size=B)]
    new[-1] = 3
    total = [a + n for a, n in zip(cached, new)]
    st = PagedState(S, kind, Hkv, 64, 16, total, total, seed=36)
    st.lens = torch.tensor(cached, dtype=torch.int32, device="cuda")
    q = st.rows(new, Hq, 2.0)
    out = run(S, st, q, new, cached, max_new=3)
    assert int(st.status.item()) == 0
    check(st, q, out, new, cached)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_calls_side_by_side(S, kind):
    """A prompt chunk, single tokens and a read-back of one cache on three streams at once, each with its own
    workspace, over and over: the results of the calls one after another."""
    st = PagedState(S, kind, 2, 128, 32, [900, 1200], [900, 1200], seed=31)
    n = [150, 70]
    st.lens = torch.tensor([750, 1130], dtype=torch.int32, device="cuda")
    q, q1, starts, first = st.rows(n, 8), st.rows([1, 1], 8), st.starts(n), st.lens.clone()
    ws, ws1 = S.alloc_paged_prefill_workspace(st.cache, 8, 220, 150), S.alloc_paged_decode_workspace(st.cache, 8)

    def outs():
        return [torch.zeros_like(q), torch.zeros_like(q1)] + [torch.zeros_like(q[:, :2]).contiguous() for _ in range(2)]

    def calls(o, streams):
        S.slim_mha_paged_prefill(st.cache, q, starts, st.lens, o[0], ws, st.status, max_new=150, stream=streams[0])
        S.slim_mha_paged_decode(st.cache, q1, st.lens, o[1], ws1, st.status, rows_extra=0, stream=streams[1])
        S.slim_mha_paged_gather(st.cache, first, starts, o[2], o[3], st.status, max_new=150, stream=streams[2])

    want = outs()
    calls(want, [None] * 3)
    streams = [torch.cuda.Stream() for _ in range(3)]
    rounds = [outs() for _ in range(6)]
    torch.cuda.synchronize()
    for o in rounds:
        calls(o, streams)
    torch.cuda.synchronize()
    for o in rounds:
        for a, b in zip(o, want):
            assert torch.equal(a, b)
    check(st, q, want[0], n, [750, 1130])
    assert int(st.status.item()) == 0


def poison(S, st, which, at):
    """An infinite key (which = 0) or value at row `at` of sequence 0, which begins a page."""
    assert at % st.page == 0
    x, ok = st.rows([1], st.Hkv), st.rows([1], st.Hkv)
    x[0, :, 5] = float("inf")
    lens = torch.full_like(st.lens, at)
    S.slim_mha_paged_append(st.cache, *((x, ok) if which == 0 else (ok, x)), st.starts([1]), lens, st.status)


@pytest.mark.parametrize("which", [0, 1])
@pytest.mark.parametrize("dh,page,cached,new,at,cap,t_hint", [
    (64, 16, 120, 28, 128, 4096, 0),      # the page begins the second key tile, which is a part of its own
    (128, 16, 120, 20, 128, 4096, 0),
    (64, 64, 120, 28, 128, 4096, 800),    # two ranges in one CTA: the second is that key tile
    (64, 128, 600, 28, 256, 4096, 0),     # a whole key tile among the cached rows
    (64, 16, 100, 60, 128, 4096, 0),      # more queries than a row tile: parts of CTAs alone
    (128, 128, 500, 60, 512, 4096, 0),
    (128, 128, 2048, 40, 128, 32768, 0),
    (64, 128, 0, 30, 0, 4096, 0),         # nothing but the page
])
def test_poisoned_page_in_parts(S, which, dh, page, cached, new, at, cap, t_hint):
    """Keys in parts that are joined, one of which holds nothing but the poisoned page for some rows: every output
    that attends the page is NaN, the others are not touched."""
    st = PagedState(S, "e4m3", 1, dh, page, [cached + new], [cap - page], seed=40)
    st.lens = torch.tensor([cached], dtype=torch.int32, device="cuda")
    poison(S, st, which, at)
    q = st.rows([new], 4)
    out = run(S, st, q, [new], [cached], max_new=new, t_hint=t_hint)
    assert S.slim_last_launch_count() == 2 and int(st.status.item()) == 0
    before = max(0, min(new, at - cached))
    assert torch.isnan(out[before:]).all() and torch.isfinite(out[:before]).all()
    check(st, q[:before], out[:before], [before], [cached])


@pytest.mark.parametrize("which", [0, 1])
@pytest.mark.parametrize("dh,G,new", [(64, 1, 3), (64, 8, 3), (128, 4, 3)])
def test_poisoned_page_few_rows(S, which, dh, G, new):
    """The form for a few rows with the page alone in the last warp's share: only the row that attends it."""
    cached = 4993 - new
    st = PagedState(S, "e4m3", 1, dh, 16, [4993], [5000], seed=41)
    st.lens = torch.tensor([cached], dtype=torch.int32, device="cuda")
    poison(S, st, which, 4992)
    q = st.rows([new], G)
    out = run(S, st, q, [new], [cached], max_new=new)
    assert S.slim_last_launch_count() == 2 and int(st.status.item()) == 0
    assert torch.isnan(out[new - 1:]).all() and torch.isfinite(out[:new - 1]).all()
    check(st, q[:new - 1], out[:new - 1], [new - 1], [cached])


@pytest.mark.parametrize("dh,page,G,new", [(64, 16, 4, 200), (128, 32, 4, 70), (128, 128, 2, 300), (64, 64, 8, 16),
                                           (128, 16, 8, 16), (64, 128, 4, 31)])
@pytest.mark.parametrize("t_hint", [1, 0])
def test_scales_of_many_pages(S, dh, page, G, new, t_hint):
    """Every page has scales of its own over many key tiles, so that each tile's scales have to be that tile's: for
    whole chunks, for one row tile (two key ranges), and split over CTAs."""
    total = 3300
    st = PagedState(S, "e4m3", 1, dh, page, [total], [total], seed=42)
    for w in (0, 1):
        f = np.exp2(st.rng.integers(-3, 4, size=(st.cache.num_pages, 1)))
        st.scales[w].mul_(torch.from_numpy(f).to(torch.float32).cuda())
        st.oracle[w].scale *= f
        st.oracle[w].values *= f[:, :, None, None]
    n, cached = [new], [total - new]
    st.lens = torch.tensor(cached, dtype=torch.int32, device="cuda")
    q = st.rows(n, G)
    want = run(S, st, q, n, cached, max_new=new, t_hint=t_hint)
    check(st, q, want, n, cached)
    for _ in range(20):
        assert torch.equal(run(S, st, q, n, cached, max_new=new, t_hint=t_hint), want)
    assert int(st.status.item()) == 0


@pytest.mark.parametrize("form", ["token", "few", "chunk"])
@pytest.mark.parametrize("dh,page", [(64, 16), (128, 128)])
@pytest.mark.parametrize("ratio", [12, 20, 26])
def test_one_huge_value_row(S, form, dh, page, ratio):
    """A value row 2^ratio times the others that hardly counts (its weight is below 2^-100) makes its page's scale as
    much larger, and its neighbours, which do count, zeros. The weights are held in f16 relative to the largest
    weight times page scale: every other page's are that much smaller. With P = 2^7·2^(s + lv - m) an f16 weight
    is off by at most 2^-25 where it is subnormal (2^-11 of it otherwise), so that the sum over value codes v8 is
    off by at most 2^-25·2^-7·max_t(p_t 2^lv_t)·Σ|v8_t|, beside the bound for ordinary pages."""
    n = {"token": 1, "few": 3, "chunk": 100}[form]
    total = 700
    st = PagedState(S, "e4m3", 1, dh, page, [0], [total], seed=43)
    k, v = st.rows([total], 1, 0.5), st.rows([total], 1)
    k[:, :, 0] = 0
    k[200, 0, 0] = -30.0 * dh ** 0.5
    v[200] *= 2.0 ** ratio
    S.slim_mha_paged_append(st.cache, k, v, st.starts([total]), st.lens, st.status)
    st.lens += total - n
    for w in (0, 1):
        st.oracle[w].values = np.nan_to_num(st.values(w), nan=0.0)
    q = st.rows([n], 4)
    q[:, :, 0] = 4.0
    if form == "token":
        out = torch.empty_like(q)
        S.slim_mha_paged_decode(st.cache, q, st.lens, out, S.alloc_paged_decode_workspace(st.cache, 4), st.status)
        torch.cuda.synchronize()
    else:
        out = run(S, st, q, [n], [total - n], max_new=n)
    assert int(st.status.item()) == 0
    K, V = (st.oracle[w].read(st.table_h[0], total) for w in (0, 1))
    lv = np.repeat(f64(st.scales[1])[st.table_h[0, :-(-total // page)], 0], page)[:total]
    o, A, D = P.attend(f64(q), K, V, [total - n + j for j in range(n)])
    for j in range(n):
        T = total - n + j + 1
        z = f64(q[j]) @ K[:T, 0].T / dh ** 0.5
        p = np.exp(z - z.max(axis=1, keepdims=True))
        p /= p.sum(axis=1, keepdims=True)
        assert (p[:, 200] < 2.0 ** -100).all()
        under = (p * lv[:T]).max(axis=1)[:, None] * np.abs(V[:T, 0] / lv[:T, None]).sum(axis=0) * 2.0 ** -32
        err = np.abs(f64(out[j]) - o[j])
        assert (err <= bound("e4m3", dh, o[j], A[j], D[j]) + under).all(), (j, (err / A[j]).max())


@pytest.mark.parametrize("form", ["token", "few", "chunk"])
@pytest.mark.parametrize("page", [16, 128])
@pytest.mark.parametrize("t_hint", [1, 0])
def test_zero_values_before_ordinary_ones(S, form, page, t_hint):
    """Thousands of rows whose values are zero (pages of the smallest scale, 2^-100), most of them with scores 2^7.5
    above those of the first ones, and then a few with ordinary values: the sum of weights holds both."""
    n = {"token": 1, "few": 3, "chunk": 100}[form]
    total, dh = 17 * 512, 64
    st = PagedState(S, "e4m3", 1, dh, page, [0], [total], seed=44)
    k, v = st.rows([total], 1, 0.02), st.rows([total], 1)
    k[:, :, 0] = 7.5 * np.log(2.0) * dh ** 0.5 / 4
    k[:64, :, 0] = 0
    v[:-128] = 0
    S.slim_mha_paged_append(st.cache, k, v, st.starts([total]), st.lens, st.status)
    st.lens += total - n
    for w in (0, 1):
        st.oracle[w].values = np.nan_to_num(st.values(w), nan=0.0)
    assert (f64(st.scales[1])[st.table_h[0, 0]] == 2.0 ** -100).all()
    q = st.rows([n], 2)
    q[:, :, 0] = 4.0
    if form == "token":
        out = torch.empty_like(q)
        S.slim_mha_paged_decode(st.cache, q, st.lens, out, S.alloc_paged_decode_workspace(st.cache, 2), st.status,
                                t_hint=t_hint)
        torch.cuda.synchronize()
    else:
        out = run(S, st, q, [n], [total - n], max_new=n, t_hint=t_hint)
    assert int(st.status.item()) == 0
    check(st, q, out, [n], [total - n])

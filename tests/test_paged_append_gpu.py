"""slim_mha_paged_append and slim_mha_paged_gather against the float64 oracle.

Tolerances. A stored bf16 value is the fp32 rotation (two products and a sum, each rounded: at most
3·2^-24 of |x| + |x'|) rounded by at most half a step, 2^-8 of it. A stored e4m3 value is rounded by
at most 2^-4 of it, or half the smallest step, 2^-10 of the scale. Values that are not rotated have
no rounding before the stored one, so their pages are compared exactly.
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


def rotated(x, n, lens, cos, sin, interleaved):
    """Oracle rotation of packed rows (float64) and the |x| + |x'| of every element."""
    y, mag = np.array(x), np.abs(x)
    if cos is None:
        return y, mag
    c, s = f64(cos), f64(sin)
    half = c.shape[1]
    i = np.arange(half)
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
    mag = mag.copy()
    mag[..., a] = mag[..., b] = np.abs(x[..., a]) + np.abs(x[..., b])
    r = 0
    for k, L in zip(n, lens):
        for j in range(k):
            y[r] = P.rotate(x[r], c[L + j], s[L + j], interleaved)
            r += 1
    return y, mag


CASES = [
    # kind, Hq, Hkv, dh, page, cached, new, rot, interleaved
    ("bf16", 4, 4, 64, 16, [0], [1], 64, False),
    ("e4m3", 4, 4, 64, 16, [0], [1], 64, False),
    ("bf16", 8, 2, 128, 64, [0, 63, 64, 65], [1, 1, 1, 1], 128, True),
    ("e4m3", 8, 2, 128, 128, [0, 127, 128, 200, 31], [1, 1, 1, 1, 0], 128, False),
    ("e4m3", 20, 20, 64, 32, [5, 0, 31], [1, 0, 1], 32, True),
    ("bf16", 6, 3, 64, 16, [0, 7, 16], [40, 0, 33], 48, False),
    ("e4m3", 6, 3, 64, 16, [0, 7, 16], [40, 0, 33], 64, True),
    ("e4m3", 7, 1, 64, 64, [3, 130], [200, 1], 64, False),
    ("e4m3", 8, 4, 128, 32, [33, 0, 95], [31, 64, 2], 16, False),
    ("bf16", 8, 8, 128, 128, [100, 0], [300, 129], 128, False),
    ("e4m3", 8, 8, 128, 128, [100, 0], [300, 129], 128, True),
    ("e4m3", 5, 5, 128, 64, [63, 1], [130, 63], 0, False),
    ("e4m3", 40, 8, 128, 16, [1, 14], [17, 100], 128, False),
    ("e4m3", 2048, 1024, 64, 16, [3, 15], [14, 1], 64, True),
    ("bf16", 8192, 64, 64, 16, [0, 15], [1, 1], 32, False),
    ("e4m3", 2, 1, 64, 16, [i % 20 for i in range(4096)], [i % 3 % 2 for i in range(4096)], 64, False),
]


@pytest.mark.parametrize("kind,Hq,Hkv,dh,page,cached,new,rot,interleaved", CASES)
@pytest.mark.parametrize("bound", ["tight", "none"])
def test_append_and_gather(S, kind, Hq, Hkv, dh, page, cached, new, rot, interleaved, bound):
    st = PagedState(S, kind, Hkv, dh, page, cached, [a + n for a, n in zip(cached, new)], seed=1)
    rows = sum(new)
    kv = st.rows(new, 2 * Hkv)  # k and v side by side: rows lie apart
    k, v = kv[:, :Hkv], kv[:, Hkv:]
    q = st.rows(new, Hq)
    q_out = torch.full_like(q, 7.0)
    cos, sin = angles(max(a + n for a, n in zip(cached, new)), rot) if rot else (None, None)
    before = [p.clone() for p in st.pages]
    S.slim_mha_paged_append(st.cache, k, v, st.starts(new), st.lens, st.status, q=q, q_out=q_out, cos=cos, sin=sin,
                            interleaved=interleaved, max_new=max(new) if bound == "tight" else 0)
    torch.cuda.synchronize()
    assert int(st.status.item()) == 0 and st.lens.tolist() == cached
    rk, mk = rotated(f64(k), new, cached, cos, sin, interleaved)
    rq, mq = rotated(f64(q), new, cached, cos, sin, interleaved)
    assert (np.abs(f64(q_out) - rq) <= 2.0 ** -8 * np.abs(rq) + 3 * 2.0 ** -24 * mq).all()
    written = np.zeros(st.pages[0].shape[:1] + (page,), dtype=bool)
    for w, x in ((0, rk), (1, f64(v))):
        r = 0
        for b, n in enumerate(new):
            st.oracle[w].write(x[r:r + n], st.table_h[b], cached[b])
            r += n
    got = [st.values(w) for w in (0, 1)]
    if kind == "e4m3":
        for w in (0, 1):
            assert np.array_equal(f64(st.scales[w]), st.oracle[w].scale), w
    r = 0
    for b, n in enumerate(new):
        for t in range(cached[b] + n):
            at = (int(st.table_h[b, t // page]), slice(None), t % page)
            written[at[0], at[2]] = True
            assert np.array_equal(got[1][at], f64(v)[r + t - cached[b]] if kind == "bf16" and t >= cached[b]
                                  else st.oracle[1].values[at])
            if t < cached[b]:
                assert np.array_equal(got[0][at], st.oracle[0].values[at])
                continue
            ref, m = rk[r + t - cached[b]], mk[r + t - cached[b]]
            if kind == "bf16":
                tol = 2.0 ** -8 * np.abs(ref) + 3 * 2.0 ** -24 * m
            else:
                tol = 2.0 ** -4 * np.abs(ref) + 2.0 ** -10 * st.oracle[0].scale[at[0], :, None] + 3 * 2.0 ** -24 * m
            assert (np.abs(got[0][at] - ref) <= tol).all()
        r += n
    # nothing else is written: other rows keep their bytes (in e4m3 also where a page's scale grew)
    for w in (0, 1):
        a = st.pages[w].view(torch.uint8).cpu().numpy()
        b0 = before[w].view(torch.uint8).cpu().numpy()
        assert np.array_equal(a.transpose(0, 2, 1, 3)[~written], b0.transpose(0, 2, 1, 3)[~written])

    # and back
    back = [a + n - a // 2 for a, n in zip(cached, new)]
    first = torch.tensor([a // 2 for a in cached], dtype=torch.int32, device=st.dev)
    total = sum(back)
    ko = torch.full((total + 3, Hkv, dh), 5.0, dtype=torch.bfloat16, device=st.dev)
    vo = torch.full_like(ko, 5.0)
    S.slim_mha_paged_gather(st.cache, first, st.starts(back, 1), ko, vo, st.status,
                            max_new=max(back) if bound == "tight" else 0)
    torch.cuda.synchronize()
    assert int(st.status.item()) == 0
    for w, o in ((0, ko), (1, vo)):
        o = f64(o)
        assert (o[:1] == 5).all() and (o[1 + total:] == 5).all()
        r = 1
        for b, n in enumerate(back):
            for t in range(cached[b] // 2, cached[b] // 2 + n):
                assert np.array_equal(o[r], got[w][int(st.table_h[b, t // page]), :, t % page])
                r += 1


@pytest.mark.parametrize("dh,page", [(64, 16), (128, 32), (128, 128)])
def test_token_by_token_is_all_at_once(S, dh, page):
    """One call per token, with magnitudes that grow and shrink, gives the scales of one call, and its values up
    to one more rounding where a value became subnormal under a later scale: at most the neighbouring value, one
    step of 2^-9 of the scale away."""
    Hkv, n = 3, page + page // 2 + 3
    growth = torch.exp2(torch.arange(n).float() % 11 - 5).view(n, 1, 1)
    a = PagedState(S, "e4m3", Hkv, dh, page, [0], [n], seed=2)
    b = PagedState(S, "e4m3", Hkv, dh, page, [0], [n], seed=2)
    k = (a.rows([n], Hkv).cpu() * growth).to(torch.bfloat16).cuda()
    v = (a.rows([n], Hkv).cpu() / growth).to(torch.bfloat16).cuda()
    cos, sin = angles(n, dh)
    S.slim_mha_paged_append(a.cache, k, v, a.starts([n]), a.lens, a.status, cos=cos, sin=sin)
    lens = torch.zeros(1, dtype=torch.int32, device="cuda")
    for j in range(n):
        S.slim_mha_paged_append(b.cache, k[j:j + 1], v[j:j + 1], b.starts([1]), lens, b.status, cos=cos, sin=sin)
        lens += 1
    torch.cuda.synchronize()
    assert int(a.status.item()) == 0 and int(b.status.item()) == 0
    used = a.table_h[0, :-(-n // page)]
    for w in (0, 1):
        assert torch.equal(a.scales[w][used], b.scales[w][used])
        x, y = a.values(w)[used], b.values(w)[used]
        sc = f64(a.scales[w])[used][:, :, None, None]
        live = np.isfinite(x)
        assert np.array_equal(live, np.isfinite(y))
        normal = live & (np.abs(x) >= 2.0 ** -6 * sc)
        assert np.array_equal(x[normal], y[normal])
        assert (np.abs(x - y)[live] <= (2.0 ** -9 * sc * np.ones_like(x))[live]).all()


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("max_new", [1, 40])
def test_skipped_sequences(S, kind, max_new):
    """Bad lengths, overflow, too many rows and bad pages are reported; nothing of the sequence is written and
    its rotated queries are zero. The others are served."""
    Hkv, dh, page = 2, 64, 16
    cached = [3, 5, 16, 2, 4]
    st = PagedState(S, kind, Hkv, dh, page, cached, [20] * 5, seed=3)
    new = [1] * 5
    cap = st.cache.cap
    lens = torch.tensor([-1, cap, cap + 1, 2, 4], dtype=torch.int32, device="cuda")
    table = st.table.clone()
    table[3, 0] = st.cache.num_pages
    cache = S.PagedKV(st.pages[0], st.pages[1], table, st.scales[0], st.scales[1])
    k, v, q = st.rows(new, Hkv), st.rows(new, Hkv), st.rows(new, 4)
    cos, sin = angles(cap, 64)
    before = [p.clone() for p in st.pages]
    q_out = torch.full_like(q, 3.0)
    S.slim_mha_paged_append(cache, k, v, st.starts(new), lens, st.status, q=q, q_out=q_out, cos=cos, sin=sin,
                            max_new=max_new)
    torch.cuda.synchronize()
    assert int(st.status.item()) == S.SLIM_DEV_BADLEN | S.SLIM_DEV_OVERFLOW | S.SLIM_DEV_BADPAGE
    assert (q_out[:3] == 0).all() and (q_out[3:] != 0).any()
    for w in (0, 1):
        now, was = st.pages[w].view(torch.uint8), before[w].view(torch.uint8)
        changed = (now != was).flatten(2).any(dim=2).any(dim=1).nonzero().flatten().tolist()
        assert changed == [int(st.table_h[4, 0])]
    # angles for fewer positions than the cache has
    st.status.zero_()
    S.slim_mha_paged_append(st.cache, k, v, st.starts(new), st.lens, st.status, cos=cos[:4], sin=sin[:4], max_new=max_new)
    torch.cuda.synchronize()
    assert int(st.status.item()) == S.SLIM_DEV_OVERFLOW
    # more rows than max_new, and starts that descend
    st.status.zero_()
    two = torch.tensor([0, 2, 1, 3, 4, 99], dtype=torch.int32, device="cuda")
    S.slim_mha_paged_append(st.cache, k, v, two, st.lens, st.status, max_new=1)
    torch.cuda.synchronize()
    assert int(st.status.item()) & S.SLIM_DEV_BADLEN


def test_gather_skips(S):
    st = PagedState(S, "e4m3", 2, 64, 16, [20, 20, 20], [32] * 3, seed=4)
    st.table[1, 0] = -1
    first = torch.tensor([16, 10, st.cache.cap - 2], dtype=torch.int32, device="cuda")
    ko = torch.full((12, 2, 64), 5.0, dtype=torch.bfloat16, device="cuda")
    vo = torch.full_like(ko, 5.0)
    S.slim_mha_paged_gather(st.cache, first, st.starts([4, 4, 4]), ko, vo, st.status)
    torch.cuda.synchronize()
    assert int(st.status.item()) == S.SLIM_DEV_BADPAGE | S.SLIM_DEV_OVERFLOW
    assert np.array_equal(f64(ko[:4]), st.oracle[0].read(st.table_h[0], 20)[16:])
    assert (ko[4:] == 0).all() and (vo[4:] == 0).all()


def test_not_finite_rows_poison_their_page(S):
    """A NaN or an infinity in a new row makes the scale of its page and head NaN, in both launch forms."""
    for n, bad in ((1, float("nan")), (1, float("inf")), (5, float("-inf"))):
        st = PagedState(S, "e4m3", 2, 64, 16, [3], [16], seed=5)
        k, v = st.rows([n], 2), st.rows([n], 2)
        k[n - 1, 1, 7] = bad
        S.slim_mha_paged_append(st.cache, k, v, st.starts([n]), st.lens, st.status)
        torch.cuda.synchronize()
        pid = int(st.table_h[0, 0])
        assert torch.isnan(st.scales[0][pid]).tolist() == [False, True]
        assert torch.isfinite(st.scales[1][pid]).all()
        # later rows do not hide it; a sequence that begins the page anew does
        S.slim_mha_paged_append(st.cache, v[:1], v[:1], st.starts([1]), st.lens + n, st.status)
        assert torch.isnan(st.scales[0][pid]).tolist() == [False, True]
        S.slim_mha_paged_append(st.cache, v[:1], v[:1], st.starts([1]), st.lens * 0, st.status)
        assert torch.isfinite(st.scales[0][pid]).all()


def test_extreme_magnitudes(S):
    """Zeros, the largest finite bf16 and values near the smallest scale."""
    st = PagedState(S, "e4m3", 4, 64, 32, [0], [32], seed=6)
    v = torch.zeros(3, 4, 64, dtype=torch.bfloat16, device="cuda")
    v[:, 1] = torch.finfo(torch.bfloat16).max
    v[:, 2] = 2.0 ** -120
    v[0, 3], v[1, 3] = 448.0, 2.0 ** -12
    S.slim_mha_paged_append(st.cache, v, v, st.starts([3]), st.lens, st.status)
    torch.cuda.synchronize()
    pid = int(st.table_h[0, 0])
    assert st.scales[1][pid].tolist() == [2.0 ** -100, 2.0 ** 120, 2.0 ** -100, 1.0]
    got = st.values(1)[pid][:, :3]
    assert (got[0] == 0).all() and (got[2] == 0).all()
    assert (np.abs(got[1] / f64(v[:, 1]) - 1) <= 2.0 ** -4).all()
    assert (got[3, 0] == 448).all() and (got[3, 1] == 0).all()


def test_queries_rotated_in_place_and_streams(S):
    """q_out may be q; calls run on the stream that is given, and can be captured."""
    st = PagedState(S, "bf16", 2, 64, 16, [9, 0], [40, 40], seed=7)
    n = [20, 7]
    k, v, q = st.rows(n, 2), st.rows(n, 2), st.rows(n, 4)
    cos, sin = angles(40, 64)
    want = torch.empty_like(q)
    S.slim_mha_paged_append(st.cache, k, v, st.starts(n), st.lens, st.status, q=q, q_out=want, cos=cos, sin=sin)
    pages = [p.clone() for p in st.pages]
    starts = st.starts(n)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    q2 = q.clone()
    s.synchronize()
    with torch.cuda.graph(g, stream=s):
        S.slim_mha_paged_append(st.cache, k, v, starts, st.lens, st.status, q=q2, q_out=q2, cos=cos, sin=sin)
    for p in st.pages:
        p.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(q2, want)
    for w in (0, 1):
        r = 0
        for b in range(2):
            for t in range(st.lens_h[b], st.lens_h[b] + n[b]):
                pid = int(st.table_h[b, t // 16])
                assert torch.equal(st.pages[w][pid, :, t % 16], pages[w][pid, :, t % 16])
                r += 1


def test_no_rows(S):
    st = PagedState(S, "bf16", 2, 64, 16, [9, 0], [40, 40], seed=8)
    e = torch.empty(0, 2, 64, dtype=torch.bfloat16, device="cuda")
    S.slim_mha_paged_append(st.cache, e, e, st.starts([0, 0]), st.lens, st.status)
    assert S.slim_last_launch_count() == 0
    S.slim_mha_paged_gather(st.cache, st.lens, st.starts([0, 0]), e, e, st.status)
    assert S.slim_last_launch_count() == 0 and int(st.status.item()) == 0


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_offsets_past_32_bits(S, kind):
    """Pools of more than 2^32 bytes, used at their far end."""
    Hkv, dh, page = 64, 128, 128
    per = Hkv * dh * page * (2 if kind == "bf16" else 1)
    num = (1 << 32) // per + 3
    dt = torch.bfloat16 if kind == "bf16" else torch.float8_e4m3fn
    pools = [torch.empty(num, Hkv, page, dh, dtype=dt, device="cuda") for _ in range(2)]
    scales = [torch.ones(num, Hkv, device="cuda") if kind == "e4m3" else None for _ in range(2)]
    table = torch.tensor([[num - 1, num - 2], [0, num - 3]], dtype=torch.int32, device="cuda")
    cache = S.PagedKV(pools[0], pools[1], table, scales[0], scales[1])
    rng = torch.Generator(device="cuda").manual_seed(1)
    new = [130, 129]
    k = torch.randn(sum(new), Hkv, dh, device="cuda", generator=rng).bfloat16()
    v = torch.randn(sum(new), Hkv, dh, device="cuda", generator=rng).bfloat16()
    starts = torch.tensor([0, 130, 259], dtype=torch.int32, device="cuda")
    lens = torch.zeros(2, dtype=torch.int32, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    S.slim_mha_paged_append(cache, k, v, starts, lens, status, max_new=130)
    ko, vo = torch.empty_like(k), torch.empty_like(v)
    S.slim_mha_paged_gather(cache, lens, starts, ko, vo, status, max_new=130)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    step = 0.0 if kind == "bf16" else 2.0 ** -4
    for a, b in ((ko, k), (vo, v)):
        assert ((a.double() - b.double()).abs() <= step * b.double().abs() + step * 2.0 ** -6 * 2.0 ** -6).all()


@pytest.mark.parametrize("n", [1, 3])
def test_largest_magnitudes_read_back(S, n):
    """Rows at bf16's largest magnitude, in both launch forms: their codes stand for finite values within a step's
    half (2^-4) of them, read back and as outputs of both attentions."""
    top = torch.finfo(torch.bfloat16).max
    st = PagedState(S, "e4m3", 3, 64, 32, [0], [32], seed=9)
    v = torch.zeros(n, 3, 64, dtype=torch.bfloat16, device="cuda")
    v[:, 0] = top
    v[:, 1] = -top
    v[:, 2] = 247 * 2.0 ** 120  # the largest that rounds to 240·2^120
    k = st.rows([n], 3)
    S.slim_mha_paged_append(st.cache, k, v, st.starts([n]), st.lens, st.status, max_new=n)
    ko, vo = torch.empty_like(v), torch.empty_like(v)
    S.slim_mha_paged_gather(st.cache, st.lens, st.starts([n]), ko, vo, st.status)
    q = st.rows([n], 3)
    out = torch.empty_like(q)
    S.slim_mha_paged_prefill(st.cache, q, st.starts([n]), st.lens, out,
                             S.alloc_paged_prefill_workspace(st.cache, 3, n), st.status)
    one = torch.empty_like(q[:1])
    S.slim_mha_paged_decode(st.cache, q[:1], st.lens, one, S.alloc_paged_decode_workspace(st.cache, 3), st.status)
    torch.cuda.synchronize()
    assert int(st.status.item()) == 0 and (st.scales[1][int(st.table_h[0, 0])] == 2.0 ** 120).all()
    for x in (vo, out, one):
        assert torch.isfinite(x).all()
        # an output is rounded to bf16 again, and its weights sum to 1 up to their rounding to f16
        assert (np.abs(f64(x) / f64(v[:1]) - 1) <= 2.0 ** -4 + (0 if x is vo else 2.0 ** -8 + 2.0 ** -10)).all()


def test_large_rows_beside_older_ones(S):
    """A row at bf16's largest magnitude behind older rows: they keep their values, under a larger scale than theirs
    and under the largest one."""
    st = PagedState(S, "e4m3", 1, 64, 16, [0], [16], seed=10)
    rows = torch.zeros(4, 1, 64, dtype=torch.bfloat16, device="cuda")
    rows[0] = 448 * 2.0 ** 119   # the largest code of the second largest scale
    rows[1] = torch.finfo(torch.bfloat16).max
    rows[2] = 240 * 2.0 ** 120
    rows[3] = -torch.finfo(torch.bfloat16).max
    lens = st.lens.clone()
    for j in range(4):
        S.slim_mha_paged_append(st.cache, rows[j:j + 1], rows[j:j + 1], st.starts([1]), lens, st.status)
        lens += 1
    ko, vo = torch.empty_like(rows), torch.empty_like(rows)
    S.slim_mha_paged_gather(st.cache, st.lens, st.starts([4]), ko, vo, st.status)
    torch.cuda.synchronize()
    want = [448 * 2.0 ** 119, 240 * 2.0 ** 120, 240 * 2.0 ** 120, -240 * 2.0 ** 120]
    for x in (ko, vo):
        assert (f64(x) == np.array(want)[:, None, None]).all()

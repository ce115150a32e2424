"""The cache's calls at the edges of their numbers: infinities and values near the
end of the range, scales and queries whose products leave fp32's normal range,
lengths beyond the table, hints that are too small.

Tolerances: those of the attention's own test (a weight is rounded to 8 bits or
more, at most 2^-8 of it, the output to bf16 once more, and the exponential is
off by less than 2^-13 of a weight); results that must not change are compared
bit by bit."""
import numpy as np
import pytest
import torch

import oracle
from test_gpu_cache import Cache, KINDS, check, offsets

pytestmark = pytest.mark.gpu

DEV = "cuda"
f64 = oracle.as_f64


def _randn(seed, *shape):
    return torch.randn(*shape, generator=torch.Generator(device=DEV).manual_seed(seed), device=DEV).to(torch.bfloat16)


@pytest.mark.parametrize("kind", list(KINDS))
@pytest.mark.parametrize("L,n,keys", [(150, 40, range(120, 128)),       # a block finishes the item
                                      (6000, 2, range(3000, 3008))])    # several blocks share it
def test_infinite_keys(cuda_lib, kind, L, n, keys):
    """Eight neighbouring keys in turn (columns that different exponentials and
    lanes handle) hold +inf. A row with a score of +inf is NaN, as inf - inf is; in
    a bf16 cache a row with one of -inf gives it no weight. (An 8-bit row with an
    infinity has that as its scale, and its scores are NaN.) Rows that do not see
    the key are as without it."""
    sa = cuda_lib
    H, G, d = 1, 2, 64
    c = Cache(kind, [L], H, d, 32, seed=50)
    k, v = c.fill(sa, 51)
    q = _randn(52, n, H * G, d)
    q[:, 0, 9] = q[:, 0, 9].abs() + 1
    q[:, 1, 9] = -q[:, 1, 9].abs() - 1
    ref = sa.sa_cache_attn(q, c.k, c.v, c.dt, offsets([n]), c.lens(), **c.args())
    for key in keys:
        bad = k.clone()
        bad[key, 0, 9] = float("inf")
        sa.sa_cache_write(bad, v, c.k, c.v, c.dt, offsets([L]), c.lens(), **c.args())
        o, lse = sa.sa_cache_attn(q, c.k, c.v, c.dt, offsets([n]), c.lens(), want_lse=True, **c.args())
        first = max(0, key - (L - n))                     # the first row that sees the key
        assert torch.equal(o[:first], ref[:first]), key
        assert torch.isnan(o[first:, 0]).all() and torch.isnan(lse[first:, 0]).all(), key
        if kind != "bf16":
            assert torch.isnan(o[first:, 1]).all() and torch.isnan(lse[first:, 1]).all(), key
            continue
        kk, vv, qq = f64(bad[:, 0]), f64(v[:, 0]), f64(q[:, 1])
        for i in range(first, n, 7):
            seen = L - n + i + 1
            want, wl = oracle.cache_attention(qq[i:i + 1], kk, vv, seen)
            mag, _ = oracle.cache_attention(qq[i:i + 1], kk, np.abs(vv), seen)
            # (the scores' own error, 2^-24 d scale sum|q||k|, is below 2^-14 here)
            lim = (2.0 ** -8 + 2.0 ** -11 + 2.0 ** -13) * mag + 2.0 ** -8 * np.abs(want)
            assert (np.abs(f64(o[i, 1]) - want[0]) <= lim[0]).all(), (key, i)
            assert abs(float(lse[i, 1]) - wl[0]) <= 2.0 ** -11 + 2.0 ** -13 + 2.0 ** -22 * abs(wl[0])
    sa.sa_device_status()


@pytest.mark.parametrize("key", [5, 24, 31, 63, 127, 130])
def test_products_beyond_fp32_give_nan(cuda_lib, key):
    """A finite query and key whose product overflows: no plausible row comes of it."""
    sa = cuda_lib
    L, H, d = 150, 1, 64
    c = Cache("bf16", [L], H, d, 32, seed=53)
    k, v = c.fill(sa, 54)
    q = _randn(55, 3, H, d)
    q[1, 0, 9] = 1e30
    k[key, 0, 9] = 1e30
    sa.sa_cache_write(k, v, c.k, c.v, c.dt, offsets([L]), c.lens(), **c.args())
    o, lse = sa.sa_cache_attn(q, c.k, c.v, c.dt, offsets([3]), c.lens(), want_lse=True, **c.args())
    assert torch.isnan(o[1]).all() and torch.isnan(lse[1]).all()


@pytest.mark.parametrize("L,n", [(150, 40), (3000, 300)])
def test_large_values_at_masked_positions(cuda_lib, L, n):
    """Finite values near the end of bf16's range that a row does not see add
    nothing to it: weights of masked positions are 0, not only small."""
    sa = cuda_lib
    H, G, d = 1, 2, 64
    c = Cache("bf16", [L], H, d, 32, seed=56)
    k, v = c.fill(sa, 57)
    q = _randn(58, n, H * G, d)
    cu = offsets([n])
    ref = sa.sa_cache_attn(q, c.k, c.v, c.dt, cu, c.lens(), **c.args())
    first = n // 2                                       # the first row that sees one of them
    v[L - n + first:] = 3e38
    sa.sa_cache_write(k, v, c.k, c.v, c.dt, offsets([L]), c.lens(), **c.args())
    o = sa.sa_cache_attn(q, c.k, c.v, c.dt, cu, c.lens(), **c.args())
    assert torch.equal(o[:first], ref[:first])
    # seen, with a score so far below the largest that the weight is 0 in fp32 (below 2^-150)
    v[L - n + first:] = 0
    k[7] = 0
    k[7, 0, 0] = -1e4
    q[:, :, 0] = q[:, :, 0].abs() + 1
    for key in range(0, 64, 5):
        kk, vv = k.clone(), v.clone()
        kk[[key, 7]], vv[key] = k[[7, key]], 0
        sa.sa_cache_write(kk, vv, c.k, c.v, c.dt, offsets([L]), c.lens(), **c.args())
        ref = sa.sa_cache_attn(q, c.k, c.v, c.dt, cu, c.lens(), **c.args())
        vv[key] = 3e38
        sa.sa_cache_write(kk, vv, c.k, c.v, c.dt, offsets([L]), c.lens(), **c.args())
        o = sa.sa_cache_attn(q, c.k, c.v, c.dt, cu, c.lens(), **c.args())
        assert torch.equal(o, ref), key
    sa.sa_device_status()


@pytest.mark.parametrize("kind", list(KINDS))
@pytest.mark.parametrize("scale", [1e-10, 1e-25, 1.3e-38, 0.0])
def test_zero_and_tiny_queries_with_small_scales(cuda_lib, kind, scale):
    """Scores that are 0 or vanish: a row is the mean of the values that it sees."""
    sa = cuda_lib
    L, n, H, G, d = 300, 40, 2, 2, 64
    c = Cache(kind, [L], H, d, 32, seed=60)
    k, v = c.fill(sa, 61)
    q = _randn(62, n, H * G, d)
    q[:, 0] = 0
    q[:, 1] = (q[:, 1].float() * 1e-37).to(torch.bfloat16)
    q[:, 2] = (q[:, 2].float() * 2.0 ** -132).to(torch.bfloat16)          # subnormal
    o, lse = sa.sa_cache_attn(q, c.k, c.v, c.dt, offsets([n]), c.lens(), scale=scale, want_lse=True, **c.args())
    check(o, lse, q, c.rows(k, v), [L], [n], True, scale=scale if scale > 0 else None)
    sa.sa_device_status()


@pytest.mark.parametrize("kind", list(KINDS))
def test_scores_of_zero_under_large_scales(cuda_lib, kind):
    """Large queries and a large scale meet keys of zero: scores of 0, not 0 times infinity."""
    sa = cuda_lib
    L, n, H, G, d = 200, 5, 1, 2, 64
    c = Cache(kind, [L], H, d, 32, seed=63)
    _, v = c.fill(sa, 64)
    k = torch.zeros_like(v)
    sa.sa_cache_write(k, v, c.k, c.v, c.dt, offsets([L]), c.lens(), **c.args())
    q = (_randn(65, n, H * G, d).float() * 1e37).to(torch.bfloat16)
    o, lse = sa.sa_cache_attn(q, c.k, c.v, c.dt, offsets([n]), c.lens(), scale=1e9, want_lse=True, **c.args())
    check(o, lse, q, c.rows(k, v), [L], [n], True, scale=1e9)
    sa.sa_device_status()


@pytest.mark.parametrize("kind", list(KINDS))
def test_lengths_beyond_the_table_mean_the_same_to_every_call(cuda_lib, kind):
    """A length beyond the table counts as the table's, in the write as in the
    attention: its new rows are the last positions of the table."""
    sa = cuda_lib
    page, width, H, G, d, n = 16, 3, 2, 2, 64, 7
    full = page * width
    q, k, v = _randn(70, n, H * G, d), _randn(71, n, H, d), _randn(72, n, H, d)
    got = []
    for L in (full, full + 1, full + 5, 10 ** 6, 2 ** 31 - 1):
        c = Cache(kind, [full], H, d, page, seed=73, extra_width=0)
        c.fill(sa, 74)
        sa.sa_cache_write(k, v, c.k, c.v, c.dt, offsets([n]), c.lens([L]), **c.args())
        kr, vr = sa.sa_cache_read(c.k, c.v, c.dt, offsets([full]), full, **c.args())
        o = sa.sa_cache_attn(q, c.k, c.v, c.dt, offsets([n]), c.lens([L]), n, **c.args())
        got.append((kr, vr, o))
    for g in got[1:]:
        for a, b in zip(g, got[0]):
            assert torch.equal(a, b)
    # lengths below 0 count as 0: nothing is written, no row sees anything
    for L in (-1, -2 ** 31):
        c = Cache(kind, [full], H, d, page, seed=73, extra_width=0)
        c.fill(sa, 74)
        before = c.k.view(torch.uint8).clone()
        sa.sa_cache_write(k, v, c.k, c.v, c.dt, offsets([n]), c.lens([L]), **c.args())
        assert torch.equal(c.k.view(torch.uint8), before)
        o, lse = sa.sa_cache_attn(q, c.k, c.v, c.dt, offsets([n]), c.lens([L]), n, want_lse=True, **c.args())
        assert (o == 0).all() and (lse == -float("inf")).all()
    sa.sa_device_status()


@pytest.mark.parametrize("kind", list(KINDS))
@pytest.mark.parametrize("causal", [True, False])
def test_hints_below_the_longest_chunk(cuda_lib, kind, causal):
    """max_q shapes the tiles only: a hint that is too small gives the same rows
    within the bound."""
    sa = cuda_lib
    kv, new, H, G, d, page = [300, 77, 150], [130, 77, 1], 2, 3, 64, 16
    c = Cache(kind, kv, H, d, page, seed=80)
    k, v = c.fill(sa, 81)
    q = _randn(82, sum(new), H * G, d)
    rows = c.rows(k, v)
    for max_q in (1, 2, 41, 129, 10 ** 6):
        o, lse = sa.sa_cache_attn(q, c.k, c.v, c.dt, offsets(new), c.lens(), max_q, causal=causal, want_lse=True, **c.args())
        check(o, lse, q, rows, kv, new, causal)
    sa.sa_device_status()


@pytest.mark.parametrize("kind", ["e4m3", "int8"])
@pytest.mark.parametrize("x", [float("inf"), -float("inf"), float("nan")])
def test_a_non_finite_number_is_its_rows_scale(cuda_lib, kind, x):
    """The row is read as NaN or infinity, its neighbours as they are."""
    sa = cuda_lib
    L, H, d = 40, 2, 64
    c = Cache(kind, [L], H, d, 16, seed=83)
    k, v = c.fill(sa, 84)
    ks, vs = c.ks.clone(), c.vs.clone()
    ref = sa.sa_cache_read(c.k, c.v, c.dt, offsets([L]), L, **c.args())
    k[7, 1, 3] = x
    v[9, 0, 60] = x
    sa.sa_cache_write(k, v, c.k, c.v, c.dt, offsets([L]), c.lens(), **c.args())
    for s, before, at, (p, h) in ((c.ks, ks, 7, (7, 1)), (c.vs, vs, 9, (9, 0))):
        pg, sl = oracle.cache_slot(c.table[0], 16, p, c.P)
        got = float(s[pg, h, sl])
        assert np.isnan(got) if np.isnan(x) else got == float("inf")
        s[pg, h, sl] = before[pg, h, sl]
        assert torch.equal(s.view(torch.int32), before.view(torch.int32))
        s[pg, h, sl] = got
    got = sa.sa_cache_read(c.k, c.v, c.dt, offsets([L]), L, **c.args())
    for a, b, (p, h) in zip(got, ref, ((7, 1), (9, 0))):
        assert not torch.isfinite(a[p, h]).any()
        keep = torch.ones(L, H, dtype=torch.bool, device=DEV)
        keep[p, h] = False
        assert torch.equal(a[keep], b[keep])


@pytest.mark.parametrize("kind", ["bf16", "int8"])
def test_offsets_beyond_32_bits(cuda_lib, kind):
    """A cache of 4.6e9 elements for each of keys and values, whose first and last
    pages are used, and operands with a token stride of 2^31 elements, against the same
    call on a cache of a few pages and dense operands: the same bits."""
    sa = cuda_lib
    H, G, d, page, L, n = 4, 2, 128, 128, 1000, 3
    used, P = -(-L // page), 70000
    small = Cache(kind, [L], H, d, page, seed=90, spare=0, extra_width=0)
    k, v = small.fill(sa, 91)
    cu, lens = offsets([n]), small.lens()
    q, kn, vn = _randn(92, n, H * G, d), _randn(93, n, H, d), _randn(94, n, H, d)
    big = dict(k_cache=torch.empty(P, H, page, d, dtype=KINDS[kind], device=DEV), v_cache=torch.empty(P, H, page, d, dtype=KINDS[kind], device=DEV))
    if kind != "bf16":
        big.update(k_scale=torch.empty(P, H, page, device=DEV), v_scale=torch.empty(P, H, page, device=DEV))
    pages = [P - 1 - i if i % 2 else i for i in range(used)]
    table = torch.tensor([pages], dtype=torch.int32, device=DEV)
    sa.sa_cache_write(k, v, table=table, cu_q=offsets([L]), kv_len=lens, **big)
    far = torch.empty(2 * 2 ** 31 + H * G * d, dtype=torch.bfloat16, device=DEV)

    def spread(x):
        y = far.as_strided(x.shape, (2 ** 31, d, 1))
        y.copy_(x)
        return y

    sa.sa_cache_write(kn, vn, small.k, small.v, small.dt, cu, lens, **small.args())
    want = sa.sa_cache_attn(q, small.k, small.v, small.dt, cu, lens, n, **small.args())
    sa.sa_cache_write(spread(kn), vn, table=table, cu_q=cu, kv_len=lens, **big)
    got = sa.sa_cache_attn(spread(q), table=table, cu_q=cu, kv_len=lens, max_q=n, **big)
    assert torch.equal(got, want)
    out = spread(torch.zeros_like(q))
    sa.sa_cache_attn(q, table=table, cu_q=cu, kv_len=lens, max_q=n, out=out, **big)
    assert torch.equal(out, want)
    kr, vr = sa.sa_cache_read(big["k_cache"], big["v_cache"], table, offsets([L]), L, big.get("k_scale"), big.get("v_scale"))
    ks, vs = sa.sa_cache_read(small.k, small.v, small.dt, offsets([L]), L, **small.args())
    assert torch.equal(kr, ks) and torch.equal(vr, vs)
    sa.sa_device_status()

"""GPU parity of the paged key/value cache and of attention over it with the
fp64 oracle.

Tolerances (derived, none fitted): a written row's codes, scales and read-back
values are equal to the oracle's exactly. Attention rounds each weight p_j (times
the row's scale in an 8-bit cache) to bf16 once, at most 2^-8 of it, and the
output once more; the exponential's error is below 2^-13 of p_j, and the fp32
score of d exact products differs by at most ds = 2^-24 d scale sum|q||k|, which
moves p_j and the sum of the weights by that factor each:
|err| <= (2^-8 + 2^-11 + 2 ds) sum_j p_j |v_j| + 2^-8 |o|."""
import numpy as np
import pytest
import torch

import oracle

pytestmark = pytest.mark.gpu

DEV = "cuda"
f64 = oracle.as_f64
KINDS = {"bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn, "int8": torch.int8}


class Cache:
    """A paged cache of S sequences whose unused slots and pages hold NaN (bf16
    and E4M3) or large codes, with its host copy."""

    def __init__(self, kind, kv, H, d, page, seed=0, spare=3, extra_width=1):
        g = np.random.default_rng(seed)
        self.kind, self.kv, self.H, self.d, self.page = kind, list(kv), H, d, page
        self.width = max(1, max(-(-L // page) for L in kv)) + extra_width
        used = [-(-L // page) for L in kv]
        self.P = sum(used) + spare
        order = g.permutation(self.P)
        self.table = np.full((len(kv), self.width), -1, dtype=np.int32)
        at = 0
        for s, n in enumerate(used):
            self.table[s, :n] = order[at:at + n]
            at += n
        shape = (self.P, H, page, d)
        if kind == "int8":
            self.k = torch.full(shape, 127, dtype=torch.int8, device=DEV)
        else:
            self.k = torch.full(shape, float("nan"), device=DEV).to(KINDS[kind])
        self.v = self.k.clone()
        self.ks = self.vs = None
        if kind != "bf16":
            self.ks = torch.full(shape[:3], float("nan"), device=DEV)
            self.vs = self.ks.clone()
        self.dt = torch.from_numpy(self.table).to(DEV)

    def lens(self, kv=None):
        return torch.tensor(self.kv if kv is None else kv, dtype=torch.int32, device=DEV)

    def args(self):
        return dict(k_scale=self.ks, v_scale=self.vs)

    def fill(self, sa, seed, gain=1.0):
        """Writes every position of every sequence; returns its rows (bf16 [sum kv, H, d])."""
        g = torch.Generator(device=DEV).manual_seed(seed)
        n = sum(self.kv)
        k, v = (torch.randn(n, self.H, self.d, generator=g, device=DEV) for _ in range(2))
        k[..., 1] *= 5
        k, v = (k * gain).to(torch.bfloat16), v.to(torch.bfloat16)
        cu = offsets(self.kv)
        sa.sa_cache_write(k, v, self.k, self.v, self.dt, cu, self.lens(), **self.args())
        return k, v

    def rows(self, k, v):
        """What the rows stand for once stored: lists per sequence of [L, H, d] float64."""
        out = []
        for x in (f64(k), f64(v)):
            if self.kind != "bf16":
                x = x.copy()
                for i in np.ndindex(x.shape[:2]):
                    c, s = oracle.cache_encode(x[i], self.kind)
                    x[i] = c * s
            out.append(np.split(x, np.cumsum(self.kv)[:-1]))
        return list(zip(*out))


def offsets(n):
    return torch.tensor(np.concatenate([[0], np.cumsum(n)]), dtype=torch.int32, device=DEV)


def check(o, lse, q, rows, kv, new, causal, row0=0, scale=None, floor=None):
    """Every row of o against the oracle; floor: absolute error of a row's sum, [H] per sequence."""
    Hq, d = q.shape[1:]
    o, lse, q = f64(o), f64(lse), f64(q)
    at = row0
    for s_, ((k, v), L, n) in enumerate(zip(rows, kv, new)):
        H = k.shape[1]
        G = Hq // H
        for i in range(n):
            vis = L - n + i + 1 if causal else L
            for h in range(H):
                qq = q[at + i, h * G:(h + 1) * G]
                ref, rl = oracle.cache_attention(qq, k[:, h], v[:, h], vis, scale)
                mag, _ = oracle.cache_attention(qq, k[:, h], np.abs(v[:, h]), vis, scale)
                sc = d ** -0.5 if scale is None else scale
                ds = 2.0 ** -24 * d * (np.abs(qq) @ np.abs(k[:vis, h]).T).max() * sc if vis > 0 else 0.0
                got = o[at + i, h * G:(h + 1) * G]
                bound = (2.0 ** -8 + 2.0 ** -11 + 2 * ds) * mag + 2.0 ** -8 * np.abs(ref)
                if floor is not None:
                    bound = bound + floor[s_][h]
                assert np.isfinite(got).all(), (at + i, h, vis)
                worst = float((np.abs(got - ref) - bound).max())
                assert worst <= 0, (at + i, h, vis, worst, float(np.abs(got - ref).max()))
                gl = lse[at + i, h * G:(h + 1) * G]
                if vis <= 0:
                    assert (gl == -np.inf).all()
                else:
                    # sum of weights: the exponential's error; the score's error
                    worst = float(np.abs(gl - rl).max())
                    assert worst <= 2.0 ** -11 + ds + 2.0 ** -22 * float(np.abs(rl).max()), (at + i, h, vis, worst)
        at += n


@pytest.mark.parametrize("kind", list(KINDS))
@pytest.mark.parametrize("d,page,H", [(64, 16, 3), (128, 48, 1), (128, 64, 8)])
def test_write_and_read(cuda_lib, kind, d, page, H):
    sa = cuda_lib
    kv = [1, 0, page, 2 * page + 5, 333]
    c = Cache(kind, kv, H, d, page)
    before = c.k.view(torch.uint8).clone()
    k, v = c.fill(sa, 7)
    k[3] = 0
    v[4] = 0
    sa.sa_cache_write(k, v, c.k, c.v, c.dt, offsets(kv), c.lens(), **c.args())
    kr, vr = sa.sa_cache_read(c.k, c.v, c.dt, offsets(kv), sum(kv), **c.args())
    rows = c.rows(k, v)
    for got, i in ((kr, 0), (vr, 1)):
        want = np.concatenate([r[i] for r in rows])
        # code * scale is formed in fp32 and rounded to bf16
        want = torch.from_numpy(want.astype(np.float32)).to(torch.bfloat16)
        assert torch.equal(got.cpu(), want)
    # slots of no position are untouched
    taken = np.zeros((c.P, page), dtype=bool)
    for s, L in enumerate(kv):
        for p in range(L):
            taken[oracle.cache_slot(c.table[s], page, p, c.P)] = True
    free = torch.from_numpy(~taken).to(DEV)
    now = c.k.view(torch.uint8)
    assert torch.equal(now.transpose(1, 2)[free], before.transpose(1, 2)[free])
    sa.sa_device_status()


def test_write_strided_offset_rows_and_bad_pages(cuda_lib):
    """Head-major operands, rows before and behind the sequences, a chunk behind
    earlier tokens, table entries that name no page, and a read into strided views."""
    sa = cuda_lib
    kv, new, page, H, d = [40, 100], [7, 33], 16, 2, 128
    c = Cache("e4m3", kv, H, d, page)
    c.table[1, 5] = c.P + 7                     # positions 80..95 of sequence 1 have no page
    c.table[1, 6] = -3                          # and 96..111
    c.dt = torch.from_numpy(c.table).to(DEV)
    g = torch.Generator(device=DEV).manual_seed(3)
    k, v = (torch.randn(H, 50, d + 8, generator=g, device=DEV).to(torch.bfloat16)[..., :d].transpose(0, 1) for _ in range(2))
    cu = torch.tensor([3, 10, 43], dtype=torch.int32, device=DEV)
    sa.sa_cache_write(k, v, c.k, c.v, c.dt, cu, c.lens(), **c.args())
    out = tuple(torch.full((H, 150, d), -1.0, dtype=torch.bfloat16, device=DEV).transpose(0, 1) for _ in range(2))
    sa.sa_cache_read(c.k, c.v, c.dt, torch.tensor([2, 42, 142], dtype=torch.int32, device=DEV), 150, out=out, **c.args())
    for got, x in zip(out, (k, v)):
        assert (got[:2] == -1).all() and (got[142:] == -1).all()
        got, x = f64(got), f64(x)
        for s, (L, n, r0, w0) in enumerate(((40, 7, 3, 2), (100, 33, 10, 42))):
            for p in range(L - n, L):
                slot = oracle.cache_slot(c.table[s], page, p, c.P)
                for h in range(H):
                    want = np.zeros(d)
                    if slot is not None:
                        codes, scale = oracle.cache_encode(x[r0 + p - (L - n), h], "e4m3")
                        want = f64(torch.from_numpy((codes * scale).astype(np.float32)).to(torch.bfloat16))
                    assert (got[w0 + p, h] == want).all(), (s, p, h)
    sa.sa_device_status()


def test_tiny_rows_quantise_without_nan(cuda_lib):
    sa = cuda_lib
    for kind in ("e4m3", "int8"):
        c = Cache(kind, [4], 1, 64, 16)
        k = torch.zeros(4, 1, 64, device=DEV)
        k[0, 0, 3] = 1e-38
        k[1, 0, 5] = 1e-40                          # subnormal
        k = k.to(torch.bfloat16)
        sa.sa_cache_write(k, k, c.k, c.v, c.dt, offsets([4]), c.lens(), **c.args())
        kr, _ = sa.sa_cache_read(c.k, c.v, c.dt, offsets([4]), 4, **c.args())
        assert torch.isfinite(kr).all() and (kr[2:] == 0).all()
        # 1e-38 is 0.85 steps of the smallest scale, 2^-126: half a step of int8 is 2^-127, E4M3 has a relative half
        # step of 2^-4; the result is rounded to bf16 once more
        half = 2.0 ** -127 if kind == "int8" else 2.0 ** -4 * 1e-38
        assert abs(float(kr[0, 0, 3]) - float(k[0, 0, 3])) <= half + 2.0 ** -8 * 1.2e-38


@pytest.mark.parametrize("kind", list(KINDS))
@pytest.mark.parametrize("H,G,d,page,kv,new,causal", [
    (2, 1, 128, 64, [1], [1], True),                                   # one token, one key
    (1, 4, 128, 64, [700], [1], True),                                 # a token over several tiles
    (2, 8, 64, 16, [129, 1, 64, 300], [1, 1, 1, 1], True),             # a batch of tokens, ragged
    (3, 3, 128, 48, [200, 5, 333], [2, 5, 130], True),                 # odd group, pages across tiles, chunks
    (1, 7, 64, 256, [600, 257], [40, 257], False),                     # a group that does not divide a tile
    (2, 1, 128, 128, [450], [300], True),                              # several query tiles
    (1, 128, 64, 32, [150], [3], True),                                # one token fills a tile
    (2, 2, 128, 32, [0, 90, 4, 0], [0, 3, 9, 2], True),                # empty sequences, rows that see nothing
])
def test_attention(cuda_lib, kind, H, G, d, page, kv, new, causal):
    sa = cuda_lib
    c = Cache(kind, kv, H, d, page, seed=1)
    k, v = c.fill(sa, 11)
    g = torch.Generator(device=DEV).manual_seed(5)
    q = torch.randn(sum(new), H * G, d, generator=g, device=DEV).to(torch.bfloat16)
    rows = c.rows(k, v)
    for max_q in (max(new), 0):
        o, lse = sa.sa_cache_attn(q, c.k, c.v, c.dt, offsets(new), c.lens(), max_q, causal=causal, want_lse=True, **c.args())
        check(o, lse, q, rows, kv, new, causal)
    o2, lse2 = sa.sa_cache_attn(q, c.k, c.v, c.dt, offsets(new), c.lens(), 0, causal=causal, want_lse=True, **c.args())
    assert torch.equal(o, o2) and torch.equal(lse, lse2)               # the same call again: the same bits
    sa.sa_device_status()


def test_attention_long_cache_and_peaks(cuda_lib):
    """A token over many tiles (so that several blocks share it) whose scores grow
    along the cache: the running maximum rises again and again."""
    sa = cuda_lib
    for kind in KINDS:
        kv, page, H, G, d = [5000, 3001], 64, 2, 2, 128
        c = Cache(kind, kv, H, d, page, seed=2)
        g = torch.Generator(device=DEV).manual_seed(6)
        n = sum(kv)
        u = torch.randn(d, generator=g, device=DEV)
        u /= u.norm()
        ramp = torch.cat([torch.linspace(0, 60, L, device=DEV) for L in kv])
        k = (torch.randn(n, H, d, generator=g, device=DEV) + ramp[:, None, None] * u).to(torch.bfloat16)
        v = torch.randn(n, H, d, generator=g, device=DEV).to(torch.bfloat16)
        sa.sa_cache_write(k, v, c.k, c.v, c.dt, offsets(kv), c.lens(), **c.args())
        q = (torch.randn(2, H * G, d, generator=g, device=DEV) * 0.5 + 8 * u).to(torch.bfloat16)
        o, lse = sa.sa_cache_attn(q, c.k, c.v, c.dt, offsets([1, 1]), c.lens(), 1, want_lse=True, **c.args())
        check(o, lse, q, c.rows(k, v), kv, [1, 1], True)
    sa.sa_device_status()


def test_attention_strides_padding_and_scale(cuda_lib):
    """Head-major q and out, rows of no sequence left as they were, a given scale,
    lengths beyond the table clamped to it."""
    sa = cuda_lib
    kv, new, page, H, G, d = [70, 200], [9, 20], 16, 2, 3, 64
    c = Cache("bf16", kv, H, d, page, seed=4, extra_width=0)
    k, v = c.fill(sa, 12)
    g = torch.Generator(device=DEV).manual_seed(8)
    q = torch.randn(H * G, 40, d + 16, generator=g, device=DEV).to(torch.bfloat16)[..., 8:8 + d].transpose(0, 1)
    out = torch.full((H * G, 40, d), 9.0, dtype=torch.bfloat16, device=DEV).transpose(0, 1)
    cu = torch.tensor([4, 13, 33], dtype=torch.int32, device=DEV)
    o, lse = sa.sa_cache_attn(q, c.k, c.v, c.dt, cu, c.lens(), 20, scale=0.2, want_lse=True, out=out)
    assert o is out and (out[:4] == 9).all() and (out[33:] == 9).all()
    check(out, lse, q, c.rows(k, v), kv, new, True, row0=4, scale=0.2)
    # a length behind the table counts as the table's: 208 positions, the last 8 of them in no written slot
    c.v[c.table[1, 12], :, 8:] = 0
    c.k[c.table[1, 12], :, 8:] = 0
    o2 = sa.sa_cache_attn(q, c.k, c.v, c.dt, cu, c.lens([70, 10 ** 6]), 20, causal=False, scale=0.2)
    o3 = sa.sa_cache_attn(q, c.k, c.v, c.dt, cu, c.lens([70, 208]), 20, causal=False, scale=0.2)
    assert torch.equal(o2[4:33], o3[4:33]) and torch.isfinite(o2[4:33]).all()
    # a table entry that names no page holds zeros
    bad = c.dt.clone()
    bad[1, 3] = c.P
    o4 = sa.sa_cache_attn(q, c.k, c.v, bad, cu, c.lens(), 20, scale=0.2)
    bad[1, 3] = -1
    o5 = sa.sa_cache_attn(q, c.k, c.v, bad, cu, c.lens(), 20, scale=0.2)
    rows = c.rows(k, v)
    for x in rows[1]:
        x[48:64] = 0
    _, lse4 = sa.sa_cache_attn(q, c.k, c.v, bad, cu, c.lens(), 20, scale=0.2, want_lse=True)
    assert torch.equal(o4[4:33], o5[4:33])
    check(o4, lse4, q, rows, kv, new, True, row0=4, scale=0.2)
    sa.sa_device_status()


def test_attention_captured_replayed_and_on_another_stream(cuda_lib):
    """A captured step replays with other lengths and fewer rows; eager calls in
    between, with their own workspace, change nothing."""
    sa = cuda_lib
    kv, page, H, G, d = [130, 260, 64], 64, 2, 4, 128
    c = Cache("int8", kv, H, d, page, seed=9)
    k, v = c.fill(sa, 13)
    rows = c.rows(k, v)
    g = torch.Generator(device=DEV).manual_seed(10)
    q = torch.randn(3, H * G, d, generator=g, device=DEV).to(torch.bfloat16)
    cu, lens = offsets([1, 1, 1]), c.lens()
    ws = torch.empty(sa.load().sa_cache_attn_workspace_size(d), dtype=torch.uint8, device=DEV)
    out = torch.zeros_like(q)
    run = lambda: sa.sa_cache_attn(q, c.k, c.v, c.dt, cu, lens, 1, out=out, workspace=ws, **c.args())
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    eager = sa.sa_cache_attn(q, c.k, c.v, c.dt, cu, lens, 1, **c.args())
    graph.replay()
    assert torch.equal(out, eager)
    lens.copy_(torch.tensor([100, 1, 33], dtype=torch.int32))
    cu.copy_(torch.tensor([0, 1, 2, 2], dtype=torch.int32))
    out.fill_(5)
    graph.replay()
    _, lse = sa.sa_cache_attn(q, c.k, c.v, c.dt, cu, lens, 1, want_lse=True, **c.args())
    check(out, lse, q, [(k_[:n], v_[:n]) for (k_, v_), n in zip(rows[:2], (100, 1))], [100, 1], [1, 1], True)
    assert (out[2] == 5).all()
    sa.sa_device_status()


@pytest.mark.parametrize("kind", list(KINDS))
def test_attention_of_many_sequences_with_a_used_workspace(cuda_lib, kind):
    """More sequences than threads, a few keys each, some empty; the workspace
    holds NaN."""
    sa = cuda_lib
    rng = np.random.default_rng(15)
    kv = [int(x) for x in rng.integers(0, 40, 1100)]
    new = [min(1, L) for L in kv]
    H, G, d = 1, 3, 64
    c = Cache(kind, kv, H, d, 16, seed=16)
    k, v = c.fill(sa, 17)
    g = torch.Generator(device=DEV).manual_seed(18)
    q = torch.randn(sum(new), H * G, d, generator=g, device=DEV).to(torch.bfloat16)
    ws = torch.full((sa.load().sa_cache_attn_workspace_size(d),), 255, dtype=torch.uint8, device=DEV)
    o, lse = sa.sa_cache_attn(q, c.k, c.v, c.dt, offsets(new), c.lens(), 1, want_lse=True, workspace=ws, **c.args())
    check(o, lse, q, c.rows(k, v), kv, new, True)
    sa.sa_device_status()


@pytest.mark.parametrize("kind", ["e4m3", "int8"])
def test_attention_of_values_and_queries_of_far_sizes(cuda_lib, kind):
    """Value rows between 2^-12 and 2^3, rows of zeros (whose scale is 1), query
    channels between 2^-20 and 1. Weights times scales are fp16 numbers in units of
    C / 2^7, C the power of two at or above the largest scale: half a step of fp16's
    subnormals, 2^-25, is 2^-32 C, which meets a code of at most M; the sum of the
    weights is at least 1. So a sum over L keys is off by up to 2^-32 C M L more than
    the relative bound says."""
    sa = cuda_lib
    kv, new, H, G, d = [300, 77], [5, 77], 2, 2, 128
    c = Cache(kind, kv, H, d, 32, seed=20)
    g = torch.Generator(device=DEV).manual_seed(21)
    n = sum(kv)
    k = torch.randn(n, H, d, generator=g, device=DEV).to(torch.bfloat16)
    v = torch.randn(n, H, d, generator=g, device=DEV) * torch.exp2(torch.randint(-12, 4, (n, H, 1), generator=g, device=DEV).float())
    v[::7] = 0
    v = v.to(torch.bfloat16)
    sa.sa_cache_write(k, v, c.k, c.v, c.dt, offsets(kv), c.lens(), **c.args())
    q = torch.randn(sum(new), H * G, d, generator=g, device=DEV) * torch.exp2(-torch.randint(0, 21, (d,), generator=g, device=DEV).float())
    q[3] *= 1e-30
    q[4] *= 1e30
    q[4] *= 1e-28
    q[6] = 0
    q = q.to(torch.bfloat16)
    o, lse = sa.sa_cache_attn(q, c.k, c.v, c.dt, offsets(new), c.lens(), want_lse=True, **c.args())
    M = oracle.stateful.CACHE_MAX[kind]
    amax = np.abs(f64(v)).max(-1)
    scales = np.split(np.where(amax > 0, amax / M, 1.0), np.cumsum(kv)[:-1])
    floor = [2.0 ** -32 * 2.0 ** np.ceil(np.log2(s.max(0))) * M * L for s, L in zip(scales, kv)]
    check(o, lse, q, c.rows(k, v), kv, new, True, floor=floor)
    sa.sa_device_status()


@pytest.mark.parametrize("kind", list(KINDS))
def test_nan_stays_nan(cuda_lib, kind):
    """A NaN in a query row reaches that row and no other; a row written with a NaN
    is read as NaN, its neighbours as they are."""
    sa = cuda_lib
    kv, H, G, d = [200], 2, 2, 64
    c = Cache(kind, kv, H, d, 16, seed=22)
    k, v = c.fill(sa, 23)
    g = torch.Generator(device=DEV).manual_seed(24)
    q = torch.randn(9, H * G, d, generator=g, device=DEV).to(torch.bfloat16)
    ref = sa.sa_cache_attn(q, c.k, c.v, c.dt, offsets([9]), c.lens(), **c.args())
    q[2, 1, 5] = float("nan")
    o, lse = sa.sa_cache_attn(q, c.k, c.v, c.dt, offsets([9]), c.lens(), want_lse=True, **c.args())
    assert torch.isnan(o[2, 1]).all() and torch.isnan(lse[2, 1])
    keep = torch.ones(9, H * G, dtype=torch.bool, device=DEV)
    keep[2, 1] = False
    assert torch.equal(o[keep], ref[keep])
    k[7, 1, 3] = float("nan")
    sa.sa_cache_write(k, v, c.k, c.v, c.dt, offsets(kv), c.lens(), **c.args())
    kr, vr = sa.sa_cache_read(c.k, c.v, c.dt, offsets(kv), 200, **c.args())
    bad = torch.isnan(kr).any(-1)
    assert bad[7, 1] and int(bad.sum()) == 1 and torch.isfinite(vr).all()


def test_attention_on_two_streams(cuda_lib):
    """Two calls at once, each with its own workspace and outputs."""
    sa = cuda_lib
    H, G, d, page = 4, 2, 128, 64
    cs, qs, refs = [], [], []
    for i, kind in enumerate(("bf16", "e4m3")):
        c = Cache(kind, [3000, 1500], H, d, page, seed=30 + i)
        c.fill(sa, 32 + i)
        g = torch.Generator(device=DEV).manual_seed(34 + i)
        q = torch.randn(2, H * G, d, generator=g, device=DEV).to(torch.bfloat16)
        cs.append((c, offsets([1, 1]), c.lens()))
        qs.append(q)
        refs.append(sa.sa_cache_attn(q, c.k, c.v, c.dt, cs[-1][1], cs[-1][2], 1, **c.args()))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cs]
    outs = [[], []]
    for _ in range(20):
        for i, (c, cu, lens) in enumerate(cs):
            with torch.cuda.stream(streams[i]):
                outs[i].append(sa.sa_cache_attn(qs[i], c.k, c.v, c.dt, cu, lens, 1, **c.args()))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(o, refs[i]) for o in outs[i])
    sa.sa_device_status()


@pytest.mark.parametrize("kind", list(KINDS))
def test_nan_keys_reach_the_rows_that_see_them(cuda_lib, kind):
    """Eight neighbouring keys in turn (columns that different exponentials and
    lanes handle): rows that see the key are NaN, the others as without it."""
    sa = cuda_lib
    kv, n, H, G, d = [150], 40, 1, 2, 64
    c = Cache(kind, kv, H, d, 32, seed=40)
    k, v = c.fill(sa, 41)
    g = torch.Generator(device=DEV).manual_seed(42)
    q = torch.randn(n, H * G, d, generator=g, device=DEV).to(torch.bfloat16)
    ref = sa.sa_cache_attn(q, c.k, c.v, c.dt, offsets([n]), c.lens(), **c.args())
    for key in range(120, 128):
        bad = k.clone()
        bad[key, 0, 9] = float("nan")
        sa.sa_cache_write(bad, v, c.k, c.v, c.dt, offsets(kv), c.lens(), **c.args())
        o, lse = sa.sa_cache_attn(q, c.k, c.v, c.dt, offsets([n]), c.lens(), want_lse=True, **c.args())
        first = key - (kv[0] - n)                       # the first row that sees the key
        assert torch.isnan(o[first:]).all() and torch.isnan(lse[first:]).all(), key
        assert torch.equal(o[:first], ref[:first]), key
    sa.sa_device_status()

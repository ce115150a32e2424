"""Host-side refusals of the cache, its attention and the decayed linear
attention: by the binding (shapes, types, layouts, devices) and by the C ABI
before any launch. No GPU needed."""
import ctypes

import pytest
import torch

import block_sparse_attention_softmax_b200 as sa
from block_sparse_attention_softmax_b200 import build as sa_build

P = ctypes.c_void_p
S, H, d, page, n_pages, width = 2, 2, 64, 16, 6, 3


@pytest.fixture(scope="module")
def lib():
    sa_build.build()
    return sa.load()


def _bf16(*shape):
    return torch.zeros(*shape, dtype=torch.bfloat16)


def _cache(dtype=torch.bfloat16):
    c = dict(k_cache=torch.zeros(n_pages, H, page, d, dtype=dtype), v_cache=torch.zeros(n_pages, H, page, d, dtype=dtype),
             table=torch.zeros(S, width, dtype=torch.int32), cu_q=torch.zeros(S + 1, dtype=torch.int32),
             kv_len=torch.zeros(S, dtype=torch.int32))
    if dtype != torch.bfloat16:
        c.update(k_scale=torch.ones(n_pages, H, page), v_scale=torch.ones(n_pages, H, page))
    return c


def _refused(match, fn, *a, **kw):
    with pytest.raises(ValueError, match=match):
        fn(*a, **kw)


def test_binding_refuses_cache_operands():
    x = _bf16(5, H, d)
    c = _cache()
    _refused("CUDA tensors", sa.sa_cache_write, x, x, **c)
    _refused("k: dtype", sa.sa_cache_write, x.float(), x, **c)
    _refused("k: shape", sa.sa_cache_write, _bf16(5, H + 1, d), x, **c)
    _refused("v has 4 rows", sa.sa_cache_write, x, x[:4], **c)
    _refused("last dimension", sa.sa_cache_write, _bf16(5, d, H).transpose(1, 2), x, **c)
    _refused("multiples of 8", sa.sa_cache_write, _bf16(5, H, d + 4)[..., :d], x, **c)
    _refused("multiples of 8", sa.sa_cache_write, _bf16(5, 1, d).expand(5, H, d), x, **c)
    _refused("k_cache: dtype", sa.sa_cache_write, x, x, **{**c, "k_cache": c["k_cache"].half()})
    _refused("v_cache: dtype", sa.sa_cache_write, x, x, **{**c, "v_cache": c["v_cache"].float()})
    _refused("v_cache: shape", sa.sa_cache_write, x, x, **{**c, "v_cache": c["v_cache"][:-1]})
    _refused("no scales", sa.sa_cache_write, x, x, k_scale=torch.ones(n_pages, H, page), **c)
    _refused("k_scale is required", sa.sa_cache_write, x, x, **{**_cache(torch.int8), "k_scale": None})
    _refused("v_scale: shape", sa.sa_cache_write, x, x, **{**_cache(torch.int8), "v_scale": torch.ones(n_pages, H)})
    _refused("table: dtype", sa.sa_cache_write, x, x, **{**c, "table": c["table"].long()})
    _refused("cu_q: shape", sa.sa_cache_write, x, x, **{**c, "cu_q": c["cu_q"][:-1]})
    _refused("kv_len: shape", sa.sa_cache_write, x, x, **{**c, "kv_len": c["cu_q"]})


def test_binding_refuses_read_and_attention_operands():
    c = _cache(torch.float8_e4m3fn)
    read = {n: c[n] for n in ("k_cache", "v_cache", "table", "k_scale", "v_scale")}
    _refused("n_rows", sa.sa_cache_read, cu_r=c["cu_q"], n_rows=-1, **read)
    _refused("expected 7", sa.sa_cache_read, cu_r=c["cu_q"], n_rows=7, out=(_bf16(6, H, d), _bf16(7, H, d)), **read)
    _refused("CUDA tensors", sa.sa_cache_read, cu_r=c["cu_q"], n_rows=7, **read)
    _refused("no multiple", sa.sa_cache_attn, _bf16(4, 3, d), **c)
    _refused("q: shape", sa.sa_cache_attn, _bf16(4, 2 * H, 128), **c)
    _refused("rows, heads, d", sa.sa_cache_attn, _bf16(1, 4, 2 * H, d), **c)
    _refused("out: 3 rows", sa.sa_cache_attn, _bf16(4, 2 * H, d), out=_bf16(3, 2 * H, d), **c)
    _refused("CUDA tensors", sa.sa_cache_attn, _bf16(4, 2 * H, d), **c)


def test_binding_refuses_decay_operands():
    B, N = 1, 10
    q = _bf16(B, H, N, d)
    ld, st = torch.zeros(H), torch.zeros(B, H, d, d)
    _refused("CUDA tensors", sa.sa_decay_attn_fwd, q, q, q, ld)
    _refused("log_decay: shape", sa.sa_decay_attn_fwd, q, q, q, torch.zeros(H + 1))
    _refused("log_decay: dtype", sa.sa_decay_attn_fwd, q, q, q, ld.double())
    _refused("state: shape", sa.sa_decay_attn_fwd, q, q, q, ld, state=st[0])
    _refused("k: shape", sa.sa_decay_attn_fwd, q, q[:, :, :-1], q, ld)
    _refused("contiguous", sa.sa_decay_attn_fwd, q.transpose(1, 2).contiguous().transpose(1, 2), q, q, ld)
    _refused("dout: dtype", sa.sa_decay_attn_bwd, q, q, q, ld, q.float())
    _refused("dstate: dtype", sa.sa_decay_attn_bwd, q, q, q, ld, q, dstate=st.double())
    t = _bf16(B, H, d)
    _refused("state: shape", sa.sa_decay_attn_step, t, t, t, ld, st[..., :-1])
    _refused(r"\[B, H, d\]", sa.sa_decay_attn_step, q, t, t, ld, st)
    _refused("CUDA tensors", sa.sa_decay_attn_step, t, t, t, ld, st)


def test_abi_refuses_cache_arguments_before_launch(lib):
    f, o = P(0x1000), P(0x2000)
    big = 1 << 40

    def write(k=f, st=128, sh=64, n_rows=4, n_seqs=2, Hkv=2, dd=64, kind=0, pages=8, pg=16, w=4, table=f, kc=f, ks=None):
        return lib.sa_cache_write(k, f, st, sh, 128, 64, n_rows, n_seqs, Hkv, dd, kind, pages, pg, w, table, f, f, kc, f, ks, ks,
                                  None)

    assert write(k=None) == -1 and write(table=None) == -1 and write(kc=None) == -1
    assert write(n_rows=-1) == -1 and write(n_seqs=0) == -1 and write(pages=0) == -1 and write(w=0) == -1
    assert write(kind=3) == -1 and write(kind=1) == -1 and write(kind=0, ks=f) == -1
    assert write(dd=96) == -2 and write(pg=24) == -2 and write(Hkv=65536) == -2
    assert write(pg=1 << 20, w=1 << 12) == -2 and write(pages=1 << 30, Hkv=64, pg=128) == -2
    assert write(st=60) == -1 and write(sh=68) == -1 and write(st=-128) == -1
    assert b"strides" in lib.sa_last_error()
    assert write(k=P(0x1008)) == -3 and write(table=P(0x1002)) == -3 and write(kc=P(0x1001)) == -3
    assert lib.sa_cache_read(f, f, None, None, 4, 2, 2, 64, 2, 8, 16, 4, f, f, 128, 64, 128, 64, f, f, None) == -1
    assert lib.sa_cache_read(f, f, None, None, 4, 2, 2, 64, 0, 8, 16, 4, f, None, 128, 64, 128, 64, f, f, None) == -1

    def attn(q=f, out=o, Hq=4, Hkv=2, max_q=1, scale=0.0, lse=None, ws=f, nws=big, n_rows=4, ost=256):
        return lib.sa_cache_attn(q, 256, 64, n_rows, 2, Hq, Hkv, 64, 0, 8, 16, 4, f, f, f, max_q, f, f, None, None, 1, scale, out,
                                 ost, 64, lse, ws, nws, None)

    assert attn(q=None) == -1 and attn(out=f) == -1 and attn(Hq=3) == -1 and attn(Hq=0) == -1
    assert attn(Hq=258) == -2 and attn(max_q=-1) == -1 and attn(scale=float("nan")) == -1
    assert attn(scale=1e-50) == -1 and attn(scale=1e39) == -1 and attn(scale=float("inf")) == -1   # not an fp32 number
    assert attn(lse=P(0x1002)) == -3 and attn(ost=12) == -1
    assert attn(n_rows=0) == 0                       # nothing to do, nothing launched
    assert lib.sa_cache_attn_workspace_size(96) == 0


def test_abi_refuses_decay_arguments_before_launch(lib):
    f, o, z = P(0x1000), P(0x2000), P(0x3000)
    big = 1 << 40
    fwd = lambda q=f, ld=f, N=8, dd=64, sc=0.0, s0=None, out=o, s1=None: lib.sa_decay_attn_fwd(
        q, f, f, ld, 1, 2, N, dd, sc, s0, out, s1, f, big, None)
    assert fwd(q=None) == -1 and fwd(N=0) == -1 and fwd(dd=32) == -2 and fwd(sc=float("nan")) == -1
    assert fwd(sc=1e-50) == -1 and fwd(N=0x7FFFFFFF) == -2
    assert lib.sa_decay_attn_workspace_size(1, 2, 2000000, 64) > 0     # no limit on a block mask applies
    assert fwd(out=f) == -1 and fwd(s0=z, s1=z) == -1 and fwd(q=P(0x1004)) == -3 and fwd(ld=P(0x1002)) == -3
    bwd = lambda dq=o, dk=z, dv=P(0x4000), ds=None, s0=None: lib.sa_decay_attn_bwd(
        f, f, f, f, f, 1, 2, 8, 64, 0.0, s0, None, dq, dk, dv, ds, f, big, None)
    assert bwd(dq=None) == -1 and bwd(dk=o) == -1 and bwd(dv=f) == -1 and bwd(ds=P(0x5000), s0=P(0x5000)) == -1
    step = lambda s=f, out=o, so=z, B=1: lib.sa_decay_attn_step(f, f, f, f, s, B, 2, 64, 0.0, out, so, None)
    assert step(s=None) == -1 and step(out=f) == -1 and step(B=0) == -1
    assert step(so=P(0x1000 + 2 * 64 * 64 * 4 - 16)) == -1    # overlaps the state without being it
    assert b"overlap" in lib.sa_last_error()


def test_abi_refuses_overlapping_ranges(lib):
    """Outputs that begin inside an input or another output, not only at its start."""
    big = 1 << 40
    nx, ns = 2 * 8 * 64 * 2, 2 * 64 * 64 * 4            # [1, 2, 8, 64] bf16, [1, 2, 64, 64] fp32
    at = lambda i, off=0: P(0x100000 * (i + 1) + off)
    names = ("q", "k", "v", "ld", "s0", "out", "s1")
    where = lambda names, kw: {n: kw.get(n, at(i)) for i, n in enumerate(names)}

    def fwd(**kw):
        x = where(names, kw)
        return lib.sa_decay_attn_fwd(x["q"], x["k"], x["v"], x["ld"], 1, 2, 8, 64, 0.0, x["s0"], x["out"], x["s1"], P(0x4), big, None)

    # (a workspace that is not aligned is what a call that overlaps nothing is refused for: nothing is launched here)
    assert fwd() == -3
    for i in (0, 1, 2):
        assert fwd(out=at(i, nx - 16)) == -1 and fwd(out=at(i, nx)) == -3
        assert fwd(s1=at(i, nx - 16)) == -1
    assert fwd(q=at(5, nx - 16)) == -1 and fwd(ld=at(5, 16)) == -1 and fwd(s0=at(6, ns - 16)) == -1 and fwd(s0=at(6, ns)) == -3
    assert fwd(s1=at(5, nx - 16)) == -1 and fwd(s1=at(4)) == -1
    assert b"overlap" in lib.sa_last_error()

    bnames = ("q", "k", "v", "ld", "do", "s0", "ds1", "dq", "dk", "dv", "ds0")

    def bwd(**kw):
        x = where(bnames, kw)
        return lib.sa_decay_attn_bwd(x["q"], x["k"], x["v"], x["ld"], x["do"], 1, 2, 8, 64, 0.0, x["s0"], x["ds1"], x["dq"], x["dk"],
                                     x["dv"], x["ds0"], P(0x4), big, None)

    assert bwd() == -3
    for i in (0, 1, 2, 4):
        assert all(bwd(**{n: at(i, nx - 16)}) == -1 for n in ("dq", "dk", "dv", "ds0"))
    for i in (5, 6):
        assert all(bwd(**{n: at(i, ns - 16)}) == -1 for n in ("dq", "dk", "dv", "ds0"))
    assert bwd(dk=at(7, nx - 16)) == -1 and bwd(dv=at(8, 16)) == -1 and bwd(ds0=at(9, nx - 16)) == -1 and bwd(dk=at(7, nx)) == -3

    n1 = 2 * 64 * 2
    snames = ("q", "k", "v", "ld", "s", "out", "so")

    def step(**kw):
        x = where(snames, kw)
        return lib.sa_decay_attn_step(x["q"], x["k"], x["v"], x["ld"], x["s"], 1, 2, 64, 0.0, x["out"], x["so"], None)

    assert all(step(out=at(i, n1 - 16)) == -1 and step(so=at(i, n1 - 16)) == -1 for i in (0, 1, 2))
    assert step(out=at(4, ns - 16)) == -1 and step(so=at(4, 16)) == -1 and step(so=at(5, 16)) == -1

    def attn(q, o, qst=256, qsh=64, ost=256, osh=64, n_rows=4):
        return lib.sa_cache_attn(q, qst, qsh, n_rows, 2, 4, 2, 64, 0, 8, 16, 4, at(3), at(4), at(5), 1, at(6), at(7), None, None, 1, 0.0,
                                 o, ost, osh, None, P(0x10), 0, None)

    # (-6: no workspace, which is asked for last)
    assert attn(at(0), at(1)) == -6 and attn(at(0), at(0)) == -1
    assert attn(at(0), at(0, 4 * 256 * 2 - 16)) == -1 and attn(at(0), at(0, 4 * 256 * 2)) == -6
    assert attn(at(0, 16), at(0)) == -1
    # parts of one packed [rows, 12, 64] buffer: apart where their heads are
    assert attn(at(0), at(0, 4 * 64 * 2), qst=768, ost=768) == -6
    assert attn(at(0), at(0, 8 * 64 * 2), qst=768, ost=768) == -6
    assert attn(at(0, 8 * 64 * 2), at(0), qst=768, ost=768) == -6
    assert attn(at(0), at(0, 3 * 64 * 2), qst=768, ost=768) == -1
    assert attn(at(0), at(0, 768 * 2), qst=768, ost=768) == -1
    assert attn(at(0, 3 * 768 * 2 + 16), at(0), qst=768, ost=768) == -1
    assert attn(at(0, 3 * 768 * 2 + 4 * 64 * 2), at(0), qst=768, ost=768) == -6
    # head-major, and a dense one inside the other's range
    assert attn(at(0), at(0, 64 * 2), qst=128, qsh=1024, ost=128, osh=1024) == -6
    assert attn(at(0), at(0, 64), qst=128, qsh=1024, ost=128, osh=1024) == -1
    assert attn(at(0), at(0, 512), qst=768, ost=256) == -1
    # a dense one in the gap between tokens of the other, and on its rows
    for a, b in (("q", "o"), ("o", "q")):
        kw = {a + "st": 4096}
        for off, want in ((512, -6), (256, -6), (255 // 8 * 8, -1), (4096 - 1024, -6), (4096 - 1016, -1), (3 * 4096 + 256, -6),
                          (3 * 4096 + 248, -1)):
            x = {a: at(0), b: at(0, 2 * off)}
            assert attn(x["q"], x["o"], **kw) == want, (a, off)
        assert attn(at(0, 2 * 1024) if a == "q" else at(0), at(0, 2 * 1024) if a == "o" else at(0), **kw) == -6
        assert attn(at(0, 2 * 1016) if a == "q" else at(0), at(0, 2 * 1016) if a == "o" else at(0), **kw) == -1

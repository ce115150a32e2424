"""The stateful calls used together: a sequence enters a cache chunk by chunk and
each chunk attends to what the cache holds, while the decayed linear branch hands
its state on; then tokens are generated one by one from a captured step.

Each call's own error is bounded in its own test; here both sides of a comparison
come from the library, so twice the bound of one of them covers the difference."""
import numpy as np
import pytest
import torch

import oracle

pytestmark = pytest.mark.gpu

DEV = "cuda"
f64 = oracle.as_f64
KINDS = {"bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn, "int8": torch.int8}


def _i32(*x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def _cache(kind, P, H, page, d):
    c = dict(k_cache=torch.zeros(P, H, page, d, device=DEV).to(KINDS[kind]), v_cache=torch.zeros(P, H, page, d, device=DEV).to(KINDS[kind]))
    if kind != "bf16":
        c.update(k_scale=torch.ones(P, H, page, device=DEV), v_scale=torch.ones(P, H, page, device=DEV))
    return c


@pytest.mark.parametrize("kind", list(KINDS))
def test_chunks_then_tokens_then_a_read(cuda_lib, kind):
    sa = cuda_lib
    H, G, d, page, N, prompt = 2, 2, 64, 32, 420, 400
    g = torch.Generator(device=DEV).manual_seed(3)
    q = torch.randn(N, H * G, d, generator=g, device=DEV).to(torch.bfloat16)
    k, v = (torch.randn(N, H, d, generator=g, device=DEV).to(torch.bfloat16) for _ in range(2))
    P = -(-N // page)
    c = _cache(kind, P, H, page, d)
    table = torch.from_numpy(np.random.default_rng(4).permutation(P).astype(np.int32)).to(DEV)[None]
    outs = []
    for a, b in ((0, 150), (150, 151), (151, 400)):
        cu, L = _i32(0, b - a), _i32(b)
        sa.sa_cache_write(k[a:b], v[a:b], table=table, cu_q=cu, kv_len=L, **c)
        outs.append(sa.sa_cache_attn(q[a:b], table=table, cu_q=cu, kv_len=L, max_q=b - a, **c))
    # single tokens from one captured step: its inputs and lengths are buffers that move on
    cu, L = _i32(0, 1), _i32(prompt + 1)
    qt, kt, vt = q[prompt:prompt + 1].clone(), k[prompt:prompt + 1].clone(), v[prompt:prompt + 1].clone()
    ot = torch.empty_like(qt)
    ws = torch.empty(sa.load().sa_cache_attn_workspace_size(d), dtype=torch.uint8, device=DEV)

    def step():
        sa.sa_cache_write(kt, vt, table=table, cu_q=cu, kv_len=L, **c)
        sa.sa_cache_attn(qt, table=table, cu_q=cu, kv_len=L, max_q=1, out=ot, workspace=ws, **c)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for t in range(prompt, N):
        for buf, x in ((qt, q), (kt, k), (vt, v)):
            buf.copy_(x[t:t + 1])
        L.fill_(t + 1)
        graph.replay()
        outs.append(ot.clone())
    pieces = f64(torch.cat(outs))
    # the whole sequence at once over the finished cache
    whole = f64(sa.sa_cache_attn(q, table=table, cu_q=_i32(0, N), kv_len=_i32(N), max_q=N, **c))
    kr, vr = (torch.empty(H, N, d, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    sa.sa_cache_read(c["k_cache"], c["v_cache"], table, _i32(0, N), N, c.get("k_scale"), c.get("v_scale"),
                     out=(kr.transpose(0, 1), vr.transpose(0, 1)))
    for t in range(N):
        for h in range(H):
            mag, _ = oracle.cache_attention(f64(q[t, h * G:(h + 1) * G]), f64(kr[h]), np.abs(f64(vr[h])), t + 1)
            lim = 2 * ((2.0 ** -8 + 2.0 ** -11 + 2.0 ** -13) * mag + 2.0 ** -8 * np.abs(whole[t, h * G:(h + 1) * G]))
            assert (np.abs(pieces[t, h * G:(h + 1) * G] - whole[t, h * G:(h + 1) * G]) <= lim).all(), (t, h)
    # what was read back feeds the dense attention: every token sees all of the sequence. The rows read are rounded to
    # bf16 once more (2^-8 of a key moves a score by at most 2^-8 scale sum|q||k|, and its weight by that factor twice)
    o = sa.sa_cache_attn(q, table=table, cu_q=_i32(0, N), kv_len=_i32(N), max_q=N, causal=False, **c)
    qh = q.transpose(0, 1).contiguous()[None]
    od = sa.sa_dense_attn_fwd(qh, kr.repeat_interleave(G, 0)[None], vr.repeat_interleave(G, 0)[None])
    a, b = f64(o), f64(od[0].transpose(0, 1))
    for t in range(0, N, 7):
        for h in range(H):
            qq = f64(q[t, h * G:(h + 1) * G])
            mag, _ = oracle.cache_attention(qq, f64(kr[h]), np.abs(f64(vr[h])), N)
            ds = 0.0 if kind == "bf16" else 2.0 ** -8 * d ** -0.5 * (np.abs(qq) @ np.abs(f64(kr[h])).T).max()
            lim = (2 * (2.0 ** -8 + 2.0 ** -11 + 2.0 ** -13) + 2 * ds + (0.0 if kind == "bf16" else 2.0 ** -8)) * mag
            lim = lim + 2.0 ** -7 * np.abs(a[t, h * G:(h + 1) * G])
            assert (np.abs(a[t, h * G:(h + 1) * G] - b[t, h * G:(h + 1) * G]) <= lim).all(), (t, h)
    sa.sa_device_status()


def test_training_and_generation_agree(cuda_lib):
    """The decayed branch trained on whole sequences gives what it gives token by
    token: forward of 300 tokens against 300 captured single steps, within both
    bounds (the products of the forward round weights and states to bf16, 2^-8 each;
    the steps stay in fp32), and the state they end in."""
    sa = cuda_lib
    B, H, N, d = 2, 3, 300, 64
    g = torch.Generator(device=DEV).manual_seed(9)
    q, k, v = (torch.randn(B, H, N, d, generator=g, device=DEV).to(torch.bfloat16) for _ in range(3))
    ld = -torch.exp(torch.linspace(-6, -1, H, device=DEV))
    o, S = sa.sa_decay_attn_fwd(q, k, v, ld, want_state=True)
    state = torch.zeros(B, H, d, d, device=DEV)
    buf = [torch.zeros(B, H, d, dtype=torch.bfloat16, device=DEV) for _ in range(4)]
    step = lambda: sa.sa_decay_attn_step(buf[0], buf[1], buf[2], ld, state, out=buf[3])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    state.zero_()
    got = []
    for t in range(N):
        for b_, x in zip(buf, (q, k, v)):
            b_.copy_(x[:, :, t])
        graph.replay()
        got.append(buf[3].clone())
    got = f64(torch.stack(got, dim=2))
    o, S, st = f64(o), f64(S), f64(state)
    q, k, v = f64(q), f64(k), f64(v)
    w = np.exp(f64(ld))
    for b in range(B):
        for h in range(H):
            i = np.arange(N)
            W = np.where(i[:, None] >= i, w[h] ** np.maximum(i[:, None] - i, 0), 0.0)
            mag = d ** -0.5 * (np.abs(q[b, h]) @ np.abs(k[b, h]).T * W) @ np.abs(v[b, h])
            assert (np.abs(o[b, h] - got[b, h]) <= (2.0 ** -7 + 2.0 ** -10) * mag + 2.0 ** -7 * np.abs(o[b, h])).all()
            magS = (np.abs(k[b, h]) * (w[h] ** (N - 1 - i))[:, None]).T @ np.abs(v[b, h])
            assert (np.abs(S[b, h] - st[b, h]) <= 2.0 ** -13 * magS).all()
    sa.sa_device_status()

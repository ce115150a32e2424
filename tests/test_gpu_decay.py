"""GPU parity of the decayed linear attention with the fp64 oracle: forward,
gradients, single tokens, and a sequence produced piece by piece.

Tolerances (derived, none fitted). The products run on bf16 operands: the weight
w_ij = e^{g (i - j)} q_i . k_j of a pair inside a chunk of 128 tokens is rounded to
bf16 once (2^-8), the state S that enters a chunk is rounded to bf16 once for the
product with q, and the output once. The state itself is kept in fp32 from
operands split into two bf16 numbers or three (2^-16 of each k_j v_j, or nothing):
  |err o| <= (2^-8 + 2^-11) (sum_j in chunk |w_ij| |v_j| + e^{..} |q_i| . |S|) + 2^-8 |o|
             + 2^-14 sum_j e^{..} (|q_i| . |k_j|) |v_j|
  |err S| <= 2^-14 sum_j e^{..} |k_j| |v_j| + 2^-18 e^{..} |S_0|
(2^-11 and 2^-14 leave room for fp32 sums of at most a few thousand terms.)"""
import numpy as np
import pytest
import torch

import oracle

pytestmark = pytest.mark.gpu

DEV = "cuda"
f64 = oracle.as_f64
CHUNK = 128


def _inputs(B, H, N, d, seed, strong=None):
    g = torch.Generator(device=DEV).manual_seed(seed)
    x = {n: torch.randn(B, H, N, d, generator=g, device=DEV).to(torch.bfloat16) for n in ("q", "k", "v", "dout")}
    x["log_decay"] = -torch.exp(torch.linspace(0.5, -7, H, device=DEV)) if strong is None else torch.full((H,), strong, device=DEV)
    x["state"] = 3 * torch.randn(B, H, d, d, generator=g, device=DEV)
    x["dstate"] = torch.randn(B, H, d, d, generator=g, device=DEV)
    return x


def _bound(a, b, c, g, s_intra, s_inter, s_upd, x0, reverse):
    """Bounds of y and of the last state for one head, as in the header."""
    if reverse:
        # against time: turned around, the incoming state without a decay of its own
        a, b, c = a[::-1], b[::-1], c[::-1]
    N, d = a.shape
    w = np.exp(g)
    lead = 0 if reverse else 1
    X = np.zeros((d, d)) if x0 is None else x0.astype(np.float64)
    absX = np.abs(X)
    absb0 = np.abs(X) * 0.0
    y = np.zeros((N, d))
    # chunks are counted from the sequence's start in either direction of time
    first = N % CHUNK if reverse and N % CHUNK else CHUNK
    t = 0
    while t < N:
        e = min(N, t + (first if t == 0 else CHUNK))
        i = np.arange(e - t)
        lag = i[:, None] - i[None, :]
        W = np.where(lag >= 0, w ** np.maximum(lag, 0), 0.0)
        far = w ** (i + lead)
        intra = np.abs(a[t:e] @ b[t:e].T) * W * s_intra
        y[t:e] = (2.0 ** -8 + 2.0 ** -11) * (intra @ np.abs(c[t:e]) + s_inter * far[:, None] * (np.abs(a[t:e]) @ np.abs(X)))
        y[t:e] += 2.0 ** -14 * (s_intra * ((np.abs(a[t:e]) @ np.abs(b[t:e]).T) * W) @ np.abs(c[t:e])
                                + s_inter * far[:, None] * (np.abs(a[t:e]) @ (absX + absb0)))
        out = w ** (len(i) - 1 - i + (1 - lead))
        wall = w ** len(i)
        X = wall * X + s_upd * (b[t:e] * out[:, None]).T @ c[t:e]
        absb0 = wall * absb0 + s_upd * (np.abs(b[t:e]) * out[:, None]).T @ np.abs(c[t:e])
        absX = wall * absX
        t = e
    return (y[::-1] if reverse else y), 2.0 ** -14 * absb0 + 2.0 ** -18 * absX


def _within(got, ref, bound, what):
    got = f64(got)
    assert np.isfinite(got).all(), what
    err = np.abs(got - ref)
    lim = bound + 2.0 ** -30
    assert (err <= lim).all(), (what, float((err - lim).max()), float(err.max()), float(np.abs(ref).max()))


def _check_fwd(sa, x, scale, with_state):
    B, H, N, d = x["q"].shape
    o, S = sa.sa_decay_attn_fwd(x["q"], x["k"], x["v"], x["log_decay"], scale, state=x["state"] if with_state else None,
                                want_state=True)
    sc = scale if scale > 0 else d ** -0.5
    for b in range(B):
        for h in range(H):
            q, k, v = (f64(x[n][b, h]) for n in ("q", "k", "v"))
            g = float(x["log_decay"][h])
            s0 = f64(x["state"][b, h]) if with_state else None
            ro, rS = oracle.decay_attention(q, k, v, g, sc, s0)
            by, bS = _bound(q, k, v, g, sc, sc, 1.0, s0, False)
            _within(o[b, h], ro, by + 2.0 ** -8 * np.abs(ro), ("o", b, h))
            _within(S[b, h], rS, bS, ("S", b, h))
    o2 = sa.sa_decay_attn_fwd(x["q"], x["k"], x["v"], x["log_decay"], scale, state=x["state"] if with_state else None)
    assert torch.equal(o, o2)
    sa.sa_device_status()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("B,H,N", [(1, 3, 1), (2, 2, 17), (1, 2, 127), (1, 3, 128), (2, 1, 129), (1, 2, 700)])
@pytest.mark.parametrize("with_state", [False, True])
def test_forward(cuda_lib, d, B, H, N, with_state):
    _check_fwd(cuda_lib, _inputs(B, H, N, d, N + d), 0.0 if N != 17 else 0.3, with_state)


@pytest.mark.parametrize("B,H,N,d", [(1, 40, 2560, 64),      # ranges that end inside heads and go on into the next
                                     (1, 1, 5000, 128),       # one head over many ranges
                                     (2, 150, 130, 64),       # several whole heads to a range
                                     (1, 2, 20000, 64)])      # long sums
def test_forward_split_over_blocks(cuda_lib, B, H, N, d):
    x = _inputs(B, H, N, d, N + H)
    if H == 2:
        x["log_decay"] = torch.tensor([0.0, -1e-4], device=DEV)
    _check_fwd(cuda_lib, x, 0.0, True)


@pytest.mark.parametrize("log_decay", [0.0, -1e-5, -0.9, -30.0, -200.0, float("-inf")])
def test_forward_extreme_decays(cuda_lib, log_decay):
    """No decay at all, decays that leave nothing of a token's neighbour, and -inf
    (each token sees only itself)."""
    _check_fwd(cuda_lib, _inputs(1, 2, 300, 64, 3, strong=log_decay), 0.0, True)


def _check_bwd(sa, x, with_state, with_dstate):
    B, H, N, d = x["q"].shape
    res = sa.sa_decay_attn_bwd(x["q"], x["k"], x["v"], x["log_decay"], x["dout"], state=x["state"] if with_state else None,
                               dstate=x["dstate"] if with_dstate else None)
    assert len(res) == (4 if with_state else 3)
    sc = d ** -0.5
    for b in range(B):
        for h in range(H):
            q, k, v, do = (f64(x[n][b, h]) for n in ("q", "k", "v", "dout"))
            g = float(x["log_decay"][h])
            s0 = f64(x["state"][b, h]) if with_state else None
            ds = f64(x["dstate"][b, h]) if with_dstate else None
            ref = oracle.decay_attention_bwd(q, k, v, g, sc, do, s0, ds)
            T = lambda t: None if t is None else t.T
            bounds = [_bound(do, v, k, g, sc, sc, 1.0, T(s0), False)[0], _bound(v, do, q, g, sc, 1.0, sc, T(ds), True)[0]]
            bv, bS = _bound(k, q, do, g, sc, 1.0, sc, ds, True)
            for got, r, lim, what in zip(res, ref, bounds + [bv], ("dq", "dk", "dv")):
                _within(got[b, h], r, lim + 2.0 ** -8 * np.abs(r), (what, b, h))
            if with_state:
                _within(res[3][b, h], ref[3], bS, ("dstate", b, h))
    sa.sa_device_status()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("B,H,N,with_state,with_dstate", [(1, 2, 1, True, True), (2, 2, 33, False, False), (1, 2, 128, True, False),
                                                          (1, 1, 200, False, True), (1, 2, 555, True, True)])
def test_backward(cuda_lib, d, B, H, N, with_state, with_dstate):
    _check_bwd(cuda_lib, _inputs(B, H, N, d, 2 * N + d), with_state, with_dstate)


@pytest.mark.parametrize("B,H,N,d", [(1, 7, 1500, 64), (1, 2, 1100, 128), (1, 300, 130, 64)])
def test_backward_split_over_blocks(cuda_lib, B, H, N, d):
    _check_bwd(cuda_lib, _inputs(B, H, N, d, N + H), True, True)


def test_used_workspace_and_two_streams(cuda_lib):
    """A workspace that holds NaN, and two calls at once with one each."""
    sa = cuda_lib
    xs = [_inputs(1, 3, 2000, 128, 50 + i) for i in range(2)]
    need = sa.load().sa_decay_attn_workspace_size(1, 3, 2000, 128)
    assert need > 0
    refs = [sa.sa_decay_attn_fwd(x["q"], x["k"], x["v"], x["log_decay"], state=x["state"], want_state=True) for x in xs]
    torch.cuda.synchronize()
    ws = [torch.full((need,), 255, dtype=torch.uint8, device=DEV) for _ in xs]
    streams = [torch.cuda.Stream() for _ in xs]
    torch.cuda.synchronize()
    for _ in range(5):
        outs = []
        for x, w, st in zip(xs, ws, streams):
            with torch.cuda.stream(st):
                outs.append(sa.sa_decay_attn_fwd(x["q"], x["k"], x["v"], x["log_decay"], state=x["state"], want_state=True, workspace=w))
        torch.cuda.synchronize()
        for (o, s), (ro, rs) in zip(outs, refs):
            assert torch.equal(o, ro) and torch.equal(s, rs)
    sa.sa_device_status()


def test_backward_against_differences(cuda_lib):
    """The directional derivative of a fixed linear functional of the outputs, by
    central differences of the 64-bit forward, against the kernels' gradients. The
    functional is bilinear along each operand, so the difference is exact; what is
    left is the gradients' own rounding, summed over N d terms."""
    sa = cuda_lib
    B, H, N, d = 1, 1, 150, 64
    x = _inputs(B, H, N, d, 77)
    x["log_decay"] = torch.full((1,), -0.02, device=DEV)
    g = sa.sa_decay_attn_bwd(x["q"], x["k"], x["v"], x["log_decay"], x["dout"], state=x["state"], dstate=x["dstate"])
    h64 = {n: f64(x[n][0, 0]) for n in ("q", "k", "v", "dout", "state", "dstate")}
    gd = float(x["log_decay"][0])
    bq = _bound(h64["dout"], h64["v"], h64["k"], gd, d ** -0.5, d ** -0.5, 1.0, h64["state"].T, False)[0]
    bk = _bound(h64["v"], h64["dout"], h64["q"], gd, d ** -0.5, 1.0, d ** -0.5, h64["dstate"].T, True)[0]
    bv, bs = _bound(h64["k"], h64["q"], h64["dout"], gd, d ** -0.5, 1.0, d ** -0.5, h64["dstate"], True)

    def loss(**y):
        o, S = oracle.decay_attention(y["q"], y["k"], y["v"], gd, d ** -0.5, y["state"])
        return (o * h64["dout"]).sum() + (S * h64["dstate"]).sum()

    rng = np.random.default_rng(1)
    base = {n: h64[n] for n in ("q", "k", "v", "state")}
    for name, grad, lim in zip(("q", "k", "v", "state"), g, (bq, bk, bv, bs)):
        u = rng.normal(size=base[name].shape)
        up, dn = dict(base), dict(base)
        up[name], dn[name] = base[name] + u, base[name] - u
        diff = (loss(**up) - loss(**dn)) / 2
        got = f64(grad[0, 0])
        tol = (np.abs(u) * (lim + 2.0 ** -8 * np.abs(got))).sum()
        assert abs((got * u).sum() - diff) <= tol + 1e-9 * abs(diff), name


@pytest.mark.parametrize("d", [64, 128])
def test_single_tokens(cuda_lib, d):
    sa = cuda_lib
    B, H = 3, 5
    x = _inputs(B, H, 4, d, d)
    state = x["state"].clone()
    keep = state.clone()
    other = torch.empty_like(state)
    t0 = [x[n][:, :, 0].contiguous() for n in ("q", "k", "v")]
    o = sa.sa_decay_attn_step(*t0, x["log_decay"], state, state_out=other)
    assert torch.equal(state, keep)
    o_in = sa.sa_decay_attn_step(*t0, x["log_decay"], state)
    assert torch.equal(o, o_in) and torch.equal(state, other)
    for b in range(B):
        for h in range(H):
            q, k, v = (f64(t[b, h])[None] for t in t0)
            ro, rS = oracle.decay_attention(q, k, v, float(x["log_decay"][h]), d ** -0.5, f64(keep[b, h]))
            # fp32 sums of d products, one rounding of e^g (2 units), one of each product and sum
            magS = np.abs(f64(keep[b, h])) + np.abs(np.outer(k[0], v[0]))
            _within(state[b, h], rS, 2.0 ** -21 * magS, "S")
            _within(o[b, h], ro[0], 2.0 ** -8 * np.abs(ro[0]) + 2.0 ** -16 * d ** -0.5 * (np.abs(q[0]) @ magS), "o")


def test_pieces_follow_each_other(cuda_lib):
    """A prompt in one call equals the prompt cut into pieces that hand the state
    on, single tokens among them, within both sides' bounds."""
    sa = cuda_lib
    B, H, N, d = 1, 2, 400, 128
    x = _inputs(B, H, N, d, 21)
    whole, S = sa.sa_decay_attn_fwd(x["q"], x["k"], x["v"], x["log_decay"], want_state=True)
    state, outs = None, []
    for a, b in ((0, 130), (130, 131), (131, 133), (133, 400)):
        t = [x[n][:, :, a:b].contiguous() for n in ("q", "k", "v")]
        if b - a == 1:
            o = sa.sa_decay_attn_step(*(y[:, :, 0].contiguous() for y in t), x["log_decay"], state).unsqueeze(2)
        else:
            o, state = sa.sa_decay_attn_fwd(*t, x["log_decay"], state=state, want_state=True)
        outs.append(o)
    pieces = torch.cat(outs, dim=2)
    for h in range(H):
        q, k, v = (f64(x[n][0, h]) for n in ("q", "k", "v"))
        g = float(x["log_decay"][h])
        ro, rS = oracle.decay_attention(q, k, v, g, d ** -0.5)
        # pieces start chunks elsewhere, where another state is rounded: bound every row by the larger of both cuts
        by, bS = _bound(q, k, v, g, d ** -0.5, d ** -0.5, 1.0, None, False)
        allS = 2.0 ** -7 * d ** -0.5 * np.abs(q).max() * np.abs(k).max() * np.abs(v).max() * d
        _within(whole[0, h], ro, by + 2.0 ** -8 * np.abs(ro), "whole")
        _within(pieces[0, h], ro, by + allS + 2.0 ** -8 * np.abs(ro), "pieces")
        _within(state[0, h], rS, 2 * bS, "state")


@pytest.mark.parametrize("N,d", [(260, 64), (2000, 128)])
def test_capture_and_side_stream(cuda_lib, N, d):
    """Forward and backward captured together replay on new inputs."""
    sa = cuda_lib
    x = _inputs(1, 3, N, d, 31)
    fwd = lambda: sa.sa_decay_attn_fwd(x["q"], x["k"], x["v"], x["log_decay"], state=x["state"], want_state=True)
    bwd = lambda: sa.sa_decay_attn_bwd(x["q"], x["k"], x["v"], x["log_decay"], x["dout"], state=x["state"], dstate=x["dstate"])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        fwd(), bwd()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        res = fwd() + bwd()
    y = _inputs(1, 3, N, d, 32)
    for n in ("q", "k", "v", "dout", "state", "dstate"):
        x[n].copy_(y[n])
    graph.replay()
    ref = fwd() + bwd()
    for a, b in zip(res, ref):
        assert torch.equal(a, b)
    sa.sa_device_status()

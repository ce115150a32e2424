"""States that the decayed linear attention hands on: their precision over long
sequences, with and without ranges that cut heads, and non-finite numbers.

The limit of the states' error (2-norm, relative). Operands in three bf16 numbers
lose nothing; two would lose up to 2^-18 of every term, evenly spread: 2^-18 / sqrt(3)
= 2.2e-6. A weight is an exponential of a rounded argument x = dist * log2(e) * g:
2^-22, and 2^-23 |x|, of which the terms that matter have x about 1; the sums are
fp32 (2^-22 for a chunk's and the range's together). 2^-20 = 9.5e-7 is above the
sum of the latter and below the former."""
import pytest
import torch

from test_gpu_decay import _check_bwd, _check_fwd, _inputs

pytestmark = pytest.mark.gpu

DEV = "cuda"
LIMIT = 2.0 ** -20


def _last(a, b, g, s0, s_upd, lead):
    """s_upd sum_j e^{g dist_j} a_j b_j^T + e^{g (dist_0 + 1 - lead)} s0 in 64 bits, dist_j the steps from token j to the
    last one, and `lead` more of them."""
    N = a.shape[0]
    dist = torch.arange(N - 1, -1, -1, device=DEV, dtype=torch.float64) + lead
    return s_upd * (a.double() * torch.exp(g.double() * dist)[:, None]).T @ b.double() + torch.exp(g.double() * N) * s0.double()


@pytest.mark.parametrize("B,H,N,d", [(4, 37, 10112, 64), (4, 37, 10112, 128),     # whole heads, 79 chunks each
                                     (1, 200, 7000, 64),                           # two heads to a range
                                     (1, 2, 40000, 64), (1, 3, 20000, 128)])       # heads cut into ranges
def test_states_of_long_sequences(cuda_lib, B, H, N, d):
    """The last state and the gradient of the first, against 64 bits, for decays
    from none at all to horizons of 100 tokens; both start from a state as large
    as what the tokens add."""
    sa = cuda_lib
    x = _inputs(B, H, N, d, N + d)
    g = -torch.logspace(-7, -2, H, device=DEV)
    g[0] = 0.0
    x["log_decay"] = g
    for n in ("state", "dstate"):
        x[n] = x[n] * min(N, 3000) ** 0.5
    _, S = sa.sa_decay_attn_fwd(x["q"], x["k"], x["v"], g, state=x["state"], want_state=True)
    dS = sa.sa_decay_attn_bwd(x["q"], x["k"], x["v"], g, x["dout"], state=x["state"], dstate=x["dstate"])[3]
    worst = {}
    for h in sorted(set(range(0, H, max(1, H // 16))) | {H - 1}):
        b = h % B
        refs = (("S", S, _last(x["k"][b, h], x["v"][b, h], g[h], x["state"][b, h], 1.0, 0)),
                ("dstate", dS, _last(x["q"][b, h].flip(0), x["dout"][b, h].flip(0), g[h], x["dstate"][b, h], d ** -0.5, 1)))
        for name, got, ref in refs:
            e = float((got[b, h].double() - ref).norm() / ref.norm())
            worst[name] = max(worst.get(name, (0.0, 0)), (e, h))
    print(worst)
    for name, (e, h) in worst.items():
        assert e <= LIMIT, (name, h, float(g[h]), e)
    sa.sa_device_status()


def test_state_of_many_single_tokens(cuda_lib):
    """4,096 tokens one by one with memories as long: the decay's own rounding, the same
    at every token, must not add up (half a step of a number below 1, 2^-25, times the
    memory would be 2^-13). What is left is each step's rounding, 2^-24 at most and
    without a sign: 2^-24 sqrt(4096) = 2^-18 in the 2-norm; the limit is twice that."""
    sa = cuda_lib
    B, H, N, d = 1, 6, 4096, 64
    x = _inputs(B, H, N, d, 11)
    g = -torch.tensor([0.0, 1e-6, 3e-5, 1e-4, 2.4e-4, 1e-3], device=DEV)
    state = x["state"] * 20
    first = state.clone()
    q, k, v = ([t.contiguous() for t in x[n].unbind(2)] for n in ("q", "k", "v"))
    for t in range(N):
        sa.sa_decay_attn_step(q[t], k[t], v[t], g, state)
    for h in range(H):
        ref = _last(x["k"][0, h], x["v"][0, h], g[h], first[0, h], 1.0, 0)
        e = float((state[0, h].double() - ref).norm() / ref.norm())
        print(h, e)
        assert e <= 2.0 ** -17, (h, float(g[h]), e)


def test_non_finite_operands(cuda_lib):
    """A NaN of a query reaches its token, of a key its token and the later ones, of a
    value its channel of the later ones and of its own group of 128 tokens; other
    heads, channels and earlier groups are as without it."""
    sa = cuda_lib
    B, H, N, d, t = 1, 2, 300, 64, 200
    x = _inputs(B, H, N, d, 90, strong=-0.01)
    run = lambda y: sa.sa_decay_attn_fwd(y["q"], y["k"], y["v"], y["log_decay"], state=y["state"], want_state=True)
    ref, refS = run(x)
    for n in ("q", "k", "v"):
        for bad in (float("nan"), float("inf")):
            y = dict(x)
            y[n] = x[n].clone()
            y[n][0, 1, t, 5] = bad
            o, S = run(y)
            assert torch.equal(o[0, 0], ref[0, 0]) and torch.equal(S[0, 0], refS[0, 0])
            o, r, S, rS = o[0, 1], ref[0, 1], S[0, 1], refS[0, 1]
            if n == "q":
                assert not torch.isfinite(o[t]).any() and torch.equal(S, rS)
                assert torch.equal(o[:t], r[:t]) and torch.equal(o[t + 1:], r[t + 1:])
            elif n == "k":
                assert not torch.isfinite(o[t:]).any() and torch.equal(o[:t], r[:t])
                assert not torch.isfinite(S[5]).any() and torch.equal(S[:5], rS[:5]) and torch.equal(S[6:], rS[6:])
            else:
                other = [c for c in range(d) if c != 5]
                assert torch.equal(o[:, other], r[:, other]) and torch.equal(S[:, other], rS[:, other])
                assert not torch.isfinite(o[t:, 5]).any() and torch.equal(o[:128, 5], r[:128, 5])
                assert not torch.isfinite(S[:, 5]).any()
    sa.sa_device_status()


@pytest.mark.parametrize("B,H,N,d", [(2, 150, 130, 128), (2, 80, 300, 64)])
def test_several_heads_to_a_range(cuda_lib, B, H, N, d):
    """Ranges of two whole heads and of heads cut unevenly, at both head sizes: forward and gradients."""
    x = _inputs(B, H, N, d, N + d)
    _check_fwd(cuda_lib, x, 0.0, True)
    _check_bwd(cuda_lib, x, True, True)


def test_tensors_beyond_32_bits(cuda_lib):
    """2.3e9 elements an operand: the last head's outputs, state and gradients."""
    sa = cuda_lib
    B, H, N, d = 2, 150, 60000, 128
    gen = torch.Generator(device=DEV).manual_seed(95)
    x = {n: torch.randn(B, H, N, d, generator=gen, device=DEV, dtype=torch.bfloat16) for n in ("q", "k", "v", "dout")}
    x["log_decay"] = torch.linspace(-0.5, -0.01, H, device=DEV)
    x["state"] = torch.randn(B, H, d, d, generator=gen, device=DEV)
    x["dstate"] = torch.randn(B, H, d, d, generator=gen, device=DEV)
    o, S = sa.sa_decay_attn_fwd(x["q"], x["k"], x["v"], x["log_decay"], state=x["state"], want_state=True)
    ref = _last(x["k"][-1, -1], x["v"][-1, -1], x["log_decay"][-1], x["state"][-1, -1], 1.0, 0)
    assert float((S[-1, -1].double() - ref).norm()) <= LIMIT * float(ref.norm())
    k, v, q = (x[n][-1, -1].double() for n in ("k", "v", "q"))
    w = torch.exp(x["log_decay"][-1].double() * torch.arange(N - 1, -1, -1, device=DEV, dtype=torch.float64))
    want = d ** -0.5 * ((k @ q[-1]) * w) @ v
    mag = d ** -0.5 * ((k.abs() @ q[-1].abs()) * w) @ v.abs()
    assert ((o[-1, -1, -1].double() - want).abs() <= (2.0 ** -8 + 2.0 ** -11) * mag + 2.0 ** -8 * want.abs()).all()
    del o, S
    dq, dk, dv, ds = sa.sa_decay_attn_bwd(x["q"], x["k"], x["v"], x["log_decay"], x["dout"], state=x["state"], dstate=x["dstate"])
    do = x["dout"][-1, -1].double()
    ref = _last(q.flip(0), do.flip(0), x["log_decay"][-1], x["dstate"][-1, -1], d ** -0.5, 1)
    assert float((ds[-1, -1].double() - ref).norm()) <= LIMIT * float(ref.norm())
    # dv of the first token: sum over all later ones
    w = w.flip(0)
    want = d ** -0.5 * ((q @ k[0]) * w) @ do
    mag = d ** -0.5 * ((q.abs() @ k[0].abs()) * w) @ do.abs()
    assert ((dv[-1, -1, 0].double() - want).abs() <= (2.0 ** -8 + 2.0 ** -11) * mag + 2.0 ** -8 * want.abs()).all()
    for g in (dq, dk, dv):
        assert torch.isfinite(g[-1, -1]).all()
    sa.sa_device_status()

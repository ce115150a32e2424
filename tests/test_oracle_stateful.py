"""Pins of the fp64 oracle of the cache, its attention and the decayed linear
attention: torch's own casts, float64 softmax attention, the quadratic form of
the recurrence, and central differences of its gradients."""
import numpy as np
import pytest
import torch

import oracle


@pytest.mark.parametrize("kind", ["e4m3", "int8"])
def test_cache_encode_against_torch_casts(kind):
    g = torch.Generator().manual_seed(5)
    for d in (64, 128):
        for gain in (1e-30, 1.0, 300.0):
            x = (torch.randn(d, generator=g) * gain).to(torch.bfloat16)
            codes, scale = oracle.cache_encode(oracle.as_f64(x), kind)
            amax = x.float().abs().max()
            M = torch.tensor(448.0 if kind == "e4m3" else 127.0)
            y = x.float() * (M / amax)
            ref = y.to(torch.float8_e4m3fn).float() if kind == "e4m3" else y.round()
            assert (torch.from_numpy(codes).float() == ref).all()
            assert scale == float(amax / M)
    codes, scale = oracle.cache_encode(np.zeros(64), kind)
    assert (codes == 0).all() and scale == 1.0


def test_cache_attention_against_float64_attention():
    rng = np.random.default_rng(3)
    q, k, v = rng.normal(size=(3, 64)), rng.normal(size=(50, 64)), rng.normal(size=(50, 64))
    o, lse = oracle.cache_attention(q, k, v, 37)
    t = torch.nn.functional.scaled_dot_product_attention(*(torch.from_numpy(x)[None] for x in (q, k[:37], v[:37])))
    assert np.abs(o - t[0].numpy()).max() < 1e-13
    assert np.abs(lse - np.log(np.exp(q @ k[:37].T / 8).sum(axis=1))).max() < 1e-12
    o, lse = oracle.cache_attention(q, k, v, 0)
    assert (o == 0).all() and (lse == -np.inf).all()


def test_cache_slot():
    assert oracle.cache_slot([4, 2], 16, 17, 5) == (2, 1)
    assert oracle.cache_slot([4, 2], 16, 32, 5) is None
    assert oracle.cache_slot([4, 5], 16, 20, 5) is None
    assert oracle.cache_slot([4, -1], 16, 20, 5) is None
    assert oracle.cache_slot([4, 2], 16, -1, 5) is None


def test_decay_attention_against_the_quadratic_form():
    rng = np.random.default_rng(4)
    N, d, g, sc = 23, 8, -0.3, 0.7
    q, k, v = (rng.normal(size=(N, d)) for _ in range(3))
    S0 = rng.normal(size=(d, d))
    o, S = oracle.decay_attention(q, k, v, g, sc, S0)
    i, j = np.arange(N)[:, None], np.arange(N)[None, :]
    W = np.where(i >= j, np.exp(g * (i - j)), 0.0)
    ref = sc * ((q @ k.T * W) @ v + np.exp(g * (np.arange(N) + 1))[:, None] * (q @ S0))
    assert np.abs(o - ref).max() < 1e-12
    refS = np.exp(g * N) * S0 + (k * np.exp(g * (N - 1 - np.arange(N)))[:, None]).T @ v
    assert np.abs(S - refS).max() < 1e-12


def test_decay_attention_gradients_against_differences():
    rng = np.random.default_rng(6)
    N, d, g, sc = 9, 5, -0.2, 0.6
    x = {n: rng.normal(size=(N, d)) for n in ("q", "k", "v")}
    x["state"] = rng.normal(size=(d, d))
    do, dS = rng.normal(size=(N, d)), rng.normal(size=(d, d))

    def loss(**y):
        o, S = oracle.decay_attention(y["q"], y["k"], y["v"], g, sc, y["state"])
        return (o * do).sum() + (S * dS).sum()

    grads = dict(zip(("q", "k", "v", "state"),
                     oracle.decay_attention_bwd(x["q"], x["k"], x["v"], g, sc, do, x["state"], dS)))
    h = 1e-5
    for name, grad in grads.items():
        for idx in np.ndindex(*grad.shape):
            up, dn = ({n: t.copy() for n, t in x.items()} for _ in range(2))
            up[name][idx] += h
            dn[name][idx] -= h
            # the loss is a polynomial of degree two in each operand: central differences are exact up to rounding
            assert abs((loss(**up) - loss(**dn)) / (2 * h) - grad[idx]) < 1e-8

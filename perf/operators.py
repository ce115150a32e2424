"""Workloads of the stateful operators: a paged key/value cache (written,
quantised and read back), attention of new tokens over that cache, and linear
attention with a decay for each head.

Each case can run in a plain form (elementary torch operations in 32 bits) or
through the package's own calls (`own`); `exact` gives the results in 64 bits.
"""
import math
import random

import numpy as np
import torch

own = False

DEV = "cuda"
BF16 = torch.bfloat16
QMAX = {"e4m3": 448.0, "int8": 127.0}
CODE = {"bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn, "int8": torch.int8}
ELEM = {"bf16": 2, "e4m3": 1, "int8": 1}


# ------------------------------------------------------------------ the cases
def _cache(name, op, kind, S, n, ctx, Hkv, G, d, page, causal=True):
    """n: new tokens of the longest sequence; ctx: cached tokens of the longest
    sequence, the new ones included; the other sequences are shorter (ragged)."""
    return {"name": name, "op": op, "kind": kind, "S": S, "n": n, "ctx": ctx, "Hkv": Hkv, "G": G, "d": d,
            "page": page, "causal": causal}


def _decay(name, op, B, H, N, d, state):
    return {"name": name, "op": op, "B": B, "H": H, "N": N, "d": d, "state": state}


def listed():
    return [
        # one generated token of each running sequence enters a bf16 cache: the smallest call, latency counts
        _cache("write_step_bf16", "write", "bf16", 48, 1, 1024, 8, 1, 128, 64),
        # a prompt enters an E4M3 cache and is read back for a pass that wants contiguous keys and values
        _cache("round_trip_e4m3", "round_trip", "e4m3", 4, 8000, 8000, 8, 1, 128, 64),
        # chunks enter an int8 cache behind earlier ones: small head, small pages, odd lengths
        _cache("round_trip_int8", "round_trip", "int8", 7, 613, 2501, 5, 1, 64, 16),
        # one sequence generates a token: the latency of a single user
        _cache("token_single", "attn", "bf16", 1, 1, 1001, 8, 4, 128, 64),
        # a batch generates a token each over long ragged contexts
        _cache("token_batch", "attn", "bf16", 64, 1, 8192, 8, 4, 128, 64),
        # the same over an E4M3 cache, longer contexts, two tokens a sequence (one drafted)
        _cache("token_batch_e4m3", "attn", "e4m3", 24, 2, 32768, 8, 8, 128, 128),
        # three latent frames of a 30 x 52 grid attend to all 21 frames (chunk-wise video generation: tokens of
        # a chunk see each other both ways)
        _cache("video_chunk", "attn", "bf16", 1, 4680, 32760, 12, 1, 128, 128, causal=False),
        # chunked prompts over an int8 cache: shared key heads, odd group, pages that do not divide a tile
        _cache("prompt_chunk_int8", "attn", "int8", 5, 517, 4099, 4, 3, 64, 48),
        # a whole 720p video of one model layer (21 x 45 x 80 tokens, 40 heads)
        _decay("decay_720p", "decay_fwd", 1, 40, 75600, 128, False),
        # a short continued prompt: small head, a state carried in
        _decay("decay_short", "decay_fwd", 2, 6, 333, 64, True),
        # a training step's forward and backward on the 480p video (21 x 30 x 52 tokens, 12 heads)
        _decay("decay_train_480p", "decay_train", 1, 12, 32760, 128, True),
        # a batch generates a token each
        _decay("decay_token", "decay_step", 32, 40, 1, 128, True),
    ]


def _log_uniform(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _draw_once(rng):
    op = rng.choice(["write", "round_trip", "attn", "attn", "attn", "decay_fwd", "decay_train", "decay_step"])
    d = rng.choice([64, 128, 128])
    if op in ("write", "round_trip", "attn"):
        # (8-bit caches are written in the round trips, which return the values that the codes stand for)
        kind = "bf16" if op == "write" else rng.choice(["bf16", "e4m3", "int8"])
        S = _log_uniform(rng, 1, 64)
        ctx = _log_uniform(rng, 1, 32768)
        if op == "attn" and rng.random() < 0.5:
            n = rng.choice([1, 1, 2, 5])
        else:
            n = _log_uniform(rng, 1, 5000)
        n = min(n, ctx)
        G = rng.choice([1, 2, 3, 4, 7, 8, 16]) if op == "attn" else 1
        return _cache(None, op, kind, S, n, ctx, rng.choice([1, 2, 4, 5, 8, 12]), G, d,
                      rng.choice([16, 32, 48, 64, 128, 256]), rng.random() < 0.7)
    if op == "decay_step":
        return _decay(None, op, _log_uniform(rng, 1, 64), rng.randint(1, 40), 1, d, True)
    return _decay(None, op, rng.choice([1, 1, 2, 3]), rng.randint(1, 40), _log_uniform(rng, 1, 75600), d,
                  rng.random() < 0.5)


def _cost(case):
    w = work(case)
    return max(w["bytes"] / 6e12, w["flops"] / 1.5e15)


def draw(rng):
    cap = {}
    for c in listed():
        cap[c["op"]] = max(cap.get(c["op"], 0.0), _cost(c))
    cap["write"] = cap["round_trip"]
    while True:
        case = _draw_once(rng)
        if _cost(case) <= cap[case["op"]] and _held(case) < 30e9:
            del case["name"]
            return case


def _held(case):
    """Bytes that a state of the case holds, roughly, with the plain form's temporaries."""
    if "S" in case:
        return 14.0 * case["S"] * (case["ctx"] + case["page"]) * case["Hkv"] * case["d"]
    return 40.0 * case["B"] * case["H"] * (case["N"] + case["d"]) * case["d"]


def _lengths(case):
    """Ragged lengths of a case's sequences: (kv_len, n) lists, the first the longest; from the sizes alone."""
    rng = random.Random(case["S"] * 1000003 + case["ctx"])
    kv, new = [], []
    for s in range(case["S"]):
        L = case["ctx"] if s == 0 else max(1, int(case["ctx"] * rng.uniform(0.4, 1.0)))
        n = case["n"] if s == 0 or case["n"] <= 5 else max(1, int(case["n"] * rng.uniform(0.4, 1.0)))
        kv.append(L)
        new.append(min(n, L))
    return kv, new


def work(case):
    if "S" in case:
        kv, new = _lengths(case)
        Hkv, Hq, d = case["Hkv"], case["Hkv"] * case["G"], case["d"]
        e = ELEM[case["kind"]]
        sc = 0 if case["kind"] == "bf16" else 4
        if case["op"] == "attn":
            if case["causal"]:
                pairs = sum(n * (L - n) + n * (n + 1) // 2 for L, n in zip(kv, new))
            else:
                pairs = sum(n * L for L, n in zip(kv, new))
            byt = 2 * sum(kv) * Hkv * (d * e + sc) + 2 * sum(new) * Hq * d * 2
            return {"bytes": byt, "flops": 4 * pairs * Hq * d}
        T = sum(new)
        byt = 2 * T * Hkv * (d * 2 + d * e + sc)
        flops = 0 if case["kind"] == "bf16" else 4 * T * Hkv * d
        if case["op"] == "round_trip":
            byt += 2 * sum(kv) * Hkv * (d * 2 + d * e + sc)
            flops += 2 * sum(kv) * Hkv * d
        return {"bytes": byt, "flops": flops}
    BH, N, d = case["B"] * case["H"], case["N"], case["d"]
    st = 4 * d * d
    if case["op"] == "decay_step":
        return {"bytes": BH * (2 * st + 4 * d * 2), "flops": BH * 5 * d * d}
    # the recurrent form's products: a rank-one update and a product of a state with a vector for each token
    byt = BH * (4 * N * d * 2 + (1 + int(case["state"])) * st)
    flops = BH * N * 4 * d * d
    if case["op"] == "decay_train":
        byt += BH * (7 * N * d * 2 + (2 + int(case["state"])) * st)
        flops += BH * N * 10 * d * d
    return {"bytes": byt, "flops": flops}


# ------------------------------------------------------------------ inputs
def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _channels(g, *shape):
    """Normal rows whose channels differ in size, a few of them by much, as keys and queries have them."""
    x = torch.randn(*shape, generator=g, device=DEV)
    gain = torch.exp(0.3 * torch.randn(shape[-1], generator=g, device=DEV))
    gain[torch.randint(shape[-1], (2,), generator=g, device=DEV)] *= 3.0
    return (x * (gain / gain.square().mean().sqrt())).to(BF16)


def _encode(x, kind):
    """(codes, scales) of rows x [..., d] of a cache kind."""
    if kind == "bf16":
        return x.to(BF16), None
    x = x.float()
    amax = x.abs().amax(dim=-1)
    # quotients of tensors: torch turns one with a number into a product with a rounded reciprocal
    M = torch.full_like(amax, QMAX[kind])
    zero = amax == 0
    a = torch.maximum(amax, M * 2.0 ** -126)
    scale = torch.where(zero, torch.ones_like(amax), a / M)
    r = torch.where(zero, torch.ones_like(amax), M / a)
    M = QMAX[kind]
    y = (x * r.unsqueeze(-1)).clamp(-M, M)
    codes = y.round().to(torch.int8) if kind == "int8" else y.to(torch.float8_e4m3fn)
    return codes, scale


def _decode(codes, scale):
    x = codes.float()
    return x if scale is None else x * scale.unsqueeze(-1)


def prepare(case, seed):
    g = _gen(seed)
    if "S" in case:
        return _prepare_cache(case, seed, g)
    B, H, N, d = case["B"], case["H"], case["N"], case["d"]
    shape = (B, H, d) if case["op"] == "decay_step" else (B, H, N, d)
    st = {"case": case, "q": _channels(g, *shape), "k": _channels(g, *shape),
          "v": torch.randn(*shape, generator=g, device=DEV).to(BF16)}
    # horizons from 8 to some 4000 tokens, spread over the heads
    half_life = 8.0 * 512.0 ** ((torch.arange(H, device=DEV, dtype=torch.float32) + 0.5) / H)
    st["log_decay"] = -math.log(2.0) / half_life
    if case["state"]:
        st["state"] = 4.0 * torch.randn(B, H, d, d, generator=g, device=DEV)
    if case["op"] == "decay_step":
        st["state_out"] = torch.empty_like(st["state"])
    if case["op"] == "decay_train":
        st["dout"] = torch.randn(*shape, generator=g, device=DEV).to(BF16)
        st["dstate"] = 0.1 * torch.randn(B, H, d, d, generator=g, device=DEV)
    return st


def _prepare_cache(case, seed, g):
    S, Hkv, G, d, page, kind = (case[x] for x in ("S", "Hkv", "G", "d", "page", "kind"))
    kv, new = _lengths(case)
    width = -(-max(kv) // page)
    used = [-(-L // page) for L in kv]
    P = sum(used) + 3
    order = np.random.default_rng(seed).permutation(P)
    table = np.zeros((S, width), dtype=np.int32)
    at = 0
    for s in range(S):
        table[s, :used[s]] = order[at:at + used[s]]
        at += used[s]
    cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    T = int(cu[-1])
    st = {"case": case, "kv": kv, "new": new, "T": T, "max_q": max(new),
          "table": torch.from_numpy(table).to(DEV), "cu_q": torch.from_numpy(cu).to(DEV),
          "kv_len": torch.tensor(kv, dtype=torch.int32, device=DEV), "k_scale": None, "v_scale": None}
    if case["op"] == "round_trip":
        st["cu_r"] = torch.from_numpy(np.concatenate([[0], np.cumsum(kv)]).astype(np.int32)).to(DEV)
        st["R"] = sum(kv)
    kc = torch.empty(P, Hkv, page, d, dtype=CODE[kind], device=DEV)
    vc = torch.empty_like(kc)
    if kind != "bf16":
        st["k_scale"] = torch.empty(P, Hkv, page, device=DEV)
        st["v_scale"] = torch.empty(P, Hkv, page, device=DEV)
    for p0 in range(0, P, 1024):
        m = min(P, p0 + 1024) - p0
        for codes, name, x in ((kc, "k_scale", _channels(g, m, Hkv, page, d)),
                               (vc, "v_scale", torch.randn(m, Hkv, page, d, generator=g, device=DEV).to(BF16))):
            c, s = _encode(x, kind)
            codes[p0:p0 + m] = c
            if s is not None:
                st[name][p0:p0 + m] = s
    st["k_cache"], st["v_cache"] = kc, vc
    if case["op"] == "attn":
        st["q"] = _channels(g, T, Hkv * G, d)
    else:
        st["k"] = _channels(g, T, Hkv, d)
        st["v"] = torch.randn(T, Hkv, d, generator=g, device=DEV).to(BF16)
    return st


# ------------------------------------------------------------------ one pass
def run(state):
    op = state["case"]["op"]
    if own:
        return _OWN[op](state)
    return _PLAIN[op](state)


def _own_write(st):
    import block_sparse_attention_softmax_b200 as sa
    sa.sa_cache_write(st["k"], st["v"], st["k_cache"], st["v_cache"], st["table"], st["cu_q"], st["kv_len"],
                      k_scale=st["k_scale"], v_scale=st["v_scale"])
    return _cache_out(st)


def _own_round_trip(st):
    import block_sparse_attention_softmax_b200 as sa
    sa.sa_cache_write(st["k"], st["v"], st["k_cache"], st["v_cache"], st["table"], st["cu_q"], st["kv_len"],
                      k_scale=st["k_scale"], v_scale=st["v_scale"])
    k, v = sa.sa_cache_read(st["k_cache"], st["v_cache"], st["table"], st["cu_r"], st["R"],
                            k_scale=st["k_scale"], v_scale=st["v_scale"])
    return {"k": k, "v": v, **_scales_out(st)}


def _own_attn(st):
    import block_sparse_attention_softmax_b200 as sa
    return sa.sa_cache_attn(st["q"], st["k_cache"], st["v_cache"], st["table"], st["cu_q"], st["kv_len"],
                            st["max_q"], k_scale=st["k_scale"], v_scale=st["v_scale"],
                            causal=st["case"]["causal"])


def _own_decay_fwd(st):
    import block_sparse_attention_softmax_b200 as sa
    return sa.sa_decay_attn_fwd(st["q"], st["k"], st["v"], st["log_decay"], state=st.get("state"), want_state=True)


def _own_decay_train(st):
    import block_sparse_attention_softmax_b200 as sa
    o, so = sa.sa_decay_attn_fwd(st["q"], st["k"], st["v"], st["log_decay"], state=st.get("state"), want_state=True)
    g = sa.sa_decay_attn_bwd(st["q"], st["k"], st["v"], st["log_decay"], st["dout"], state=st.get("state"),
                             dstate=st["dstate"])
    return (o, so) + tuple(g)


def _own_decay_step(st):
    import block_sparse_attention_softmax_b200 as sa
    o = sa.sa_decay_attn_step(st["q"], st["k"], st["v"], st["log_decay"], st["state"], state_out=st["state_out"])
    return o, st["state_out"]


def _cache_out(st):
    return {"k_cache": st["k_cache"], "v_cache": st["v_cache"]}


def _scales_out(st):
    return {} if st["k_scale"] is None else {"k_scale": st["k_scale"], "v_scale": st["v_scale"]}


# ------------------------------------------------------------------ plain forms
def _slots(st):
    """(page, slot) of every new token, on the device."""
    page = st["case"]["page"]
    cu, kv = st["cu_q"].long(), st["kv_len"].long()
    n = cu[1:] - cu[:-1]
    s = torch.repeat_interleave(torch.arange(n.numel(), device=DEV), n, output_size=st["T"])
    pos = kv[s] - n[s] + torch.arange(st["T"], device=DEV) - cu[s]
    return st["table"][s, pos // page].long(), pos % page


def _put(dst, pg, slot, x):
    # 8-bit floats are moved as bytes: indexed stores do not take them
    if dst.dtype == torch.float8_e4m3fn:
        dst, x = dst.view(torch.uint8), x.view(torch.uint8)
    dst[pg, :, slot] = x


def _plain_write(st):
    pg, slot = _slots(st)
    for x, c, s in (("k", "k_cache", "k_scale"), ("v", "v_cache", "v_scale")):
        codes, scale = _encode(st[x], st["case"]["kind"])
        _put(st[c], pg, slot, codes)
        if scale is not None:
            st[s][pg, :, slot] = scale
    return _cache_out(st)


def _rows(st, name, s):
    """Keys or values [Hkv, kv_len, d] of sequence s in 32 bits."""
    page = st["case"]["page"]
    L = st["kv"][s]
    pages = st["table"][s, :-(-L // page)].long()
    c = st[name + "_cache"]
    c = c.view(torch.uint8)[pages].view(c.dtype) if c.dtype == torch.float8_e4m3fn else c[pages]
    sc = None if st[name + "_scale"] is None else st[name + "_scale"][pages]
    x = _decode(c, sc)                                        # [pages, Hkv, page, d]
    return x.transpose(0, 1).flatten(1, 2)[:, :L]


def _plain_round_trip(st):
    pg, slot = _slots(st)
    for x, c, s in (("k", "k_cache", "k_scale"), ("v", "v_cache", "v_scale")):
        codes, scale = _encode(st[x], st["case"]["kind"])
        _put(st[c], pg, slot, codes)
        if scale is not None:
            st[s][pg, :, slot] = scale
    k, v = (torch.cat([_rows(st, x, s).transpose(0, 1) for s in range(len(st["kv"]))]).to(BF16) for x in "kv")
    return {"k": k, "v": v, **_scales_out(st)}


def _plain_attn(st):
    case = st["case"]
    Hkv, G, d = case["Hkv"], case["G"], case["d"]
    out = torch.empty(st["T"], Hkv * G, d, dtype=BF16, device=DEV)
    at = 0
    for s, (L, n) in enumerate(zip(st["kv"], st["new"])):
        k, v = _rows(st, "k", s), _rows(st, "v", s)
        q = st["q"][at:at + n].float().view(n, Hkv, G, d).permute(1, 2, 0, 3)     # [Hkv, G, n, d]
        step = max(1, int(2 ** 28 // (Hkv * G * L)))
        for i in range(0, n, step):
            qi = q[:, :, i:i + step]
            m = qi.shape[2]
            x = (qi.reshape(Hkv, G * m, d) @ k.transpose(1, 2)).view(Hkv, G, m, L) / math.sqrt(d)
            if case["causal"]:
                last = L - n + i + torch.arange(m, device=DEV)
                x.masked_fill_(torch.arange(L, device=DEV)[None, :] > last[:, None], float("-inf"))
            x = torch.exp(x - x.amax(dim=-1, keepdim=True))
            o = (x.view(Hkv, G * m, L) @ v).view(Hkv, G, m, d) / x.sum(dim=-1, keepdim=True)
            out[at + i:at + i + m] = o.permute(2, 0, 1, 3).reshape(m, Hkv * G, d).to(BF16)
        at += n
    return out


def _chunk_weights(ld, C):
    """Of a chunk of C tokens: decay between its tokens [H, C, C] (lower triangle), from the state before it to
    its tokens [H, C], from its tokens to the state behind it [H, C], and over the whole chunk [H]."""
    i = torch.arange(C, device=DEV, dtype=torch.float32)
    dist = i[:, None] - i[None, :]
    ld = ld[:, None]
    D = torch.exp(ld[:, :, None] * dist.clamp(min=0)) * (dist >= 0)
    return D, torch.exp(ld * (i + 1)), torch.exp(ld * (C - 1 - i)), torch.exp(ld[:, 0] * C)


def _plain_scan(q, k, v, ld, state, C=128):
    """o_t = q_t S_t with S_t = e^ld S_{t-1} + k_t v_t^T, in chunks; 32-bit operands. Returns (o, last state)."""
    B, H, N, d = q.shape
    S = torch.zeros(B, H, d, d, device=DEV) if state is None else state
    out = torch.empty_like(v)
    W = _chunk_weights(ld, C)
    for a in range(0, N, C):
        b = min(N, a + C)
        D, win, wout, wall = W if b - a == C else _chunk_weights(ld, b - a)
        qc, kc, vc = q[:, :, a:b], k[:, :, a:b], v[:, :, a:b]
        out[:, :, a:b] = (qc @ kc.transpose(2, 3) * D) @ vc + (qc @ S) * win[:, :, None]
        S = S * wall[:, None, None] + (kc * wout[:, :, None]).transpose(2, 3) @ vc
    return out, S


def _plain_decay_fwd(st):
    q, k, v = (st[x].float() for x in "qkv")
    o, S = _plain_scan(q / math.sqrt(q.shape[-1]), k, v, st["log_decay"], st.get("state"))
    return o.to(BF16), S


def _plain_decay_train(st):
    q, k, v, do = (st[x].float() for x in ("q", "k", "v", "dout"))
    ld, s0, ds1 = st["log_decay"], st.get("state"), st["dstate"]
    q = q / math.sqrt(q.shape[-1])
    o, S = _plain_scan(q, k, v, ld, s0)
    # dq_t = S_t do_t: the same recurrence with values and keys exchanged
    dq, _ = _plain_scan(do, v, k, ld, None if s0 is None else s0.transpose(2, 3))
    # E_t = e^ld E_{t+1} + q_t do_t^T, backwards; the incoming gradient of the last state stands one token behind
    # the last, without a decay of its own
    fl = lambda x: x.flip(2)
    decay = torch.exp(ld)[:, None, None]
    E = ds1 / decay
    dv, E1 = _plain_scan(fl(k), fl(q), fl(do), ld, E)
    dk, _ = _plain_scan(fl(v), fl(do), fl(q), ld, E.transpose(2, 3))
    g = [(dq / math.sqrt(q.shape[-1])).to(BF16), fl(dk).to(BF16), fl(dv).to(BF16)]
    if s0 is not None:
        g.append(E1 * decay)
    return (o.to(BF16), S) + tuple(g)


def _plain_decay_step(st):
    q, k, v = (st[x].float() for x in "qkv")
    S = st["state"] * torch.exp(st["log_decay"])[:, None, None] + k.unsqueeze(3) * v.unsqueeze(2)
    o = (q.unsqueeze(2) @ S).squeeze(2) / math.sqrt(q.shape[-1])
    return o.to(BF16), S


_OWN = {"write": _own_write, "round_trip": _own_round_trip, "attn": _own_attn, "decay_fwd": _own_decay_fwd,
        "decay_train": _own_decay_train, "decay_step": _own_decay_step}
_PLAIN = {"write": _plain_write, "round_trip": _plain_round_trip, "attn": _plain_attn, "decay_fwd": _plain_decay_fwd,
          "decay_train": _plain_decay_train, "decay_step": _plain_decay_step}


# ------------------------------------------------------------------ 64 bits
def _nearest_e4m3(y):
    """Nearest E4M3 value (ties to even, saturating) of 64-bit numbers: 4 significant bits from 2^-6 on, steps of
    2^-9 below."""
    _, e = torch.frexp(y.abs().clamp(min=2.0 ** -6))
    step = torch.ldexp(torch.ones_like(y), e - 4)
    return (torch.round(y / step) * step).clamp(-448.0, 448.0)


def _exact_rows(x, kind):
    """(values, scales) that a cache row of bf16 numbers x stands for, in 64 bits. The two 32-bit numbers M / a and
    x M / a are part of the definition."""
    x = x.double()
    if kind == "bf16":
        return x, None
    M = QMAX[kind]
    amax = x.abs().amax(dim=-1)
    some = amax > 0
    amax = amax.clamp(min=M * 2.0 ** -126)
    r = torch.where(some, M / amax, torch.ones_like(amax)).float().double()
    y = (x * r.unsqueeze(-1)).float().double()
    codes = torch.round(y).clamp(-M, M) if kind == "int8" else _nearest_e4m3(y)
    scale = torch.where(some, amax / M, torch.ones_like(amax))
    return codes * scale.unsqueeze(-1), scale


def _exact_cache(st):
    """Caches and scales after the new tokens entered, token by token position computed on the host."""
    case = st["case"]
    page, kind = case["page"], case["kind"]
    table = st["table"].cpu().numpy()
    idx = []
    for s, (L, n) in enumerate(zip(st["kv"], st["new"])):
        for p in range(L - n, L):
            idx.append((int(table[s, p // page]), p % page))
    pg, sl = (torch.tensor(t, device=DEV) for t in zip(*idx))
    out = {}
    for x in "kv":
        c = st[x + "_cache"].double()
        if kind != "bf16":
            sc = st[x + "_scale"].double()
            c = c * sc.unsqueeze(-1)
        val, scale = _exact_rows(st[x], kind)
        c[pg, :, sl] = val
        out[x] = c
        if kind != "bf16":
            sc[pg, :, sl] = scale
            out[x + "_scale"] = sc
    return out


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op in ("write", "round_trip"):
        c = _exact_cache(st)
        if op == "write":
            return {"k_cache": c["k"], "v_cache": c["v"]}
        page = case["page"]
        table = st["table"].cpu().numpy()
        out = {}
        for x in "kv":
            rows = []
            for s, L in enumerate(st["kv"]):
                p = np.arange(L)
                rows.append(c[x][torch.from_numpy(table[s, p // page].astype(np.int64)).to(DEV), :,
                                 torch.from_numpy(p % page).to(DEV)])
            out[x] = torch.cat(rows)
        if case["kind"] != "bf16":
            out["k_scale"], out["v_scale"] = c["k_scale"], c["v_scale"]
        return out
    if op == "attn":
        return _exact_attn(st)
    return _exact_decay(st)


def _exact_attn(st):
    case = st["case"]
    Hkv, G, d, page = case["Hkv"], case["G"], case["d"], case["page"]
    if work(case)["flops"] > 3e12 or work(case)["bytes"] > 12e9:
        return None
    table = st["table"].cpu().numpy()
    out = torch.empty(st["T"], Hkv * G, d, dtype=torch.float64, device=DEV)
    at = 0
    for s, (L, n) in enumerate(zip(st["kv"], st["new"])):
        p = np.arange(L)
        pg = torch.from_numpy(table[s, p // page].astype(np.int64)).to(DEV)
        sl = torch.from_numpy(p % page).to(DEV)
        kv = []
        for x in ("k", "v"):
            c = st[x + "_cache"]
            c = c.view(torch.uint8)[pg, :, sl].view(c.dtype).double() if c.element_size() == 1 else c[pg, :, sl].double()
            if st[x + "_scale"] is not None:
                c = c * st[x + "_scale"][pg, :, sl].double().unsqueeze(-1)
            kv.append(c)                                       # [L, Hkv, d]
        k, v = kv
        for h in range(Hkv):
            q = st["q"][at:at + n, h * G:(h + 1) * G].double().reshape(n * G, d)
            step = max(G, int(2 ** 27 // L) // G * G)
            for i in range(0, n * G, step):
                z = torch.einsum("id,jd->ij", q[i:i + step], k[:, h]) * d ** -0.5
                if case["causal"]:
                    tok = torch.arange(i, min(n * G, i + step), device=DEV) // G
                    z = torch.where(torch.arange(L, device=DEV)[None] <= (L - n + tok)[:, None], z,
                                    torch.full_like(z, -math.inf))
                z = torch.softmax(z, dim=1)
                o = z @ v[:, h]
                r = torch.arange(i, i + o.shape[0], device=DEV)
                out[at + r // G, h * G + r % G] = o
        at += n
    return out


def _exact_recurrence(a, b, c, ld, init, reverse):
    """y_t = R_t^T a_t with R_t = e^ld R_{t -+ 1} + b_t c_t^T along time or against it, in 64 bits, in blocks of 96
    tokens; returns y and the last R."""
    B, H, N, d = a.shape
    if reverse:
        a, b, c = a.flip(2), b.flip(2), c.flip(2)
    R = torch.zeros(B, H, d, d, dtype=torch.float64, device=DEV) if init is None else init.double()
    y = torch.zeros(B, H, N, d, dtype=torch.float64, device=DEV)
    for s in range(0, N, 96):
        e = min(N, s + 96)
        t = torch.arange(1, e - s + 1, device=DEV, dtype=torch.float64)
        lag = t[:, None] - t[None, :]
        w = torch.where(lag >= 0, torch.exp(ld[:, None, None] * lag.clamp(min=0)), torch.zeros_like(lag))
        sc = torch.einsum("bhid,bhjd->bhij", a[:, :, s:e], b[:, :, s:e]) * w
        y[:, :, s:e] = sc @ c[:, :, s:e]
        y[:, :, s:e] += torch.exp(ld[:, None] * t)[None, :, :, None] * torch.einsum("bhik,bhkd->bhid", a[:, :, s:e], R)
        left = torch.exp(ld[:, None] * (e - s - t))[None, :, :, None]
        R = R * torch.exp(ld * (e - s))[None, :, None, None]
        R = R + torch.einsum("bhjk,bhjd->bhkd", b[:, :, s:e] * left, c[:, :, s:e])
    return (y.flip(2) if reverse else y), R


def _exact_decay(st):
    op = st["case"]["op"]
    q, k, v = (st[x].double() for x in "qkv")
    ld = st["log_decay"].double()
    s0 = st.get("state")
    d = q.shape[-1]
    if op == "decay_step":
        S = s0.double() * torch.exp(ld)[None, :, None, None] + torch.einsum("bhk,bhd->bhkd", k, v)
        return torch.einsum("bhk,bhkd->bhd", q, S) * d ** -0.5, S
    o, S = _exact_recurrence(q, k, v, ld, s0, False)
    o *= d ** -0.5
    if op == "decay_fwd":
        return o, S
    do = st["dout"].double() * d ** -0.5
    dq, _ = _exact_recurrence(do, v, k, ld, None if s0 is None else s0.transpose(2, 3), False)
    ahead = st["dstate"].double() * torch.exp(-ld)[None, :, None, None]
    dv, E = _exact_recurrence(k, q, do, ld, ahead, True)
    dk, _ = _exact_recurrence(v, do, q, ld, ahead.transpose(2, 3), True)
    g = (dq, dk, dv)
    if s0 is not None:
        g += (E * torch.exp(ld)[None, :, None, None],)
    return (o, S) + g

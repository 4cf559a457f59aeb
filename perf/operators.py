"""Cases that measure the position and shared-prefix operators.

Two operators that sit in front of and beside jagged attention:

* rope: rotary positions of Q and K rows ([T, H, d], token-major), forward and
  its gradient (the inverse rotation);
* prefix: attention of a jagged batch whose samples come in groups that share
  a long prefix of keys (one user's history, many candidate ads), each sample
  also having a few keys of its own; softmax or an element-wise activation,
  forward and gradients.

``run`` computes them in plain torch operations (``own = False``) or through
the package's calls (``own = True``).
"""

import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------- cases

def _rope(name, op="rope_fwd", dtype="bf16", T=64, samples=0, med=0, H=8, Hk=8, d=128, rot=128,
          layout="half", scaling="none", far=0, packed=False, lens=1):
    c = dict(op=op, dtype=dtype, T=T, samples=samples, med=med, H=H, Hk=Hk, d=d, rot=rot,
             layout=layout, scaling=scaling, far=far, packed=packed, lens=lens)
    return dict(c, name=name) if name else c


def _prefix(name, op="prefix_fwd", dtype="bf16", act="softmax", G=1, cand=(1, 1), q=(1, 1),
            p=(1, 1), kv=(0, 0), H=8, Hkv=8, d=128, window=0, gain=2.0, lens=1):
    c = dict(op=op, dtype=dtype, act=act, G=G, cand_lo=cand[0], cand_hi=cand[1], q_lo=q[0],
             q_hi=q[1], p_lo=p[0], p_hi=p[1], kv_lo=kv[0], kv_hi=kv[1], H=H, Hkv=Hkv, d=d,
             window=window, gain=gain, lens=lens)
    return dict(c, name=name) if name else c


def listed():
    return [
        # the newest event of each of 64 users, ranked one step at a time: latency
        _rope("rope_step", T=64, far=100000, layout="half"),
        # the windowed self-attention batch (256 samples, median 200 events, 4 heads), Q and K
        # taken from one packed projection
        _rope("rope_selfattn_packed", samples=256, med=200, T=0, H=4, Hk=4, packed=True, lens=1),
        # event times in seconds as positions, part of each head, float32, odd row count
        _rope("rope_far_f32", dtype="f32", T=40009, H=2, Hk=2, d=32, rot=24, layout="interleaved",
              scaling="by_parts", far=2000000000),
        # gradients of a training batch's Q and K, float32 as the attention backward gives them
        _rope("rope_train_grad", op="rope_bwd", dtype="f32", samples=512, med=200, T=0, H=8, Hk=8,
              scaling="linear", lens=4),
        # one user, 16 candidates against a history of 4096 events: latency
        _prefix("prefix_step", cand=(16, 16), p=(4096, 4096), H=4, Hkv=4),
        # one user's ranking request: 512 candidates with 8-64 context keys each
        _prefix("prefix_rank", cand=(512, 512), p=(16384, 16384), kv=(8, 64)),
        # requests of 24 users served together, ragged everywhere, shared key heads
        _prefix("prefix_users_gqa", G=24, cand=(1, 128), q=(1, 4), p=(1, 8192), kv=(0, 64), Hkv=2),
        # candidate sequences with a causal window of their own, SiLU weights, 64-wide heads
        _prefix("prefix_silu_window", act="silu", G=8, cand=(16, 64), q=(16, 64), p=(200, 4096),
                kv=(-1, -1), H=4, Hkv=4, d=64, window=256, gain=1.0),
        # the tiny float32 configuration's heads
        _prefix("prefix_tiny_f32", dtype="f32", G=4, cand=(1, 8), q=(1, 16), p=(0, 1000),
                kv=(0, 64), H=2, Hkv=2, d=32, gain=1.5),
        # the largest: two users, 512 candidates of 4 tokens, histories of 32768 events
        _prefix("prefix_long", G=2, cand=(512, 512), q=(4, 4), p=(32768, 32768), kv=(8, 64)),
        # training on impressions grouped by request: 32 users, ragged
        _prefix("prefix_train", op="prefix_bwd", G=32, cand=(8, 32), q=(1, 8), p=(64, 2048),
                kv=(8, 128)),
        # the same with GELU weights, longer histories and more impressions per user
        _prefix("prefix_train_gelu", op="prefix_bwd", act="gelu_tanh", G=4, cand=(256, 256),
                q=(4, 4), p=(8192, 8192), kv=(8, 64), H=4, Hkv=4, gain=1.0),
    ]


def _spread(rng, lo, hi):
    """An integer of [lo, hi], even in its logarithm (lo >= 1)."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def _draw_rope(rng):
    d = rng.choice((16, 32, 40, 64, 96, 128))
    rot = 2 * rng.randint(1, d // 2) if rng.random() < 0.5 else d
    jagged = rng.random() < 0.5
    c = _rope("", op=rng.choice(("rope_fwd", "rope_fwd", "rope_bwd")),
              dtype=rng.choice(("bf16", "bf16", "f32")), H=_spread(rng, 1, 16),
              Hk=rng.choice((0, 1, 2, 4, 8)), d=d, rot=rot,
              layout=rng.choice(("half", "interleaved")),
              scaling=rng.choice(("none", "linear", "ntk", "by_parts")), packed=rng.random() < 0.3,
              lens=rng.randint(1, 1 << 20), T=0 if jagged else _spread(rng, 1, 100000),
              samples=_spread(rng, 1, 300) if jagged else 0, med=_spread(rng, 1, 400) if jagged else 0,
              far=0 if jagged else rng.choice((4096, 1000000, 2000000000)))
    return c


def _draw_prefix(rng):
    f32 = rng.random() < 0.2
    H = rng.choice((1, 2, 4, 8))
    Hkv = rng.choice([n for n in (1, 2, 4, 8) if n <= H])
    qs, cs = _spread(rng, 1, 32), _spread(rng, 1, 256)
    ph, kvh = _spread(rng, 1, 20000), rng.choice((0, 1, 33, 64, 128))
    kv = (-1, -1) if rng.random() < 0.2 else (min(kvh, rng.choice((0, 1, 8))), kvh)
    return _prefix("", op=rng.choice(("prefix_fwd", "prefix_fwd", "prefix_bwd")),
                   dtype="f32" if f32 else "bf16",
                   act=rng.choice(("softmax", "softmax", "silu", "gelu_tanh")),
                   G=_spread(rng, 1, 32), cand=(max(1, cs // rng.choice((1, 8))), cs),
                   q=(max(1, qs // rng.choice((1, 4))), qs), p=(ph // rng.choice((1, 10)), ph), kv=kv,
                   H=H, Hkv=Hkv, d=rng.choice((16, 32, 40, 64, 128)) if f32 else rng.choice((64, 128)),
                   window=rng.choice((0, 0, 1, 20, 256)), gain=rng.choice((1.0, 1.5, 2.0)),
                   lens=rng.randint(1, 1 << 20))


def draw(rng):
    top = {op: max(work(c)["flops"] for c in listed() if c["op"] == op)
           for op in ("prefix_fwd", "prefix_bwd")}
    while True:
        c = _draw_rope(rng) if rng.random() < 0.4 else _draw_prefix(rng)
        if c["op"].startswith("rope"):
            if 0 < _rope_rows(c)[-1] <= 200000 and work(c)["bytes"] <= 2.0e9:
                return c
            continue
        lq, lkv, grp, lp = _lengths(c)
        rows = np.add.reduceat(lq, np.searchsorted(grp, np.arange(c["G"])))
        area = c["G"] * c["H"] * int(rows.max()) * max(1, int(lp.max()))
        slow = 40 if c["dtype"] == "f32" else 1   # float32 products run on the CUDA cores
        if area <= 6e8 and work(c)["flops"] * slow <= top[c["op"]]:
            return c


def _loguniform(rng, lo, hi, n):
    if lo == hi:
        return np.full(n, lo, dtype=np.int64)
    a = np.exp(rng.uniform(math.log(lo + 1.0), math.log(hi + 1.0), size=n)) - 1.0
    return np.clip(np.rint(a), lo, hi).astype(np.int64)


def _rope_rows(c):
    """Offsets of the samples a rope case's rows belong to."""
    if not c["samples"]:
        return np.arange(c["T"] + 1)
    rng = np.random.Generator(np.random.PCG64(c["lens"]))
    n = np.clip(np.rint(np.exp(math.log(c["med"]) + rng.standard_normal(c["samples"]))), 0, 2048)
    return np.concatenate([[0], np.cumsum(n.astype(np.int64))])


def _lengths(c):
    """Per sample: queries, own keys, group; per group: prefix length."""
    rng = np.random.Generator(np.random.PCG64(c["lens"]))
    cand = _loguniform(rng, c["cand_lo"], c["cand_hi"], c["G"])
    lp = _loguniform(rng, c["p_lo"], c["p_hi"], c["G"])
    B = int(cand.sum())
    lq = _loguniform(rng, c["q_lo"], c["q_hi"], B)
    lkv = lq.copy() if c["kv_lo"] < 0 else _loguniform(rng, c["kv_lo"], c["kv_hi"], B)
    return lq, lkv, np.repeat(np.arange(c["G"]), cand), lp


def _pairs(c):
    lq, lkv, grp, lp = _lengths(c)
    n = int((lq * lp[grp]).sum())
    if not c["window"]:
        return n + int((lq * lkv).sum())
    for a, b in zip(lq.tolist(), lkv.tolist()):
        i = np.arange(a)
        n += int(np.maximum(0, np.minimum(i + 1, b) - np.maximum(0, i + 1 - c["window"])).sum())
    return n


def work(case):
    c = case
    e = 2 if c["dtype"] == "bf16" else 4
    if c["op"].startswith("rope"):
        T = int(_rope_rows(c)[-1])
        # one sine and cosine per row and pair of columns, four products and two sums per pair
        return {"bytes": 2 * T * (c["H"] + c["Hk"]) * c["d"] * e + 8 * T,
                "flops": T * (c["H"] + c["Hk"]) * (c["rot"] // 2) * 6}
    lq, lkv, _, lp = _lengths(c)
    tq, tk, tp = int(lq.sum()), int(lkv.sum()), int(lp.sum())
    row_q, row_k = c["H"] * c["d"] * e, c["Hkv"] * c["d"] * e
    sm = c["act"] == "softmax"
    if c["op"] == "prefix_fwd":
        return {"bytes": 2 * tq * row_q + 2 * (tk + tp) * row_k + (4 * tq * c["H"] if sm else 0),
                "flops": 4 * c["d"] * c["H"] * _pairs(c)}
    return {"bytes": (4 if sm else 3) * tq * row_q + 4 * (tk + tp) * row_k + (4 * tq * c["H"] if sm else 0),
            "flops": 10 * c["d"] * c["H"] * _pairs(c)}


# ------------------------------------------------------------------ inputs

_SCALED = dict(factor=4.0, orig_len=4096, lo=1.0, hi=32.0)


def _freqs(c):
    """Radians per position of each pair of columns (float64, the scaling applied)."""
    n = c["rot"]
    base = 10000.0
    if c["scaling"] == "ntk" and n > 2:
        base *= _SCALED["factor"] ** (n / (n - 2.0))
    f = base ** (-np.arange(0, n, 2, dtype=np.float64) / n)
    if c["scaling"] == "linear":
        f = f / _SCALED["factor"]
    if c["scaling"] == "by_parts":
        turns = _SCALED["orig_len"] * f / (2 * math.pi)
        keep = np.clip((turns - _SCALED["lo"]) / (_SCALED["hi"] - _SCALED["lo"]), 0.0, 1.0)
        f = f / _SCALED["factor"] * (1.0 - keep) + f * keep
    return f


def _amplitude(c):
    return 0.1 * math.log(_SCALED["factor"]) + 1.0 if c["scaling"] == "by_parts" else 1.0


def _inputs_rope(c, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    dt = DTYPES[c["dtype"]]
    off = _rope_rows(c)
    T, H, Hk, d = int(off[-1]), c["H"], c["Hk"], c["d"]
    if c["packed"]:   # rows of one projection: Q heads, K heads, then as many V heads
        w = torch.randn((T, H + 2 * Hk, d), generator=g, device="cuda").to(dt)
        q, k = w[:, :H], w[:, H:H + Hk]
    else:
        q = torch.randn((T, H, d), generator=g, device="cuda").to(dt)
        k = torch.randn((T, Hk, d), generator=g, device="cuda").to(dt)
    s = dict(case=c, q=q, k=k if Hk else None, T=T)
    if c["samples"]:   # positions count from each sample's start, after 100 events seen before
        s["offsets"] = torch.from_numpy(off.astype(np.int32)).cuda()
        s["starts"] = torch.full((c["samples"],), 100, dtype=torch.int32, device="cuda")
        pos = np.arange(T) - np.repeat(off[:-1], np.diff(off)) + 100
        s["pos"] = torch.from_numpy(pos.astype(np.int64)).cuda()
    else:
        s["pos"] = torch.randint(0, c["far"], (T,), generator=g, device="cuda", dtype=torch.int64)
    s["freqs"] = torch.from_numpy(_freqs(c)).cuda()
    return s


def _unit(n, heads, d, gain, g, dt):
    """Rows as an RMS norm leaves them, times a gain."""
    x = torch.randn((n, heads, d), generator=g, device="cuda")
    return (x * (gain * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6))).to(dt)


def _inputs_prefix(c, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    dt = DTYPES[c["dtype"]]
    lq, lkv, grp, lp = _lengths(c)
    tq, tk, tp = int(lq.sum()), int(lkv.sum()), int(lp.sum())
    H, Hkv, d = c["H"], c["Hkv"], c["d"]
    s = dict(case=c, lq=lq, lkv=lkv, grp=grp, lp=lp)
    s["q"] = _unit(tq, H, d, c["gain"], g, dt)
    s["kp"], s["vp"] = _unit(tp, Hkv, d, 1.0, g, dt), _unit(tp, Hkv, d, 1.0, g, dt)
    s["k"], s["v"] = _unit(tk, Hkv, d, 1.0, g, dt), _unit(tk, Hkv, d, 1.0, g, dt)
    if c["op"] == "prefix_bwd":
        s["do"] = torch.randn((tq, H, d), generator=g, device="cuda").to(dt)
    return s


def _padded(lengths, width):
    """[n, width] row indices of ragged rows laid end to end, and which are real."""
    start = np.cumsum(lengths) - lengths
    j = np.arange(max(1, width))
    real = j[None, :] < lengths[:, None]
    return (torch.from_numpy(np.where(real, start[:, None] + j, 0)).cuda(),
            torch.from_numpy(real).cuda())


def _layout(s):
    """Index tensors of the plain form: ragged rows as padded blocks and back."""
    c, lq, lkv, grp, lp = s["case"], s["lq"], s["lkv"], s["grp"], s["lp"]
    rows = np.bincount(grp, weights=lq, minlength=c["G"]).astype(np.int64)
    R, L = int(rows.max()), int(lq.max())
    s["gq"], _ = _padded(rows, R)
    s["gk"], s["gk_ok"] = _padded(lp, int(lp.max()))
    s["sq"], _ = _padded(lq, L)
    s["sk"], s["sk_ok"] = _padded(lkv, int(lkv.max()))
    i = torch.arange(s["sq"].shape[1], device="cuda")[:, None]
    j = torch.arange(s["sk"].shape[1], device="cuda")[None, :]
    see = (j <= i) & (j > i - c["window"]) if c["window"] else (j >= 0) & (i >= 0)
    s["s_ok"] = s["sk_ok"][:, None, :] & see[None]
    at = lambda n, w: torch.from_numpy(  # noqa: E731  (token -> place in the padded blocks)
        np.concatenate([b * w + np.arange(x) for b, x in enumerate(n)])).cuda()
    s["g_at"], s["s_at"] = at(rows, max(1, R)), at(lq, max(1, L))


def prepare(case, seed):
    c = case
    if c["op"].startswith("rope"):
        s = _inputs_rope(c, seed)
        if own:
            import recommender_model_attention_gb300 as gd
            s["rope"] = gd.Rope(c["rot"], layout=c["layout"], scaling=c["scaling"],
                                scale=_amplitude(c), **_SCALED)
        return s
    s = _inputs_prefix(c, seed)
    _layout(s)
    if c["op"] == "prefix_bwd" and c["act"] == "softmax":
        # what the forward kept for the gradients
        s["o"], s["lse"] = _plain_prefix_fwd(s)
    if own:
        import recommender_model_attention_gb300 as gd
        off = lambda n: np.concatenate([[0], np.cumsum(n)]).astype(np.int32)  # noqa: E731
        s["plan"] = gd.PrefixPlan(off(s["lq"]), off(s["lkv"]), off(np.bincount(s["grp"], minlength=c["G"])),
                                  off(s["lp"]), c["H"], c["d"], kv_heads=c["Hkv"],
                                  mask="causal_window" if c["window"] else "none",
                                  window=c["window"])
    return s


# -------------------------------------------------------------- plain forms

def _plain_rope(s, x, back):
    c = s["case"]
    n = c["rot"]
    angle = s["pos"].double()[:, None] * s["freqs"]   # far positions need more than 32 bits
    cos = (torch.cos(angle).float() * _amplitude(c))[:, None]
    sin = (torch.sin(angle).float() * (-_amplitude(c) if back else _amplitude(c)))[:, None]
    y = x.float().clone()
    if c["layout"] == "half":
        a, b = x[..., :n // 2].float(), x[..., n // 2:n].float()
        y[..., :n // 2] = a * cos - b * sin
        y[..., n // 2:n] = a * sin + b * cos
    else:
        a, b = x[..., 0:n:2].float(), x[..., 1:n:2].float()
        y[..., 0:n:2] = a * cos - b * sin
        y[..., 1:n:2] = a * sin + b * cos
    return y.to(x.dtype)


def _act(x, kind):
    """act(x) and act'(x)."""
    if kind == "silu":
        t = 1.0 / (1.0 + torch.exp(-x))
        return x * t, t * (1.0 + x * (1.0 - t))
    t = torch.tanh(math.sqrt(2.0 / math.pi) * (x + 0.044715 * x * x * x))
    du = math.sqrt(2.0 / math.pi) * (1.0 + 3 * 0.044715 * x * x)
    return 0.5 * x * (1.0 + t), 0.5 * (1.0 + t) + 0.5 * x * (1.0 - t * t) * du


def _heads(x, at, Hkv):
    """Rows x[at] ([n, w, H, d]) as [n, Hkv, (H / Hkv) w, d] in float32."""
    n, w = at.shape
    y = x[at].float().permute(0, 2, 1, 3)
    return y.reshape(n, Hkv, (y.shape[1] // Hkv) * w, y.shape[3])


def _tokens(y, at, H):
    """The inverse of _heads for the rows that are real: [T, H, ...]."""
    n, w = y.shape[0], y.shape[1] * y.shape[2] // H
    y = y.reshape((n, H, w) + tuple(y.shape[3:])).transpose(1, 2)
    return y.reshape((n * w, H) + tuple(y.shape[3:]))[at]


def _blocks(t, at, Hkv):
    """Per-token values [T, H] in the row order of _heads: [n, Hkv, rows, 1]."""
    n, w = at.shape
    y = t[at].permute(0, 2, 1)
    return y.reshape(n, Hkv, (y.shape[1] // Hkv) * w, 1)


def _parts(s):
    """Query rows, keys, values and what is masked, for the prefix and the own part."""
    c = s["case"]
    rep = c["H"] // c["Hkv"]
    yield ("gq", "g_at", _heads(s["kp"], s["gk"], c["Hkv"]) if s["kp"].shape[0] else None,
           _heads(s["vp"], s["gk"], c["Hkv"]) if s["kp"].shape[0] else None,
           ~s["gk_ok"][:, None, None, :])
    yield ("sq", "s_at", _heads(s["k"], s["sk"], c["Hkv"]) if s["k"].shape[0] else None,
           _heads(s["v"], s["sk"], c["Hkv"]) if s["k"].shape[0] else None,
           ~s["s_ok"].repeat(1, rep, 1)[:, None])


def _plain_prefix_fwd(s):
    c, alpha = s["case"], s["case"]["d"] ** -0.5
    H, Hkv = c["H"], c["Hkv"]
    o, m, l = [], [], []
    for rows, at, k, v, hidden in _parts(s):
        if k is None:
            continue
        x = _heads(s["q"], s[rows], Hkv) @ k.transpose(-1, -2) * alpha
        if c["act"] != "softmax":
            o.append(_tokens(_act(x, c["act"])[0].masked_fill_(hidden, 0.0) @ v, s[at], H))
            continue
        x = x.masked_fill_(hidden, -math.inf)
        top = x.amax(-1, keepdim=True)
        e = torch.exp(x - top.clamp_min(-1e30))
        o.append(_tokens(e @ v, s[at], H))
        m.append(_tokens(top, s[at], H))
        l.append(_tokens(e.sum(-1, keepdim=True), s[at], H))
    if c["act"] != "softmax":
        return sum(o, torch.zeros_like(s["q"], dtype=torch.float32)).to(s["q"].dtype)
    if not m:   # no key anywhere
        return torch.zeros_like(s["q"]), torch.full(s["q"].shape[:2], -math.inf, device="cuda")
    top = torch.stack(m).amax(0).clamp_min(-1e30)
    w = [torch.exp(x - top) for x in m]
    total = sum(a * b for a, b in zip(w, l))
    out = sum(a * b for a, b in zip(w, o)) / torch.where(total > 0, total, 1.0)
    lse = torch.where(total > 0, torch.log(total) + top, -math.inf)[..., 0]
    return out.to(s["q"].dtype), lse


def _plain_prefix_bwd(s):
    c, alpha = s["case"], s["case"]["d"] ** -0.5
    H, Hkv, dt = c["H"], c["Hkv"], s["q"].dtype
    sm = c["act"] == "softmax"
    dq, grads = 0.0, []
    if sm:
        delta = (s["do"].float() * s["o"].float()).sum(-1)
    for (rows, at, k, v, hidden), ok in zip(_parts(s), (s["gk_ok"], s["sk_ok"])):
        if k is None:
            grads += [s["kp" if rows == "gq" else "k"].clone(), s["vp" if rows == "gq" else "v"].clone()]
            continue
        # padded query rows repeat a real row: their upstream gradient is dropped below
        real = torch.zeros(s[rows].numel(), device="cuda").index_fill_(0, s[at], 1.0).view(s[rows].shape)
        q, do = _heads(s["q"], s[rows], Hkv), _heads(s["do"], s[rows], Hkv)
        keep = real[:, None, :].expand(-1, H // Hkv, -1).reshape(real.shape[0], 1, -1, 1)
        x = q @ k.transpose(-1, -2) * alpha
        dp = do @ v.transpose(-1, -2)
        if sm:
            p = torch.exp(x - _blocks(s["lse"].clamp_min(-1e30), s[rows], Hkv)).masked_fill_(hidden, 0.0) * keep
            ds = p * (dp - _blocks(delta, s[rows], Hkv)) * alpha
        else:
            p, ds = _act(x, c["act"])
            p = p.masked_fill_(hidden, 0.0) * keep
            ds = (ds * dp * alpha).masked_fill_(hidden, 0.0) * keep
        dq = dq + _tokens(ds @ k, s[at], H)
        flat = lambda y: y.transpose(1, 2)[ok].to(dt)  # noqa: E731  ([n, w, Hkv, d] -> real rows)
        grads += [flat(ds.transpose(-1, -2) @ q), flat(p.transpose(-1, -2) @ do)]
    return [dq.to(dt) if torch.is_tensor(dq) else torch.zeros_like(s["q"])] + grads


def run(state):
    s = state
    c = s["case"]
    op = c["op"]
    if op.startswith("rope"):
        if own:
            import recommender_model_attention_gb300 as gd
            f = gd.gdpa_rope_fwd if op == "rope_fwd" else gd.gdpa_rope_bwd
            if "offsets" in s:
                return f(s["rope"], s["q"], s["k"], offsets=s["offsets"], starts=s["starts"])
            return f(s["rope"], s["q"], s["k"], positions=s["pos"])
        out = _plain_rope(s, s["q"], op == "rope_bwd")
        return out if s["k"] is None else (out, _plain_rope(s, s["k"], op == "rope_bwd"))
    if own:
        import recommender_model_attention_gb300 as gd
        args = (s["plan"], s["q"], s["kp"], s["vp"], s["k"], s["v"])
        if op == "prefix_fwd":
            if c["act"] == "softmax":
                return gd.gdpa_prefix_softmax_fwd(*args)
            return gd.gdpa_prefix_fwd(*args, act=c["act"])
        if c["act"] == "softmax":
            return gd.gdpa_prefix_softmax_bwd(*args, s["o"], s["do"], s["lse"])
        return gd.gdpa_prefix_bwd(*args, s["do"], act=c["act"])
    return _plain_prefix_fwd(s) if op == "prefix_fwd" else _plain_prefix_bwd(s)


# ------------------------------------------------------------------ 64 bits

def _exact_rope(c, seed):
    s = _inputs_rope(c, seed)
    amp = _amplitude(c)
    turn = 1.0 if c["op"] == "rope_fwd" else -1.0
    # each pair (a, b) as the complex number a + i b, turned by e^(i angle)
    z = torch.polar(torch.full_like(s["freqs"], amp).expand(s["T"], -1).contiguous(),
                    turn * s["pos"].double()[:, None] * s["freqs"][None, :])[:, None]
    outs = []
    for x in (s["q"], s["k"]):
        if x is None:
            continue
        x, n = x.double(), c["rot"]
        if c["layout"] == "half":
            w = torch.complex(x[..., :n // 2].contiguous(), x[..., n // 2:n].contiguous()) * z
            y = torch.cat([w.real, w.imag, x[..., n:]], -1)
        else:
            w = torch.view_as_complex(x[..., :n].reshape(x.shape[0], x.shape[1], n // 2, 2).contiguous()) * z
            y = torch.cat([torch.view_as_real(w).reshape(x.shape[0], x.shape[1], n), x[..., n:]], -1)
        outs.append(y)
    return outs[0] if len(outs) == 1 else tuple(outs)


def _exact_act(x, kind):
    if kind == "silu":
        return x * torch.sigmoid(x), torch.sigmoid(x) + x * torch.sigmoid(x) * torch.sigmoid(-x)
    u = 0.7978845608028654 * x * (1.0 + 0.044715 * x ** 2)
    th = torch.tanh(u)
    return x * (1.0 + th) / 2, (1.0 + th) / 2 + x / 2 * 0.7978845608028654 * (1.0 + 0.134145 * x ** 2) / torch.cosh(u) ** 2


def _exact_prefix(c, seed):
    """Group by group and head by head: all keys a group's rows can see side by side, the rest masked."""
    if 10 * c["d"] * c["H"] * _pairs(c) > 1e13:
        return None
    s = _inputs_prefix(c, seed)
    lq, lkv, grp, lp = s["lq"], s["lkv"], s["grp"], s["lp"]
    alpha, rep, bwd, sm = c["d"] ** -0.5, c["H"] // c["Hkv"], c["op"] == "prefix_bwd", c["act"] == "softmax"
    if bwd and sm:
        _layout(s)
        s["o"], s["lse"] = _plain_prefix_fwd(s)   # inputs of the gradients
    x64 = {n: s[n].double() for n in ("q", "kp", "vp", "k", "v") + (("do",) if bwd else ())}
    o, lse = torch.zeros_like(x64["q"]), torch.full(x64["q"].shape[:2], -math.inf, device="cuda", dtype=torch.float64)
    grads = {n: torch.zeros_like(x64[n]) for n in ("q", "kp", "vp", "k", "v")} if bwd else None
    q0, k0, p0 = 0, 0, 0
    for g in range(c["G"]):
        mine = grp == g
        nq, nk, npre = int(lq[mine].sum()), int(lkv[mine].sum()), int(lp[g])
        sample_q = torch.from_numpy(np.repeat(np.arange(mine.sum()), lq[mine])).cuda()
        sample_k = torch.from_numpy(np.repeat(np.arange(mine.sum()), lkv[mine])).cuda()
        place = lambda n: torch.from_numpy(np.concatenate([np.arange(a) for a in n] + [np.zeros(0, np.int64)]).astype(np.int64)).cuda()  # noqa: E731
        i, j = place(lq[mine])[:, None], place(lkv[mine])[None, :]
        see = sample_q[:, None] == sample_k[None, :]
        if c["window"]:
            see = see & (j <= i) & (i - j < c["window"])
        see = torch.cat([torch.ones((nq, npre), dtype=torch.bool, device="cuda"), see], 1)
        Q, Ks, Ps = slice(q0, q0 + nq), slice(k0, k0 + nk), slice(p0, p0 + npre)
        for h in range(c["H"]):
            e = h // rep
            key = torch.cat([x64["kp"][Ps, e], x64["k"][Ks, e]])
            val = torch.cat([x64["vp"][Ps, e], x64["v"][Ks, e]])
            x = alpha * torch.mm(x64["q"][Q, h], key.t())
            if not bwd:
                if sm:
                    x = torch.where(see, x, -math.inf)
                    lse[Q, h] = torch.logsumexp(x, 1)
                    o[Q, h] = torch.mm(torch.nan_to_num(torch.exp(x - lse[Q, h][:, None])), val)
                else:
                    o[Q, h] = torch.mm(torch.where(see, _exact_act(x, c["act"])[0], 0.0), val)
                continue
            dout = x64["do"][Q, h]
            dp = torch.mm(dout, val.t())
            if sm:
                p = torch.where(see, torch.exp(x - s["lse"][Q, h].double()[:, None]), 0.0)
                ds = p * (dp - (dout * s["o"][Q, h].double()).sum(1, keepdim=True))
            else:
                p, slope = _exact_act(x, c["act"])
                p, ds = torch.where(see, p, 0.0), torch.where(see, slope * dp, 0.0)
            grads["q"][Q, h] = alpha * torch.mm(ds, key)
            dkey, dval = alpha * torch.mm(ds.t(), x64["q"][Q, h]), torch.mm(p.t(), dout)
            grads["kp"][Ps, e] += dkey[:npre]
            grads["vp"][Ps, e] += dval[:npre]
            grads["k"][Ks, e] += dkey[npre:]
            grads["v"][Ks, e] += dval[npre:]
        q0, k0, p0 = q0 + nq, k0 + nk, p0 + npre
    if bwd:
        return [grads[n] for n in ("q", "kp", "vp", "k", "v")]
    return (o, lse) if sm else o


def exact(case, seed):
    return _exact_rope(case, seed) if case["op"].startswith("rope") else _exact_prefix(case, seed)

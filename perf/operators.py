"""Measured cases of the cache and window-attention operators.

Three operators that a serving or training program of this package uses beside
the layer itself:

- ``append``: rotary position embedding of new q / k rows and the append of
  k / v to a cache (contiguous or paged; in the working type, or in 8 bits
  with one scale per block of tokens and kv head);
- ``attend``: one query token per sequence against such a cache, over the whole
  sequence or over a sliding window plus the first ("sink") tokens;
- ``window``: causal attention of whole sequences over a sliding window plus
  sink tokens, forward alone or with its gradients.

``run`` computes a case in plain torch (``own`` false) or through the package's
entry points (``own`` true).
"""
import math

import numpy as np
import torch

own = False

QMAX = {"i8": 127.0, "e4m3": 448.0}


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one decode step's append for 64 sequences of a paged bf16 cache: latency
        dict(name="append_token_paged_bf16", op="append", B=64, n=1, ragged=False, Hq=8, Hkv=2, d=64, cap=2048, page=64,
             fmt="native", block=0, dtype="bf16", base=500000.0),
        # chunked prefill into a contiguous cache behind a prefix, ragged chunk lengths
        dict(name="append_chunk_ragged_bf16", op="append", B=3, n=517, ragged=True, Hq=32, Hkv=8, d=128, cap=2048, page=0,
             fmt="native", block=0, dtype="bf16", base=500000.0),
        # a batch of prompts quantised into a paged int8 cache, and the values read back
        dict(name="append_prefill_paged_i8", op="append", B=4, n=4096, ragged=False, Hq=16, Hkv=4, d=32, cap=8192, page=64,
             fmt="i8", block=64, dtype="bf16", base=10000.0),
        # chunks of odd length into an e4m3 cache whose last block is partly filled
        dict(name="append_chunk_e4m3", op="append", B=2, n=1001, ragged=True, Hq=32, Hkv=8, d=128, cap=4096, page=0,
             fmt="e4m3", block=32, dtype="bf16", base=500000.0),
        # the decode workload of the package (64 x 16384 tokens), its cache in int8
        dict(name="attend_b64_l16384_i8", op="attend", B=64, full=True, Hq=8, Hkv=2, d=64, cap=16384, page=0, fmt="i8", block=64,
             dtype="bf16", window=0, sinks=0),
        # a serving batch of ragged lengths, paged e4m3 cache, heads of 128
        dict(name="attend_ragged_paged_e4m3", op="attend", B=16, full=False, Hq=32, Hkv=8, d=128, cap=8192, page=64, fmt="e4m3",
             block=32, dtype="bf16", window=0, sinks=0),
        # a single short conversation: latency
        dict(name="attend_b1_short_i8", op="attend", B=1, full=True, Hq=16, Hkv=4, d=32, cap=1008, page=0, fmt="i8", block=16,
             dtype="bf16", window=0, sinks=0),
        # streaming with a window and four sink tokens over a long bf16 cache
        dict(name="attend_window_bf16", op="attend", B=32, full=False, Hq=8, Hkv=2, d=64, cap=32768, page=0, fmt="native", block=0,
             dtype="bf16", window=4096, sinks=4),
        # prefill of a long prompt of a sliding-window layer
        dict(name="window_prefill_s16384", op="window", B=1, S=16384, Hq=8, Hkv=2, d=64, dtype="bf16", window=1024, sinks=4,
             train=False),
        # a training step of a grouped-query layer with heads of 128
        dict(name="window_train_s4096_d128", op="window", B=1, S=4096, Hq=32, Hkv=8, d=128, dtype="bf16", window=1024, sinks=0,
             train=True),
        # a short training step of odd length: latency
        dict(name="window_train_s301_d32", op="window", B=2, S=301, Hq=16, Hkv=4, d=32, dtype="bf16", window=100, sinks=3,
             train=True),
        # a long training step with a wide window and a few more sinks
        dict(name="window_train_s8192_d64", op="window", B=1, S=8192, Hq=8, Hkv=2, d=64, dtype="bf16", window=4096, sinks=16,
             train=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    Hq, Hkv, d = rng.choice([(8, 2, 64), (16, 4, 32), (32, 8, 128), (12, 4, 64), (8, 8, 128), (16, 1, 64), (6, 3, 32)])
    op = rng.choice(["append", "attend", "window"])
    base = rng.choice([10000.0, 500000.0])
    fmt = rng.choice(["native", "i8", "e4m3"])
    block = 0 if fmt == "native" else rng.choice([16, 32, 64])
    page = rng.choice([0, 64, 128])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    window = rng.choice([0, 1]) * _log(rng, 16, 4096)
    sinks = rng.choice([0, 1, 4, 37]) if window else 0
    if op == "append":
        n = _log(rng, 1, 2000)
        room = rng.randint(1, 1000)
        return dict(op=op, B=_log(rng, 1, 16), n=n, ragged=rng.random() < 0.5, Hq=Hq, Hkv=Hkv, d=d, cap=-(-(n + room) // 128) * 128,
                    page=page, fmt=fmt, block=block, dtype="bf16" if fmt != "native" else dtype, base=base)
    if op == "attend":
        cap = -(-_log(rng, 1, 20000) // 128) * 128
        most = max(1, min(64, 64 * 16384 * 128 // (cap * Hkv * d * (4 if dtype == "f32" else 2))))
        return dict(op=op, B=_log(rng, 1, most), full=rng.random() < 0.3, Hq=Hq, Hkv=Hkv, d=d, cap=cap, page=page, fmt=fmt,
                    block=block, dtype=dtype, window=window, sinks=sinks)
    S = _log(rng, 16, 1500 if dtype == "f32" else 4096)
    B = _log(rng, 1, max(1, min(4, 8192 // S)))
    return dict(op=op, B=B, S=S, Hq=Hq, Hkv=Hkv, d=d, dtype=dtype, window=window, sinks=sinks, train=rng.random() < 0.6)


# ------------------------------------------------------------------ state
def _dt(c):
    return torch.float32 if c["dtype"] == "f32" else torch.bfloat16


def _randn(g, shape, dtype):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).to(dtype)


def _pool_of(dense, table, page):
    """[B, Hkv, cap, d] -> pool [n_pages, Hkv, page, d] in the table's order."""
    B, H, cap, d = dense.shape
    pages = dense.view(B, H, cap // page, page, d).permute(0, 2, 1, 3, 4).reshape(-1, H, page, d)
    pool = torch.empty_like(pages)
    pool[table.view(-1).long()] = pages
    return pool


def _make_cache(c, g, rng, lens):
    """Cache tensors holding random rows everywhere (rows past a sequence's length are what an earlier one left there)."""
    B, H, cap, d, page = c["B"], c["Hkv"], c["cap"], c["d"], c["page"]
    s = {"len": torch.from_numpy(lens.astype(np.int32)).cuda()}
    if page:
        s["table"] = torch.from_numpy(rng.permutation(B * (cap // page)).astype(np.int32).reshape(B, -1)).cuda()
    for name in ("k", "v"):
        if c["fmt"] == "native":
            x = _randn(g, (B, H, cap, d), _dt(c))
            s[name] = _pool_of(x, s["table"], page) if page else x
            continue
        x = _randn(g, (B, H, cap // c["block"], c["block"], d), torch.bfloat16)
        # blocks differ in size, as keys of different heads and tokens do
        x = x * torch.exp(0.5 * torch.randn(x.shape[:3] + (1, 1), generator=g, device="cuda")).to(x.dtype)
        scale = x.abs().amax((3, 4)).float() / QMAX[c["fmt"]]
        x = x.float() / scale[..., None, None]
        x = (x.round().clamp(-127, 127).to(torch.int8) if c["fmt"] == "i8" else x.clamp(-448, 448).to(torch.float8_e4m3fn))
        x = x.view(B, H, cap, d)
        if page:
            raw = x.view(torch.uint8) if c["fmt"] == "e4m3" else x
            x = _pool_of(raw, s["table"], page).view(x.dtype)
            scale = _pool_of(scale.view(B, H, cap // c["block"], 1), s["table"], page // c["block"]).squeeze(-1)
        s[name], s[name + "_scale"] = x.contiguous(), scale.contiguous()
    return s


def prepare(case, seed):
    c = dict(case)
    rng = np.random.RandomState((seed * 7919 + 17) % (1 << 31))
    g = torch.Generator(device="cuda").manual_seed(seed * 104729 + 5)
    dt = _dt(c)
    if c["op"] == "append":
        B, n, cap = c["B"], c["n"], c["cap"]
        new = rng.randint(max(1, n // 2), n + 1, B) if c["ragged"] else np.full(B, n)
        s = _make_cache(c, g, rng, rng.randint(0, cap - n + 1, B))
        # packed rows q | k | v, as one projection leaves them
        x = _randn(g, (B, n, c["Hq"] + 2 * c["Hkv"], c["d"]), dt)
        s["q"], s["knew"], s["vnew"] = x.split([c["Hq"], c["Hkv"], c["Hkv"]], 2)
        s["len0"], s["new"] = s["len"].clone(), torch.from_numpy(new.astype(np.int32)).cuda() if c["ragged"] else None
        s["q_out"] = torch.zeros(B, n, c["Hq"], c["d"], dtype=dt, device="cuda")
        if c["fmt"] != "native":
            s["k_read"], s["v_read"] = (torch.zeros(B, c["Hkv"], cap, c["d"], dtype=dt, device="cuda") for _ in range(2))
    elif c["op"] == "attend":
        B, cap = c["B"], c["cap"]
        s = _make_cache(c, g, rng, np.full(B, cap) if c["full"] else rng.randint(max(1, cap // 4), cap + 1, B))
        s["q"] = _randn(g, (B, c["Hq"], c["d"]), dt)
    else:
        B, S = c["B"], c["S"]
        s = {"q": _randn(g, (B, S, c["Hq"], c["d"]), dt)}
        s["k"], s["v"] = (_randn(g, (B, S, c["Hkv"], c["d"]), dt) for _ in range(2))
        if c["train"]:
            s["dout"] = _randn(g, (B, S, c["Hq"], c["d"]), dt)
    s["case"] = c
    if own:
        _handles(s)
    return s


# ------------------------------------------------------------------ the package's operators
def _handles(s):
    """What a program keeps beside its tensors: the layer's configuration and the cache's handle (pointers and a workspace)."""
    from compressed_latent_grouped_b200 import binding, device
    c = s["case"]
    s["cfg"] = binding.make_config(c["Hq"] * c["d"], 1, c["Hq"], c["Hkv"], conv_width=0, qk_mean=0, value_shift=0,
                                   rope_base=c.get("base", 0.0), dtype=binding.F32 if c["dtype"] == "f32" else binding.BF16)
    if c["op"] != "window":
        # (the pool of a single sequence may have been gathered into another order of strides)
        s["k"], s["v"] = s["k"].contiguous(), s["v"].contiguous()
        s["cache"] = device.DeviceKVCache.wrap(s["cfg"], s["k"], s["v"], s["len"], k_scale=s.get("k_scale"),
                                               v_scale=s.get("v_scale"), block_table=s.get("table"))


def _run_own(s):
    from compressed_latent_grouped_b200 import device
    c = s["case"]
    if c["op"] == "append":
        s["len"].copy_(s["len0"])
        s["cache"].append_rope(s["knew"], s["vnew"], q=s["q"], q_out=s["q_out"], n_valid=s["new"])
        if c["fmt"] == "native":
            return {"q": s["q_out"], "k": s["k"], "v": s["v"], "len": s["len"]}
        s["cache"].read(0, c["cap"], s["k_read"], s["v_read"])
        return {"q": s["q_out"], "k": s["k_read"], "v": s["v_read"], "len": s["len"]}
    if c["op"] == "attend":
        return s["cache"].attend(s["q"], window=c["window"], sinks=c["sinks"])
    if not c["train"]:
        return device.window_attention(s["cfg"], s["q"], s["k"], s["v"], window=c["window"], sinks=c["sinks"])
    out, stats = device.window_attention(s["cfg"], s["q"], s["k"], s["v"], window=c["window"], sinks=c["sinks"], with_stats=True)
    dq, dk, dv = device.window_attention_backward(s["cfg"], s["q"], s["k"], s["v"], out, stats, s["dout"], window=c["window"],
                                                  sinks=c["sinks"])
    return {"out": out, "dq": dq, "dk": dk, "dv": dv}


# ------------------------------------------------------------------ plain forms
def _rope(x, pos, base):
    """Pairs (i, i + d/2) turn by pos * base^(-2i/d); angles in 64 bits."""
    half = x.shape[-1] // 2
    theta = base ** (-2.0 * torch.arange(half, device=x.device, dtype=torch.float64) / x.shape[-1])
    ang = pos.double()[..., None, None] * theta
    cos, sin = ang.cos().float(), ang.sin().float()
    a, b = x[..., :half].float(), x[..., half:].float()
    return torch.cat([a * cos - b * sin, a * sin + b * cos], -1)


def _dense(s, name):
    """Cache rows [B, Hkv, cap, d] as fp32 codes (8 bits) or values, and the scales per token (None for the working type)."""
    x, scale, c = s[name], s.get(name + "_scale"), s["case"]
    if c["page"]:
        t = s["table"].long()
        B, P = t.shape
        raw = x.view(torch.uint8) if x.dtype == torch.float8_e4m3fn else x
        x = raw[t].permute(0, 2, 1, 3, 4).reshape(B, c["Hkv"], c["cap"], c["d"]).view(x.dtype)
        scale = None if scale is None else scale[t].permute(0, 2, 1, 3).reshape(B, c["Hkv"], -1)
    return x.float(), None if scale is None else scale


def _append_plain(s, name, new):
    """new [B, n, Hkv, d] (fp32, rotated) joins the cache; 8-bit caches also return their values [B, Hkv, cap, d]."""
    c = s["case"]
    B, n, cap = c["B"], c["n"], c["cap"]
    count = s["new"] if s["new"] is not None else torch.full_like(s["len0"], n)
    t = torch.arange(cap, device="cuda")[None]
    start, end = s["len0"][:, None], (s["len0"] + count)[:, None]
    fresh = ((t >= start) & (t < end))[:, None, :, None]
    at = (t - start).clamp(0, n - 1).long()[:, None, :, None].expand(B, c["Hkv"], cap, c["d"])
    x = torch.gather(new.permute(0, 2, 1, 3), 2, at)
    old, scale = _dense(s, name)
    if scale is None:
        x = torch.where(fresh, x, old).to(s[name].dtype)
    else:
        blk, qmax = c["block"], QMAX[c["fmt"]]
        split = lambda y: y.unflatten(2, (cap // blk, blk))  # noqa: E731
        amax = split(torch.where(fresh, x.abs(), 0.0)).amax((3, 4))
        held = (torch.arange(0, cap, blk, device="cuda")[None] < start)[:, None]
        hit = split(fresh).any(3).squeeze(-1)
        s_old = torch.where(held, scale, 0.0)
        s_new = torch.where(hit, torch.maximum(s_old, amax / qmax), scale)
        per = lambda y: y.repeat_interleave(blk, 2)[..., None]  # noqa: E731
        safe = torch.where(s_new > 0, s_new, 1.0)
        again = old * per(torch.where(hit & (s_new > s_old), s_old / safe, 1.0))
        stays = t[:, None, :, None] < start[:, None, :, None]
        code = torch.where(fresh, x / per(safe), torch.where(stays, again, old))
        code = code.round().clamp(-127, 127) if c["fmt"] == "i8" else code.clamp(-448, 448)
        x = code.to(s[name].dtype)
        value = torch.where((t < end)[:, None, :, None], x.float() * per(s_new), 0.0).to(_dt(c))
    if c["page"]:
        raw = x.view(torch.uint8) if x.dtype == torch.float8_e4m3fn else x
        pool = _pool_of(raw, s["table"], c["page"]).view(x.dtype)
        s[name].view(torch.uint8).copy_(pool.view(torch.uint8))
        if scale is not None:
            s[name + "_scale"].copy_(_pool_of(s_new[..., None], s["table"], c["page"] // c["block"]).squeeze(-1))
    else:
        s[name].view(torch.uint8).copy_(x.view(torch.uint8))
        if scale is not None:
            s[name + "_scale"].copy_(s_new)
    return s[name] if scale is None else value


def _visible(q_pos, k_pos, window, sinks):
    seen = k_pos <= q_pos
    return seen & ((k_pos > q_pos - window) | (k_pos < sinks)) if window else seen


def _softmax(sc, seen):
    sc = torch.where(seen, sc, -math.inf)
    top = sc.amax(-1, keepdim=True)
    p = torch.exp(sc - torch.where(top == -math.inf, 0.0, top))
    total = p.sum(-1, keepdim=True)
    return p / torch.where(total > 0, total, 1.0)


def _run_plain(s):
    c = s["case"]
    if c["op"] == "append":
        pos = s["len0"][:, None] + torch.arange(c["n"], device="cuda")[None]
        inside = (torch.arange(c["n"], device="cuda")[None] < (s["new"][:, None] if s["new"] is not None else c["n"]))
        q = torch.where(inside[..., None, None], _rope(s["q"], pos, c["base"]), 0.0).to(_dt(c))
        k = _append_plain(s, "k", _rope(s["knew"], pos, c["base"]))
        v = _append_plain(s, "v", s["vnew"].float())
        s["len"] = s["len0"] + (s["new"] if s["new"] is not None else c["n"])
        return {"q": q, "k": k, "v": v, "len": s["len"]}
    G, d = c["Hq"] // c["Hkv"], c["d"]
    if c["op"] == "attend":
        k, ks = _dense(s, "k")
        v, vs = _dense(s, "v")
        if ks is not None:
            k, v = (y * z.repeat_interleave(c["block"], 2)[..., None] for y, z in ((k, ks), (v, vs)))
        q = s["q"].float().view(c["B"], c["Hkv"], G, d)
        seen = _visible(s["len"].long()[:, None] - 1, torch.arange(c["cap"], device="cuda")[None], c["window"], c["sinks"])
        p = _softmax(torch.matmul(q, k.transpose(-1, -2)) / math.sqrt(d), seen[:, None, None])
        return torch.matmul(p, v).reshape(c["B"], c["Hq"], d).to(_dt(c))
    B, S, H = c["B"], c["S"], c["Hkv"]
    rows = lambda x: x.float().view(B, S, H, G, d).permute(0, 2, 3, 1, 4)  # noqa: E731
    keys = lambda x: x.float().permute(0, 2, 1, 3)[:, :, None]  # noqa: E731
    back = lambda x: x.permute(0, 3, 1, 2, 4).reshape(B, S, H * G, d).to(_dt(c))  # noqa: E731
    q, k, v = rows(s["q"]), keys(s["k"]), keys(s["v"])
    t = torch.arange(S, device="cuda")
    p = _softmax(torch.matmul(q, k.transpose(-1, -2)) / math.sqrt(d), _visible(t[:, None], t[None], c["window"], c["sinks"]))
    o = torch.matmul(p, v)
    if not c["train"]:
        return back(o)
    do = rows(s["dout"])
    ds = p * (torch.matmul(do, v.transpose(-1, -2)) - (do * o).sum(-1, keepdim=True)) / math.sqrt(d)
    dv = torch.matmul(p.transpose(-1, -2), do).sum(2).permute(0, 2, 1, 3).to(_dt(c))
    dk = torch.matmul(ds.transpose(-1, -2), q).sum(2).permute(0, 2, 1, 3).to(_dt(c))
    return {"out": back(o), "dq": back(torch.matmul(ds, k)), "dk": dk, "dv": dv}


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ------------------------------------------------------------------ floors
def _pairs(S, window, sinks):
    """Visible (query, key) pairs of a sequence of S tokens."""
    t = np.arange(S, dtype=np.int64)
    if not window:
        return int((t + 1).sum())
    lo = np.maximum(t - window + 1, 0)
    return int((t + 1 - lo + np.minimum(lo, sinks)).sum())


def work(case):
    c = case
    es = 4 if c["dtype"] == "f32" else 2
    row = c["Hkv"] * c["d"]
    if c["op"] == "append":
        # half to all of a ragged chunk: three quarters on average
        tokens = c["B"] * c["n"] * (0.75 if c["ragged"] else 1.0)
        cell = es if c["fmt"] == "native" else 1
        b = tokens * (2 * c["Hq"] * c["d"] * es + 2 * row * (es + cell))
        if c["fmt"] != "native":   # the values of every held token, read back
            held = c["B"] * (c["cap"] - c["n"]) / 2 + tokens
            b += held * 2 * row * (1 + es)
        return {"bytes": b, "flops": tokens * (c["Hq"] + c["Hkv"]) * c["d"] * 3}
    if c["op"] == "attend":
        tokens = c["cap"] * (1.0 if c["full"] else 0.625)
        if c["window"]:
            tokens = min(tokens, c["window"] + c["sinks"])
        cell = es if c["fmt"] == "native" else 1 + 4.0 / (c["block"] * c["d"])
        return {"bytes": c["B"] * (tokens * 2 * row * cell + 2 * c["Hq"] * c["d"] * es),
                "flops": 4.0 * c["B"] * c["Hq"] * c["d"] * tokens}
    pairs = c["B"] * c["Hq"] * _pairs(c["S"], c["window"], c["sinks"])
    io = c["B"] * c["S"] * (c["Hq"] * 2 + c["Hkv"] * 2) * c["d"] * es
    return {"bytes": io * (1 if not c["train"] else 3), "flops": pairs * c["d"] * (4.0 if not c["train"] else 14.0)}


# ------------------------------------------------------------------ 64 bits
def _values64(s, name):
    """Codes and scales [B, Hkv, cap, d] in 64 bits, page by page."""
    c = s["case"]
    x = s[name].double()
    sc = s[name + "_scale"].double() if name + "_scale" in s else None
    if c["page"]:
        order = s["table"].long().cpu().tolist()
        x = torch.stack([torch.cat([x[p] for p in row], 1) for row in order])
        sc = None if sc is None else torch.stack([torch.cat([sc[p] for p in row], 1) for row in order])
    return x, sc


def _turned64(x, pos, base):
    d = x.shape[-1]
    z = torch.complex(x[..., : d // 2].double(), x[..., d // 2:].double())
    rate = torch.exp(torch.arange(d // 2, device=x.device, dtype=torch.float64) * (-2.0 * math.log(base) / d))
    a = pos.double()[:, None] * rate
    z = z * torch.polar(torch.ones_like(a), a)[:, None]
    return torch.cat([z.real, z.imag], -1)


def _exact_append(s):
    c = s["case"]
    out = {"q": torch.zeros(c["B"], c["n"], c["Hq"], c["d"], dtype=torch.float64, device="cuda"), "len": None}
    for name in ("k", "v"):
        x, sc = _values64(s, name)
        for b in range(c["B"]):
            first, n = int(s["len0"][b]), int(s["new"][b]) if s["new"] is not None else c["n"]
            pos = torch.arange(first, first + n, device="cuda")
            out["q"][b, :n] = _turned64(s["q"][b, :n], pos, c["base"])
            rows = s["knew" if name == "k" else "vnew"][b, :n]
            rows = (_turned64(rows, pos, c["base"]) if name == "k" else rows.double()).transpose(0, 1)
            if sc is None:
                x[b, :, first:first + n] = rows
                continue
            blk, qmax = c["block"], QMAX[c["fmt"]]
            for j in range(first // blk, (first + n - 1) // blk + 1):
                lo, hi = max(first, j * blk), min(first + n, (j + 1) * blk)
                part = rows[:, lo - first:hi - first]
                before = sc[b, :, j] if j * blk < first else torch.zeros_like(sc[b, :, j])
                s1 = torch.maximum(before, part.abs().amax((1, 2)) / qmax)
                code = (lambda y: y.round()) if c["fmt"] == "i8" else (lambda y: y.float().to(torch.float8_e4m3fn).double())
                held = x[b, :, j * blk:lo]
                x[b, :, j * blk:lo] = torch.where((s1 > before)[:, None, None], code(held * (before / s1)[:, None, None]), held)
                x[b, :, lo:hi] = code(part / s1[:, None, None])
                sc[b, :, j] = s1
        if sc is None:
            page = c["page"]
            out[name] = x if not page else _pool_of(x, s["table"], page)
        else:
            end = s["len0"] + (s["new"] if s["new"] is not None else c["n"])
            keep = (torch.arange(c["cap"], device="cuda")[None] < end[:, None])[:, None, :, None]
            out[name] = x * sc.repeat_interleave(c["block"], 2)[..., None] * keep
    return out


def exact(case, seed):
    if case["op"] == "append" and case["fmt"] != "native" and case["B"] * case["n"] / case["block"] > 3000:
        return None
    s = prepare(case, seed)
    c = s["case"]
    if c["op"] == "append":
        return _exact_append(s)
    G, d = c["Hq"] // c["Hkv"], c["d"]
    if c["op"] == "attend":
        out = torch.zeros(c["B"], c["Hq"], d, dtype=torch.float64, device="cuda")
        (k, ks), (v, vs) = _values64(s, "k"), _values64(s, "v")
        for b in range(c["B"]):
            L = int(s["len"][b])
            keep = [t for t in ([0, L] if not c["window"] else [max(0, L - c["window"]), L])]
            idx = torch.arange(keep[0], keep[1], device="cuda")
            if c["window"]:
                idx = torch.cat([torch.arange(min(c["sinks"], keep[0]), device="cuda"), idx])
            for h in range(c["Hkv"]):
                kk, vv = k[b, h, idx], v[b, h, idx]
                if ks is not None:
                    kk, vv = kk * ks[b, h, idx // c["block"]][:, None], vv * vs[b, h, idx // c["block"]][:, None]
                w = torch.softmax(s["q"][b, h * G:(h + 1) * G].double() @ kk.T / math.sqrt(d), -1)
                out[b, h * G:(h + 1) * G] = w @ vv
        return out
    if c["B"] * c["Hq"] * c["S"] ** 2 * d > 4e11:
        return None
    names = ("out", "dq", "dk", "dv")
    got = {n: torch.zeros(c["B"], c["S"], c["Hkv"] if n in ("dk", "dv") else c["Hq"], d, dtype=torch.float64, device="cuda") for n in names}
    i = torch.arange(c["S"], device="cuda")
    hidden = i[None] > i[:, None]
    if c["window"]:
        hidden |= (i[:, None] - i[None] >= c["window"]) & (i[None] >= c["sinks"])
    for b in range(c["B"]):
        for h in range(c["Hq"]):
            q, k, v = s["q"][b, :, h].double(), s["k"][b, :, h // G].double(), s["v"][b, :, h // G].double()
            z = (q @ k.T / math.sqrt(d)).masked_fill_(hidden, -math.inf)
            p = torch.softmax(z, -1)
            got["out"][b, :, h] = p @ v
            if c["train"]:
                do = s["dout"][b, :, h].double()
                e = do @ v.T
                e = p * (e - (e * p).sum(-1, keepdim=True)) / math.sqrt(d)
                got["dq"][b, :, h] = e @ k
                got["dk"][b, :, h // G] += e.T @ q
                got["dv"][b, :, h // G] += p.T @ do
    return got if c["train"] else got["out"]

"""float64 references of the operators on finished query / key / value rows."""
from __future__ import annotations

import numpy as np
import torch

from compressed_latent_grouped_b200 import binding as B

QMAX = {"i8": 127.0, "e4m3": 448.0}
# largest rounding error relative to the value, and below the normal range absolute
CODE_ERR = {"i8": (0.0, 0.5), "e4m3": (2.0 ** -4, 2.0 ** -10)}   # in units of the scale


def config(Hq, Hkv, d, dtype="bf16", base=0.0):
    return B.make_config(Hq * d, 1, Hq, Hkv, conv_width=0, qk_mean=0, value_shift=0, rope_base=base,
                         dtype=B.F32 if dtype == "f32" else B.BF16)


def torch_dtype(dtype):
    return torch.float32 if dtype == "f32" else torch.bfloat16


def f64(t):
    return t.detach().to("cpu", torch.float64).numpy()


def rotate(x, pos, base):
    """x [..., n, H, d] float64, pos [n]: pair (i, i + d/2) turns by pos base^(-2i/d)."""
    if base == 0.0:
        return x
    d = x.shape[-1]
    theta = base ** (-2.0 * np.arange(d // 2) / d)
    a = np.asarray(pos, dtype=np.float64)[:, None, None] * theta
    lo, hi = x[..., : d // 2], x[..., d // 2:]
    return np.concatenate([lo * np.cos(a) - hi * np.sin(a), lo * np.sin(a) + hi * np.cos(a)], -1)


def rotate_slack(x):
    """Bound on the fp32 rotation's error: (|a| + |b|) 2^-21.  The angle (a
    fraction of a turn held in fp32, at most half a turn) is off by 2^-25 turns
    = 2^-22.3 rad, sine and cosine add at most 2^-23 and the two products and
    the sum a rounding of 2^-24 each: below 2^-21 together."""
    d = x.shape[-1]
    s = np.abs(x[..., : d // 2]) + np.abs(x[..., d // 2:])
    return np.concatenate([s, s], -1) * 2.0 ** -21


def half_step(dtype):
    return torch.finfo(torch_dtype(dtype)).eps / 2


def assert_within(got, ref, tol, what=""):
    got, ref, tol = np.broadcast_arrays(np.asarray(got, np.float64), ref, tol)
    bad = ~(np.abs(got - ref) <= tol)
    if bad.any():
        i = np.unravel_index(np.argmax(np.where(bad, np.abs(got - ref) - tol, -1)), got.shape)
        raise AssertionError(f"{what}: {bad.sum()} of {bad.size} outside; at {i} got {got[i]!r}, "
                             f"reference {ref[i]!r}, tolerance {tol[i]:.3e}")


def dense_rows(x, table):
    """Cache or scale tensor as [batch, Hkv, tokens, ...] on the host."""
    x = x.detach().to("cpu")
    if x.dtype == torch.float8_e4m3fn:
        x = x.float()
    x = x.to(torch.float64).numpy()
    if table is None:
        return x
    t = table.cpu().numpy()
    return np.stack([np.concatenate([x[p] for p in row], 1) for row in t])


def cache_values(c, table=None):
    """k, v of a DeviceKVCache as float64 [batch, Hkv, cap, d]."""
    out = []
    for name in ("k", "v"):
        x = dense_rows(getattr(c, name), table)
        if c.block:
            x = x * np.repeat(dense_rows(getattr(c, name + "_scale"), table), c.block, 2)[..., None]
        out.append(x)
    return out


def seen(t, s, window, sinks):
    """Whether the query at position t sees key s (broadcast)."""
    ok = s <= t
    return ok & ((s > t - window) | (s < sinks)) if window else ok


def attend(q, k, v, keys):
    """One query row per head over the listed keys: q [Hq, d], k, v [Hkv, cap, d].
    Returns (out, weighted |v|, largest sum |q_i k_i| / sqrt(d))."""
    Hq, d = q.shape
    G = Hq // k.shape[0]
    out, mag, top = np.zeros((Hq, d)), np.zeros((Hq, d)), 0.0
    for h in range(Hq):
        if len(keys) == 0:
            continue
        kk, vv = k[h // G, keys], v[h // G, keys]
        s = kk @ q[h] / np.sqrt(d)
        p = np.exp(s - s.max())
        p /= p.sum()
        out[h], mag[h] = p @ vv, p @ np.abs(vv)
        top = max(top, (np.abs(kk) @ np.abs(q[h])).max() / np.sqrt(d))
    return out, mag, top


def attention_slack(d, n, top):
    """Relative error of softmax sums in fp32: scores are off by (d + 3) 2^-24
    of sum |q k| / sqrt(d) (in the exponent), in the numerator and in the
    denominator; sums over n terms by n 2^-24 each; exponentials (in base 2, an
    argument of up to 2 top log2 e rounded to 2^-24, and the hardware's 2^-22)."""
    return 2 * (d + 3 + 4) * 2.0 ** -24 * top + (2 * n + 32) * 2.0 ** -24

"""ccgqa_window_attention and its backward against float64: every pair's
probability and score gradient, with the bounds that the kernels' roundings
allow element by element."""
import math

import numpy as np
import pytest
import torch

from compressed_latent_grouped_b200 import binding as B
from compressed_latent_grouped_b200.device import Graph, window_attention, window_attention_backward
from rows_ref import attention_slack, config, torch_dtype

pytestmark = pytest.mark.gpu


def visible(S, window, sinks, device="cuda"):
    t, s = torch.arange(S, device=device)[:, None], torch.arange(S, device=device)[None]
    ok = s <= t
    return ok & ((s > t - window) | (s < sinks)) if window else ok


def reference(q, k, v, window, sinks, dout=None):
    """float64 values and error bounds, one (sequence, head) at a time.

    Bounds, for inputs in bf16: probabilities are rounded to bf16 before P V
    and P^T dO (2^-8 of each, and below 2^-13 for the exponential), score
    gradients before dS k and dS^T q (2^-8), D = dO.o takes the rounded output
    (its own bound, times |dO|), and each result is rounded once (2^-8).  fp32
    inputs: 2^-24 in place of 2^-8, and the sums' error (attention_slack)."""
    Bn, S, Hq, d = q.shape
    G = Hq // k.shape[2]
    f32 = q.dtype == torch.float32
    hs, pr = (2.0 ** -24, 0.0) if f32 else (2.0 ** -8, 2.0 ** -8 * (1 + 2.0 ** -8) + 2.0 ** -13)
    ok = visible(S, window, sinks)
    n = int(ok.sum(1).max())
    z = lambda x: torch.zeros(x.shape, dtype=torch.float64, device=x.device)  # noqa: E731
    ref = dict(out=z(q), dq=z(q), dk=z(k), dv=z(v))
    tol = dict(out=z(q), dq=z(q), dk=z(k), dv=z(v))
    for b in range(Bn):
        for h in range(Hq):
            g = h // G
            Q, K, V = q[b, :, h].double(), k[b, :, g].double(), v[b, :, g].double()
            s = (Q @ K.T / math.sqrt(d)).masked_fill(~ok, -math.inf)
            p = torch.softmax(s, -1)
            top = float((Q.abs() @ K.abs().T / math.sqrt(d)).masked_fill(~ok, 0).max())
            rel = attention_slack(d, n, top)
            o = p @ V
            t_o = (pr + rel) * (p @ V.abs()) + hs * o.abs()
            ref["out"][b, :, h], tol["out"][b, :, h] = o, t_o
            if dout is None:
                continue
            dO = dout[b, :, h].double()
            e, e_abs = dO @ V.T, dO.abs() @ V.abs().T
            D, D_err = (dO * o).sum(-1, keepdim=True), (dO.abs() * t_o).sum(-1, keepdim=True)
            D_abs = (dO * o).abs().sum(-1, keepdim=True)
            dS = p * (e - D)
            err = p * (D_err + (rel + (d + 8) * 2.0 ** -24) * (e_abs + D_abs)) + dS.abs() * (0 if f32 else 2.0 ** -8 * 1.01 + 2.0 ** -13)
            c = 1 / math.sqrt(d)
            ref["dq"][b, :, h] = dS @ K * c
            tol["dq"][b, :, h] = err @ K.abs() * c + (dS.abs() @ K.abs()) * c * n * 2.0 ** -24
            ref["dk"][b, :, g] += dS.T @ Q * c
            tol["dk"][b, :, g] += err.T @ Q.abs() * c + (dS.abs().T @ Q.abs()) * c * S * G * 2.0 ** -24
            ref["dv"][b, :, g] += p.T @ dO
            tol["dv"][b, :, g] += (p.T @ dO.abs()) * (pr + rel + S * G * 2.0 ** -24)
    for m in ("dq", "dk", "dv"):
        tol[m] += ref[m].abs() * hs + 1e-30
    tol["out"] += 1e-30
    return ref, tol


def close(got, ref, tol, what):
    d = (got.double() - ref).abs()
    bad = ~(d <= tol)
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.numel()} outside, worst "
                           f"{float((d / tol).nan_to_num(1e9).max()):.2f} of the bound at "
                           f"{tuple(int(x) for x in bad.nonzero()[0])}")


def inputs(Bn, S, Hq, Hkv, d, dtype, seed=0, layout="bthd", scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = torch_dtype(dtype)
    r = lambda *s: (torch.randn(s, generator=g, device="cuda") * scale).to(dt)  # noqa: E731
    if layout == "packed":
        q, k, v = r(Bn, S, Hq + 2 * Hkv, d).split([Hq, Hkv, Hkv], 2)
    elif layout == "bhtd":
        q, k, v = (r(Bn, H, S, d).transpose(1, 2) for H in (Hq, Hkv, Hkv))
    else:
        q, k, v = r(Bn, S, Hq, d), r(Bn, S, Hkv, d), r(Bn, S, Hkv, d)
    return q, k, v, r(Bn, S, Hq, d)


CASES = [
    # B, S, Hq, Hkv, d, dtype, window, sinks, layout
    (1, 1, 4, 2, 64, "bf16", 0, 0, "bthd"),
    (2, 2, 4, 1, 32, "bf16", 1, 1, "packed"),
    (1, 63, 8, 2, 64, "bf16", 16, 0, "bthd"),
    (2, 64, 3, 1, 64, "bf16", 17, 4, "bhtd"),
    (1, 65, 8, 8, 128, "bf16", 64, 65, "packed"),
    (2, 301, 16, 4, 32, "bf16", 100, 3, "bthd"),
    (1, 333, 8, 2, 64, "bf16", 0, 0, "packed"),
    (1, 500, 12, 4, 64, "bf16", 77, 130, "bhtd"),
    (1, 700, 16, 1, 64, "bf16", 129, 37, "bthd"),
    (1, 1025, 6, 3, 32, "bf16", 512, 4, "bthd"),
    (1, 777, 8, 2, 128, "bf16", 256, 1, "bthd"),
    (2, 260, 5, 1, 128, "bf16", 1, 0, "packed"),
    (1, 130, 24, 1, 32, "bf16", 33, 70, "bthd"),
    (1, 90, 64, 1, 64, "bf16", 20, 2, "bthd"),
    (1, 70, 100, 1, 32, "bf16", 20, 2, "bthd"),
    (1, 40, 160, 1, 16, "bf16", 9, 3, "bthd"),
    (2, 200, 4, 2, 16, "bf16", 40, 5, "packed"),
    (1, 1500, 8, 2, 64, "bf16", 2000, 5, "bthd"),
    (1, 1, 2, 1, 16, "f32", 0, 0, "bthd"),
    (2, 65, 4, 2, 32, "f32", 20, 3, "packed"),
    (1, 301, 6, 2, 64, "f32", 100, 70, "bhtd"),
    (1, 257, 4, 1, 128, "f32", 0, 0, "bthd"),
    (1, 130, 72, 1, 16, "f32", 65, 1, "bthd"),
]


@pytest.mark.parametrize("Bn,S,Hq,Hkv,d,dtype,window,sinks,layout", CASES)
def test_forward_and_gradients(Bn, S, Hq, Hkv, d, dtype, window, sinks, layout):
    cfg = config(Hq, Hkv, d, dtype)
    q, k, v, do = inputs(Bn, S, Hq, Hkv, d, dtype, layout=layout)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    kw = dict(window=window, sinks=sinks, dev_err=err)
    ref, tol = reference(q, k, v, window, sinks, do)
    out, stats = window_attention(cfg, q, k, v, with_stats=True, **kw)
    close(out, ref["out"], tol["out"], "out")
    assert torch.equal(window_attention(cfg, q, k, v, **kw), out), "with and without statistics"
    if layout == "packed":      # gradients into one packed tensor, as q, k, v came
        dq, dk, dv = torch.full((Bn, S, Hq + 2 * Hkv, d), 3.0, dtype=q.dtype, device="cuda").split([Hq, Hkv, Hkv], 2)
    elif layout == "bhtd":
        dq, dk, dv = (torch.empty(Bn, H, S, d, dtype=q.dtype, device="cuda").transpose(1, 2) for H in (Hq, Hkv, Hkv))
    else:
        dq = dk = dv = None
    got = window_attention_backward(cfg, q, k, v, out, stats, do, dq=dq, dk=dk, dv=dv, **kw)
    again = window_attention_backward(cfg, q, k, v, out, stats, do, **kw)
    for m, x, y in zip(("dq", "dk", "dv"), got, again):
        close(x, ref[m], tol[m], m)
        assert torch.equal(x, y), f"{m}: equal calls, other bits"
    assert int(err) == 0


def test_large_scores():
    """Scores of several hundred: running maxima that grow along the keys."""
    q, k, v, do = inputs(1, 400, 8, 2, 64, "bf16", seed=3, scale=6.0)
    k = k * torch.linspace(0.1, 2.0, 400, device="cuda")[None, :, None, None]
    k = k.bfloat16()
    cfg = config(8, 2, 64)
    ref, tol = reference(q, k, v, 150, 4, do)
    out, stats = window_attention(cfg, q, k, v, window=150, sinks=4, with_stats=True)
    close(out, ref["out"], tol["out"], "out")
    for m, x in zip(("dq", "dk", "dv"), window_attention_backward(cfg, q, k, v, out, stats, do, window=150, sinks=4)):
        close(x, ref[m], tol[m], m)


def test_far_sinks_of_a_long_sequence():
    """A long sequence, a short window: most key tiles are never visited."""
    q, k, v, do = inputs(1, 4000, 4, 2, 64, "bf16", seed=4)
    cfg = config(4, 2, 64)
    ref, tol = reference(q, k, v, 70, 66, do)
    out, stats = window_attention(cfg, q, k, v, window=70, sinks=66, with_stats=True)
    close(out, ref["out"], tol["out"], "out")
    for m, x in zip(("dq", "dk", "dv"), window_attention_backward(cfg, q, k, v, out, stats, do, window=70, sinks=66)):
        close(x, ref[m], tol[m], m)


def test_gradients_are_those_of_the_output():
    """fp32 gradients against central differences of the float64 function."""
    cfg = config(4, 2, 32, "f32")
    q, k, v, do = inputs(1, 50, 4, 2, 32, "f32", seed=5)
    out, stats = window_attention(cfg, q, k, v, window=13, sinks=2, with_stats=True)
    grads = window_attention_backward(cfg, q, k, v, out, stats, do, window=13, sinks=2)
    ok = visible(50, 13, 2)

    def loss(q, k, v):
        K, V = (x.repeat_interleave(2, 2) for x in (k, v))
        p = torch.softmax((torch.einsum("bthd,bshd->bhts", q, K) / math.sqrt(32)).masked_fill(~ok, -math.inf), -1)
        return float((torch.einsum("bhts,bshd->bthd", p, V) * do.double()).sum())

    x = [t.double() for t in (q, k, v)]
    g = torch.Generator(device="cuda").manual_seed(1)
    for i in range(3):
        for _ in range(3):
            u = torch.randn(x[i].shape, generator=g, device="cuda", dtype=torch.float64)
            h = 1e-4
            up, dn = list(x), list(x)
            up[i], dn[i] = x[i] + h * u, x[i] - h * u
            diff = (loss(*up) - loss(*dn)) / (2 * h)
            ours = float((grads[i].double() * u).sum())
            # the difference is off by h^2 times a third derivative of order |u|^3, the gradient by fp32
            assert abs(diff - ours) <= 1e-4 * float((grads[i].double() * u).abs().sum())


def test_streams_graph_and_empty():
    cfg = config(8, 2, 64)
    q, k, v, do = inputs(1, 600, 8, 2, 64, "bf16", seed=6)
    kw = dict(window=200, sinks=4)
    out, stats = window_attention(cfg, q, k, v, with_stats=True, **kw)
    ref = window_attention_backward(cfg, q, k, v, out, stats, do, **kw)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    runs = []
    for s in (s1, s2, s1, s2):
        with torch.cuda.stream(s):
            o, st = window_attention(cfg, q, k, v, with_stats=True, **kw)
            runs.append((o, *window_attention_backward(cfg, q, k, v, o, st, do, **kw)))
    torch.cuda.synchronize()
    for r in runs:
        assert all(torch.equal(a, b) for a, b in zip(r, (out, *ref)))
    o2, st2 = torch.empty_like(out), torch.empty_like(stats)
    grads = [torch.empty_like(x) for x in ref]
    ws = torch.empty(B.ccgqa_window_attention_backward_workspace_size(cfg, 1, 600), dtype=torch.uint8, device="cuda")
    win, rows = B.ccgqa_window(200, 4), B.make_rows

    def step():
        B.ccgqa_window_attention(cfg, win, rows(q), rows(k), rows(v), 1, 600, rows(o2), st2)
        B.ccgqa_window_attention_backward(cfg, win, rows(q), rows(k), rows(v), rows(o2), st2, rows(do), 1, 600,
                                          *(rows(x) for x in grads), ws)
    g = Graph(step, s1)
    for _ in range(3):
        for x in (o2, st2, *grads):
            x.fill_(float("nan"))
        ws.fill_(255)
        torch.cuda.synchronize()
        g.launch()
        torch.cuda.synchronize()
        assert torch.equal(o2, out) and all(torch.equal(a, b) for a, b in zip(grads, ref))
    g.close()
    e = window_attention(cfg, q[:, :0], k[:, :0], v[:, :0])
    assert e.shape == (1, 0, 8, 64)


def test_prompt_then_tokens():
    """The prompt by window attention, then tokens by cache attention, one
    window: the last row of either is the same function of the same rows."""
    from compressed_latent_grouped_b200.device import DeviceKVCache
    cfg = config(8, 2, 64, base=1e4)
    q, k, v, _ = inputs(2, 300, 8, 2, 64, "bf16", seed=7, layout="packed")
    c = DeviceKVCache(cfg, 2, 320)
    kr = torch.empty(2, 300, 2, 64, dtype=torch.bfloat16, device="cuda")
    qr = c.append_rope(k, v, q=q, k_out=kr)
    out = window_attention(cfg, qr, kr, v, window=90, sinks=4)
    last = c.attend(qr[:, -1].contiguous(), window=90, sinks=4)
    ref, tol = reference(qr, kr, v, 90, 4)
    close(out, ref["out"], tol["out"], "prompt")
    close(last, ref["out"][:, -1], tol["out"][:, -1], "token")
    assert c.error_bits() == 0
    assert np.array_equal(c.k[:, :, :300].float().cpu().numpy(), kr.transpose(1, 2).float().cpu().numpy())


def test_recorded_calls_keep_their_memory():
    """What calls allocate while the library's graph records stays with the graph."""
    from compressed_latent_grouped_b200.device import DeviceKVCache
    cfg = config(8, 2, 64)
    q, k, v, do = inputs(1, 900, 8, 2, 64, "bf16", seed=8)
    kw = dict(window=300, sinks=4)
    c = DeviceKVCache(cfg, 1, 4096)
    c.append_rope(k, v)
    qt = q[:, -1].contiguous()
    grads = [torch.empty_like(x) for x in (q, k, v)]
    row = torch.empty_like(qt)
    s = torch.cuda.Stream()

    def step():
        out, stats = window_attention(cfg, q, k, v, with_stats=True, **kw)
        window_attention_backward(cfg, q, k, v, out, stats, do, dq=grads[0], dk=grads[1], dv=grads[2], **kw)
        c.attend(qt, out=row)

    with torch.cuda.stream(s):
        step()
    torch.cuda.synchronize()
    ref = [x.clone() for x in (*grads, row)]
    g = Graph(step, s)
    with torch.cuda.stream(s):          # the stream's pool is drawn on by others meanwhile
        others = [torch.full((n,), 255, dtype=torch.uint8, device="cuda") for n in (1 << 12, 1 << 20, 1 << 22, 1 << 24)
                  for _ in range(6)]
    for _ in range(3):
        for x in (*grads, row):
            x.fill_(float("nan"))
        torch.cuda.synchronize()
        g.launch()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip((*grads, row), ref))
        assert all(bool((o == 255).all()) for o in others)
    g.close()


def test_python_refusals():
    cfg = config(8, 2, 64)
    q, k, v, do = inputs(2, 40, 8, 2, 64, "bf16")
    out, stats = window_attention(cfg, q, k, v, with_stats=True)
    two_way = config(8, 2, 64)
    two_way.causal = 0
    bad = [
        lambda: window_attention(cfg, q[0], k, v), lambda: window_attention(cfg, q, k[:, :39], v),
        lambda: window_attention(cfg, q, k, v.float()), lambda: window_attention(cfg, q, k.cpu(), v),
        lambda: window_attention(cfg, q, k, v, window=-3), lambda: window_attention(cfg, q, k, v, sinks=1 << 40),
        lambda: window_attention(cfg, q, k, v, out=out[:1]), lambda: window_attention(two_way, q, k, v),
        lambda: window_attention(cfg, q, k, v, dev_err=torch.zeros(1, device="cuda")),
        lambda: window_attention(cfg, q, k[:, :1].expand(2, 40, 2, 64), v),       # keys that share memory
        lambda: window_attention_backward(cfg, q, k, v, out, stats[:-1], do),
        lambda: window_attention_backward(cfg, q, k, v, out, None, do),
        lambda: window_attention_backward(cfg, q, k, v, out, stats, do[:, :, :4]),
        lambda: window_attention_backward(cfg, q, k, v, out, stats, torch.ones(1, 1, 1, 1, dtype=q.dtype, device="cuda").expand_as(do)),
        lambda: window_attention_backward(cfg, q, k, v, out, stats, do, dk=torch.empty_like(q)),
    ]
    n = B.ccgqa_launch_count()
    for i, f in enumerate(bad):
        with pytest.raises(B.CCGQAError):
            f()
            pytest.fail(f"call {i} was accepted")
    assert B.ccgqa_launch_count() == n
    with pytest.raises(RuntimeError):
        window_attention(cfg, q.cpu(), k.cpu(), v.cpu())


@pytest.mark.parametrize("Bn,S,Hq,Hkv,d,window,sinks", [
    (1, 2048, 16, 4, 64, 0, 0),          # tiles of very different length
    (2, 1900, 16, 4, 128, 700, 5),       # a tile's partial sums in two CTAs
    (1, 2500, 16, 4, 32, 1000, 200),     # every query sees the first tile and a half
    (5, 700, 16, 2, 64, 65, 0),          # short tiles, several of them in a CTA
    (3, 900, 12, 4, 32, 0, 0),
    (2, 1300, 10, 2, 128, 0, 0),         # groups of five: rows left over in every block
])
def test_gradients_of_shared_out_tiles(Bn, S, Hq, Hkv, d, window, sinks):
    """Enough blocks that tiles are cut across CTAs and CTAs take several tiles."""
    cfg = config(Hq, Hkv, d)
    q, k, v, do = inputs(Bn, S, Hq, Hkv, d, "bf16", seed=7, layout="packed")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    kw = dict(window=window, sinks=sinks, dev_err=err)
    ref, tol = reference(q, k, v, window, sinks, do)
    out, stats = window_attention(cfg, q, k, v, with_stats=True, **kw)
    close(out, ref["out"], tol["out"], "out")
    got = window_attention_backward(cfg, q, k, v, out, stats, do, **kw)
    again = window_attention_backward(cfg, q, k, v, out, stats, do, **kw)
    for m, x, y in zip(("dq", "dk", "dv"), got, again):
        close(x, ref[m], tol[m], m)
        assert torch.equal(x, y), f"{m}: equal calls, other bits"
    assert int(err) == 0


@pytest.mark.parametrize("Bn,S,Hq,Hkv,d,window,sinks", [
    (1, 89, 8, 2, 64, 0, 0),             # one tile per head, of three blocks
    (3, 383, 6, 3, 32, 20, 0),           # more tiles than shares of two blocks
    (40, 300, 4, 4, 128, 60, 0),         # several whole tiles in a CTA
    (70, 130, 8, 2, 32, 0, 0),
])
def test_gradients_of_whole_tiles(Bn, S, Hq, Hkv, d, window, sinks):
    """Tiles too short to be cut: each in one CTA, no sums to join."""
    cfg = config(Hq, Hkv, d)
    q, k, v, do = inputs(Bn, S, Hq, Hkv, d, "bf16", seed=11)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    kw = dict(window=window, sinks=sinks, dev_err=err)
    ref, tol = reference(q, k, v, window, sinks, do)
    out, stats = window_attention(cfg, q, k, v, with_stats=True, **kw)
    got = window_attention_backward(cfg, q, k, v, out, stats, do, **kw)
    for m, x in zip(("dq", "dk", "dv"), got):
        close(x, ref[m], tol[m], m)
    assert int(err) == 0


@pytest.mark.parametrize("Bn,S,Hq,Hkv,d,window,sinks", [
    (1, 2500, 128, 16, 128, 300, 0),     # pairs of tiles for one round, the rest by themselves
    (2, 1800, 40, 20, 128, 77, 9),
    (1, 3601, 64, 16, 32, 250, 3),       # threes of tiles
    (3, 1501, 45, 9, 32, 130, 0),        # groups of five: rows left over in every tile
])
def test_tiles_left_over(Bn, S, Hq, Hkv, d, window, sinks):
    """More query tiles than whole rounds of the GPU hold; a few heads of each group against float64."""
    cfg = config(Hq, Hkv, d)
    q, k, v, _ = inputs(Bn, S, Hq, Hkv, d, "bf16", seed=3)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = window_attention(cfg, q, k, v, window=window, sinks=sinks, dev_err=err)
    assert int(err) == 0
    G = Hq // Hkv
    for g in {0, Hkv // 2, Hkv - 1}:
        for h in {g * G, g * G + G - 1}:
            ref, tol = reference(q[:, :, h:h + 1], k[:, :, g:g + 1], v[:, :, g:g + 1], window, sinks)
            close(out[:, :, h:h + 1], ref["out"], tol["out"], f"head {h}")
    ok = visible(S, window, sinks)               # and every row is some mean of values it sees
    top = torch.stack([v[b, :, :].float().abs().amax(-1) for b in range(Bn)])
    for b in range(Bn):
        for g in range(Hkv):
            bound = torch.where(ok, top[b, :, g][None], torch.zeros((), device="cuda")).amax(1)
            assert (out[b, :, g * G:(g + 1) * G].float().abs().amax((1, 2)) <= bound * (1 + 2.0 ** -6)).all()


@pytest.mark.parametrize("Bn,S,Hq,Hkv,d,window,sinks", [
    (2, 2000, 32, 8, 64, 0, 0),          # seven query tiles per CTA, of every length
    (1, 3000, 24, 8, 128, 1000, 37),     # groups of three: rows left over
    (3, 1500, 32, 8, 32, 900, 0),
    (2, 1700, 32, 8, 64, 200, 300),      # short windows: D formed tile by tile
    (4, 640, 64, 16, 128, 1, 0),         # tiles of one block
])
def test_gradients_of_many_query_tiles(Bn, S, Hq, Hkv, d, window, sinks):
    """CTAs that take several query tiles one after another; some heads against float64."""
    cfg = config(Hq, Hkv, d)
    q, k, v, do = inputs(Bn, S, Hq, Hkv, d, "bf16", seed=5)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    kw = dict(window=window, sinks=sinks, dev_err=err)
    out, stats = window_attention(cfg, q, k, v, with_stats=True, **kw)
    got = window_attention_backward(cfg, q, k, v, out, stats, do, **kw)
    again = window_attention_backward(cfg, q, k, v, out, stats, do, **kw)
    assert int(err) == 0
    for x, y in zip(got, again):
        assert torch.equal(x, y), "equal calls, other bits"
    G = Hq // Hkv
    for g in {0, Hkv // 2, Hkv - 1}:
        hs, kv = slice(g * G, g * G + G), slice(g, g + 1)
        ref, tol = reference(q[:, :, hs], k[:, :, kv], v[:, :, kv], window, sinks, do[:, :, hs])
        for m, x, sl in zip(("dq", "dk", "dv"), got, (hs, kv, kv)):
            close(x[:, :, sl], ref[m], tol[m], f"{m}, kv head {g}")

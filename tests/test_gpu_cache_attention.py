"""ccgqa_cache_attention against float64: caches in the working type and in 8
bits, contiguous and paged, whole sequences and windows with sinks."""
import numpy as np
import pytest
import torch

from compressed_latent_grouped_b200 import binding as B
from compressed_latent_grouped_b200.device import DeviceKVCache, Graph
from rows_ref import (QMAX, assert_within, attend, attention_slack, cache_values, config, f64, half_step,
                      rotate, seen, torch_dtype)

pytestmark = pytest.mark.gpu


def make(Hq, Hkv, d, dtype, fmt, block, cap, page, lens, seed=0, spread=1.0):
    """A cache of random rows with stale, non-finite rows behind each sequence."""
    rng = np.random.RandomState(seed)
    batch = len(lens)
    table, n_pages = None, 0
    if page:
        n_pages = batch * (cap // page) + 2
        table = torch.from_numpy(rng.permutation(n_pages)[: batch * (cap // page)].astype(np.int32).reshape(batch, -1)).cuda()
    c = DeviceKVCache(config(Hq, Hkv, d, dtype), batch, cap, fmt=fmt, block=block, block_table=table, page_size=page, n_pages=n_pages)
    g = torch.Generator(device="cuda").manual_seed(seed + 1)
    for x, sc in ((c.k, c.k_scale), (c.v, c.v_scale)):
        r = torch.randn(x.shape, generator=g, device="cuda")
        if fmt == "native":
            x.copy_(r)
            continue
        r = (r * 40).round().clamp(-127, 127) if fmt == "i8" else (r * 100).clamp(-448, 448)
        x.view(torch.uint8).copy_(r.to(x.dtype).view(torch.uint8))
        sc.copy_(torch.exp(torch.randn(sc.shape, generator=g, device="cuda") * spread) * (0.025 if fmt == "i8" else 0.01))
    c.len.copy_(torch.tensor(lens, dtype=torch.int32))
    q = torch.randn(batch, Hq, d, generator=g, device="cuda").to(torch_dtype(dtype))
    return c, table, q


def poison(c, table, lens, window, sinks):
    """NaN into every row, and scale, that no query sees."""
    block = c.block or 1
    for b, L in enumerate(lens):
        see = seen(L - 1, np.arange(c.cap), window, sinks)
        for t0 in range(0, c.cap, block):
            if c.block and not see[t0:t0 + block].any():
                for sc in (c.k_scale, c.v_scale):
                    i, j = (b, t0 // block) if table is None else (int(table[b, t0 // c.k.shape[2]]), t0 % c.k.shape[2] // block)
                    sc[i, :, j] = float("nan")
        hidden = np.flatnonzero(~see)
        if len(hidden) == 0 or c.k.dtype == torch.int8:
            continue
        page = c.k.shape[2]
        hid = torch.from_numpy(hidden).cuda()
        for x in (c.k, c.v):
            raw = x.view(torch.uint8) if c.block else x
            val = 0x7f if c.block else float("nan")
            if table is None:
                raw[b, :, hid] = val
            else:
                raw[table[b, hid // page].long(), :, hid % page] = val


def compare(q, out, k, v, keys, dtype, fmt, what=""):
    """One sequence's heads against float64 over the listed keys."""
    k, v = np.nan_to_num(k), np.nan_to_num(v)
    ref, mag, top = attend(f64(q), k, v, keys)
    rel = attention_slack(q.shape[-1], len(keys), top)
    if dtype == "bf16" and fmt == "i8" and len(keys):
        # q as 16-bit integers: each element off by at most 2^-15 of its head's largest, so a score by
        # that times sum |k| / sqrt(d), and a probability's numerator and denominator by it each
        rel = rel + 2 * 2.0 ** -15 * np.abs(f64(q)).max(-1, keepdims=True) * np.abs(k[:, keys]).sum(-1).max() / np.sqrt(q.shape[-1])
    tol = np.abs(ref) * half_step(dtype) + mag * rel
    if dtype == "bf16":
        tol = tol + mag * (2.0 ** -8 if fmt == "native" else 2.0 ** -11) * (1 + 2.0 ** -8)
        if fmt != "native" and len(keys):
            # a weight below fp16's normal range is off by 2^-25 of the largest weight's unit:
            # times the code, summed over the keys
            tol = tol + len(keys) * 2.0 ** -25 * np.abs(v[:, keys]).max() * QMAX[fmt]
    assert_within(f64(out), ref, tol + 1e-30, what)


def check(c, table, q, out, lens, window, sinks, dtype, fmt, what=""):
    k, v = cache_values(c, table)
    for b, L in enumerate(lens):
        keys = np.flatnonzero(seen(L - 1, np.arange(c.cap), window, sinks))
        compare(q[b], out[b], k[b], v[b], keys, dtype, fmt, f"{what} sequence {b}")


CASES = [
    # Hq, Hkv, d, dtype, fmt, block, cap, page, lens, window, sinks
    (8, 2, 64, "bf16", "native", 0, 512, 0, (512, 1, 0, 77), 0, 0),
    (8, 2, 64, "bf16", "i8", 64, 4096, 0, (4096, 3001, 64), 0, 0),
    (16, 4, 32, "bf16", "i8", 16, 1008, 0, (1008,), 0, 0),
    (16, 4, 32, "bf16", "i8", 16, 1008, 16, (1008, 17, 15), 0, 0),
    (32, 8, 128, "bf16", "e4m3", 32, 2048, 64, (2048, 1999), 0, 0),
    (3, 1, 64, "bf16", "e4m3", 16, 256, 128, (255, 2), 0, 0),
    (16, 1, 64, "bf16", "i8", 32, 640, 0, (633,), 0, 0),
    (20, 1, 32, "bf16", "native", 0, 320, 32, (301, 33), 0, 0),
    (40, 2, 16, "bf16", "e4m3", 16, 128, 0, (128, 5), 0, 0),
    (4, 4, 16, "bf16", "i8", 128, 256, 256, (129,), 0, 0),
    (8, 8, 128, "bf16", "native", 0, 1024, 0, (1000, 513), 0, 0),
    (12, 4, 128, "f32", "native", 0, 512, 64, (511, 0, 1), 0, 0),
    (8, 2, 64, "f32", "i8", 32, 2048, 0, (2047,), 0, 0),
    (6, 3, 32, "f32", "e4m3", 16, 320, 32, (320, 77), 0, 0),
    (5, 1, 16, "f32", "native", 0, 160, 0, (159,), 0, 0),
    # windows: shorter and longer than the sequence, sinks in and out of it, odd borders
    (8, 2, 64, "bf16", "native", 0, 4096, 0, (4001, 100, 16), 129, 4),
    (8, 2, 64, "bf16", "i8", 16, 2048, 16, (2047, 333, 1), 37, 37),
    (32, 8, 128, "bf16", "e4m3", 64, 4096, 64, (4096, 1025), 1000, 0),
    (16, 4, 32, "bf16", "i8", 64, 1024, 64, (1000, 999), 1, 0),
    (16, 2, 16, "bf16", "native", 0, 512, 32, (510, 40), 33, 1),
    (4, 2, 128, "bf16", "native", 0, 2048, 128, (1500,), 700, 2000),
    (8, 2, 64, "f32", "i8", 16, 1024, 16, (1001, 50), 65, 5),
    (4, 1, 128, "f32", "native", 0, 512, 0, (512,), 16, 16),
]


@pytest.mark.parametrize("Hq,Hkv,d,dtype,fmt,block,cap,page,lens,window,sinks", CASES)
def test_attention(Hq, Hkv, d, dtype, fmt, block, cap, page, lens, window, sinks):
    c, table, q = make(Hq, Hkv, d, dtype, fmt, block, cap, page, lens)
    poison(c, table, lens, window, sinks)
    keep = [x.view(torch.uint8).clone() for x in (c.k, c.v)]
    out = c.attend(q, window=window, sinks=sinks)
    again = c.attend(q, out=torch.full_like(q, 7.0), window=window, sinks=sinks)
    torch.cuda.synchronize()
    assert c.error_bits() == 0
    assert torch.equal(out, again), "equal calls, other bits"
    assert all(torch.equal(a, x.view(torch.uint8)) for a, x in zip(keep, (c.k, c.v))) and c.len.tolist() == list(lens)
    check(c, table, q, out, lens, window, sinks, dtype, fmt)


@pytest.mark.parametrize("fmt", ["i8", "e4m3"])
def test_blocks_of_very_different_size(fmt):
    """Scales over twelve orders of magnitude, blocks of zeros and large scores:
    each weight is rounded where it matters."""
    c, _, q = make(8, 2, 64, "bf16", fmt, 16, 512, 0, (512, 300), spread=0.5)
    g = torch.Generator().manual_seed(5)
    c.v_scale.mul_(torch.pow(10.0, torch.randint(-9, 4, c.v_scale.shape, generator=g).float()).cuda())
    c.v_scale[:, :, 3] = 0
    c.k_scale[:, :, 7] = 0
    q = (q * 8).bfloat16()
    out = c.attend(q)
    assert c.error_bits() == 0
    k, v = cache_values(c)
    for b, L in enumerate((512, 300)):
        ref, mag, top = attend(f64(q[b]), k[b], v[b], np.arange(L))
        # fp16's subnormal steps: 2^-25 of the largest weight p sv, times the code, per key
        G = 4
        sv = np.repeat(f64(c.v_scale[b]), 16, 1)
        extra = np.zeros_like(ref)
        for h in range(8):
            s = k[b, h // G, :L] @ f64(q[b, h]) / 8
            p = np.exp(s - s.max())
            extra[h] = L * 2.0 ** -25 * QMAX[fmt] * (p * sv[h // G, :L]).max() / p.sum() * 2
        assert_within(f64(out[b]), ref, np.abs(ref) * 2.0 ** -8 + mag * (2.0 ** -11 * 1.01 + attention_slack(64, L, top)) + extra)


def test_queries_of_extreme_size():
    c, _, q = make(4, 2, 32, "bf16", "i8", 16, 64, 0, (64,) * 4)
    q[0] = 0
    q[1] *= 2.0 ** -100
    q[2] = q[2] * 2.0 ** 60
    q[3, 0] = float("nan")
    out = c.attend(q)
    torch.cuda.synchronize()
    k, v = cache_values(c)
    for b in (0, 1):
        assert_within(f64(out[b]), v[b].mean(1).repeat(2, 0), np.abs(v[b]).mean(1).repeat(2, 0) * 2.0 ** -7)
    for h in range(4):      # one key takes all
        best = np.argmax(k[2, h // 2] @ f64(q[2, h]))
        assert_within(f64(out[2, h]), v[2, h // 2, best], np.abs(v[2, h // 2, best]) * (2.0 ** -8 + 2.0 ** -10))
    assert out[3, 0].isnan().all() and out[3, 1:].isfinite().all()


@pytest.mark.parametrize("dtype,fmt", [("bf16", "native"), ("bf16", "i8"), ("f32", "native"), ("f32", "e4m3")])
def test_device_checks(dtype, fmt):
    c, table, q = make(8, 2, 64, dtype, fmt, 16, 256, 32, (200, 257, -3, 256))
    lens = (200, 0, 0, 256)
    out = c.attend(q)
    torch.cuda.synchronize()
    assert c.error_bits() == B.DEVERR_CAPACITY
    assert not out[1].any() and not out[2].any()
    check(c, table, q, out, lens, 0, 0, dtype, fmt)
    # a missing page: its tokens count as absent; one that is not needed is not looked at
    c.dev_err.zero_()
    c.len.copy_(torch.tensor([200, 31, 0, 256], dtype=torch.int32))
    c.block_table[0, 2] = 1 << 20
    c.block_table[1, 1:] = -1
    c.block_table[3, 4] = -7
    out = c.attend(q)
    torch.cuda.synchronize()
    assert c.error_bits() == B.DEVERR_INDEX
    k, v = cache_values(c, c.block_table.clamp(0, c.k.shape[0] - 1))
    for b, keys in ((0, np.r_[0:64, 96:200]), (1, np.arange(31)), (3, np.r_[0:128, 160:256])):
        compare(q[b], out[b], k[b], v[b], keys, dtype, fmt, f"sequence {b}")
    c.dev_err.zero_()
    c.attend(q, window=60, sinks=20)       # sequence 0 sees [140, 200) and [0, 20): page 2 is outside
    torch.cuda.synchronize()
    assert c.error_bits() == 0


def test_infinite_scores_and_values():
    c, _, q = make(4, 2, 32, "bf16", "native", 0, 64, 0, (64, 64))
    c.v[0, 0, 5, 3] = float("inf")
    c.k[1, 1, 9] = float("nan")
    out = c.attend(q)
    torch.cuda.synchronize()
    assert out[0, :2, 3].isinf().all() and out[0, :2, :3].isfinite().all() and out[0, 2:].isfinite().all()
    assert out[1, 2:].isnan().all() and out[1, :2].isfinite().all()


@pytest.mark.parametrize("fmt", ["native", "i8"])
def test_streams_and_graphs(fmt):
    """Calls of one handle that overlap on two streams, and two recorded graphs
    of it, keep apart."""
    c, _, q = make(8, 2, 64, "bf16", fmt, 64, 8192, 0, (8192, 8000))
    p = q.flip(0).contiguous()
    ref_q, ref_p = c.attend(q), c.attend(p, window=5000)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    oq, op = [torch.empty_like(q) for _ in range(20)], [torch.empty_like(q) for _ in range(20)]
    for i in range(20):
        c.attend(q, out=oq[i], stream=s1)
        c.attend(p, out=op[i], window=5000, stream=s2)
    torch.cuda.synchronize()
    assert all(torch.equal(x, ref_q) for x in oq) and all(torch.equal(x, ref_p) for x in op)
    g1, g2 = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g1, stream=s1):
        a = c.attend(q)
    with torch.cuda.graph(g2, stream=s2):
        b = c.attend(p, window=5000)
    for _ in range(10):
        with torch.cuda.stream(s1):
            g1.replay()
        with torch.cuda.stream(s2):
            g2.replay()
    torch.cuda.synchronize()
    assert torch.equal(a, ref_q) and torch.equal(b, ref_p)


def test_pools_past_32_bits():
    """Pages whose elements lie past 2^32 bytes and elements."""
    pages, page = 1 << 17, 256
    cfg = config(4, 2, 64, "bf16", 1e4)
    table = torch.tensor([[pages - 1, 0, pages // 2 + 1, pages - 2]], dtype=torch.int32).cuda()
    c = DeviceKVCache(cfg, 1, 1024, fmt="i8", block=64, block_table=table, page_size=page, n_pages=pages)
    assert c.k.numel() >= 1 << 32
    d = DeviceKVCache(cfg, 1, 1024, fmt="i8", block=64)
    g = torch.Generator(device="cuda").manual_seed(8)
    x = torch.randn(1, 1000, 8, 64, generator=g, device="cuda").bfloat16()
    q, k, v = x.split([4, 2, 2], 2)
    for h in (c, d):
        h.append_rope(k, v)
    qq = q[:, -1].contiguous()
    assert torch.equal(c.attend(qq), d.attend(qq))
    assert all(torch.equal(a, b) for a, b in zip(c.read(0, 1000), d.read(0, 1000)))
    assert c.error_bits() == 0


@pytest.mark.parametrize("fmt,page", [("native", 0), ("i8", 64), ("e4m3", 0)])
def test_a_chunk_then_tokens(fmt, page):
    """A prompt in two chunks, then tokens one at a time, each appended with its
    rotation and attended: against attention over the values read back."""
    Hq, Hkv, d, base, cap = 8, 2, 64, 5e5, 256
    table = torch.randperm(8).int().view(2, 4).cuda() if page else None
    c = DeviceKVCache(config(Hq, Hkv, d, "bf16", base), 2, cap, fmt=fmt, block=32, block_table=table, page_size=page, n_pages=8)
    g = torch.Generator(device="cuda").manual_seed(6)
    x = torch.randn(2, 160, Hq + 2 * Hkv, d, generator=g, device="cuda").bfloat16()
    q, k, v = x.split([Hq, Hkv, Hkv], 2)
    c.append_rope(k[:, :70], v[:, :70])
    c.append_rope(k[:, 70:150], v[:, 70:150], n_valid=torch.tensor([80, 53], dtype=torch.int32).cuda())
    lens = [150, 123]
    for t in range(150, 160):
        qt = c.append_rope(k[:, t:t + 1], v[:, t:t + 1], q=q[:, t:t + 1])
        out = c.attend(qt[:, 0], window=100, sinks=3)
        lens = [n + 1 for n in lens]
        assert c.len.tolist() == lens
        check(c, table, qt[:, 0], out, lens, 100, 3, "bf16", fmt, f"token {t}")
        for b in range(2):
            ref = rotate(f64(q[b, t:t + 1]), [lens[b] - 1], base)
            assert_within(f64(qt[b]), ref, np.abs(ref) * 2.0 ** -8 + 1e-5, "query")
    assert c.error_bits() == 0


@pytest.mark.parametrize("d", [16, 32, 64, 128])
@pytest.mark.parametrize("fmt", ["native", "i8", "e4m3"])
@pytest.mark.parametrize("page,window,sinks", [(0, 0, 0), (16, 0, 0), (64, 301, 20)])
def test_fp32_layers(d, fmt, page, window, sinks):
    """Lengths around a warp's, a tile's and a split's share of the tokens; groups that fill a chunk of heads and do not."""
    Hq, Hkv = (4, 1) if page == 0 else (14, 2)
    block = {"native": 0, "i8": 16, "e4m3": 16 if page == 16 else 64}[fmt]
    lens = (0, 1, 15, 16, 17, 63, 65, 128, 1023, 2047, 2048)
    c, table, q = make(Hq, Hkv, d, "f32", fmt, block, 2048, page, lens, seed=d)
    poison(c, table, lens, window, sinks)
    out = c.attend(q, window=window, sinks=sinks)
    again = c.attend(q, out=torch.full_like(q, 7.0), window=window, sinks=sinks)
    torch.cuda.synchronize()
    assert c.error_bits() == 0
    assert torch.equal(out, again), "equal calls, other bits"
    check(c, table, q, out, lens, window, sinks, "f32", fmt)


@pytest.mark.parametrize("fmt", ["native", "e4m3"])
def test_fp32_layers_and_bad_pages(fmt):
    """Pages that are not in the pool count as absent, beside pages that are."""
    lens = (400, 77)
    c, table, q = make(8, 2, 64, "f32", fmt, 16 if fmt == "e4m3" else 0, 512, 16, lens)
    good = table.clone()
    table[0, 3] = -1
    table[0, 24] = c.k.shape[0]
    table[1, 4] = 1 << 30
    out = c.attend(q)
    torch.cuda.synchronize()
    assert c.error_bits() == B.DEVERR_INDEX
    k, v = cache_values(c, good)
    for b, L in enumerate(lens):
        gone = {0: (3, 24), 1: (4,)}[b]
        keys = np.array([t for t in range(L) if t // 16 not in gone])
        compare(q[b], out[b], k[b], v[b], keys, "f32", fmt, f"sequence {b}")

"""The pieces of a decoding loop outside the built-in step (session_extend, kv_write, kv_read, kv_export, attend,
sample) against plain 64-bit forms of the same definitions."""
import math

import numpy as np
import pytest
import torch

import oracle
import quantized_decode_step_gb300 as mag
from tests.helpers import device_bytes

pytestmark = pytest.mark.gpu

KV_NAMES = {mag.KV_FP16: "fp16", mag.KV_INT8: "int8", mag.KV_INT4: "int4"}
ALL_KV = tuple(KV_NAMES)


@pytest.fixture(scope="module", autouse=True)
def built():
    mag.build()
    assert torch.cuda.is_available()
    torch.cuda.init()


def make(kv=mag.KV_FP16, heads=4, kv_heads=2, dim=64, layers=1, pool_blocks=64, sessions=4, max_context=2048, seed=0,
         stream=1, flags=0):
    class Shape:
        n_layers, hidden, n_heads, n_kv_heads, head_dim = layers, 256, heads, kv_heads, dim
        ffn, vocab, rms_eps, rope_base = 256, 0, 1e-5, 10000.0

    order = None if flags & mag.FLAG_ELASTIC_POOL else np.random.default_rng(seed).permutation(pool_blocks)
    cfg = mag.make_config(Shape, kv_dtype=kv, pool_blocks=pool_blocks, max_sessions=sessions, max_batch=1,
                          max_context=max_context, pool_order=order, flags=flags)
    return mag.Context(cfg, stream)


def half(rng, *shape, std=1.0):
    return torch.from_numpy((rng.standard_normal(shape) * std).astype(np.float16))


def as_stored(x, kv):
    """What fp16 vectors [..., d] read back as, from the oracle's quantisers: fp16 of the exact s q (+ m)."""
    a = x.numpy()
    if kv == mag.KV_FP16 or a.size == 0:
        return x
    flat = np.ascontiguousarray(a.reshape(-1, a.shape[-1]))
    if kv == mag.KV_INT8:
        q, s = oracle.kv_quant_int8(flat)
        v = q.astype(np.float64).reshape(flat.shape) * s.view(np.float16).astype(np.float64).reshape(-1, 1)
    else:
        packed, sm = oracle.kv_quant_int4(flat)
        packed = packed.reshape(flat.shape[0], -1)
        sm = sm.view(np.float16).astype(np.float64).reshape(flat.shape[0], -1, 2)
        q = np.stack((packed & 15, packed >> 4), -1).reshape(flat.shape[0], -1, 32).astype(np.float64)
        v = (q * sm[..., :1] + sm[..., 1:]).reshape(flat.shape)
    return torch.from_numpy(v.astype(np.float16).reshape(a.shape))


# ------------------------------------------------------------------------------------------------ the cache
@pytest.mark.parametrize("kv", ALL_KV, ids=KV_NAMES.get)
@pytest.mark.parametrize("kv_heads,dim", [(1, 64), (2, 128), (5, 64), (8, 128)])
def test_write_stores_the_bytes_of_append(kv, kv_heads, dim):
    """Two layers, three sessions of odd lengths, rows inside a wider merged buffer: the pool's bytes equal those of
    mag_kv_append of the same tokens."""
    rng = np.random.default_rng(kv * 100 + kv_heads)
    n = [1, 37, 16]
    rows = sum(n)
    k, v = half(rng, 2, rows, kv_heads, dim), half(rng, 2, rows, kv_heads, dim)
    k[0, 3] = 0.0                      # a vector of zeros
    k[1, 5, 0, :32] = 0.75             # a constant group
    v[0, 7, 0, 0] = 60000.0            # an outlier
    v[1, 2, 0, :2] = torch.tensor([-0.0, 0.0])
    a = make(kv, kv_heads=kv_heads, heads=kv_heads, dim=dim, layers=2)
    b = make(kv, kv_heads=kv_heads, heads=kv_heads, dim=dim, layers=2)
    sa, sb = [a.session_open() for _ in n], [b.session_open() for _ in n]
    at = 0
    for s, c in zip(sa, n):
        kk, vv = k[:, at:at + c].contiguous().cuda(), v[:, at:at + c].contiguous().cuda()
        a.kv_append(s, c, kk, vv)
        a.sync()
        at += c
    b.session_extend(sb, n)
    width = kv_heads * dim
    for layer in range(2):
        wide = torch.zeros((rows, 2 * width + 24), dtype=torch.float16, device="cuda")
        wide[:, 8:8 + width] = k[layer].reshape(rows, -1).cuda()
        wide[:, 16 + width:16 + 2 * width] = v[layer].reshape(rows, -1).cuda()
        b.kv_write(layer, sb, n, wide[:, 8:], wide[:, 16 + width:], ld=wide.stride(0))
        b.sync()
    pa, na = a.debug_pool()
    pb, nb = b.debug_pool()
    assert na == nb and torch.equal(device_bytes(pa, na), device_bytes(pb, nb))


@pytest.mark.parametrize("kv", [mag.KV_INT8, mag.KV_INT4], ids=KV_NAMES.get)
def test_write_decides_codes_like_division(kv):
    """Vectors made for quotients halfway between two codes, next to it, and of every magnitude down to fp16's smallest
    number: what is read back equals the oracle's quantisers' to the bit."""
    rng = np.random.default_rng(17)
    n, h, d = 3000, 8, 128
    x = rng.standard_normal((n, h, d)) * np.exp2(rng.integers(-24, 9, (n, h, 1)))
    # the scale's own multiples and half multiples: integers and halves below a maximum of 127 (or 15 steps) times a power of two
    unit = np.exp2(rng.integers(-10, 6, (n // 2, h, 1)))
    top = 127 if kv == mag.KV_INT8 else 15
    x[::2] = rng.integers(-2 * top, 2 * top + 1, (n // 2, h, d)) * 0.5 * unit
    x[::2, :, ::32] = top * unit
    if kv == mag.KV_INT4:
        x[::2] = np.abs(x[::2])
        x[::2, :, 1::32] = 0.0
        x[1::4] += rng.standard_normal((len(x[1::4]), h, 1)) * 100
    x = torch.from_numpy(np.clip(x, -60000, 60000).astype(np.float16))
    x[5, 0] = 6e-8
    x[7, 1, 3] = 6e-8
    ctx = make(kv, heads=h, kv_heads=h, dim=d, pool_blocks=200, max_context=n + 16)
    sid = ctx.session_open()
    ctx.session_extend([sid], [n])
    xd = x.cuda()
    for step in (n, 100):  # as one call, and as calls of few rows
        for at in range(0, n, step):
            if step != n:
                ctx.session_truncate(sid, at)
                ctx.session_extend([sid], [step])
            ctx.kv_write(0, [sid], [step], xd[at:at + step], xd[at:at + step])
        out = torch.empty((2, n, h, d), dtype=torch.float16, device="cuda")
        ctx.kv_read(0, [sid], [n], out[0], out[1])
        ctx.sync()
        want = as_stored(x, kv)
        assert torch.equal(out[0].cpu(), want) and torch.equal(out[1].cpu(), want)


@pytest.mark.parametrize("kv", ALL_KV, ids=KV_NAMES.get)
@pytest.mark.parametrize("kv_heads,dim", [(1, 64), (3, 128), (8, 128)])
def test_read_gives_the_stored_values(kv, kv_heads, dim):
    """Newest tokens of several sessions into a strided buffer whose other bytes stay, and spans of one session in
    every layer, against the oracle's quantisers: equal to the bit."""
    rng = np.random.default_rng(7 + kv + dim)
    lens = [50, 1, 33]
    ctx = make(kv, heads=kv_heads, kv_heads=kv_heads, dim=dim, layers=3)
    sids, ks, vs = [], [], []
    for c in lens:
        sid = ctx.session_open()
        k, v = half(rng, 3, c, kv_heads, dim, std=3), half(rng, 3, c, kv_heads, dim)
        ctx.kv_append(sid, c, k.cuda(), v.cuda())
        ctx.sync()
        sids.append(sid)
        ks.append(as_stored(k, kv))
        vs.append(as_stored(v, kv))
    new = [19, 0, 33]
    width = kv_heads * dim
    for layer in range(3):
        out = torch.full((2, sum(new), width + 16), 7.0, dtype=torch.float16, device="cuda")
        ctx.kv_read(layer, sids, new, out[0], out[1], ld=width + 16)
        ctx.sync()
        for x, ref in ((out[0], ks), (out[1], vs)):
            want = torch.cat([r[layer, len(r[layer]) - m:] for r, m in zip(ref, new)])
            assert torch.equal(x[:, :width].cpu().reshape(want.shape), want)
            assert (x[:, width:] == 7).all()
    for first, n in ((0, 50), (13, 1), (15, 2), (16, 16), (31, 19), (49, 1)):
        out = torch.full((2, 3, n, kv_heads, dim), 7.0, dtype=torch.float16, device="cuda")
        ctx.kv_export(sids[0], first, n, out[0], out[1])
        ctx.sync()
        assert torch.equal(out[0].cpu(), ks[0][:, first:first + n])
        assert torch.equal(out[1].cpu(), vs[0][:, first:first + n])


def test_export_moves_a_session():
    """A session of an FP16 pool exported, closed, and appended to a new session: the same values, other blocks."""
    rng = np.random.default_rng(3)
    ctx = make(layers=2, pool_blocks=8)
    sid = ctx.session_open()
    k, v = half(rng, 2, 77, 2, 64).cuda(), half(rng, 2, 77, 2, 64).cuda()
    ctx.kv_append(sid, 77, k, v)
    out = torch.empty((2, 2, 77, 2, 64), dtype=torch.float16, device="cuda")
    ctx.kv_export(sid, 0, 77, out[0], out[1])
    ctx.session_close(sid)
    sid = ctx.session_open()
    ctx.kv_append(sid, 77, out[0], out[1])
    again = torch.empty_like(out)
    ctx.kv_export(sid, 0, 77, again[0], again[1])
    ctx.sync()
    assert torch.equal(again[0], k) and torch.equal(again[1], v)


def test_extend_is_all_or_nothing():
    ctx = make(pool_blocks=4, max_context=60)
    a, b = ctx.session_open(), ctx.session_open()
    ctx.session_extend([a, b], [17, 0])
    assert (ctx.session_length(a), ctx.session_length(b)) == (17, 0)
    with pytest.raises(mag.MagError) as e:
        ctx.session_extend([b, a], [16, 30])  # 1 + 1 blocks of 2 fit; 16 more of b do not
        ctx.session_extend([b, a], [33, 1])
    assert e.value.status == mag.ERR_KV_FULL
    lengths = ctx.session_length(a), ctx.session_length(b)
    free = ctx.memory_stats()["pool_blocks_free"]
    with pytest.raises(mag.MagError) as e:
        ctx.session_extend([b, a], [1, 100])
    assert e.value.status == mag.ERR_CONTEXT_FULL
    assert (ctx.session_length(a), ctx.session_length(b)) == lengths
    assert ctx.memory_stats()["pool_blocks_free"] == free


# ------------------------------------------------------------------------------------------------ attention
def reference(q, k, v, pos0, window, scale):
    """q [n, Hq, d], k and v [len, Hkv, d] (what the cache reads back as); returns the output in 64 bits and, per
    element, sum_j w_j |v_j - o|: how far a relative error of every weight can move it."""
    q, k, v = q.double(), k.double(), v.double()
    n, hq, d = q.shape
    g = hq // k.shape[1]
    k, v = k.repeat_interleave(g, 1), v.repeat_interleave(g, 1)
    s = torch.einsum("nhd,khd->hnk", q, k) * scale
    p = pos0 + torch.arange(n).view(1, n, 1)
    j = torch.arange(k.shape[0]).view(1, 1, -1)
    hidden = (j > p) | ((j <= p - window) if window else torch.zeros_like(j, dtype=torch.bool))
    w = torch.softmax(s.masked_fill(hidden, -math.inf), -1)
    o = torch.einsum("hnk,khd->nhd", w, v)
    spread = torch.empty_like(o)
    for h in range(hq):
        spread[:, h] = torch.stack([(w[h, i, :, None] * (v[:, h] - o[i, h]).abs()).sum(0) for i in range(n)])
    return o, spread


def check(out, o, spread, group):
    """fp16 output and weights, each off by at most half a step, 2^-11 of it. The output adds 2^-11 |o|. With weights
    w_j (1 + e_j), |e_j| <= 2^-11, in the products: sessions of up to 16 packed rows add up the rounded weights, so o
    moves by sum_j w_j e_j (v_j - o), at most 2^-11 of the spread; the others add up the unrounded ones, so it
    moves by sum_j w_j e_j v_j, at most 2^-11 (|o| + spread). What is left, the scores and exponentials in fp32
    (about 2^-18 of a weight) and weights below fp16's normal range (2^-25 each of a sum of at least 2^7), is within a
    tenth of that on these sizes; 2^-24 is half of fp16's smallest step, twice."""
    rows = o.shape[0]
    out = out.double().cpu()
    assert torch.isfinite(out).all()
    many = rows * group > 16
    tol = 1.1 * 2.0 ** -11 * ((2 if many else 1) * o.abs() + spread) + 2.0 ** -24
    bad = (out - o).abs() > tol
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()}, worst {((out - o).abs() / tol).max():.2f} times"


def attend_case(kv, heads, kv_heads, dim, priors, new, window=0, scale=None, std=1.0, seed=0, layers=1, layer=0,
                extra=0, ctx=None):
    rng = np.random.default_rng(seed)
    lens = [p + n for p, n in zip(priors, new)]
    if ctx is None:
        ctx = make(kv, heads, kv_heads, dim, layers, pool_blocks=sum(-(-n // 16) for n in lens) + 3,
                   sessions=len(lens), max_context=max(max(lens), 1), seed=seed)
    sids, ks, vs = [], [], []
    for n in lens:
        sid = ctx.session_open()
        k, v = half(rng, layers, n, kv_heads, dim, std=std), half(rng, layers, n, kv_heads, dim)
        if n:
            ctx.kv_append(sid, n, k.cuda(), v.cuda())
            ctx.sync()
        sids.append(sid)
        ks.append(as_stored(k, kv)[layer])
        vs.append(as_stored(v, kv)[layer])
    rows = sum(new)
    q = half(rng, rows, heads, dim, std=std)
    width = heads * dim
    qd = torch.zeros((rows, width + 8 * extra), dtype=torch.float16, device="cuda")
    qd[:, :width] = q.reshape(rows, width).cuda()
    out = torch.full((rows, width + 8 * extra), 7.0, dtype=torch.float16, device="cuda")
    ctx.attend(layer, sids, new, qd, out, ldq=qd.stride(0), ldo=out.stride(0), window=window, scale=scale)
    ctx.sync()
    assert (out[:, width:] == 7).all()
    got = out[:, :width].reshape(rows, heads, dim)
    at = 0
    for i, m in enumerate(new):
        if m:
            check(got[at:at + m], *reference(q[at:at + m], ks[i], vs[i], lens[i] - m, window,
                                             dim ** -0.5 if scale is None else scale), heads // kv_heads)
        at += m
    return ctx, sids, qd, out


@pytest.mark.parametrize("kv", ALL_KV, ids=KV_NAMES.get)
@pytest.mark.parametrize("heads,kv_heads,dim", [(1, 1, 64), (4, 2, 128), (8, 1, 128), (6, 2, 64), (5, 1, 128)])
@pytest.mark.parametrize("prior,new", [(0, 1), (0, 2), (15, 1), (16, 1), (100, 3), (257, 1)])
def test_attend_few_tokens(kv, heads, kv_heads, dim, prior, new):
    attend_case(kv, heads, kv_heads, dim, [prior], [new], seed=prior)


@pytest.mark.parametrize("kv", ALL_KV, ids=KV_NAMES.get)
@pytest.mark.parametrize("heads,kv_heads,dim", [(2, 2, 64), (4, 1, 128), (8, 1, 64), (3, 1, 128), (14, 2, 128)])
@pytest.mark.parametrize("prior,new", [(0, 17), (0, 128), (5, 33), (300, 64), (129, 130), (64, 301)])
def test_attend_chunk(kv, heads, kv_heads, dim, prior, new):
    attend_case(kv, heads, kv_heads, dim, [prior], [new], seed=new)


@pytest.mark.parametrize("kv", ALL_KV, ids=KV_NAMES.get)
@pytest.mark.parametrize("window", [1, 2, 15, 16, 17, 100, 128, 1000])
@pytest.mark.parametrize("prior,new", [(200, 1), (400, 5), (150, 140)])
def test_attend_window(kv, window, prior, new):
    attend_case(kv, 4, 2, 128, [prior], [new], window=window, seed=window)


@pytest.mark.parametrize("kv", ALL_KV, ids=KV_NAMES.get)
@pytest.mark.parametrize("dim", [64, 128])
def test_attend_sessions_of_every_size(kv, dim):
    """Sixteen sessions, among them empty, left-out, single-token and chunk ones, in one call."""
    priors = [0, 0, 3, 700, 16, 15, 31, 1, 90, 64, 250, 8, 0, 33, 511, 2]
    new = [0, 1, 0, 1, 2, 1, 1, 4, 70, 17, 1, 130, 260, 1, 3, 16]
    attend_case(kv, 8, 2, dim, priors, new, seed=11, extra=3)


@pytest.mark.parametrize("kv", ALL_KV, ids=KV_NAMES.get)
@pytest.mark.parametrize("new", [1, 6, 200])
def test_attend_long_and_sharp(kv, new):
    """Thousands of keys and scores of a hundred and more: a running maximum that moves late."""
    attend_case(kv, 4, 1, 128, [5000], [new], std=3.0, seed=5)


def test_attend_other_layer_and_scale():
    for layer in (0, 2):
        attend_case(mag.KV_INT8, 4, 2, 64, [70, 10], [40, 1], layers=3, layer=layer, scale=0.3, seed=layer)
    attend_case(mag.KV_FP16, 4, 2, 64, [70], [40], scale=0.0)
    attend_case(mag.KV_FP16, 4, 2, 64, [70], [3], scale=-0.125)


def test_attend_ignores_what_a_recycled_block_holds():
    """A closed session's infinities and NaN stay in its blocks; the next session's last block and tile hold them past
    its end."""
    for new in (1, 40):
        ctx = make(mag.KV_FP16, 4, 2, 128, pool_blocks=12, max_context=192)
        sid = ctx.session_open()
        bad = torch.full((1, 192, 2, 128), math.nan, dtype=torch.float16, device="cuda")
        bad[:, ::2] = math.inf
        ctx.kv_append(sid, 192, bad, bad)
        ctx.sync()
        ctx.session_close(sid)
        attend_case(mag.KV_FP16, 4, 2, 128, [90 - new], [new], ctx=ctx)


def test_attend_splits_merge_and_repeat_to_the_bit():
    """Long caches split over many blocks: repeated calls, and other calls between them on the same workspace, give the
    same bits."""
    ctx, sids, q, out = attend_case(mag.KV_INT4, 4, 2, 128, [6000, 3000], [1, 2], seed=21)
    first = out.clone()
    for _ in range(3):
        other = torch.empty_like(out[:2])
        ctx.attend(0, [sids[1]], [2], q[1:], other)
        out.zero_()
        ctx.attend(0, sids, [1, 2], q, out)
        ctx.sync()
        assert torch.equal(out, first)


def test_attend_captured_graph_replays():
    """write + attend captured on the context's stream; replays on new q, k, v equal eager calls."""
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        ctx = make(mag.KV_INT8, 4, 2, 128, pool_blocks=300, max_context=4800, stream=stream.cuda_stream)
        rng = np.random.default_rng(4)
        sid = ctx.session_open()
        k, v = half(rng, 1, 4000, 2, 128).cuda(), half(rng, 1, 4000, 2, 128).cuda()
        ctx.kv_append(sid, 4000, k, v)
        ctx.session_extend([sid], [20])
        nk, nv, q = (half(rng, 20, h, 128).cuda() for h in (2, 2, 4))
        out, eager = torch.empty_like(q), torch.empty_like(q)
        ctx.kv_write(0, [sid], [20], nk, nv)
        ctx.attend(0, [sid], [20], q, eager)
        ctx.sync()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            ctx.kv_write(0, [sid], [20], nk, nv)
            ctx.attend(0, [sid], [20], q, out)
        for i in range(3):
            for t in (nk, nv, q):
                t.copy_(half(rng, *t.shape).cuda())
            graph.replay()
            ctx.sync()
            ctx.kv_write(0, [sid], [20], nk, nv)
            ctx.attend(0, [sid], [20], q, eager)
            ctx.sync()
            assert torch.equal(out, eager)


@pytest.mark.parametrize("kv", ALL_KV, ids=KV_NAMES.get)
@pytest.mark.parametrize("group,new", [(1, 15), (1, 16), (1, 17), (1, 127), (1, 128), (1, 129), (1, 256), (1, 257), (3, 5),
                                       (3, 6), (3, 42), (3, 43), (3, 85), (3, 86), (8, 2), (8, 3), (8, 16), (8, 17),
                                       (8, 32), (8, 33)])
def test_attend_at_every_tile_border(kv, group, new):
    """Packed rows on both sides of 16, 128 and 256, over keys that are cut into several blocks' parts, with and without a
    window."""
    for dim, window in ((64, 0), (128, 700)):
        attend_case(kv, group, 1, dim, [2100], [new], window=window, seed=new)


def test_attend_two_graphs_and_calls_share_the_workspace():
    """Two captured graphs of one context, replayed in turn with a call between them, give the bits of eager calls."""
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        ctx, sids, q, out = attend_case(mag.KV_INT8, 4, 1, 128, [3000, 2500, 2000], [3, 30, 200], seed=8, ctx=make(
            mag.KV_INT8, 4, 1, 128, pool_blocks=520, max_context=3100, stream=stream.cuda_stream))
        eager = [torch.empty_like(out) for _ in range(2)]
        calls = ((sids[:2], [3, 30], q), (sids[1:], [30, 200], q[3:]))
        for c, e in zip(calls, eager):
            ctx.attend(0, *c, e)
        ctx.sync()
        graphs, outs = [], []
        for c in calls:
            o, g = torch.empty_like(out), torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=stream):
                ctx.attend(0, *c, o)
            graphs.append(g)
            outs.append(o)
        for _ in range(3):
            for i, (g, o, n) in enumerate(zip(graphs, outs, (33, 230))):
                o.zero_()
                g.replay()
                ctx.attend(0, sids, [3, 30, 200], q, out)
                ctx.sync()
                assert torch.equal(o[:n], eager[i][:n])


def test_what_a_capture_refuses():
    """A context's first attend (it makes the workspace) and every session_extend; the capture goes on."""
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        ctx = make(mag.KV_FP16, 4, 2, 64, stream=stream.cuda_stream)
        sid = ctx.session_open()
        ctx.session_extend([sid], [20])
        k, q = torch.zeros((20, 2, 64), device="cuda").half(), torch.zeros((20, 4, 64), device="cuda").half()
        out = torch.ones_like(q)
        ctx.kv_write(0, [sid], [20], k, k)
        ctx.sync()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            for call in (lambda: ctx.attend(0, [sid], [20], q, out), lambda: ctx.session_extend([sid], [1])):
                with pytest.raises(mag.MagError) as e:
                    call()
                assert e.value.status == mag.ERR_INVALID_ARG
            ctx.kv_write(0, [sid], [20], k, k)
        graph.replay()
        ctx.sync()
        assert ctx.session_length(sid) == 20
        ctx.attend(0, [sid], [20], q, out)
        ctx.sync()
        assert (out == 0).all()


def test_attend_without_memory_for_the_workspace():
    ctx = make(mag.KV_FP16, 4, 2, 64)
    sid = ctx.session_open()
    ctx.session_extend([sid], [20])
    k, q = torch.ones((20, 2, 64), device="cuda").half(), torch.zeros((20, 4, 64), device="cuda").half()
    ctx.kv_write(0, [sid], [20], k, k)
    out = torch.zeros_like(q)
    before = ctx.memory_stats()["other_device_bytes"]
    for skip in range(3):
        mag.debug_fail_allocations(skip, 1)
        try:
            with pytest.raises(mag.MagError) as e:
                ctx.attend(0, [sid], [20], q, out)
        finally:
            mag.debug_fail_allocations(0, 0)
        assert e.value.status == mag.ERR_OOM and ctx.memory_stats()["other_device_bytes"] == before
    ctx.attend(0, [sid], [20], q, out)
    ctx.sync()
    assert (out == 1).all() and ctx.memory_stats()["other_device_bytes"] > before


@pytest.mark.parametrize("kv", ALL_KV, ids=KV_NAMES.get)
def test_elastic_pool_grows_under_extension(kv):
    """Sessions of an elastic pool, which maps its blocks as they are asked for: extended, written, attended and read."""
    rng = np.random.default_rng(3)
    ctx = make(kv, 4, 2, 64, pool_blocks=2048, max_context=20000, flags=mag.FLAG_ELASTIC_POOL)
    mapped = ctx.memory_stats()["pool_blocks_mapped"]
    n = min(19000, (mapped + 1) * 16 + 5)
    sid = ctx.session_open()
    k, v = half(rng, n, 2, 64), half(rng, n, 2, 64)
    ctx.session_extend([sid], [n])
    ctx.kv_write(0, [sid], [n], k.cuda(), v.cuda())
    kr, vr = torch.empty((2, n, 2, 64), dtype=torch.float16, device="cuda")
    ctx.kv_read(0, [sid], [n], kr, vr)
    q = half(rng, 3, 4, 64)
    out = torch.empty((3, 4, 64), dtype=torch.float16, device="cuda")
    ctx.attend(0, [sid], [3], q.cuda(), out)
    ctx.sync()
    ks, vs = as_stored(k, kv), as_stored(v, kv)
    assert torch.equal(kr.cpu(), ks) and torch.equal(vr.cpu(), vs)
    check(out, *reference(q, ks, vs, n - 3, 0, 0.125), 2)


# ------------------------------------------------------------------------------------------------ sampling
def sample_reference(logits, t, k, p, m, u, allowed):
    """One row in 64 bits; returns (token, probability)."""
    x = np.where(allowed, logits.astype(np.float64), -np.inf)
    x[np.isnan(x)] = -np.inf
    order = np.argsort(-x, kind="stable")
    order = order[x[order] > -np.inf]
    if len(order) == 0:
        return -1, math.nan
    if not t > 0:
        return int(order[0]), 1.0
    with np.errstate(invalid="ignore"):
        w = np.exp((x[order] - x[order[0]]) / np.float64(np.float32(t)))
    w[x[order] == x[order[0]]] = 1.0
    n = len(w)
    if 0 < k < n:
        n = k
    total = w[:n].sum()
    if p < 1:
        n = min(n, int((np.cumsum(w[:n]) < np.float64(np.float32(p)) * total).sum()) + 1)
    if m > 0:
        n = min(n, max(1, int((w >= np.float64(np.float32(m))).sum())))
    c = np.cumsum(w[:n])
    i = min(int((c <= np.float64(np.float32(u)) * c[-1]).sum()), n - 1)
    return int(order[i]), w[i] / c[-1]


def sample_case(logits, t=None, k=None, p=None, m=None, u=None, allowed=None, seed=0, ld=None):
    rows, vocab = logits.shape
    rng = np.random.default_rng(seed)
    u = rng.random(rows, dtype=np.float32) if u is None else np.asarray(u, np.float32)
    dev = {}
    for name, val, dt in (("temperature", t, np.float32), ("top_k", k, np.int32), ("top_p", p, np.float32),
                          ("min_p", m, np.float32)):
        dev[name] = None if val is None else torch.from_numpy(np.broadcast_to(np.asarray(val, dt), (rows,)).copy()).cuda()
    words = None
    if allowed is not None:
        padded = np.zeros((rows, -(-vocab // 32) * 32), np.uint8)
        padded[:, :vocab] = allowed
        words = torch.from_numpy(np.packbits(padded, axis=1, bitorder="little").view(np.int32).copy()).cuda()
    ld = vocab if ld is None else ld
    buf = torch.full((rows, ld), 1e4, dtype=torch.from_numpy(logits[:0]).dtype, device="cuda")
    buf[:, :vocab] = torch.from_numpy(logits).cuda()
    token = torch.full((rows,), -7, dtype=torch.int32, device="cuda")
    prob = torch.full((rows,), -7.0, dtype=torch.float32, device="cuda")
    mag.sample(buf, rows, vocab, torch.from_numpy(u).cuda(), token, prob=prob, ld=ld,
               dtype=mag.LOGITS_F16 if logits.dtype == np.float16 else mag.LOGITS_F32, allowed=words, **dev)
    torch.cuda.synchronize()
    got, gp = token.cpu().numpy(), prob.cpu().numpy()
    at = lambda v, r, off: off if v is None else float(np.broadcast_to(v, (rows,))[r])  # noqa: E731
    for r in range(rows):
        ref, rp = sample_reference(logits[r], at(t, r, 1.0), int(at(k, r, 0)), at(p, r, 1.0), at(m, r, 0.0), u[r],
                                   np.ones(vocab, bool) if allowed is None else allowed[r])
        assert got[r] == ref, (r, got[r], ref)
        # Rounded to fp32 (2^-24 of it) from a quotient whose terms are good to 2^-30 of themselves, and whose upper one is
        # rounded to units of 2^-40 of the row's largest weight: off by 2^-41 of that, and the sum is at least that.
        assert (math.isnan(rp) and math.isnan(gp[r])) or abs(gp[r] - rp) <= rp * (2.0 ** -24 + 2.0 ** -28) + 2.0 ** -41, (
            r, gp[r], rp)
    return got, gp


def rows_of(rng, rows, vocab, dtype, std=2.5):
    return (rng.standard_normal((rows, vocab)) * std).astype(dtype)


@pytest.mark.parametrize("dtype", [np.float16, np.float32])
@pytest.mark.parametrize("rows,vocab", [(1, 1), (3, 2), (2, 31), (5, 33), (4, 1000), (1, 5001), (200, 777), (2, 128256),
                                        (20, 20000), (30, 1), (160, 40), (22, 128256), (5, 200000)])
def test_sample_cuts(dtype, rows, vocab):
    rng = np.random.default_rng(rows + vocab)
    x = rows_of(rng, rows, vocab, dtype)
    sample_case(x, seed=1)
    sample_case(x, t=0.7, seed=2)
    sample_case(x, t=0.9, k=5, seed=3)
    sample_case(x, t=1.3, p=0.8, seed=4)
    sample_case(x, t=1.0, m=0.05, seed=5)
    sample_case(x, t=rng.uniform(0.3, 2, rows), k=rng.integers(0, vocab + 2, rows), p=rng.uniform(0, 1.1, rows),
                m=rng.uniform(-0.1, 0.5, rows), seed=6)


@pytest.mark.parametrize("dtype", [np.float16, np.float32])
def test_sample_strides_and_masks(dtype):
    rng = np.random.default_rng(9)
    for ld in (501, 508, 640):
        for copies in (1, 5, 30):
            x = rows_of(rng, 6 * copies, 501, dtype)
            share = np.tile(np.array([[1.0], [0.5], [0.01], [0.0], [0.9], [0.002]]), (copies, 1))
            allowed = rng.random((6 * copies, 501)) < share
            allowed[4, np.argsort(-x[4].astype(np.float64))[:5]] = False
            sample_case(x, t=0.8, k=[0, 3, 0, 4, 10, 0] * copies, p=0.9, allowed=allowed, ld=ld, seed=ld)
            sample_case(x, t=0.8, m=[0, 0.1, 0, 0.9, 1e-3, 0] * copies, allowed=allowed, ld=ld, seed=ld)


@pytest.mark.parametrize("dtype", [np.float16, np.float32])
def test_sample_ties(dtype):
    """Equal logits go by index: in what top-k and top-p keep, and in the token that u picks."""
    x = np.zeros((24, 4096), dtype)
    u = [0.0, 0.25, 0.5, 0.999, 0.0, 0.5, 0.75, 1 - 2.0 ** -24] * 3
    got, prob = sample_case(x, u=u)
    assert list(got) == [int(4096 * np.float32(v)) for v in u]
    got, _ = sample_case(x, k=16, u=u)
    assert list(got) == [int(16 * np.float32(v)) for v in u]
    got, _ = sample_case(x, p=0.5, u=u)
    assert list(got) == [int(2048 * np.float32(v)) for v in u]
    x[:, 100:3000] = 2.0
    x[:, 7] = -0.0
    sample_case(x, t=0.5, k=2950, u=u)
    sample_case(x, t=0.5, p=0.9999, u=u)
    sample_case(x, m=1.0, u=u)


@pytest.mark.parametrize("dtype", [np.float16, np.float32])
def test_sample_numbers_outside_the_unit_interval(dtype):
    """No uniform number takes the draw out of what the cuts keep."""
    x = rows_of(np.random.default_rng(6), 6, 4000, dtype)
    u = torch.tensor([math.nan, -1.0, 1.0, 2.0, math.inf, -math.inf], device="cuda")
    token = torch.full((6,), -7, dtype=torch.int32, device="cuda")
    mag.sample(torch.from_numpy(x).cuda(), 6, 4000, u, token, stream=torch.cuda.current_stream().cuda_stream,
               dtype=mag.LOGITS_F32 if dtype == np.float32 else mag.LOGITS_F16,
               top_k=torch.full((6,), 5, dtype=torch.int32, device="cuda"))
    for row, t in zip(x, token.cpu().tolist()):
        assert t in np.argsort(-row.astype(np.float64), kind="stable")[:5]


def test_sample_captured_on_another_stream():
    rng = np.random.default_rng(12)
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        x, u = torch.from_numpy(rows_of(rng, 5, 3000, np.float16)).cuda(), torch.rand(5, device="cuda")
        token, eager = torch.empty((2, 5), dtype=torch.int32, device="cuda")
        p = torch.full((5,), 0.9, device="cuda")
        mag.sample(x, 5, 3000, u, eager, top_p=p, stream=stream.cuda_stream)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            mag.sample(x, 5, 3000, u, token, top_p=p, stream=stream.cuda_stream)
        for _ in range(3):
            x.copy_(torch.from_numpy(rows_of(rng, 5, 3000, np.float16)))
            u.copy_(torch.rand(5))
            graph.replay()
            mag.sample(x, 5, 3000, u, eager, top_p=p, stream=stream.cuda_stream)
            stream.synchronize()
            assert torch.equal(token, eager)


@pytest.mark.parametrize("dtype", [np.float16, np.float32])
@pytest.mark.parametrize("rows,vocab", [(1, 128256), (3, 20000), (160, 9000)])
def test_sample_crowds(dtype, rows, vocab):
    """Thousands of tokens within a hair of each other, or equal, at and below the top: cuts and draws inside them."""
    rng = np.random.default_rng(vocab)
    flat = np.full((rows, vocab), 1.5, dtype)
    steps = (rng.integers(0, 4, (rows, vocab)) * 0.5).astype(dtype)
    peak = steps.copy()
    peak[:, vocab // 3] = 9.0
    narrow = rows_of(rng, rows, vocab, dtype, std=1e-3)
    for x in (flat, steps, peak, narrow):
        sample_case(x, seed=1)
        sample_case(x, k=vocab // 2, seed=2)
        sample_case(x, t=0.7, k=vocab - 1, p=0.6, seed=3)
        sample_case(x, t=2.0, p=0.3, m=0.4, seed=4)
        sample_case(x, t=1e4, p=0.9, seed=5)
        sample_case(x, t=0.05, k=3000, m=0.9, seed=6)
        sample_case(x, k=1000, p=0.99, seed=7)


def test_sample_more_equal_tokens_than_16_bits_count():
    """Rows of which most tokens are equal, many rows at a time: counts past 65,535, of even and odd patterns, at the top
    and below it."""
    rng = np.random.default_rng(5)
    x = rows_of(rng, 24, 131000, np.float16)
    for r in range(24):
        few = rng.permutation(131000)[:65536 + 2000 * r]
        x[r, few] = np.array([0x3C00 + r % 2], np.uint16).view(np.float16)[0] * (1 if r % 3 else -1)
    x[::5, 77] = 14.0
    sample_case(x, t=0.8, seed=1)
    sample_case(x, t=1.2, k=rng.integers(0, 131000, 24), p=rng.uniform(0.1, 1.1, 24), m=rng.uniform(-0.1, 0.2, 24), seed=2)


@pytest.mark.parametrize("copies", [1, 4, 20])
@pytest.mark.parametrize("dtype", [np.float16, np.float32])
def test_sample_extremes(dtype, copies):
    rng = np.random.default_rng(12)
    nan = np.nan
    x = np.concatenate([rows_of(rng, 9, 300, dtype)] * copies)
    for at in range(0, 9 * copies, 9):
        extreme_rows(x[at:at + 9], dtype)
    got, prob = sample_case(x, seed=3)
    assert got[0] == got[1] == -1 and got[2] in (5, 17, 200)
    for t in (0.0, -1.0, nan, 1e-30, 1e-6, 1e6, 1e30):
        sample_case(x, t=t, seed=4)
    for p in (0.0, -3.0, 1e-9, 1.0, 5.0):
        sample_case(x, p=p, seed=5)
    for m in (2.0, 1.0, -1.0, 0.999, 1e-9):
        sample_case(x, m=m, seed=6)
    sample_case(x, k=-5, seed=7)
    sample_case(x, k=2 ** 31 - 1, seed=8)
    sample_case(x, k=7, m=0.5, seed=9)


def extreme_rows(x, dtype):
    inf, nan = np.inf, np.nan
    x[0, :] = -inf
    x[1, :] = nan
    x[2, [5, 17, 200]] = inf
    x[3, 10] = nan
    x[4, :] = 65504 if dtype == np.float16 else 3e38
    x[5, :] = -65504 if dtype == np.float16 else -3e38
    x[5, 3] = 1
    x[6, 100:] = -inf
    x[7, ::2] = 60000.0
    x[7, 1::2] = 6e-8


def test_sample_shares_of_many_draws():
    """Frequencies over 4096 evenly spaced u follow the shares to one part in 4096 a token."""
    x = np.broadcast_to(np.array([2.0, 1.0, 0.0, -1.0, 3.0], np.float32), (4096, 5)).copy()
    u = (np.arange(4096) + 0.5) / 4096
    got, _ = sample_case(x, u=u)
    w = np.exp(x[0].astype(np.float64))
    assert np.abs(np.bincount(got, minlength=5) / 4096 - w / w.sum()).max() <= 1.5 / 4096


# ------------------------------------------------------------------------------------------------ together
@pytest.mark.parametrize("kv", ALL_KV, ids=KV_NAMES.get)
def test_generation_loop(kv):
    """A two-layer decoder of the caller's own (an attention layer with a bias, no FFN): a prompt as one chunk, then
    tokens one at a time, each drawn by mag_sample. The same tokens fed as one chunk give the same last outputs."""
    L, H, HK, D, V, hid = 2, 4, 2, 64, 500, 256
    gen = torch.Generator().manual_seed(kv + 1)
    rand = lambda *s: (torch.randn(*s, generator=gen) / math.sqrt(s[-1])).half().cuda()  # noqa: E731
    emb, head = rand(V, hid) * 16, rand(V, hid) * 12
    wqkv, bias, wo = [rand((H + 2 * HK) * D, hid) for _ in range(L)], [rand(1, (H + 2 * HK) * D) for _ in range(L)], \
        [rand(hid, H * D) for _ in range(L)]

    def forward(ctx, sids, counts, tokens):
        ctx.session_extend(sids, counts)
        x = emb[tokens].float()
        for layer in range(L):
            qkv = (x.half() @ wqkv[layer].T + bias[layer]).contiguous()
            ctx.kv_write(layer, sids, counts, qkv[:, H * D:], qkv[:, (H + HK) * D:], ld=qkv.stride(0))
            o = torch.empty((len(tokens), H * D), dtype=torch.float16, device="cuda")
            ctx.attend(layer, sids, counts, qkv, o, ldq=qkv.stride(0))
            x = x + (o @ wo[layer].T).float()
        return (x.half() @ head.T).contiguous()

    ctx = make(kv, H, HK, D, layers=L, pool_blocks=40, sessions=4)
    sids = [ctx.session_open(), ctx.session_open()]
    prompts = [[5, 6, 7, 8, 9] * 7, [100, 3]]
    logits = forward(ctx, sids, [35, 2], torch.tensor(sum(prompts, []), device="cuda"))
    last = logits[[34, 36]].contiguous()
    history, outs = [list(p) for p in prompts], []
    rng = np.random.default_rng(0)
    for _ in range(20):
        u = torch.from_numpy(rng.random(2, dtype=np.float32)).cuda()
        token = torch.empty(2, dtype=torch.int32, device="cuda")
        temp, top_p = torch.full((2,), 0.8, device="cuda"), torch.full((2,), 0.95, device="cuda")
        mag.sample(last, 2, V, u, token, temperature=temp, top_p=top_p)
        ids = token.cpu().tolist()
        for i in range(2):
            ref, _ = sample_reference(last[i].cpu().numpy(), 0.8, 0, 0.95, 0.0, float(u[i].cpu()), np.ones(V, bool))
            assert ids[i] == ref
            history[i].append(ids[i])
        last = forward(ctx, sids, [1, 1], token.long())
        outs.append(last)
    ctx.sync()
    # each whole sequence as one chunk of a fresh session
    for i in range(2):
        sid = ctx.session_open()
        whole = forward(ctx, [sid], [len(history[i])], torch.tensor(history[i], device="cuda"))
        ctx.sync()
        assert ctx.session_length(sid) == ctx.session_length(sids[i])
        ref = whole[-1].float()
        # quantised caches hold the same codes but for roundings of q, k, v at the last bit of fp16
        assert float((outs[-1][i].float() - ref).norm() / ref.norm()) < 2e-2
        ctx.session_close(sid)


def test_sample_on_the_steps_logits():
    """mag_decode_step's fp16 logits go into mag_sample as they lie."""
    from synth import driver
    from synth.workloads import TINY, Workload
    from dataclasses import replace
    wl = Workload("tiny-vocab", replace(TINY, vocab=512), mag.KV_FP16, 2, (30, 9))
    ctx, sids = driver.setup(wl, 1)
    x = torch.from_numpy(driver.step_inputs(wl, 1)).cuda()
    logits = torch.empty((2, 512), dtype=torch.float16, device="cuda")
    ctx.decode_step(sids, x, logits)
    ctx.sync()
    sample_case(logits.cpu().numpy(), t=0.1, k=40, p=0.9)
    # attention over the step's own cache: one more token written and attended by hand
    n = ctx.session_length(sids[0])
    ctx.session_extend([sids[0]], [0])
    q = torch.randn(1, 4, 64, device="cuda").half()
    out = torch.empty_like(q)
    ctx.attend(0, [sids[0]], [1], q, out)
    kv = torch.empty((2, 1, n, 2, 64), dtype=torch.float16, device="cuda")
    ctx.kv_export(sids[0], 0, n, kv[0], kv[1])
    ctx.sync()
    check(out, *reference(q.cpu(), kv[0, 0].cpu(), kv[1, 0].cpu(), n - 1, 0, 0.125), 2)


# ------------------------------------------------------------------------------------------------ refusals
def test_refusals():
    ctx = make(mag.KV_INT8, 4, 2, 64, layers=2)
    sid, other = ctx.session_open(), ctx.session_open()
    ctx.session_extend([sid], [20])
    buf = torch.zeros((64, 512), dtype=torch.float16, device="cuda")
    far = torch.zeros((64, 512), dtype=torch.float16, device="cuda")

    def refused(call, *args, **kw):
        with pytest.raises(mag.MagError) as e:
            call(*args, **kw)
        assert e.value.status == mag.ERR_INVALID_ARG, e.value

    for call in (ctx.kv_write, ctx.kv_read, ctx.attend):
        for layer in (-1, 2):
            refused(call, layer, [sid], [4], buf, far)
        refused(call, 0, [], [], buf, far)
        refused(call, 0, [sid] * 17, [1] * 17, buf, far)
        refused(call, 0, [sid, sid], [1, 1], buf, far)
        refused(call, 0, [3], [1], buf, far)       # not open
        refused(call, 0, [-1], [1], buf, far)
        refused(call, 0, [sid], [21], buf, far)    # more than it holds
        refused(call, 0, [sid], [-1], buf, far)
        refused(call, 0, [other], [1], buf, far)   # empty
        refused(call, 0, [sid], [4], None, far)
        refused(call, 0, [sid], [4], buf, None)
        refused(call, 0, [sid], [4], buf.data_ptr() + 2, far)
        refused(call, 0, [sid], [4], buf, far.data_ptr() + 8)
        call(0, [sid, other], [0, 0], None, None)  # nothing to do
    for ld in (127, 129, 120, 0, -128):
        refused(ctx.kv_write, 0, [sid], [4], buf, far, ld=ld)
        refused(ctx.kv_read, 0, [sid], [4], buf, far, ld=ld)
    for ld in (255, 257, 248, 0):
        refused(ctx.attend, 0, [sid], [4], buf, far, ldq=ld)
        refused(ctx.attend, 0, [sid], [4], buf, far, ldo=ld)
    refused(ctx.attend, 0, [sid], [4], buf, far, window=-1)
    refused(ctx.attend, 0, [sid], [4], buf, far, scale=math.nan)
    refused(ctx.attend, 0, [sid], [4], buf, far, scale=math.inf)
    refused(ctx.kv_export, other, 0, 1, buf, far)
    refused(ctx.kv_export, sid, 10, 11, buf, far)
    refused(ctx.kv_export, sid, -1, 2, buf, far)
    refused(ctx.kv_export, sid, 0, -1, buf, far)
    refused(ctx.kv_export, sid, 0, 4, None, far)
    ctx.kv_export(sid, 20, 0, None, None)
    refused(ctx.session_extend, [sid, sid], [1, 1])
    refused(ctx.session_extend, [sid], [-1])
    refused(ctx.session_extend, [3], [1])
    refused(ctx.session_extend, [], [])
    with pytest.raises(ValueError):
        ctx.attend(0, [sid], [1, 1], buf, far)
    ctx.sync()
    assert ctx.session_length(sid) == 20


def test_bad_table_entry_is_reported_not_followed():
    """A block id outside the pool is not used: the calls finish, and the next sync says so."""
    ctx = make(mag.KV_FP16, 4, 2, 64)
    sid = ctx.session_open()
    ctx.session_extend([sid], [40])
    k = torch.zeros((40, 2, 64), dtype=torch.float16, device="cuda")
    q = torch.zeros((40, 4, 64), dtype=torch.float16, device="cuda")
    ctx.kv_write(0, [sid], [40], k, k)
    ctx.sync()
    for call in (lambda: ctx.kv_write(0, [sid], [40], k, k), lambda: ctx.kv_read(0, [sid], [40], k, k.clone()),
                 lambda: ctx.attend(0, [sid], [40], q, q.clone()), lambda: ctx.attend(0, [sid], [1], q, q.clone())):
        ctx.debug_set_table_entry(sid, 1, 1 << 20)
        call()
        with pytest.raises(mag.MagError) as e:
            ctx.sync()
        assert e.value.status == mag.ERR_CORRUPT
        ctx.sync()

"""Measured cases of the operators that a decoding loop outside the built-in step is made of.

Three kinds of operator, each in two forms: the plain one (elementary torch operations) and, with ``own`` set, the
library's calls:

* ``store`` / ``read``: one layer's new keys and values of several sessions written into the block pool, quantised to
  its precision as they are written, and read back as fp16 (``kv_write``, ``kv_read``);
* ``attend``: causal grouped-query attention of the sessions' newest tokens over that pool (``attend``);
* ``sample``: the next token of every row of logits by temperature, top-k, top-p and min-p from given uniform numbers
  (``sample``).

A cache is held as the pool holds it: blocks of 16 tokens in a shuffled order, fp16 values, int8 codes with one fp16
scale per (token, head), or 4-bit codes with an fp16 (scale, min) per 32 values. What a quantised cache reads back as
is the fp16 nearest to scale * code (+ min); attention is defined over those values.
"""
import math
import random

import torch

own = False

BLOCK = 16
KV_TYPES = ("fp16", "int8", "int4")


# ------------------------------------------------------------------------------------------------ cases
def listed():
    return [
        # the keys and values of one decode step of 16 sessions: the smallest write, where the launch is what counts
        dict(name="store_step16_int8", op="store", kv="int8", heads=32, kv_heads=8, dim=128, sessions=16, prior_lo=20,
             prior_hi=2048, new_lo=1, new_hi=1, spread=1, merged=True),
        # three prompts' chunks of uneven length, behind caches of their own, as a batched prefill writes them
        dict(name="store_chunks_int4", op="store", kv="int4", heads=32, kv_heads=8, dim=128, sessions=3, prior_lo=100,
             prior_hi=3000, new_lo=700, new_hi=4000, spread=2, merged=True),
        # a tool call's worth of tokens taken out of a cache, from an odd position
        dict(name="read_span_int4", op="read", kv="int4", heads=32, kv_heads=8, dim=128, layers=1, first=13,
             tokens=1237, spread=3),
        # a long session read back before its blocks are given to another one (four layers of it)
        dict(name="read_session_int8", op="read", kv="int8", heads=32, kv_heads=8, dim=128, layers=4, first=0,
             tokens=38863, spread=4),
        # one decode token of one session: latency
        dict(name="attend_step_fp16", op="attend", kv="fp16", heads=32, kv_heads=8, dim=128, sessions=1,
             prior_lo=2048, prior_hi=2048, new_lo=1, new_hi=1, window=0, spread=5, merged=True),
        # a decode step of 16 sessions of uneven length
        dict(name="attend_step16_int8", op="attend", kv="int8", heads=32, kv_heads=8, dim=128, sessions=16,
             prior_lo=500, prior_hi=20000, new_lo=1, new_hi=1, window=0, spread=6, merged=True),
        # four draft tokens checked at the end of a long 4-bit cache
        dict(name="attend_drafts_long_int4", op="attend", kv="int4", heads=32, kv_heads=8, dim=128, sessions=1,
             prior_lo=77726, prior_hi=77726, new_lo=4, new_hi=4, window=0, spread=7, merged=True),
        # a prompt chunk behind a short cache
        dict(name="attend_chunk_fp16", op="attend", kv="fp16", heads=32, kv_heads=8, dim=128, sessions=1,
             prior_lo=800, prior_hi=800, new_lo=512, new_hi=512, window=0, spread=8, merged=True),
        # a long chunk at the end of a long session: the largest
        dict(name="attend_chunk_long_fp16", op="attend", kv="fp16", heads=32, kv_heads=8, dim=128, sessions=1,
             prior_lo=19431, prior_hi=19431, new_lo=4096, new_hi=4096, window=0, spread=9, merged=True),
        # the next token of one session under every cut at once
        dict(name="sample_one", op="sample", rows=1, vocab=128256, type="fp16", cuts="all", mask=False, pad=0),
        # a decode step's 16 rows drawn from whole distributions (temperature only), logits in fp32
        dict(name="sample_step16_full_fp32", op="sample", rows=16, vocab=128256, type="fp32", cuts="none", mask=False,
             pad=0),
        # many requests with settings of their own, some of them bound to a set of allowed tokens
        dict(name="sample_many_mixed", op="sample", rows=256, vocab=128256, type="fp16", cuts="mixed", mask=True,
             pad=0),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.99)))))))


def draw(rng):
    op = rng.choice(("store", "read", "attend", "attend", "sample", "sample"))
    if op == "sample":
        rows = _log(rng, 1, 256)
        return dict(op=op, rows=rows, vocab=_log(rng, 16, 130000), type=rng.choice(("fp16", "fp32")),
                    cuts=rng.choice(("none", "all", "mixed", "mixed")), mask=rng.random() < 0.4,
                    pad=rng.choice((0, 0, 1, 8, 37)))
    kv = rng.choice(KV_TYPES)
    kv_heads, group, dim = rng.choice((1, 2, 4, 5, 8)), rng.choice((1, 2, 3, 4, 5, 8)), rng.choice((64, 128, 128))
    case = dict(op=op, kv=kv, heads=kv_heads * group, kv_heads=kv_heads, dim=dim)
    spread = rng.randrange(1 << 20)
    if op == "read":
        return dict(case, layers=rng.randint(1, 4), first=rng.randint(0, 200), tokens=_log(rng, 1, 38863),
                    spread=spread)
    sessions = _log(rng, 1, 16)
    if op == "store":
        hi = _log(rng, 1, 4096)
        return dict(case, sessions=sessions, prior_lo=1, prior_hi=_log(rng, 1, 4000), new_lo=rng.randint(1, hi),
                    new_hi=hi, spread=spread, merged=rng.random() < 0.5)
    # attention: the tokens that the sessions' lengths leave room for, so that no drawn case passes the largest listed
    prior_hi = rng.choice((0, *[_log(rng, 1, 40000)] * 5))
    room = max(1, int(3e9 / (sessions * case["heads"] * (prior_hi + 1500))))
    hi = min(_log(rng, 1, 2048), room)
    return dict(case, sessions=sessions, prior_lo=rng.randint(0, prior_hi), prior_hi=prior_hi,
                new_lo=rng.randint(1, hi), new_hi=hi, window=rng.choice((0, 0, _log(rng, 1, 20000))), spread=spread,
                merged=rng.random() < 0.5)


def _sizes(case):
    """The sessions' (tokens before, new tokens), spread over the case's ranges."""
    rng = random.Random(case["spread"])
    return [(_log(rng, max(1, case["prior_lo"]), max(1, case["prior_hi"])) if case["prior_hi"] else 0,
             _log(rng, case["new_lo"], case["new_hi"])) for _ in range(case["sessions"])]


def _vector_bytes(case):
    d = case["dim"]
    return {"fp16": 2 * d, "int8": d + 2, "int4": d // 2 + 4 * (d // 32)}[case["kv"]]


def _keys(prior, new, window):
    """Keys that `new` tokens after `prior` ones attend to, summed over the tokens, and how many different ones."""
    if not window:
        return new * prior + new * (new + 1) // 2, prior + new
    total = sum(min(window, prior + t + 1) for t in range(new))
    return total, min(prior + new, window + new - 1)


def work(case):
    op = case["op"]
    if op == "sample":
        size = 2 if case["type"] == "fp16" else 4
        mask = case["vocab"] / 8 if case["mask"] else 0
        return {"bytes": case["rows"] * (case["vocab"] * size + mask + 28), "flops": 4 * case["rows"] * case["vocab"]}
    h, d, vec = case["kv_heads"], case["dim"], _vector_bytes(case)
    if op == "read":
        n = 2 * case["layers"] * case["tokens"] * h
        return {"bytes": n * (vec + 2 * d), "flops": 2 * n * d}
    sizes = _sizes(case)
    if op == "store":  # fp16 in, the stored form out, and once more for reading it back
        n = 2 * sum(new for _, new in sizes) * h
        return {"bytes": n * (2 * d + vec) + n * (vec + 2 * d), "flops": 8 * n * d}
    pairs = keys = rows = 0
    for prior, new in sizes:
        p, k = _keys(prior, new, case["window"])
        pairs, keys, rows = pairs + p, keys + k, rows + new
    return {"bytes": 2 * keys * h * vec + 4 * rows * case["heads"] * d, "flops": 4 * pairs * case["heads"] * d}


# ------------------------------------------------------------------------------------------------ the cache, in torch
def _quantise(x, kv):
    """fp16 [..., d] as the pool stores it: (codes or values, scales)."""
    if kv == "fp16":
        return x, None
    f = x.float()
    if kv == "int8":
        s = (f.abs().amax(-1) / 127.0).half()
        q = torch.round(f / s.float().unsqueeze(-1)).clamp(-127, 127)
        return torch.where(s.unsqueeze(-1) == 0, torch.zeros_like(q), q).to(torch.int8), s
    g = f.unflatten(-1, (-1, 32))
    lo, hi = g.aminmax(dim=-1)
    s, m = ((hi - lo) / 15.0).half(), lo.half()
    q = torch.round((g - m.float().unsqueeze(-1)) / s.float().unsqueeze(-1)).clamp(0, 15)
    q = torch.where(s.unsqueeze(-1) == 0, torch.zeros_like(q), q).to(torch.uint8).flatten(-2)
    return q[..., 0::2] | (q[..., 1::2] << 4), torch.stack((s, m), -1)


def _values(codes, scales, kv):
    """The fp16 values that stored codes stand for."""
    if kv == "fp16":
        return codes
    if kv == "int8":
        return (codes.float() * scales.float().unsqueeze(-1)).half()
    q = torch.stack((codes & 15, codes >> 4), -1).flatten(-2).unflatten(-1, (-1, 32)).float()
    s, m = scales.float().unbind(-1)
    return (s.unsqueeze(-1) * q + m.unsqueeze(-1)).flatten(-2).half()


def _pool(case, layers, lengths, seed):
    """Empty blocks for sessions of these lengths: data and scales [layers, blocks, 2, heads, 16, ..] and the sessions'
    block ids [sessions, most blocks], shuffled."""
    h, d, kv = case["kv_heads"], case["dim"], case["kv"]
    per = [-(-n // BLOCK) for n in lengths]
    order = list(range(sum(per)))
    random.Random(seed).shuffle(order)
    table = torch.zeros((len(per), max(per)), dtype=torch.int64)
    at = 0
    for i, n in enumerate(per):
        table[i, :n] = torch.tensor(order[at:at + n], dtype=torch.int64)
        at += n
    shape = (layers, sum(per), 2, h, BLOCK)
    if kv == "fp16":
        data, scales = torch.zeros(shape + (d,), dtype=torch.float16, device="cuda"), None
    elif kv == "int8":
        data = torch.zeros(shape + (d,), dtype=torch.int8, device="cuda")
        scales = torch.zeros(shape, dtype=torch.float16, device="cuda")
    else:
        data = torch.zeros(shape + (d // 2,), dtype=torch.uint8, device="cuda")
        scales = torch.zeros(shape + (d // 32, 2), dtype=torch.float16, device="cuda")
    return {"data": data, "scales": scales, "table": table.cuda(), "order": order}


def _pool_write(pool, layer, sess, pos, k, v, kv):
    """Rows of keys and values [rows, heads, d] into the blocks of (session, position)."""
    block, slot = pool["table"][sess, pos // BLOCK], pos % BLOCK
    for part, x in enumerate((k, v)):
        codes, scales = _quantise(x, kv)
        pool["data"][layer, block, part, :, slot] = codes
        if scales is not None:
            pool["scales"][layer, block, part, :, slot] = scales


def _pool_read(pool, layers, sess, pos, part, kv):
    """fp16 [layers, *pos.shape, heads, d] of (session, position); `sess` and `pos` of one shape."""
    block, slot = pool["table"][sess, pos // BLOCK], pos % BLOCK
    codes = pool["data"][:layers, block, part, :, slot]  # the indexed axes come first
    scales = None if pool["scales"] is None else pool["scales"][:layers, block, part, :, slot]
    return _values(codes, scales, kv).movedim(pos.dim(), 0)


# ------------------------------------------------------------------------------------------------ inputs
def _context(case, layers, pool, max_context, sessions):
    """The library's context over a pool of the same size and block order."""
    import quantized_decode_step_gb300 as mag

    class Shape:
        n_layers, hidden, n_heads, n_kv_heads, head_dim = layers, 256, case["heads"], case["kv_heads"], case["dim"]
        ffn, vocab, rms_eps, rope_base = 256, 0, 1e-5, 10000.0

    cfg = mag.make_config(Shape, kv_dtype=KV_TYPES.index(case["kv"]), pool_blocks=len(pool["order"]),
                          max_sessions=sessions, max_batch=1, max_context=max_context, pool_order=pool["order"])
    # torch's default stream is the legacy one, whose handle as an argument is cudaStreamLegacy = 1
    return mag.Context(cfg, torch.cuda.current_stream().cuda_stream or 1)


def _normal(gen, *shape):
    return torch.randn(*shape, generator=gen, device="cuda", dtype=torch.float32).half()


def _keys_values(gen, case, *lead):
    """Keys and values as a trained layer has them: a few large channels in the keys, values without."""
    h, d = case["kv_heads"], case["dim"]
    k, v = _normal(gen, *lead, h, d), _normal(gen, *lead, h, d)
    k[..., 0:d:29] *= 3
    return k, v


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    op = case["op"]
    if op == "sample":
        return _prepare_sample(case, gen)
    if op == "read":
        n = case["first"] + case["tokens"]
        pool = _pool(case, case["layers"], [n], seed)
        state = dict(case=case, pool=pool, sess=torch.zeros(case["tokens"], dtype=torch.int64, device="cuda"),
                     pos=torch.arange(case["first"], n, device="cuda"))
        ctx = None
        if own:
            ctx = _context(case, case["layers"], pool, n, 1)
            state["sid"] = ctx.session_open()
        k, v = _keys_values(gen, case, case["layers"], n)
        every = torch.arange(n, device="cuda")
        for layer in range(case["layers"]):
            _pool_write(pool, layer, torch.zeros_like(every), every, k[layer], v[layer], case["kv"])
        if own:
            ctx.kv_append(state["sid"], n, k, v)
            ctx.sync()
        state.update(ctx=ctx)
        return state

    sizes = _sizes(case)
    lengths = [p + n for p, n in sizes]
    h, d, hq = case["kv_heads"], case["dim"], case["heads"]
    rows = sum(n for _, n in sizes)
    pool = _pool(case, 1, lengths, seed)
    state = dict(case=case, pool=pool, new=[n for _, n in sizes], ctx=None,
                 sess=torch.tensor([i for i, (_, n) in enumerate(sizes) for _ in range(n)], device="cuda"),
                 pos=torch.tensor([p + t for p, n in sizes for t in range(n)], device="cuda"),
                 turn=torch.tensor([t for _, n in sizes for t in range(n)], device="cuda"),
                 length=torch.tensor(lengths, device="cuda"))
    # the new tokens' q, k and v: rows of one merged projection, or tensors of their own
    q, (k, v) = _normal(gen, rows, hq, d), _keys_values(gen, case, rows)
    if case["merged"]:
        qkv = torch.cat((q, k, v), 1)
        q, k, v = qkv[:, :hq], qkv[:, hq:hq + h], qkv[:, hq + h:]
    state.update(q=q, k=k, v=v)
    if own:
        state["ctx"] = _context(case, 1, pool, max(lengths), len(sizes))
        state["sids"] = [state["ctx"].session_open() for _ in sizes]
    at = 0
    for i, (prior, new) in enumerate(sizes):  # what the cache holds already; for attention, the new tokens as well
        pk, pv = _keys_values(gen, case, prior)
        if op == "attend":
            pk, pv = torch.cat((pk, k[at:at + new])), torch.cat((pv, v[at:at + new]))
        at += new
        pos = torch.arange(len(pk), device="cuda")
        _pool_write(pool, 0, torch.full_like(pos, i), pos, pk, pv, case["kv"])
        if own:
            state["ctx"].kv_append(state["sids"][i], len(pk), pk, pv)
    if own:  # the new tokens' places in the cache
        if op == "store":
            state["ctx"].session_extend(state["sids"], state["new"])
        state["ctx"].sync()
    return state


def _prepare_sample(case, gen):
    rows, vocab = case["rows"], case["vocab"]
    # a language model's logits: most tokens far down, some tens of them near the top
    x = torch.randn(rows, vocab + case["pad"], generator=gen, device="cuda") * 2.2
    few = min(vocab, 40)
    top = torch.randint(0, vocab, (rows, few), generator=gen, device="cuda")
    x.scatter_add_(1, top, 6 * torch.rand(rows, few, generator=gen, device="cuda"))
    x = x.half() if case["type"] == "fp16" else x

    def uniform(lo, hi):
        return lo + (hi - lo) * torch.rand(rows, generator=gen, device="cuda")

    state = dict(case=case, logits=x[:, :vocab], uniform=torch.rand(rows, generator=gen, device="cuda"),
                 temperature=uniform(0.5, 1.5), top_k=None, top_p=None, min_p=None, allowed=None)
    if case["cuts"] == "all":
        state.update(top_k=uniform(1, 200).int(), top_p=uniform(0.7, 1.0), min_p=uniform(0.0, 0.1))
    elif case["cuts"] == "mixed":  # every row its own choice of cuts, some rows greedy
        on = torch.rand(4, rows, generator=gen, device="cuda")
        zero = torch.zeros(rows, device="cuda")
        state.update(temperature=torch.where(on[0] < 0.1, zero, state["temperature"]),
                     top_k=torch.where(on[1] < 0.5, uniform(1, 1000).int(), 0),
                     top_p=torch.where(on[2] < 0.6, uniform(0.5, 1.0), zero + 1),
                     min_p=torch.where(on[3] < 0.3, uniform(0.0, 0.2), zero))
    if case["mask"]:  # a bit for every token: nine in ten rows may use most of them, the others few
        most = torch.where(torch.rand(rows, 1, generator=gen, device="cuda") < 0.9, 0.95, 0.01)
        bits = torch.rand(rows, -(-vocab // 32), 32, generator=gen, device="cuda") < most.unsqueeze(-1)
        words = (bits.long() << torch.arange(32, device="cuda")).sum(-1)
        state["allowed"] = torch.where(words >= 1 << 31, words - (1 << 32), words).int()
    return state


# ------------------------------------------------------------------------------------------------ one pass
def run(state):
    op = state["case"]["op"]
    if op == "sample":
        return _run_sample(state)
    if op == "read":
        return _run_read(state)
    if op == "store":
        return _run_store(state)
    return _run_attend(state)


def _run_store(s):
    case, k, v = s["case"], s["k"], s["v"]
    rows, h, d = k.shape
    if own:
        s["ctx"].kv_write(0, s["sids"], s["new"], k, v, ld=k.stride(0))
        out = torch.empty((2, rows, h, d), dtype=torch.float16, device="cuda")
        s["ctx"].kv_read(0, s["sids"], s["new"], out[0], out[1])
        return {"k": out[0], "v": out[1]}
    _pool_write(s["pool"], 0, s["sess"], s["pos"], k, v, case["kv"])
    return {"k": _pool_read(s["pool"], 1, s["sess"], s["pos"], 0, case["kv"])[0],
            "v": _pool_read(s["pool"], 1, s["sess"], s["pos"], 1, case["kv"])[0]}


def _run_read(s):
    case = s["case"]
    if own:
        out = torch.empty((2, case["layers"], case["tokens"], case["kv_heads"], case["dim"]), dtype=torch.float16,
                          device="cuda")
        s["ctx"].kv_export(s["sid"], case["first"], case["tokens"], out[0], out[1])
        return {"k": out[0], "v": out[1]}
    return {"k": _pool_read(s["pool"], case["layers"], s["sess"], s["pos"], 0, case["kv"]),
            "v": _pool_read(s["pool"], case["layers"], s["sess"], s["pos"], 1, case["kv"])}


def _run_attend(s):
    case, q = s["case"], s["q"]
    rows, hq, d = q.shape
    if own:
        out = torch.empty((rows, hq, d), dtype=torch.float16, device="cuda")
        s["ctx"].attend(0, s["sids"], s["new"], q, out, ldq=q.stride(0), window=case["window"])
        return out
    # every session padded to the longest cache and to the most new tokens
    h, n_s = case["kv_heads"], len(s["new"])
    most, longest = max(s["new"]), s["pool"]["table"].shape[1] * BLOCK
    key = torch.arange(longest, device="cuda")
    sess = torch.arange(n_s, device="cuda").unsqueeze(1).expand(n_s, longest)
    k = _pool_read(s["pool"], 1, sess, key.expand(n_s, longest), 0, case["kv"])[0].float()  # [S, N, H, d]
    v = _pool_read(s["pool"], 1, sess, key.expand(n_s, longest), 1, case["kv"])[0].float()
    qf = torch.zeros((n_s, most, hq, d), device="cuda")
    qf[s["sess"], s["turn"]] = q.float()
    qpos = torch.full((n_s, most), -1, device="cuda")
    qpos[s["sess"], s["turn"]] = s["pos"]
    qf = qf.view(n_s, most, h, hq // h, d).permute(0, 2, 1, 3, 4).reshape(n_s, h, -1, d)
    score = torch.matmul(qf, k.permute(0, 2, 3, 1)).mul_(1.0 / math.sqrt(d))  # [S, H, T G, N]
    back = qpos.unsqueeze(-1) - key  # how far each key lies behind each token
    keep = (back >= 0) & (back < (case["window"] or longest + 1))
    score = score.view(n_s, h, most, hq // h, longest)
    score.masked_fill_(~keep.view(n_s, 1, most, 1, longest), -math.inf)
    score.sub_(score.amax(-1, keepdim=True)).exp_()
    total = score.sum(-1, keepdim=True)
    out = torch.matmul(score.view(n_s, h, -1, longest), v.permute(0, 2, 1, 3)).view(n_s, h, most, hq // h, d)
    out = (out / total).half().permute(0, 2, 1, 3, 4).reshape(n_s, most, hq, d)
    return out[s["sess"], s["turn"]]


def _run_sample(s):
    x, u = s["logits"], s["uniform"]
    rows, vocab = x.shape
    if own:
        import quantized_decode_step_gb300 as mag
        token = torch.empty(rows, dtype=torch.int32, device="cuda")
        prob = torch.empty(rows, dtype=torch.float32, device="cuda")
        mag.sample(x, rows, vocab, u, token, prob=prob, ld=x.stride(0),
                   dtype=mag.LOGITS_F16 if x.dtype == torch.float16 else mag.LOGITS_F32,
                   temperature=s["temperature"], top_k=s["top_k"], top_p=s["top_p"], min_p=s["min_p"],
                   allowed=s["allowed"], stream=torch.cuda.current_stream().cuda_stream)
        return {"token": token, "prob": prob}
    # cumulative sums of a whole vocabulary, compared with a number: in 64 bits
    x = x.float()
    if s["allowed"] is not None:
        bit = torch.arange(vocab, device="cuda")
        x = torch.where((s["allowed"][:, bit // 32] >> (bit % 32)) & 1 == 1, x, -math.inf)
    x, index = torch.sort(x, dim=1, descending=True, stable=True)
    rank = torch.arange(vocab, device="cuda")
    t = s["temperature"].double().unsqueeze(1)
    greedy = t <= 0
    w = ((x.double() - x[:, :1].double()) / torch.where(greedy, 1.0, t)).exp()
    w = torch.where(greedy & (rank > 0), 0.0, w)
    if s["top_k"] is not None:
        k = s["top_k"].unsqueeze(1)
        w = torch.where((k <= 0) | (rank < k), w, 0.0)
    c = w.cumsum(1)
    kept = w > 0
    if s["top_p"] is not None:
        kept &= (c - w < s["top_p"].double().unsqueeze(1) * c[:, -1:]) | (s["top_p"].unsqueeze(1) >= 1) | (rank == 0)
    if s["min_p"] is not None:
        kept &= (w >= s["min_p"].double().unsqueeze(1)) | (rank == 0)
    w = torch.where(kept, w, 0.0)
    c = w.cumsum(1)
    n = kept.sum(1, keepdim=True)
    at = torch.minimum((c <= u.double().unsqueeze(1) * c[:, -1:]).sum(1, keepdim=True), n - 1).clamp(min=0)
    token = torch.where(x[:, :1] == -math.inf, -1, index.gather(1, at))  # no token allowed: -1, and no probability
    return {"token": token[:, 0].int(), "prob": (w.gather(1, at) / c[:, -1:])[:, 0].float()}


# ------------------------------------------------------------------------------------------------ in 64 bits
def _as_read(x, kv):
    """What fp16 rows read back as once stored, from the format's definition, in 64 bits (unrounded)."""
    x = x.double()
    if kv == "fp16":
        return x
    if kv == "int8":
        s = (x.abs().amax(-1, keepdim=True) / 127).half().double()
        return torch.nan_to_num(x / s, nan=0.0, posinf=0.0, neginf=0.0).round().clamp(-127, 127) * s
    g = x.reshape(x.shape[:-1] + (x.shape[-1] // 32, 32))
    m = g.amin(-1, keepdim=True)
    s = ((g.amax(-1, keepdim=True) - m) / 15).half().double()
    return (torch.nan_to_num((g - m) / s, nan=0.0, posinf=0.0, neginf=0.0).round().clamp(0, 15) * s + m).reshape(x.shape)


def exact(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    op = case["op"]
    if op == "sample":
        return _exact_sample(_prepare_sample(case, gen))
    kv, h, d, hq = case["kv"], case["kv_heads"], case["dim"], case["heads"]
    if op == "read":
        k, v = _keys_values(gen, case, case["layers"], case["first"] + case["tokens"])
        return {"k": _as_read(k[:, case["first"]:], kv), "v": _as_read(v[:, case["first"]:], kv)}
    sizes = _sizes(case)
    rows = sum(n for _, n in sizes)
    q, (k, v) = _normal(gen, rows, hq, d), _keys_values(gen, case, rows)
    if op == "store":
        return {"k": _as_read(k, kv), "v": _as_read(v, kv)}
    out = torch.empty((rows, hq, d), dtype=torch.float64, device="cuda")
    at = 0
    for prior, new in sizes:
        pk, pv = _keys_values(gen, case, prior)
        # attention is over what the cache reads back as: fp16
        fk = _as_read(torch.cat((pk, k[at:at + new])), kv).half().double()
        fv = _as_read(torch.cat((pv, v[at:at + new])), kv).half().double()
        col = torch.arange(prior + new, device="cuda")
        for t0 in range(0, new, 512):
            t1 = min(new, t0 + 512)
            pos = torch.arange(prior + t0, prior + t1, device="cuda").unsqueeze(1)
            hidden = (col > pos) | ((pos - col >= case["window"]) if case["window"] else col < 0)
            for head in range(hq):
                z = q[at + t0:at + t1, head].double() @ fk[:, head * h // hq].T / math.sqrt(d)
                z[hidden] = -math.inf
                out[at + t0:at + t1, head] = (z - z.logsumexp(1, keepdim=True)).exp() @ fv[:, head * h // hq]
        at += new
    return out


def _exact_sample(s):
    """Row by row: the sorted tokens, the three cuts as lengths of their prefix, and the place of u in what is left."""
    x = s["logits"].double()
    rows, vocab = x.shape
    if s["allowed"] is not None:
        word = s["allowed"].long()
        x[((word.repeat_interleave(32, 1)[:, :vocab] >> (torch.arange(vocab, device="cuda") % 32)) & 1) == 0] = -math.inf
    tokens, probs = [], []
    given = {m: None if s[m] is None else s[m].tolist() for m in ("uniform", "temperature", "top_k", "top_p", "min_p")}
    for r in range(rows):
        order = torch.sort(x[r], descending=True, stable=True)[1]
        order = order[x[r][order] > -math.inf]
        t = given["temperature"][r]
        if not len(order):
            tokens.append(-1)
            probs.append(math.nan)
            continue
        if t <= 0:
            tokens.append(int(order[0]))
            probs.append(1.0)
            continue
        z = x[r][order] / t
        if given["top_k"] is not None and given["top_k"][r] > 0:
            z = z[:given["top_k"][r]]
        share = (z - z.logsumexp(0)).exp()
        n = len(share)
        if given["top_p"] is not None and given["top_p"][r] < 1:
            n = min(n, int((share.cumsum(0) < given["top_p"][r]).sum()) + 1)
        if given["min_p"] is not None:
            n = min(n, max(1, int((share >= given["min_p"][r] * share[0]).sum())))
        c = share[:n].cumsum(0)
        i = min(int((c <= given["uniform"][r] * c[-1]).sum()), n - 1)
        tokens.append(int(order[i]))
        probs.append(float(share[i] / c[-1]))
    return {"token": torch.tensor(tokens, dtype=torch.int32, device="cuda"),
            "prob": torch.tensor(probs, dtype=torch.float64, device="cuda")}

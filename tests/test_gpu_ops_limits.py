"""The pieces of a decoding loop at the edges of what they accept."""
import math

import numpy as np
import pytest
import torch

import quantized_decode_step_gb300 as mag
from tests.test_gpu_ops import (ALL_KV, KV_NAMES, as_stored, check, extreme_rows, half, make, reference, rows_of,
                                sample_case)

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    mag.build()
    assert torch.cuda.is_available()
    torch.cuda.init()


# ------------------------------------------------------------------------------------------------ after a failure
def test_calls_after_a_refused_allocation():
    """A context whose pool no device holds is refused (4 TB: the allocation fails at once and takes nothing). The calls of
    another context, and sampling, go on as if it had not been asked for."""
    ctx = make(mag.KV_FP16, 4, 2, 128, pool_blocks=200, max_context=3000)
    rng = np.random.default_rng(1)
    sid = ctx.session_open()
    k, v, q = (half(rng, 2100, h, 128) for h in (2, 2, 4))
    ctx.session_extend([sid], [2100])

    class Large:
        n_layers, hidden, n_heads, n_kv_heads, head_dim = 64, 256, 4, 4, 128
        ffn, vocab, rms_eps, rope_base = 256, 0, 1e-5, 10000.0

    def refused():
        with pytest.raises(mag.MagError) as e:
            mag.Context(mag.make_config(Large, kv_dtype=mag.KV_FP16, pool_blocks=1 << 21, max_sessions=1, max_batch=1,
                                        max_context=64), 1)
        assert e.value.status == mag.ERR_OOM

    refused()
    ctx.kv_write(0, [sid], [2100], k.cuda(), v.cuda())
    back = torch.empty((2, 2100, 2, 128), dtype=torch.float16, device="cuda")
    refused()
    ctx.kv_read(0, [sid], [2100], back[0], back[1])
    ctx.sync()
    assert torch.equal(back[0].cpu(), k) and torch.equal(back[1].cpu(), v)
    for new in (1, 30, 200):  # a kernel each, their keys cut into several blocks' parts
        out = torch.full((new, 4, 128), math.nan, dtype=torch.float16, device="cuda")
        refused()
        ctx.attend(0, [sid], [new], q[:new].cuda(), out)
        ctx.sync()
        check(out, *reference(q[:new], k, v, 2100 - new, 0, 128 ** -0.5), 2)
    for rows in (1, 30):
        refused()
        sample_case((rng.standard_normal((rows, 3000)) * 2.5).astype(np.float16), p=0.9, seed=rows)
    src = torch.randn((64, 256), device="cuda")
    codes, sm = torch.zeros(64 * 128, dtype=torch.uint8, device="cuda"), torch.zeros(64 * 8 * 4, dtype=torch.uint8, device="cuda")
    refused()
    mag.quantize_w4g32(src, 64, 256, codes, sm)
    torch.cuda.synchronize()


# ------------------------------------------------------------------------------------------------ waits that run out
@pytest.mark.parametrize("kv", ALL_KV, ids=KV_NAMES.get)
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("new", [30, 200])
@pytest.mark.parametrize("polls", [0, 1, 3])
def test_attend_waits_give_up_then_context_recovers(kv, dim, new, polls):
    """Every wait between the roles of the kernels for more than 16 packed rows gives up at its first poll (as if what it waits
    for were stuck), or after one or three, where most waits end in time and some warps' do not: mag_sync says so, or
    the result is right. With the limit restored the same call gives the bits that it gave before. The kernel for
    fewer rows has no waits and works throughout."""
    rng = np.random.default_rng(new)
    n = 9000 + new
    ctx = make(kv, 16, 8, dim, pool_blocks=n // 16 + 2, max_context=n)
    sid = ctx.session_open()
    k, v = half(rng, 1, n, 8, dim), half(rng, 1, n, 8, dim)
    ctx.kv_append(sid, n, k.cuda(), v.cuda())
    q = half(rng, new, 16, dim).cuda()
    want, few = torch.empty_like(q), torch.empty_like(q[:1])
    ctx.attend(0, [sid], [new], q, want)
    ctx.attend(0, [sid], [1], q, few)
    ctx.sync()
    ctx.set_wait_limit(polls)
    for _ in range(3):
        out = torch.empty_like(q)
        ctx.attend(0, [sid], [new], q, out)
        if polls:
            try:
                ctx.sync()
                assert torch.equal(out, want)
            except mag.MagError as e:
                assert e.status == mag.ERR_TIMEOUT and "gave up" in str(e)
        else:
            with pytest.raises(mag.MagError) as e:
                ctx.sync()
            assert e.value.status == mag.ERR_TIMEOUT and "gave up" in str(e.value)
        ctx.sync()  # the error word was read and cleared
        one = torch.empty_like(few)
        ctx.attend(0, [sid], [1], q, one)
        ctx.sync()
        assert torch.equal(one, few)
    ctx.set_wait_limit(-1)
    for _ in range(2):
        out = torch.empty_like(q)
        ctx.attend(0, [sid], [new], q, out)
        ctx.sync()
        assert torch.equal(out, want)


@pytest.mark.parametrize("polls", [0, 1, 3])
def test_chunk_waits_give_up_then_context_recovers(polls):
    """The same of the prefill GEMM's roles: a chunk times out or gives the bits that it gave before, and gives them
    again with the limit restored."""
    import synth
    from synth import driver
    from synth.workloads import TINY, Workload
    wl = Workload("tiny-wait", TINY, mag.KV_FP16, 1, (128,), chunk=64)
    ctx, sids = driver.setup(wl, 3, extra_tokens=60)
    sid, p = sids[0], wl.prior[0]
    x = torch.from_numpy(synth.hidden_f16(3, 48, TINY.hidden, tag="chunk")).cuda()

    def chunk():
        out = torch.empty(TINY.hidden, dtype=torch.float16, device="cuda")
        ctx.session_truncate(sid, p)
        ctx.prefill_chunk(sid, 48, x, out)
        ctx.sync()
        return out

    want = chunk()
    ctx.set_wait_limit(polls)
    for _ in range(5):
        try:
            got = chunk()
            assert polls and torch.equal(got, want)
        except mag.MagError as e:
            assert e.status == mag.ERR_TIMEOUT
    ctx.set_wait_limit(-1)
    assert torch.equal(chunk(), want) and torch.equal(chunk(), want)


# ------------------------------------------------------------------------------------------------ scores far from zero
@pytest.mark.parametrize("kv", ALL_KV, ids=KV_NAMES.get)
@pytest.mark.parametrize("scale", [128 ** -0.5, 1.0, -1.0], ids=["default", "one", "minus"])
@pytest.mark.parametrize("prior,new", [(700, 2), (700, 30), (2500, 2), (2500, 30), (300, 200), (2500, 150)])
def test_attend_scores_far_from_zero(kv, scale, prior, new):
    """Scores of up to 2^37 that lie 2^20 and more apart, or are equal: a token's output is the mean of the values whose score is
    its largest, to the rounding of the output and, of a mean of n, of weights 1 / n in fp16."""
    rng = np.random.default_rng(prior + new)
    n = prior + new
    # constant key vectors: exact in an INT4 pool, and multiples of the same stored scale in an INT8 one
    level = torch.from_numpy((rng.integers(-200, 201, n) * 128).astype(np.float16))
    k = level.view(n, 1, 1).expand(n, 2, 128).contiguous()
    v, q = half(rng, n, 2, 128), torch.full((new, 4, 128), 2.0 ** 15, dtype=torch.float16)
    q[1::2] = -2.0 ** 15
    ctx = make(kv, 4, 2, 128, pool_blocks=n // 16 + 2, max_context=n)
    sid = ctx.session_open()
    ctx.session_extend([sid], [n])
    ctx.kv_write(0, [sid], [n], k.cuda(), v.cuda())
    out = torch.empty((new, 4, 128), dtype=torch.float16, device="cuda")
    ctx.attend(0, [sid], [new], q.cuda(), out, scale=scale)
    ctx.sync()
    check(out, *reference(q, as_stored(k, kv), as_stored(v, kv), prior, 0, scale), 2)


@pytest.mark.parametrize("shift", range(20, 36))
@pytest.mark.parametrize("new", [1, 20, 130])
def test_attend_rising_scores_of_any_size(new, shift):
    """Scores around 2^shift that rise by steps of fp32, so that they pass the running maximum by less than, about, and more
    than what they may: the output is a mean of its keys' values, 1 and 3."""
    n, dims = 1000 + new, 1 << max(0, shift - 30)
    a = min(15, shift // 2)
    k, q = torch.zeros((n, 1, 64), dtype=torch.float16), torch.zeros((new, 1, 64), dtype=torch.float16)
    k[..., :dims], q[..., :dims] = 2.0 ** a, 2.0 ** min(15, shift - a)
    k[:, 0, 63], q[..., 63] = (torch.arange(n) % 1024).half(), 2.0 ** (shift - 23)
    v = torch.ones((n, 1, 64), dtype=torch.float16)
    v[::2] = 3.0
    ctx = make(mag.KV_FP16, 1, 1, 64, pool_blocks=n // 16 + 2, max_context=n)
    sid = ctx.session_open()
    ctx.session_extend([sid], [n])
    ctx.kv_write(0, [sid], [n], k.cuda(), v.cuda())
    out = torch.empty((new, 1, 64), dtype=torch.float16, device="cuda")
    ctx.attend(0, [sid], [new], q.cuda(), out, scale=1.0)
    ctx.sync()
    # half a step of fp16 at 3 is 2^-10; the weights' roundings move a mean of 1 and 3 no further than they differ
    assert torch.isfinite(out).all() and (out >= 1 - 2.0 ** -10).all() and (out <= 3 + 2.0 ** -8).all(), out.unique()


@pytest.mark.parametrize("new", [1, 20, 130])
def test_attend_scores_that_pass_the_maximum_by_just_what_they_may(new):
    """Around 2^26, where steps of fp32 are as large as what a score may pass the running maximum by before it is raised: two
    scores one step apart, in turn along the keys, from eight starts (the scaled step is 8 or 16)."""
    n = 100000 + new
    k, q = torch.zeros((n, 1, 64), dtype=torch.float16), torch.zeros((new, 1, 64), dtype=torch.float16)
    k[..., 0], q[..., 0] = 2.0 ** 11, 2.0 ** 15
    k[:, 0, 1], q[..., 1] = ((torch.arange(n) // 256) % 2).half(), 8.0
    k[..., 2] = 1.0
    v = torch.ones((n, 1, 64), dtype=torch.float16)
    v[::2] = 3.0
    ctx = make(mag.KV_FP16, 1, 1, 64, pool_blocks=n // 16 + 2, max_context=n)
    sid = ctx.session_open()
    ctx.session_extend([sid], [n])
    ctx.kv_write(0, [sid], [n], k.cuda(), v.cuda())
    for start in range(8):
        q[..., 2] = 8.0 * start
        out = torch.empty((new, 1, 64), dtype=torch.float16, device="cuda")
        ctx.attend(0, [sid], [new], q.cuda(), out, scale=1.0)
        ctx.sync()
        assert torch.isfinite(out).all() and (out >= 1 - 2.0 ** -10).all() and (out <= 3 + 2.0 ** -8).all(), start


# ------------------------------------------------------------------------------------------------ small probabilities
@pytest.mark.parametrize("dtype", [np.float16, np.float32])
@pytest.mark.parametrize("rows,vocab", [(1, 50), (3, 20000), (30, 300), (30, 40000), (160, 300)])
@pytest.mark.parametrize("k", [0, 5, 2000])
def test_sample_probability_of_an_unlikely_token(dtype, rows, vocab, k):
    """Four tokens down to 2^-38 of the largest one's weight, the last of them drawn (u = 1): its probability is good to
    2^-24, the rounding of the quotient, and what the weights are good to, 2^-28, of itself."""
    rng = np.random.default_rng(vocab)
    x = np.full((rows, vocab), -np.inf, dtype)
    far = rng.uniform(10.0, 26.0, rows).astype(dtype)
    for r in range(rows):
        at = rng.permutation(vocab)[:4]
        x[r, at] = np.array([0.0, -1.5, -4.25, -far[r]], dtype)
    token = torch.full((rows,), -7, dtype=torch.int32, device="cuda")
    prob = torch.empty(rows, dtype=torch.float32, device="cuda")
    mag.sample(torch.from_numpy(x).cuda(), rows, vocab, torch.ones(rows, device="cuda"), token, prob=prob,
               dtype=mag.LOGITS_F16 if dtype == np.float16 else mag.LOGITS_F32,
               top_k=torch.full((rows,), k, dtype=torch.int32, device="cuda") if k else None)
    torch.cuda.synchronize()
    w = np.exp(np.where(np.isfinite(x), x, -np.inf).astype(np.float64))
    for r, (t, p) in enumerate(zip(token.cpu().tolist(), prob.cpu().tolist())):
        assert x[r, t] == -far[r]
        assert abs(p / (w[r, t] / w[r].sum()) - 1) <= 2.0 ** -24 + 2.0 ** -28, (r, p, w[r, t] / w[r].sum())


# ------------------------------------------------------------------------------------------------ the sum of the weights
@pytest.mark.parametrize("kv", ALL_KV, ids=KV_NAMES.get)
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("new", [1, 30, 200, 300])
def test_attend_equal_values_come_back(kv, dim, new):
    """Every value 1: the output is 1 whatever the weights, if their sum adds what the products take, which it does up to 128
    packed rows. One key in 16 has the largest weight, the others half of it times 1 + 0.95 2^-11, which fp16 rounds
    down by almost half a step; the sum of the weights before that rounding, by which longer chunks divide, is 0.84 2^-11
    larger, and the output then the number below 1, or 1."""
    n = 1500 + new
    k, v = torch.ones((n, 1, dim), dtype=torch.float16), torch.ones((n, 1, dim), dtype=torch.float16)
    k[::16] = 0
    one = float(as_stored(v, kv)[0, 0, 0])
    want = math.log(0.5 * (1 + 0.95 * 2.0 ** -11)) / one
    q = torch.zeros((new, 2, dim), dtype=torch.float16)
    q[..., 0] = want
    q[..., 1] = want - float(np.float16(want))  # the two together: want to 2^-25
    ctx = make(kv, 2, 1, dim, pool_blocks=n // 16 + 2, max_context=n)
    sid = ctx.session_open()
    ctx.session_extend([sid], [n])
    ctx.kv_write(0, [sid], [n], k.cuda(), v.cuda())
    out = torch.empty((new, 2, dim), dtype=torch.float16, device="cuda")
    ctx.attend(0, [sid], [new], q.cuda(), out, scale=1.0)
    ctx.sync()
    if 2 * new <= 128:
        assert (out.cpu() == one).all(), out.unique()
    else:  # and half a step for the output's own rounding
        assert ((out.cpu().double() - one).abs() <= one * 2.0 ** -10).all(), out.unique()


@pytest.mark.parametrize("kv", ALL_KV, ids=KV_NAMES.get)
@pytest.mark.parametrize("dim,group,new", [(64, 1, 17), (128, 4, 5), (64, 8, 16), (128, 2, 60), (128, 1, 128)])
@pytest.mark.parametrize("prior", [40, 2300])
def test_attend_up_to_128_rows_to_the_weights_rounding(kv, dim, group, new, prior):
    """Sums of the rounded weights: with weights w_j (1 + e_j), |e_j| <= 2^-11, in both the products and the sum, o moves by at most
    2^-11 sum_j w_j |v_j - o|, and its own rounding adds 2^-11 |o|; a tenth of that for fp32's part, and half of fp16's smallest
    step twice."""
    rng = np.random.default_rng(prior + new)
    n = prior + new
    k, v, q = half(rng, n, 2, dim), half(rng, n, 2, dim), half(rng, new, 2 * group, dim)
    v[..., ::3] += 4.0  # an o that is large next to what the values differ by
    ctx = make(kv, 2 * group, 2, dim, pool_blocks=n // 16 + 2, max_context=n)
    sid = ctx.session_open()
    ctx.session_extend([sid], [n])
    ctx.kv_write(0, [sid], [n], k.cuda(), v.cuda())
    out = torch.empty((new, 2 * group, dim), dtype=torch.float16, device="cuda")
    ctx.attend(0, [sid], [new], q.cuda(), out)
    ctx.sync()
    o, spread = reference(q, as_stored(k, kv), as_stored(v, kv), prior, 0, dim ** -0.5)
    tol = 1.1 * 2.0 ** -11 * (o.abs() + spread) + 2.0 ** -24
    assert ((out.double().cpu() - o).abs() <= tol).all()


def test_attend_refuses_a_scale_whose_base_2_form_overflows():
    """Scores are taken in powers of two: a finite scale of which log2(e) times is not gave NaN."""
    ctx = make(mag.KV_FP16, 4, 2, 64)
    sid = ctx.session_open()
    ctx.session_extend([sid], [20])
    k, q = torch.zeros((20, 2, 64), device="cuda").half(), torch.zeros((20, 4, 64), device="cuda").half()
    ctx.kv_write(0, [sid], [20], k, k + 1)
    out = torch.zeros_like(q)
    for scale in (2.5e38, -3.4e38):
        with pytest.raises(mag.MagError) as e:
            ctx.attend(0, [sid], [20], q, out, scale=scale)
        assert e.value.status == mag.ERR_INVALID_ARG
    for new in (1, 20):
        ctx.attend(0, [sid], [new], q, out[:new], scale=2.3e38)
        ctx.sync()
        assert (out[:new] == 1).all()


# ------------------------------------------------------------------------------------------------ sizes between the other tests'
@pytest.mark.parametrize("kv", ALL_KV, ids=KV_NAMES.get)
@pytest.mark.parametrize("kv_heads,dim", [(1, 64), (3, 128), (8, 128)])
@pytest.mark.parametrize("lens,new", [((300, 1, 258, 2, 7, 900), (299, 1, 5, 2, 3, 721)), ((517,), (513,)),
                                      ((130, 131, 129, 133), (130, 129, 127, 128))])
def test_write_of_many_rows_of_several_sessions(kv, kv_heads, dim, lens, new):
    """More than 512 rows, where a block of the kernel takes four neighbouring rows, of two sessions or the last ones: what is
    read back equals the oracle's quantisers', older tokens stay."""
    rng = np.random.default_rng(sum(new))
    ctx = make(kv, kv_heads, kv_heads, dim, pool_blocks=sum(-(-n // 16) for n in lens) + 1, sessions=len(lens),
               max_context=max(lens))
    sids, ks, vs = [ctx.session_open() for _ in lens], [], []
    for sid, n in zip(sids, lens):
        k, v = half(rng, n, kv_heads, dim, std=2), half(rng, n, kv_heads, dim)
        ctx.kv_append(sid, n, k.cuda(), v.cuda())
        ctx.sync()
        ks.append(k)
        vs.append(v)
    rows, width = sum(new), kv_heads * dim
    nk, nv = half(rng, rows, kv_heads, dim), half(rng, rows, kv_heads, dim, std=3)
    wide = torch.zeros((2, rows, width + 8), dtype=torch.float16, device="cuda")
    wide[0, :, :width], wide[1, :, :width] = nk.view(rows, -1).cuda(), nv.view(rows, -1).cuda()
    ctx.kv_write(0, sids, new, wide[0], wide[1], ld=width + 8)
    at = 0
    for sid, n, m, k, v in zip(sids, lens, new, ks, vs):
        out = torch.empty((2, n, kv_heads, dim), dtype=torch.float16, device="cuda")
        ctx.kv_read(0, [sid], [n], out[0], out[1])
        ctx.sync()
        for got, old, fresh in ((out[0], k, nk), (out[1], v, nv)):
            assert torch.equal(got.cpu(), as_stored(torch.cat((old[:n - m], fresh[at:at + m])), kv))
        at += m


@pytest.mark.parametrize("dtype,rows,vocab", [(np.float32, 152, 128256), (np.float32, 153, 131071), (np.float32, 160, 131072),
                                              (np.float16, 153, 131071), (np.float16, 20, 131072), (np.float16, 2, 540672),
                                              (np.float32, 2, 270336), (np.float32, 9, 131072)])
def test_sample_largest_rows(dtype, rows, vocab):
    """Rows of a real vocabulary in the kernels for many rows, next to the border between kernels, and the largest that are
    taken: whole distributions, equal logits (the largest sums), and cuts."""
    rng = np.random.default_rng(vocab)
    x = rows_of(rng, rows, vocab, dtype)
    x[1::3] = dtype(0.5)
    x[2::3] *= dtype(0.01)
    sample_case(x, t=1.5, seed=1)
    sample_case(x, t=0.7, p=0.95, seed=2)
    sample_case(x, t=rng.uniform(0.3, 2, rows), k=rng.integers(0, vocab + 2, rows), p=rng.uniform(0, 1.1, rows),
                m=rng.uniform(-0.1, 0.5, rows), seed=3)


def test_sample_bins_as_wide_as_their_adds_allow():
    """131,071 equal fp32 logits just below the largest, many rows: one bin takes all their weights, whose limbs of 15 bits are
    nearly full."""
    x = np.full((152, 131071), np.float32(-2.0 ** -20), np.float32)
    x[:, 100] = 0.0
    u = (np.arange(152) + 0.5) / 152
    sample_case(x, u=u)
    sample_case(x, p=0.5, u=u)
    sample_case(x, k=131070, u=u)


# ------------------------------------------------------------------------------------------------ rows that are counted by value
COUNTED = [(39, 40001), (45, 65536), (160, 50021), (40, 131071)]  # fp16, many long rows
EITHER = [(38, 131071), (160, 40000)]                             # their neighbours, which are not


@pytest.mark.parametrize("rows,vocab", COUNTED + EITHER)
def test_sample_counted_cuts(rows, vocab):
    rng = np.random.default_rng(rows + vocab)
    x = rows_of(rng, rows, vocab, np.float16)
    sample_case(x, seed=1)
    sample_case(x, t=0.9, k=5, seed=3)
    sample_case(x, t=1.3, p=0.8, seed=4)
    sample_case(x, m=0.05, seed=5)
    sample_case(x, t=rng.uniform(0.3, 2, rows), k=rng.integers(0, vocab + 2, rows), p=rng.uniform(0, 1.1, rows),
                m=rng.uniform(-0.1, 0.5, rows), seed=6)
    sample_case(x, t=rng.uniform(0.3, 2, rows), k=rng.integers(400, 1100, rows), p=rng.uniform(0.5, 1.1, rows), seed=7)


@pytest.mark.parametrize("rows,vocab", COUNTED)
def test_sample_counted_crowds_and_ties(rows, vocab):
    """Equal and nearly equal logits: cuts and draws inside them, by index."""
    rng = np.random.default_rng(vocab)
    flat = np.full((rows, vocab), 1.5, np.float16)
    steps = (rng.integers(0, 4, (rows, vocab)) * 0.5).astype(np.float16)
    peak = steps.copy()
    peak[:, vocab // 3] = 9.0
    for x in (flat, steps, peak):
        sample_case(x, seed=1)
        sample_case(x, k=vocab // 2, seed=2)
        sample_case(x, t=2.0, p=0.3, m=0.4, seed=4)
        sample_case(x, t=0.05, k=3000, m=0.9, seed=6)


def test_sample_counted_more_equal_tokens_than_16_bits():
    """Counts past 65,535, of even and odd patterns, at the top and below it: such a row is not counted."""
    rng = np.random.default_rng(5)
    x = rows_of(rng, 40, 131000, np.float16)
    for r in range(40):
        few = rng.permutation(131000)[:65536 + 1500 * r]
        x[r, few] = np.array([0x3C00 + r % 2], np.uint16).view(np.float16)[0] * (1 if r % 3 else -1)
    x[::5, 77] = 14.0
    sample_case(x, t=0.8, seed=1)
    sample_case(x, t=1.2, k=rng.integers(0, 131000, 40), p=rng.uniform(0.1, 1.1, 40), m=rng.uniform(-0.1, 0.2, 40), seed=2)


def test_sample_counted_strides_and_masks():
    rng = np.random.default_rng(9)
    for ld in (41001, 41008, 41024):
        x = rows_of(rng, 42, 41001, np.float16)
        allowed = rng.random((42, 41001)) < np.tile(np.array([[1.0], [0.5], [0.01], [0.0], [0.9], [0.002]]), (7, 1))
        allowed[4, np.argsort(-x[4].astype(np.float64))[:5]] = False
        sample_case(x, t=0.8, k=[0, 3, 0, 4, 10, 0] * 7, p=0.9, allowed=allowed, ld=ld, seed=ld)
        sample_case(x, t=0.8, m=[0, 0.1, 0, 0.9, 1e-3, 0] * 7, allowed=allowed, ld=ld, seed=ld)


def test_sample_counted_extremes():
    rng = np.random.default_rng(12)
    x = rows_of(rng, 45, 40100, np.float16)
    for at in range(0, 45, 9):
        extreme_rows(x[at:at + 9], np.float16)
    got, _ = sample_case(x, seed=3)
    assert got[0] == got[1] == -1 and got[2] in (5, 17, 200)
    for t in (0.0, float("nan"), 1e-30, 1e-6, 1e6, 1e30):
        sample_case(x, t=t, seed=4)
    for p in (0.0, 1e-9, 5.0):
        sample_case(x, p=p, seed=5)
    for m in (2.0, 1.0, 0.999, 1e-9):
        sample_case(x, m=m, seed=6)
    sample_case(x, k=2 ** 31 - 1, seed=8)
    sample_case(x, k=1500, m=0.5, seed=9)
    token, n = torch.full((45,), -7, dtype=torch.int32, device="cuda"), 40100
    u = torch.tensor([math.nan, -1.0, 1.0, 2.0, math.inf] * 9, device="cuda")
    mag.sample(torch.from_numpy(x).cuda(), 45, n, u, token, top_k=torch.full((45,), 1200, dtype=torch.int32, device="cuda"))
    for r, t in enumerate(token.cpu().tolist()):
        ok = np.flatnonzero(x[r] > -np.inf)
        assert (t == -1) if len(ok) == 0 else t in ok[np.argsort(-x[r][ok].astype(np.float64), kind="stable")[:1200]]

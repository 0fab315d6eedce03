"""The pieces of a decoding loop at the edges of what they accept."""
import math

import numpy as np
import pytest
import torch

import quantized_decode_step_gb300 as mag
from tests.test_gpu_ops import ALL_KV, KV_NAMES, check, half, make, reference, sample_case

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

"""The pieces of a decoding loop at the edges of what they accept."""
import math

import numpy as np
import pytest
import torch

import quantized_decode_step_gb300 as mag
from tests.test_gpu_ops import check, half, make, reference, sample_case

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

"""Refusals of the stateless sampler and of null contexts, which need no GPU."""
import ctypes

import pytest

import quantized_decode_step_gb300 as mag


@pytest.fixture(scope="module")
def lib():
    mag.build()
    return mag.lib()


def test_sample_refusals(lib):
    p = mag.SampleParams()
    x = 4096  # an address that is never followed

    def call(logits=x, dtype=mag.LOGITS_F16, rows=1, vocab=16, ld=16, uniform=x, token=x):
        return lib.mag_sample(logits, dtype, rows, vocab, ld, ctypes.byref(p), uniform, token, None, None)

    assert call(rows=0) == mag.OK
    assert call(rows=0, logits=None, uniform=None, token=None) == mag.OK
    for bad in (dict(rows=-1), dict(vocab=0), dict(vocab=-1), dict(ld=15), dict(dtype=2), dict(dtype=-1),
                dict(logits=None), dict(uniform=None), dict(token=None), dict(logits=x + 1),
                dict(logits=x + 2, dtype=mag.LOGITS_F32)):
        assert call(**bad) == mag.ERR_INVALID_ARG, bad
    assert call(vocab=540673, ld=540673) == mag.ERR_UNSUPPORTED
    assert call(vocab=270337, ld=270337, dtype=mag.LOGITS_F32) == mag.ERR_UNSUPPORTED
    assert call(rows=0, vocab=540672, ld=540672) == mag.OK


def test_null_context(lib):
    one = (ctypes.c_int32 * 1)(0)
    assert lib.mag_session_extend(None, 1, one, one) == mag.ERR_INVALID_ARG
    assert lib.mag_kv_write(None, 0, 1, one, one, None, None, 0) == mag.ERR_INVALID_ARG
    assert lib.mag_kv_read(None, 0, 1, one, one, None, None, 0) == mag.ERR_INVALID_ARG
    assert lib.mag_kv_export(None, 0, 0, 1, None, None) == mag.ERR_INVALID_ARG
    assert lib.mag_attend(None, 0, 1, one, one, None, 0, None, 0, 0, 1.0) == mag.ERR_INVALID_ARG


def test_lists_of_unlike_length():
    with pytest.raises(ValueError):
        mag._Lists([1, 2], [3])
    a = mag._Lists([5, 6], [7, 8])
    assert a.n == 2 and list((ctypes.c_int32 * 4).from_address(a.ids)) == [5, 6, 7, 8] and a.counts == a.ids + 8


def test_sample_refuses_misaligned_arrays(lib):
    x = 4096
    for name in ("uniform", "token", "prob", "temperature", "top_k", "top_p", "min_p", "allowed"):
        at = dict(uniform=x, token=x, prob=x)
        p = mag.SampleParams()
        if name in at:
            at[name] = x + 2
        else:
            setattr(p, name, x + 2)
        assert lib.mag_sample(x, mag.LOGITS_F16, 1, 16, 16, ctypes.byref(p), at["uniform"], at["token"], at["prob"],
                              None) == mag.ERR_INVALID_ARG, name

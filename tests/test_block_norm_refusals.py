"""What moe_block_norm and moe_reduce_norm refuse, on the host and before any
launch (addresses here are never dereferenced)."""
import ctypes

import pytest

from mixture_experts_routed_moe_amd import _lib

A = 1 << 20          # a 16-byte aligned address
F16, BF16, F32, FP8 = 0, 1, 2, 3
NULL, SHAPE, DTYPE, UNSUPPORTED = 1, 2, 3, 4


def _norm(y=A, residual=A, gamma_post=A, gate=None, kind=0, alpha=1.0, gamma_pre=A, eps=1e-6, T=4,
          H=256, dtype=BF16, res_dtype=BF16, residual_out=A, h=A, quant=0, codes=None, scales=None,
          reduce=None):
    args = [residual, gamma_post, gate, kind, alpha, gamma_pre, eps, T, H, dtype, res_dtype,
            residual_out, h, quant, codes, scales, None]
    if reduce is None:
        return _lib.lib().moe_block_norm(y, *args)
    rows, pos, w, K = reduce
    return _lib.lib().moe_reduce_norm(y, rows, pos, w, K, *args)


@pytest.mark.parametrize("bad, status", [
    (dict(residual=None), NULL),
    (dict(y=None), NULL),                                  # gamma_post and residual_out without y
    (dict(y=None, gamma_post=None), NULL),
    (dict(y=None, gamma_post=None, residual_out=None, gate=A, kind=1), NULL),
    (dict(gate=A), NULL), (dict(kind=3), NULL),
    (dict(gamma_pre=None), NULL),                          # h without gamma_pre
    (dict(residual_out=None, h=None), NULL),
    (dict(quant=1), NULL), (dict(quant=1, codes=A), NULL), (dict(codes=A, scales=A), NULL),
    (dict(kind=4, gate=A), UNSUPPORTED), (dict(kind=-1, gate=A), UNSUPPORTED),
    (dict(quant=5, codes=A, scales=A), UNSUPPORTED),
    (dict(T=-1), SHAPE), (dict(H=0), SHAPE), (dict(H=16385), SHAPE), (dict(T=1 << 22), SHAPE),
    (dict(eps=0.0), SHAPE), (dict(eps=-1.0), SHAPE), (dict(eps=float("nan")), SHAPE),
    (dict(dtype=FP8, res_dtype=FP8), DTYPE), (dict(dtype=7), DTYPE),
    (dict(res_dtype=F16), DTYPE), (dict(dtype=F32, res_dtype=BF16), DTYPE),
    (dict(quant=3, codes=A, scales=A, H=24), SHAPE),       # a cut 32-block
    (dict(quant=4, codes=A + 8, scales=A), SHAPE),
    (dict(quant=4, codes=A, scales=A, residual=A + 2), SHAPE),
])
def test_block_norm_refuses(bad, status):
    assert _norm(**bad) == status
    assert _lib.lib().moe_last_error()


@pytest.mark.parametrize("bad, status", [
    (dict(reduce=(8, None, A, 2)), NULL), (dict(y=None, reduce=(8, A, A, 2)), NULL),
    (dict(reduce=(-1, A, A, 2)), SHAPE), (dict(reduce=(8, A, A, 0)), SHAPE),
    (dict(reduce=(8, A, A, 65)), SHAPE), (dict(reduce=(8, A, A, 2), H=320), SHAPE),
    (dict(reduce=(8, A, A, 2), residual=None), NULL), (dict(reduce=(8, A, A, 2), dtype=FP8), DTYPE),
])
def test_reduce_norm_refuses(bad, status):
    assert _norm(**bad) == status


def test_no_tokens_launch_nothing():
    assert _norm(T=0) == 0
    assert _norm(T=0, reduce=(0, A, None, 2)) == 0

"""The calls that run a quantized layer refuse what they do not take, before any device work; and
the helpers of their GPU tests against hand-written values."""
import ctypes

import numpy as np
import pytest
import torch

from tests.gpu_helpers import unpack_np
from tests.running_helpers import layer_np, norm_np, pack_np

INVALID, UNSUPPORTED, WORKSPACE = 1, 4, 7
P = ctypes.c_void_p(4096)


def _linear(x=P, xt=0, T=4, m=8, n=16, codes=P, scales=P, zeros=P, bits=4, group=0, perm=None, y=P,
            yt=0, ws=P, nws=1 << 40):
    from post_weight_quantization_22_b200 import gq as G
    return G.LIB.gq_linear(x, xt, T, m, n, codes, scales, zeros, bits, group, perm, y, yt, ws, nws,
                           None)


def _quantized(q=P, s=P, T=4, m=8, n=16, codes=P, scales=P, zeros=P, bits=4, group=0, perm=None,
               y=P, yt=0, ws=P, nws=1 << 40):
    from post_weight_quantization_22_b200 import gq as G
    return G.LIB.gq_linear_quantized(q, s, T, m, n, codes, scales, zeros, bits, group, perm, y, yt,
                                     ws, nws, None)


def _norm(x=P, r=None, xt=0, g=P, gt=0, T=4, n=16, eps=1e-6, sum=None, y=None, q=P, s=P):
    from post_weight_quantization_22_b200 import gq as G
    return G.LIB.gq_rmsnorm_quantize(x, r, xt, g, gt, T, n, eps, sum, y, q, s, None)


@pytest.mark.parametrize("kw", [
    dict(T=-1), dict(T=1 << 31), dict(m=0), dict(m=(1 << 24) + 1), dict(n=0), dict(n=32769),
    dict(bits=1), dict(bits=9), dict(group=-1), dict(group=7), dict(group=256), dict(x=None),
    dict(codes=None), dict(scales=None), dict(zeros=None), dict(y=None), dict(xt=2), dict(yt=2),
    dict(x=ctypes.c_void_p(4097)), dict(codes=ctypes.c_void_p(4098)),
    dict(scales=ctypes.c_void_p(4098)), dict(perm=ctypes.c_void_p(4098)),
    dict(xt=1, x=ctypes.c_void_p(4098)), dict(yt=1, y=ctypes.c_void_p(4098)),
])
def test_linear_rejects_bad_arguments(kw):
    assert _linear(**kw) == INVALID
    if not {"x", "xt"} & set(kw):
        assert _quantized(**kw) == INVALID


def test_linear_rejects_groups_the_quantizer_does_not_write():
    assert _linear(group=8) == UNSUPPORTED and _quantized(group=1) == UNSUPPORTED


def test_quantized_rows_need_their_scales():
    assert _quantized(s=None) == INVALID and _quantized(q=None) == INVALID


def test_no_tokens_is_no_work():
    assert _linear(T=0, x=None, y=None) == 0 and _quantized(T=0, q=None, s=None, y=None) == 0
    assert _norm(T=0, x=None, q=None, s=None) == 0


@pytest.mark.parametrize("kw", [
    dict(T=-1), dict(T=1 << 31), dict(n=0), dict(n=32769), dict(eps=-1e-9), dict(eps=float("nan")),
    dict(eps=float("inf")), dict(x=None), dict(g=None), dict(q=None), dict(s=None),
    dict(q=None, s=None), dict(xt=3), dict(gt=3), dict(sum=P, y=P), dict(x=ctypes.c_void_p(4097)),
    dict(r=ctypes.c_void_p(4097)), dict(xt=1, y=ctypes.c_void_p(4098)),
    dict(gt=1, g=ctypes.c_void_p(4098)), dict(s=ctypes.c_void_p(4098)),
])
def test_norm_rejects_bad_arguments(kw):
    assert _norm(**kw) == INVALID


@pytest.mark.parametrize("kw", [
    dict(m=0), dict(n=0), dict(n=32769), dict(bits=1), dict(bits=9), dict(codes=None),
    dict(perm=None), dict(out=None), dict(out=P), dict(perm=ctypes.c_void_p(4098)),
])
def test_order_codes_rejects_bad_arguments(kw):
    from post_weight_quantization_22_b200 import gq as G
    a = dict(codes=P, m=8, n=16, bits=4, perm=P, out=ctypes.c_void_p(8192))
    a.update(kw)
    assert G.LIB.gq_order_codes(a["codes"], a["m"], a["n"], a["bits"], a["perm"], a["out"],
                                None) == INVALID


def test_workspace_queries():
    from post_weight_quantization_22_b200 import gq as G
    assert G.gq_linear_workspace_size(1, 4096, 4096) == 0          # one token needs none
    assert G.gq_linear_workspace_size(-1, 8, 8) == 0
    assert G.gq_linear_workspace_size(8, 8, 32769) == 0
    assert G.gq_linear_workspace_size(1, 4096, 4096, torch.int8) == 0
    assert G.LIB.gq_linear_workspace_size(1, 8, 8, 5, 0) == 0
    assert G.LIB.gq_linear_workspace_size(1, 8, 8, 0, 2) == 0


def test_many_tokens_need_their_workspace():
    from post_weight_quantization_22_b200 import gq as G
    m = 4096
    need = G.gq_linear_workspace_size(64, m, 16, torch.float32)
    assert need >= 3 * 64 * 16 * 2                      # three bf16 parts of the tokens
    assert G.gq_linear_workspace_size(64, m, 16, torch.bfloat16) == 256
    assert G.gq_linear_workspace_size(64, m, 16, torch.bfloat16, ordered=True) > 256
    assert G.gq_linear_workspace_size(64, m, 17, torch.bfloat16) > 256
    assert G.gq_linear_workspace_size(48, 256, 16, torch.bfloat16) == 0  # few rows: none
    assert _linear(T=64, m=m, ws=None, nws=0) == WORKSPACE
    assert _linear(T=64, m=m, xt=1, nws=need - 1) == WORKSPACE
    assert _linear(T=64, m=m, ws=ctypes.c_void_p(4096 + 128)) == WORKSPACE
    assert _quantized(T=64, m=m, ws=None, nws=0) == WORKSPACE


def test_binding_refuses_cpu_tensors_and_wrong_shapes():
    from post_weight_quantization_22_b200 import gq as G
    x = torch.zeros(2, 16)
    with pytest.raises(ValueError):
        G.gq_linear(x, torch.zeros(4, 2, dtype=torch.int32), torch.ones(4, 1),
                    torch.zeros(4, 1, dtype=torch.uint8), 4)
    with pytest.raises(ValueError):
        G.gq_linear_quantized(x.to(torch.int8), torch.ones(2), torch.zeros(4, 2, dtype=torch.int32),
                              torch.ones(4, 1), torch.zeros(4, 1, dtype=torch.uint8), 4)
    with pytest.raises(ValueError):
        G.gq_rmsnorm_quantize(x, torch.ones(16))
    with pytest.raises(ValueError):
        G.gq_order_codes(torch.zeros(4, 2, dtype=torch.int32), 16, 4,
                         torch.arange(16, dtype=torch.int32))


def test_pack_helper_against_the_layout():
    # 3-bit codes 1, 6, 7, ..: bits 0-2, 3-5, 6-8 of the stream; code 10 spans two words
    codes = np.arange(22).reshape(2, 11) % 8
    p = pack_np(codes, 3)
    assert p.shape == (2, 2)
    assert p[0, 0] & 0x1FF == 0b010_001_000
    assert np.array_equal(unpack_np(p, 11, 3), codes)
    for bits in range(2, 9):
        c, s, z, w = layer_np(3, 45, bits, 16, bits)
        assert np.array_equal(unpack_np(pack_np(c, bits), 45, bits), c)
        assert w[1, 20] == float(s[1, 1]) * (int(c[1, 20]) - int(z[1, 1]))


def test_norm_helper_by_hand():
    x = np.array([[3.0, -4.0], [0.0, 0.0], [np.inf, 1.0]])
    h, v, q, s = norm_np(x, None, np.array([1.0, 2.0]), 0.0, torch.float32)
    rms = np.sqrt(12.5)
    assert np.allclose(v[0], [3 / rms, -8 / rms])
    assert q[0].tolist() == [48, -127]            # 127 * 3 / 8 = 47.6
    assert np.isclose(s[0], 8 / rms / 127)
    assert q[1].tolist() == [0, 0] and q[2].tolist() == [0, 0] and np.isnan(s[2])

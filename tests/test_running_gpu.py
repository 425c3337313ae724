"""The operators that run a quantized layer (packed products, norm with 8-bit rows) against plain
fp64 forms, at the sizes, groups, widths and values where they can go wrong."""
import numpy as np
import pytest
import torch

from tests.gpu_helpers import run_gpu
from tests.running_helpers import check_linear, layer_np, norm_np, to_cuda

pytestmark = pytest.mark.gpu

GROUPS = (0, 16, 32, 64, 128)
# (T, m, n): one of everything, partial words, tiles and units, one token to many
SIZES = ((1, 1, 1), (1, 33, 31), (2, 16, 32), (5, 17, 100), (8, 130, 257), (9, 48, 128),
         (16, 128, 1000), (31, 65, 129), (33, 250, 384), (64, 128, 512), (100, 300, 136),
         (129, 256, 1024), (260, 129, 640), (300, 257, 333))


def _x(T, n, dtype, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(T, n, generator=g, device="cuda")
    x[:, ::7] *= 10
    return x.to(dtype)


def _rows(T, n, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    q = torch.randint(-127, 128, (T, n), generator=g, device="cuda").to(torch.int8)
    return q, torch.rand(T, generator=g, device="cuda") + 0.01


def _guarded(T, m, dtype):
    """A T x m output with guard rows around it."""
    buf = torch.full((T + 2, m), 7.0, dtype=dtype, device="cuda")
    return buf, buf[1:T + 1]


def _whole(buf):
    assert bool((buf[0] == 7).all()) and bool((buf[-1] == 7).all())


@pytest.mark.parametrize("bits", range(2, 9))
@pytest.mark.parametrize("group", GROUPS)
def test_linear_matches_fp64(bits, group):
    from post_weight_quantization_22_b200 import gq as G
    for i, (T, m, n) in enumerate(SIZES):
        c, s, z, w = layer_np(m, n, bits, group, 100 * bits + i, extreme=i % 3 == 2)
        dev = to_cuda(c, s, z, bits)
        for dtype, out in ((torch.bfloat16, torch.bfloat16), (torch.float32, torch.float32),
                           (torch.bfloat16, torch.float32)):
            x = _x(T, n, dtype, i)
            buf, y = _guarded(T, m, out)
            G.gq_linear(x, *dev, bits, group, y=y)
            check_linear(y, x.double().cpu().numpy(), w)
            _whole(buf)


@pytest.mark.parametrize("bits", range(2, 9))
@pytest.mark.parametrize("group", GROUPS)
def test_linear_quantized_matches_fp64(bits, group):
    from post_weight_quantization_22_b200 import gq as G
    for i, (T, m, n) in enumerate(SIZES):
        c, s, z, w = layer_np(m, n, bits, group, 200 * bits + i, extreme=i % 3 == 2)
        dev = to_cuda(c, s, z, bits)
        q, qs = _rows(T, n, i)
        for out in (torch.float32, torch.bfloat16):
            buf, y = _guarded(T, m, out)
            G.gq_linear_quantized(q, qs, *dev, bits, group, y=y)
            check_linear(y, q.double().cpu().numpy(), w, qs.double().cpu().numpy())
            _whole(buf)


@pytest.mark.parametrize("T", (1, 40, 200))
@pytest.mark.parametrize("dtype", (torch.bfloat16, torch.float32, torch.int8))
def test_long_rows_and_many_rows(T, dtype):
    """The widest layer (n = 32768) and one with many rows."""
    from post_weight_quantization_22_b200 import gq as G
    for m, n, bits, group in ((40, 32768, 3, 128), (24, 32767, 4, 0), (9000, 96, 2, 32)):
        c, s, z, w = layer_np(m, n, bits, group, m)
        dev = to_cuda(c, s, z, bits)
        if dtype == torch.int8:
            q, qs = _rows(T, n, 5)
            y = G.gq_linear_quantized(q, qs, *dev, bits, group, y_dtype=torch.float32)
            check_linear(y, q.double().cpu().numpy(), w, qs.double().cpu().numpy())
        else:
            x = _x(T, n, dtype, 5)
            y = G.gq_linear(x, *dev, bits, group, y_dtype=torch.float32)
            check_linear(y, x.double().cpu().numpy(), w)


@pytest.mark.parametrize("T", (1, 7, 200))
def test_unaligned_inputs(T):
    """Views that start one element behind an aligned address, with rows that are aligned in
    themselves."""
    from post_weight_quantization_22_b200 import gq as G
    m, n, bits, group = 70, 256, 4, 64
    c, s, z, w = layer_np(m, n, bits, group, 3)
    dev = to_cuda(c, s, z, bits)
    for dtype in (torch.bfloat16, torch.float32):
        x = _x(1, T * n + 1, dtype, T).view(-1)[1:].view(T, n)
        assert x.data_ptr() % 16
        y = G.gq_linear(x, *dev, bits, group, y_dtype=torch.float32)
        check_linear(y, x.double().cpu().numpy(), w)
    q, qs = _rows(1, T * n + 1, T)
    q = q.view(-1)[1:].view(T, n)
    qs = torch.rand(T, device="cuda")
    y = G.gq_linear_quantized(q, qs, *dev, bits, group, y_dtype=torch.float32)
    check_linear(y, q.double().cpu().numpy(), w, qs.double().cpu().numpy())
    # packed words, scales, zero points and the output at odd places of larger buffers
    codes = torch.cat([dev[0].new_zeros(1), dev[0].view(-1)])[1:].view_as(dev[0])
    scales = torch.cat([dev[1].new_zeros(1), dev[1].view(-1)])[1:].view_as(dev[1])
    zeros = torch.cat([dev[2].new_zeros(1), dev[2].view(-1)])[1:].view_as(dev[2])
    x = _x(T, n, torch.bfloat16, T)
    y = torch.zeros(T * m + 1, dtype=torch.bfloat16, device="cuda")[1:].view(T, m)
    G.gq_linear(x, codes, scales, zeros, bits, group, y=y)
    check_linear(y, x.double().cpu().numpy(), w)


@pytest.mark.parametrize("T", (1, 12, 150))
@pytest.mark.parametrize("bits,group", ((3, 16), (4, 128), (8, 32), (5, 64)))
def test_ordered_layers(T, bits, group):
    """Groups along an order: codes repacked once, inputs taken through the permutation."""
    from post_weight_quantization_22_b200 import gq as G
    m, n = 150, 600
    c, s, z, w = layer_np(m, n, bits, group, 17)   # in processing order
    perm = np.random.default_rng(1).permutation(n).astype(np.int32)
    orig = np.empty_like(c)
    orig[:, perm] = c                              # code of original column perm[k] is c[:, k]
    codes, scales, zeros = to_cuda(orig, s, z, bits)
    p = torch.from_numpy(perm).cuda()
    packed = G.gq_order_codes(codes, n, bits, p)
    assert torch.equal(packed, to_cuda(c, s, z, bits)[0])
    for dtype in (torch.bfloat16, torch.float32):
        x = _x(T, n, dtype, T)
        y = G.gq_linear(x, packed, scales, zeros, bits, group, perm=p, y_dtype=torch.float32)
        check_linear(y, x.double().cpu().numpy()[:, perm], w)
    q, qs = _rows(T, n, T)
    y = G.gq_linear_quantized(q, qs, packed, scales, zeros, bits, group, perm=p)
    check_linear(y, q.double().cpu().numpy()[:, perm], w, qs.double().cpu().numpy())


@pytest.mark.parametrize("bits", range(2, 9))
def test_order_codes_every_width(bits):
    from post_weight_quantization_22_b200 import gq as G
    for m, n in ((1, 1), (3, 31), (5, 33), (2, 1000)):
        c, s, z, _ = layer_np(m, n, bits, 0, n)
        perm = np.random.default_rng(n).permutation(n).astype(np.int32)
        got = G.gq_order_codes(to_cuda(c, s, z, bits)[0], n, bits, torch.from_numpy(perm).cuda())
        assert torch.equal(got, to_cuda(c[:, perm], s, z, bits)[0])


@pytest.mark.parametrize("T", (3, 90))
def test_non_finite_tokens_stay_in_their_rows(T):
    from post_weight_quantization_22_b200 import gq as G
    m, n, bits, group = 64, 256, 4, 64
    c, s, z, w = layer_np(m, n, bits, group, 9)
    c[0, 5] = z[0, 0]                               # 0 * inf
    w = s.astype(np.float64)[:, np.arange(n) // group] * (c - z[:, np.arange(n) // group].astype(int))
    dev = to_cuda(c, s, z, bits)
    for dtype in (torch.bfloat16, torch.float32):
        x = _x(T, n, dtype, 1)
        clean = G.gq_linear(x, *dev, bits, group)
        x[1, 5] = float("inf")
        x[2, 7] = float("nan")
        x[0, 9] = torch.finfo(dtype).max / 2 ** 12
        y = G.gq_linear(x, *dev, bits, group)
        with np.errstate(all="ignore"):
            ref = x.double().cpu().numpy() @ w.T
        assert np.array_equal(np.isnan(y.cpu().float().numpy()), np.isnan(ref))
        assert np.array_equal(np.isinf(y.cpu().float().numpy()[1]), np.isinf(ref[1]))
        assert torch.equal(y[3:], clean[3:])
        check_linear(y[:1], x[:1].double().cpu().numpy(), w)
    q, qs = _rows(T, n, 2)
    qs[1] = float("nan")
    y = G.gq_linear_quantized(q, qs, *dev, bits, group)
    assert bool(y[1].isnan().all()) and not bool(y[0].isnan().any()) and not bool(y[2:].isnan().any())


def test_empty_and_repeated_calls_give_equal_bits():
    from post_weight_quantization_22_b200 import gq as G
    m, n, bits, group = 300, 1000, 3, 128
    c, s, z, _ = layer_np(m, n, bits, group, 4)
    dev = to_cuda(c, s, z, bits)
    assert G.gq_linear(torch.empty(0, n, device="cuda"), *dev, bits, group).shape == (0, m)
    for T in (1, 20, 500):
        x = _x(T, n, torch.float32, T)
        first = G.gq_linear(x, *dev, bits, group)
        for _ in range(3):
            assert torch.equal(G.gq_linear(x, *dev, bits, group), first)


def test_two_streams_and_a_captured_graph():
    from post_weight_quantization_22_b200 import gq as G
    m, n, bits, group = 256, 1024, 4, 128
    c, s, z, w = layer_np(m, n, bits, group, 6)
    dev = to_cuda(c, s, z, bits)
    gamma = torch.ones(n, device="cuda")
    xs = {T: _x(T, n, torch.float32, T) for T in (1, 70)}
    ref = {T: G.gq_linear(x, *dev, bits, group) for T, x in xs.items()}
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    got = []
    for _ in range(5):
        for st, T in ((a, 1), (b, 70)):
            got.append((T, G.gq_linear(xs[T], *dev, bits, group, stream=st)))
    torch.cuda.synchronize()
    assert all(torch.equal(y, ref[T]) for T, y in got)
    # captured: norm, 8-bit product and fp32 product, replayed on new inputs
    x = xs[70].clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        r = G.gq_rmsnorm_quantize(x, gamma, 1e-6)
        y1 = G.gq_linear_quantized(r["q"], r["qscale"], *dev, bits, group)
        y2 = G.gq_linear(x, *dev, bits, group)
    for seed in (1, 2):
        x.copy_(_x(70, n, torch.float32, seed))
        graph.replay()
        r2 = G.gq_rmsnorm_quantize(x, gamma, 1e-6)
        assert torch.equal(y1, G.gq_linear_quantized(r2["q"], r2["qscale"], *dev, bits, group))
        assert torch.equal(y2, G.gq_linear(x, *dev, bits, group))


def test_a_layer_of_the_quantizer_runs():
    """What gq_quantize_layer writes, natural, per-row and in act-order with groups, multiplied
    with the calibration tokens."""
    from post_weight_quantization_22_b200 import gq as G, synth
    W, X, _ = synth.workload("q_proj_4096x4096", m=96, n=320, T=200)
    for bits, group, order in ((4, 64, None), (3, 0, None), (4, 32, "act")):
        g = run_gpu(W, X, bits=bits, group=group, order=order)
        assert g["status"] == (0, 0)
        scales, zeros = torch.from_numpy(g["scales"]).cuda(), torch.from_numpy(
            g["zeros"].astype(np.uint8)).cuda()
        of = np.zeros(320, dtype=int) if not group else np.arange(320) // group
        if order:
            at = np.empty(320, dtype=int)
            at[g["perm"]] = of
            of = at                                  # group of original column c
        w = g["scales"].astype(np.float64)[:, of] * (g["codes"] - g["zeros"][:, of])
        codes, p = g["codes_dev"], None
        if order:
            p = torch.from_numpy(g["perm"].astype(np.int32)).cuda()
            codes = G.gq_order_codes(codes, 320, bits, p)
        x = X.cuda()
        y = G.gq_linear(x, codes, scales, zeros, bits, group, perm=p, y_dtype=torch.float32)
        check_linear(y, x.double().cpu().numpy(), w)


# ---------------------------------------------------------------------------------------------
# norm
# ---------------------------------------------------------------------------------------------

def _check_norm(r, x, res, gamma, eps):
    h, v, q, s = norm_np(x.double().cpu().numpy(), None if res is None else res.double().cpu().numpy(),
                         gamma.double().cpu().numpy(), eps, x.dtype)
    if r["sum"] is not None:
        assert np.array_equal(r["sum"].double().cpu().numpy(), h)
    if r["y"] is not None:
        # fp64 up to the one rounding of the output (through fp32 for bf16: 2^-24 more)
        half = torch.finfo(x.dtype).eps / 2 + 2.0 ** -23
        got = r["y"].double().cpu().numpy()
        assert np.all(np.abs(got - v) <= half * np.abs(v) + 1e-38)
    if r["q"] is not None:
        assert np.array_equal(r["q"].cpu().numpy().astype(np.int64), q)
        got = r["qscale"].double().cpu().numpy()
        assert np.all(np.abs(got - s) <= 2.0 ** -23 * s + 1e-38)


@pytest.mark.parametrize("n", (1, 7, 8, 64, 255, 1000, 1003, 4096, 5000, 14336, 32768))
@pytest.mark.parametrize("dtype", (torch.bfloat16, torch.float32))
def test_norm_matches_fp64(n, dtype):
    from post_weight_quantization_22_b200 import gq as G
    for T, gt, use_res, forms in ((1, dtype, True, "q"), (5, torch.float32, True, "yq"),
                                  (33, torch.bfloat16, False, "y"), (300, dtype, True, "q")):
        x, gamma = _x(T, n, dtype, n + T), (1 + 0.3 * _x(1, n, torch.float32, 3)[0]).to(gt)
        res = _x(T, n, dtype, n + T + 1) if use_res else None
        buf, y = _guarded(T, n, dtype)
        q = torch.full((T + 2, n), 99, dtype=torch.int8, device="cuda")
        s = torch.full((T + 2,), 7.0, device="cuda")
        r = G.gq_rmsnorm_quantize(x, gamma, 1e-5, residual=res,
                                  y=y if "y" in forms else None,
                                  q=q[1:-1] if "q" in forms else None,
                                  qscale=s[1:-1] if "q" in forms else None)
        _check_norm(r, x, res, gamma, 1e-5)
        _whole(buf)
        assert bool((q[0] == 99).all()) and bool((q[-1] == 99).all()) and float(s[0]) == float(s[-1]) == 7


@pytest.mark.parametrize("dtype", (torch.bfloat16, torch.float32))
def test_norm_codes_at_borders(dtype):
    """Values that are exactly half way between two codes go to the even one, and their neighbours
    to their own side."""
    from post_weight_quantization_22_b200 import gq as G
    k = torch.arange(0, 127, dtype=torch.float32, device="cuda")
    half = torch.cat([k + 0.5, -(k + 0.5), torch.tensor([127.0], device="cuda")])
    rows = []
    for f in (1.0, 3.0, 0.1875, 2.0 ** -60, 2.0 ** 60):
        rows += [half * f]
        if dtype == torch.float32:
            inf = torch.tensor(float("inf"), device="cuda")
            up = torch.nextafter(half, inf)
            up[-1] = 127.0
            down = torch.nextafter(half, -inf)
            down[-1] = 127.0
            rows += [up * f, down * f]
    x = torch.stack(rows).to(dtype)
    gamma = torch.ones(x.shape[1], device="cuda")
    r = G.gq_rmsnorm_quantize(x, gamma, 0.0)
    _check_norm(r, x, None, gamma, 0.0)


@pytest.mark.parametrize("dtype", (torch.bfloat16, torch.float32))
def test_norm_extreme_values(dtype):
    """Zero rows, infinities and NaN, the type's largest and smallest values."""
    from post_weight_quantization_22_b200 import gq as G
    n = 1000
    x = _x(12, n, dtype, 0)
    x[1] = 0
    x[2, 5] = float("inf")
    x[3, 6] = float("nan")
    x[4, 7] = -float("inf")
    x[5] *= torch.finfo(dtype).max / 64
    x[6] *= torch.finfo(dtype).tiny
    x[7] = torch.finfo(dtype).tiny * 2.0 ** -5
    x[8] = 0
    x[8, 999] = torch.finfo(dtype).max
    gamma = torch.ones(n, dtype=torch.float32, device="cuda")
    gamma[::3] = -2.5
    gamma[1] = 1e30
    for eps in (0.0, 1e-6):
        r = G.gq_rmsnorm_quantize(x, gamma, eps)
        h, v, q, s = norm_np(x.double().cpu().numpy(), None, gamma.double().cpu().numpy(), eps, dtype)
        got = r["qscale"].double().cpu().numpy()
        assert np.array_equal(np.isnan(got), np.isnan(s) | ((eps == 0) & (np.abs(h).max(1) == 0)))
        ok = np.isfinite(s)
        assert np.array_equal(r["q"].cpu().numpy()[ok].astype(int), q[ok])
        assert not r["q"][2:5].any()
        with np.errstate(over="ignore"):
            s32 = s.astype(np.float32).astype(np.float64)
        assert np.allclose(got[ok], s32[ok], rtol=2.0 ** -22, atol=2.0 ** -148)


def test_norm_in_place_and_other_streams():
    from post_weight_quantization_22_b200 import gq as G
    for n in (1003, 4096):
        for dtype in (torch.bfloat16, torch.float32):
            x, res = _x(37, n, dtype, 1), _x(37, n, dtype, 2)
            gamma = torch.rand(n, device="cuda")
            want = G.gq_rmsnorm_quantize(x, gamma, 1e-6, residual=res, y=torch.empty_like(x),
                                         q=torch.empty(37, n, dtype=torch.int8, device="cuda"),
                                         qscale=torch.empty(37, device="cuda"))
            # the residual stream in place, the output over the input
            x2, r2 = x.clone(), res.clone()
            st = torch.cuda.Stream()
            torch.cuda.synchronize()
            got = G.gq_rmsnorm_quantize(x2, gamma, 1e-6, residual=r2, sum=r2, y=x2, stream=st)
            torch.cuda.synchronize()
            assert torch.equal(got["sum"], want["sum"]) and torch.equal(got["y"], want["y"])
            x3, r3 = x.clone(), res.clone()
            got = G.gq_rmsnorm_quantize(x3, gamma, 1e-6, residual=r3, sum=x3)
            assert torch.equal(x3, want["sum"]) and torch.equal(r3, res)
            assert torch.equal(got["q"], want["q"]) and torch.equal(got["qscale"], want["qscale"])


def test_norm_unaligned_rows():
    from post_weight_quantization_22_b200 import gq as G
    for dtype in (torch.bfloat16, torch.float32):
        n, T = 512, 9
        x = _x(1, T * n + 1, dtype, 3).view(-1)[1:].view(T, n)
        res = _x(1, T * n + 1, dtype, 4).view(-1)[1:].view(T, n)
        gamma = torch.rand(n + 1, device="cuda")[1:]
        q = torch.empty(T * n + 1, dtype=torch.int8, device="cuda")[1:].view(T, n)
        r = G.gq_rmsnorm_quantize(x, gamma, 1e-6, residual=res, q=q,
                                  qscale=torch.empty(T + 1, device="cuda")[1:])
        _check_norm(r, x, res, gamma, 1e-6)


def test_norm_feeds_the_product():
    """The residual, norm, 8-bit rows and product as a decoder runs them, against the formula on
    the values that the rows stand for."""
    from post_weight_quantization_22_b200 import gq as G
    m, n, bits, group = 200, 512, 4, 128
    c, s, z, w = layer_np(m, n, bits, group, 8)
    dev = to_cuda(c, s, z, bits)
    for T in (1, 50):
        x, res = _x(T, n, torch.bfloat16, T), _x(T, n, torch.bfloat16, T + 1)
        gamma = (1 + 0.1 * _x(1, n, torch.float32, 5)[0]).to(torch.bfloat16)
        r = G.gq_rmsnorm_quantize(x, gamma, 1e-6, residual=res)
        y = G.gq_linear_quantized(r["q"], r["qscale"], *dev, bits, group, y_dtype=torch.float32)
        _, v, q, qs = norm_np(x.double().cpu().numpy(), res.double().cpu().numpy(),
                              gamma.double().cpu().numpy(), 1e-6, torch.bfloat16)
        check_linear(y, q.astype(np.float64), w, qs.astype(np.float32).astype(np.float64))
        # and the rows are within half a step of the norm
        got = r["q"].double().cpu().numpy() * r["qscale"].double().cpu().numpy()[:, None]
        assert np.all(np.abs(got - v) <= (0.5 + 127 * 2.0 ** -23) * qs[:, None])


@pytest.mark.parametrize("dtype", (torch.bfloat16, torch.int8))
def test_more_tiles_than_sms(dtype):
    """Several tiles one after another on every SM."""
    from post_weight_quantization_22_b200 import gq as G
    m, n, bits, group, T = 2500, 200, 4, 32, 5000
    c, s, z, w = layer_np(m, n, bits, group, 12)
    dev = to_cuda(c, s, z, bits)
    if dtype == torch.int8:
        q, qs = _rows(T, n, 1)
        y = G.gq_linear_quantized(q, qs, *dev, bits, group)
        check_linear(y, q.double().cpu().numpy(), w, qs.double().cpu().numpy())
    else:
        x = _x(T, n, dtype, 1)
        check_linear(G.gq_linear(x, *dev, bits, group), x.double().cpu().numpy(), w)


def test_layer_quantizer_output():
    """LayerQuantizer.output: the quantized layer on its calibration tokens, natural order and
    act-order with groups, against the dequantized weights."""
    from post_weight_quantization_22_b200 import gq as G, synth
    from post_weight_quantization_22_b200.pipeline import LayerQuantizer
    from tests.gpu_helpers import unpack_np
    m, n = 96, 256
    W, X, _ = synth.workload("q_proj_4096x4096", m=m, n=n, T=300)
    for order in (None, "act"):
        cfg = G.QuantCfg(bits=4, group_size=64)
        lq = LayerQuantizer(m, n, cfg, order=order)
        lq.run(W.cuda().contiguous(), X.cuda().contiguous())
        y = lq.output(X.cuda().contiguous())
        codes = unpack_np(lq.codes.cpu().numpy().view(np.uint32), n, 4)
        at = np.arange(n) if order is None else np.argsort(lq.perm.cpu().numpy())
        of = at // 64
        w = lq.scales.double().cpu().numpy()[:, of] * (codes - lq.zeros.cpu().numpy().astype(int)[:, of])
        assert y.dtype == torch.bfloat16
        check_linear(y, X.double().numpy(), w)


def test_block_forward_runs_every_layer_of_an_input():
    """BlockQuantizer.forward: residual, norm, 8-bit rows and q, k, v on them; and the same as one
    stacked product."""
    from post_weight_quantization_22_b200 import gq as G, synth
    from post_weight_quantization_22_b200.pipeline import BlockQuantizer, QuantizedLinear
    from tests.gpu_helpers import unpack_np
    layers = (("q", 128, 256, "attn"), ("k", 64, 256, "attn"), ("v", 64, 256, "attn"),
              ("o", 96, 128, "o"))
    bq = BlockQuantizer(layers, G.QuantCfg(bits=2, group_size=64))
    g = torch.Generator(device="cuda").manual_seed(3)
    Ws = {name: (0.02 * torch.randn(m, n, generator=g, device="cuda")).bfloat16()
          for name, m, n, _ in layers}
    Xs = {k: torch.randn(400, n, generator=g, device="cuda").bfloat16()
          for k, n in (("attn", 256), ("o", 128))}
    bq.run(Ws, Xs)
    assert bq.status() == 0
    gamma = (1 + 0.1 * torch.randn(256, generator=g, device="cuda")).bfloat16()
    for T in (1, 20, 70):
        x = torch.randn(T, 256, generator=g, device="cuda").bfloat16()
        res = torch.randn(T, 256, generator=g, device="cuda").bfloat16()
        out = bq.forward("attn", x, gamma, residual=res)
        assert set(out) == {"sum", "q", "k", "v"}
        h, v, q, qs = norm_np(x.double().cpu().numpy(), res.double().cpu().numpy(),
                              gamma.double().cpu().numpy(), 1e-6, torch.bfloat16)
        assert np.array_equal(out["sum"].double().cpu().numpy(), h)
        for name in "qkv":
            o = bq.out[name]
            codes = unpack_np(o["codes"].cpu().numpy().view(np.uint32), 256, 2)
            of = np.arange(256) // 64
            w = o["scales"].double().cpu().numpy()[:, of] * (
                codes - o["zeros"].cpu().numpy().astype(int)[:, of])
            check_linear(out[name], q.astype(np.float64), w, qs.astype(np.float32).astype(np.float64))
        one = QuantizedLinear.stack([bq.linear(name) for name in "qkv"])
        r = G.gq_rmsnorm_quantize(x, gamma, 1e-6, residual=res)
        y = one(r["q"], r["qscale"])
        assert torch.equal(y, torch.cat([out[name] for name in "qkv"], 1))
        plain = bq.forward("attn", x, gamma, residual=res, quantized=False)
        assert torch.equal(plain["sum"], out["sum"]) and plain["q"].dtype == torch.bfloat16
    with pytest.raises(ValueError):
        bq.forward("mlp", x, gamma)
    with pytest.raises(ValueError):
        QuantizedLinear.stack([bq.linear("q"), bq.linear("o")])
    with pytest.raises(ValueError):
        QuantizedLinear(bq.out["q"]["codes"], bq.out["q"]["scales"], bq.out["q"]["zeros"], 256,
                        G.QuantCfg(bits=2, clip="unbounded"))


@pytest.mark.parametrize("bits", (2, 4, 6, 8))
@pytest.mark.parametrize("dtype", (torch.bfloat16, torch.float32))
def test_half_a_chunk_at_the_end_of_many_tiles(bits, dtype):
    """Widths that end inside a packed chunk of 128 columns (an odd number of 64-column stages),
    with several tiles for every pair of SMs."""
    from post_weight_quantization_22_b200 import gq as G
    for m, n, T, group in ((2560, 192, 4000, 64), (2560, 64, 4000, 0), (2600, 448, 2100, 32)):
        c, s, z, w = layer_np(m, n, bits, group, n + bits)
        dev = to_cuda(c, s, z, bits)
        x = _x(T, n, dtype, 1)
        first = G.gq_linear(x, *dev, bits, group, y_dtype=torch.float32)
        rows = np.r_[0:40, T - 40:T]
        check_linear(first[rows], x.double().cpu().numpy()[rows], w)
        ref = x.double() @ torch.from_numpy(w).cuda().T
        A = x.double().abs() @ torch.from_numpy(np.abs(w)).cuda().T
        # the bound of check_linear (fp32 output) for the rest
        sums = 3 * 256 * 2.0 ** -23 + (n / 16 + 18) * 2.0 ** -24
        assert bool(((first.double() - ref).abs() <= 2.0 ** -24 * ref.abs() + 1.01 * sums * A).all())
        for _ in range(5):
            assert torch.equal(G.gq_linear(x, *dev, bits, group, y_dtype=torch.float32), first)


def _check_on_gpu(y, x, w, xscale=None):
    """check_linear's bounds, computed on the GPU in fp64."""
    x, w = x.double(), torch.from_numpy(w).cuda()
    ref, A = x @ w.T, x.abs() @ w.abs().T
    if xscale is not None:
        ref, A = ref * xscale.double()[:, None], A * xscale.double()[:, None]
    n, half = x.shape[1], torch.finfo(y.dtype).eps / 2
    sums = 3 * 256 * 2.0 ** -23 + (n / 16 + 18) * 2.0 ** -24
    assert bool(((y.double() - ref).abs() <= half * ref.abs() + (1 + half) * sums * A + 1e-38).all())
    rel = float((y.double() - ref).norm() / ref.norm())
    assert rel <= half + 3 * 16 * 2.0 ** -23 + (n / 16 + 18) * 2.0 ** -24, rel


@pytest.mark.parametrize("bits", range(2, 9))
@pytest.mark.parametrize("group", GROUPS)
def test_wide_layers(bits, group):
    """Layers with rows enough for pairs of CTAs (3400 rows, 520 tokens) and for single CTAs that
    take whole rows by TMA (2500 rows, 40 and 90 tokens), in every width and group."""
    from post_weight_quantization_22_b200 import gq as G
    for T, m, n in ((520, 3400, 256), (40, 2500, 320), (90, 2500, 192)):
        c, s, z, w = layer_np(m, n, bits, group, bits + T, extreme=T == 90)
        dev = to_cuda(c, s, z, bits)
        for dtype in (torch.bfloat16, torch.float32):
            x = _x(T, n, dtype, T)
            buf, y = _guarded(T, m, torch.float32)
            G.gq_linear(x, *dev, bits, group, y=y)
            _check_on_gpu(y, x, w)
            _whole(buf)
        q, qs = _rows(T, n, T)
        buf, y = _guarded(T, m, torch.bfloat16)
        G.gq_linear_quantized(q, qs, *dev, bits, group, y=y)
        _check_on_gpu(y, q, w, qs)
        _whole(buf)


def test_wide_layer_captured_and_on_two_streams():
    """The tcgen05 kernels in a graph (their workspace in the graph's pool) and on two streams at
    once."""
    from post_weight_quantization_22_b200 import gq as G
    bits, group, n = 4, 64, 512
    c, s, z, w = layer_np(3000, n, bits, group, 2)
    dev = to_cuda(c, s, z, bits)
    xs = {T: _x(T, n, torch.bfloat16, T) for T in (100, 800)}
    q, qs = _rows(800, n, 1)
    ref = {T: G.gq_linear(x, *dev, bits, group) for T, x in xs.items()}
    ref_q = G.gq_linear_quantized(q, qs, *dev, bits, group)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ya = G.gq_linear(xs[100], *dev, bits, group)
        yb = G.gq_linear(xs[800], *dev, bits, group)
        yc = G.gq_linear_quantized(q, qs, *dev, bits, group)
    for _ in range(2):
        graph.replay()
        assert torch.equal(ya, ref[100]) and torch.equal(yb, ref[800]) and torch.equal(yc, ref_q)
    st = (torch.cuda.Stream(), torch.cuda.Stream())
    torch.cuda.synchronize()
    got = [(T, G.gq_linear(xs[T], *dev, bits, group, stream=st[i % 2]))
           for i, T in enumerate((100, 800) * 4)]
    torch.cuda.synchronize()
    assert all(torch.equal(y, ref[T]) for T, y in got)


def test_workspace_status_after_a_product():
    from post_weight_quantization_22_b200 import gq as G
    c, s, z, w = layer_np(2500, 128, 4, 64, 2)
    dev = to_cuda(c, s, z, 4)
    x = _x(64, 128, torch.float32, 1)
    ws = torch.full((G.gq_linear_workspace_size(64, 2500, 128, torch.float32),), 255,
                    dtype=torch.uint8, device="cuda")
    y = G.gq_linear(x, *dev, 4, 64, ws=ws)
    assert G.gq_workspace_status(ws)[0] == 0
    _check_on_gpu(y, x, w)
    with pytest.raises(G.GQError) as e:
        G.gq_linear(x, *dev, 4, 64, ws=ws[:-1])
    assert e.value.code == 7

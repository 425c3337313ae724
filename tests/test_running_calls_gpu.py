"""The running calls as programs make them around other work: side streams, kept layers, status
words, waits that run out."""
import numpy as np
import pytest
import torch

from tests.running_helpers import check_linear, layer_np, norm_np, to_cuda

pytestmark = pytest.mark.gpu

BUSY = 200_000_000  # clock cycles for which the current stream is kept busy: a tenth of a second


def _weights(codes, scales, zeros, n, bits, group, perm=None):
    """The fp64 weights of a quantizer's result buffers."""
    from tests.gpu_helpers import unpack_np
    c = unpack_np(codes.cpu().numpy().view(np.uint32), n, bits)
    at = np.arange(n) if perm is None else np.argsort(perm.cpu().numpy())
    of = at // (group or n)
    return scales.double().cpu().numpy()[:, of] * (c - zeros.cpu().numpy().astype(int)[:, of])


@pytest.mark.parametrize("T", (5, 300))
def test_output_on_a_side_stream(T):
    """An ordered layer with groups quantized and run on a stream of its own, while the current
    stream is busy and takes memory back into use right behind the call."""
    from post_weight_quantization_22_b200 import gq as G, synth
    from post_weight_quantization_22_b200.pipeline import LayerQuantizer
    m, n = 96, 256
    W, X, _ = synth.workload("q_proj_4096x4096", m=m, n=n, T=300)
    W, X = W.cuda().contiguous(), X.cuda().contiguous()
    lq = LayerQuantizer(m, n, G.QuantCfg(bits=4, group_size=64), order="act")
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda._sleep(BUSY)
    lq.run(W, X, stream=side)
    y = lq.output(X[:T], stream=side)
    for _ in range(8):
        torch.full((m, n // 8), -1, dtype=torch.int32, device="cuda")
    side.synchronize()
    w = _weights(lq.codes, lq.scales, lq.zeros, n, 4, 64, lq.perm)
    check_linear(y, X[:T].double().cpu().numpy(), w)


@pytest.mark.parametrize("T", (3, 200))
def test_forward_on_a_side_stream(T):
    """BlockQuantizer.forward in both modes on a stream of its own, the current stream busy and
    taking memory back into use right behind the call; every output against the formula."""
    from post_weight_quantization_22_b200 import gq as G
    from post_weight_quantization_22_b200.pipeline import BlockQuantizer
    layers = (("q", 128, 256, "attn"), ("k", 64, 256, "attn"), ("v", 64, 256, "attn"))
    bq = BlockQuantizer(layers, G.QuantCfg(bits=3, group_size=64))
    g = torch.Generator(device="cuda").manual_seed(3)
    Ws = {name: (0.02 * torch.randn(m, n, generator=g, device="cuda")).bfloat16()
          for name, m, n, _ in layers}
    bq.run(Ws, {"attn": torch.randn(400, 256, generator=g, device="cuda").bfloat16()})
    gamma = (1 + 0.1 * torch.randn(256, generator=g, device="cuda")).bfloat16()
    x, res = (torch.randn(T, 256, generator=g, device="cuda").bfloat16() for _ in range(2))
    h, v, q, qs = norm_np(x.double().cpu().numpy(), res.double().cpu().numpy(),
                          gamma.double().cpu().numpy(), 1e-6, torch.bfloat16)
    side = torch.cuda.Stream()
    for quantized in (True, False):
        torch.cuda.synchronize()
        torch.cuda._sleep(BUSY)
        out = bq.forward("attn", x, gamma, residual=res, quantized=quantized, stream=side)
        for _ in range(8):
            torch.full_like(x, float("nan"))
        side.synchronize()
        assert np.array_equal(out["sum"].double().cpu().numpy(), h)
        for name, _, n, _ in layers:
            o = bq.out[name]
            w = _weights(o["codes"], o["scales"], o["zeros"], n, 3, 64)
            if quantized:
                check_linear(out[name], q.astype(np.float64), w, qs.astype(np.float32).astype(np.float64))
            else:
                # the norm's rows in bf16 are off by half a step at most (and 2^-23: they are
                # rounded from fp32), the product of them as check_linear says: sums of at most
                # 3 * 256 truncated additions a run, n / 16 + 18 of 2^-24, half a step of y
                ref, A = v @ w.T, np.abs(v) @ np.abs(w).T
                half = torch.finfo(torch.bfloat16).eps / 2
                sums = 3 * 256 * 2.0 ** -23 + (n / 16 + 18) * 2.0 ** -24
                off = (half + 2.0 ** -23 + (1 + half) * sums) * A
                got = out[name].double().cpu().numpy()
                assert np.all(np.abs(got - ref) <= half * (np.abs(ref) + off) + off + 1e-38)


def test_a_kept_ordered_layer_stays_what_it_was():
    """A repacked layer after the quantizer has written another order, other grids and codes."""
    from post_weight_quantization_22_b200 import gq as G, synth
    from post_weight_quantization_22_b200.pipeline import LayerQuantizer
    m, n = 96, 256
    W, X, _ = synth.workload("q_proj_4096x4096", m=m, n=n, T=300)
    W, X = W.cuda().contiguous(), X.cuda().contiguous()
    lq = LayerQuantizer(m, n, G.QuantCfg(bits=4, group_size=64), order="act")
    lq.run(W, X)
    layer, w = lq.linear(), _weights(lq.codes, lq.scales, lq.zeros, n, 4, 64, lq.perm)
    first = layer(X)
    check_linear(first, X.double().cpu().numpy(), w)
    perm = lq.perm.clone()
    lq.run((3 * W.flip(1)).contiguous(), X.flip(1).contiguous())
    assert not torch.equal(lq.perm, perm)
    assert torch.equal(layer(X), first)


@pytest.mark.parametrize("T", (64, 300))
def test_status_word_of_a_misaligned_matrix(T):
    """A bf16 matrix off the 16-byte boundaries that tensor maps need: the call asks for a workspace
    as for an aligned one and leaves its status word clean."""
    from post_weight_quantization_22_b200 import gq as G
    m, n, bits, group = 4096, 256, 4, 64
    c, s, z, w = layer_np(m, n, bits, group, T)
    dev = to_cuda(c, s, z, bits)
    g = torch.Generator(device="cuda").manual_seed(T)
    x = torch.randn(T * n + 1, generator=g, device="cuda").bfloat16()[1:].view(T, n)
    assert x.data_ptr() % 16 == 2
    need = G.gq_linear_workspace_size(T, m, n, torch.bfloat16)
    assert need > 0
    ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda")
    y = G.gq_linear(x, *dev, bits, group, y_dtype=torch.float32, ws=ws)
    check_linear(y, x.double().cpu().numpy(), w)
    assert G.gq_workspace_status(ws)[0] == 0


@pytest.mark.parametrize("dtype", (torch.bfloat16, torch.float32))
@pytest.mark.parametrize("form,T,m,n", (("one CTA a tile", 64, 4096, 256),
                                        ("a cluster a tile", 64, 2048, 2048),
                                        ("pairs of CTAs", 1024, 2560, 512)))
def test_a_wait_of_the_product_runs_out(form, T, m, n, dtype):
    """With the test setting the first CTA never announces its second stage: every wait that needs
    it gives up, the kernel returns, the status word says GQ_ERR_TIMEOUT, and the next call on the
    same workspace is clean and right."""
    import time
    from post_weight_quantization_22_b200 import gq as G
    bits, group = 4, 64
    c, s, z, w = layer_np(m, n, bits, group, 11)
    dev = to_cuda(c, s, z, bits)
    g = torch.Generator(device="cuda").manual_seed(T)
    x = torch.randn(T, n, generator=g, device="cuda").to(dtype)
    ws = torch.zeros(G.gq_linear_workspace_size(T, m, n, dtype), dtype=torch.uint8, device="cuda")
    y = torch.empty(T, m, device="cuda")
    torch.cuda.synchronize()
    G.gq_debug_wait_test(16384, True)
    try:
        t0 = time.perf_counter()
        G.gq_linear(x, *dev, bits, group, y=y, ws=ws)
        torch.cuda.synchronize()
        elapsed = time.perf_counter() - t0
    finally:
        G.gq_debug_wait_test()
    print(f"{form}: {elapsed:.3f} s")
    assert G.gq_workspace_status(ws)[0] == 5           # GQ_ERR_TIMEOUT
    assert G.gq_linear_status() == 5 and G.gq_linear_status() == 0
    assert elapsed < 30.0
    G.gq_linear(x, *dev, bits, group, y=y, ws=ws)
    assert G.gq_workspace_status(ws)[0] == 0 and G.gq_linear_status() == 0
    rows = np.r_[0:8, T - 8:T]
    check_linear(y[rows], x.double().cpu().numpy()[rows], w)


def test_a_timeout_is_seen_without_a_workspace():
    """Calls that bring no workspace of their own, through the pipeline's objects and in a replayed
    graph: the device's status tells of a wait that ran out, once."""
    from post_weight_quantization_22_b200 import gq as G
    from post_weight_quantization_22_b200.pipeline import BlockQuantizer
    m, n, T = 4096, 256, 64
    bq = BlockQuantizer((("q", m, n, "attn"),), G.QuantCfg(bits=4, group_size=64))
    g = torch.Generator(device="cuda").manual_seed(1)
    W = (0.02 * torch.randn(m, n, generator=g, device="cuda")).bfloat16()
    bq.run({"q": W}, {"attn": torch.randn(400, n, generator=g, device="cuda").bfloat16()})
    layer = bq.linear("q")
    x = torch.randn(T, n, generator=g, device="cuda").bfloat16()
    gamma = torch.ones(n, device="cuda")
    G.gq_linear_status()                               # what ran before
    first = layer(x)
    assert layer.status() == 0 and bq.status() == 0
    graph = torch.cuda.CUDAGraph()
    G.gq_debug_wait_test(16384, True)
    try:
        layer(x)
        assert layer.status() == 5                     # GQ_ERR_TIMEOUT
        bq.forward("attn", x, gamma)
        assert bq.status() == 5
        with torch.cuda.graph(graph):
            layer(x)
    finally:
        G.gq_debug_wait_test()
    assert layer.status() == 0
    graph.replay()
    assert G.gq_linear_status() == 5
    side = torch.cuda.Stream()
    assert torch.equal(layer(x), first) and layer.status() == 0 and layer.status(side) == 0


def test_workspace_arguments_are_checked():
    from post_weight_quantization_22_b200 import gq as G
    c, s, z, _ = layer_np(4096, 128, 4, 64, 2)
    dev = to_cuda(c, s, z, 4)
    x = torch.zeros(64, 128, device="cuda")
    need = G.gq_linear_workspace_size(64, 4096, 128, torch.float32)
    for ws in (torch.zeros(need, dtype=torch.uint8), torch.zeros(need, device="cuda"),
               torch.zeros(1, dtype=torch.uint8, device="cuda").expand(need)):
        with pytest.raises(ValueError):
            G.gq_linear(x, *dev, 4, 64, ws=ws)
    G.gq_linear(x, *dev, 4, 64, ws=torch.zeros(2, need, dtype=torch.uint8, device="cuda")[1])


def test_norm_rows_far_below_one():
    """bf16 rows whose 1 / rms leaves fp32, and products h gamma below fp32's normal range in rows
    that eps does not hold down: y is the formula's, rounded once."""
    from post_weight_quantization_22_b200 import gq as G
    n = 256
    g = torch.Generator(device="cuda").manual_seed(0)
    base = torch.randn(n, generator=g, device="cuda").clamp(-3, 3)
    odd = torch.arange(n, device="cuda") % 2 == 1
    x = torch.stack([(base.double() * 2.0 ** e).float() for e in (-131, -120, -126, -95, -60, 0, 100)]).bfloat16()
    gammas = []
    gammas.append(torch.full((n,), 2.0 ** 40, device="cuda"))               # max|u| near 2^-80
    gammas.append(torch.where(odd, 1 + 2.0 ** -7, 2.0 ** -50 * (1 + 2.0 ** -6)))
    gammas.append(1 + 0.1 * torch.randn(n, generator=g, device="cuda"))
    for gamma in gammas:
        gamma = gamma.bfloat16()
        for eps in (0.0, 1e-6):
            r = G.gq_rmsnorm_quantize(x, gamma, eps, y=torch.empty_like(x),
                                      q=torch.empty(len(x), n, dtype=torch.int8, device="cuda"),
                                      qscale=torch.empty(len(x), device="cuda"))
            h, v, q, s = norm_np(x.double().cpu().numpy(), None, gamma.double().cpu().numpy(), eps,
                                 torch.bfloat16)
            # half a step of bf16 relative to the value and 2^-23 for roundings in fp32 on the way;
            # below the normal range half of the smallest step, 2^-133, and a quarter for the way
            half = torch.finfo(torch.bfloat16).eps / 2 + 2.0 ** -23
            got = r["y"].double().cpu().numpy()
            off = np.abs(got - v) - (half * np.abs(v) + 0.75 * 2.0 ** -133)
            assert np.all(off <= 0), (eps, np.argwhere(~(off <= 0))[:4], float(off.max()))
            assert np.array_equal(r["q"].cpu().numpy().astype(int), q)


@pytest.mark.parametrize("dtype", (torch.bfloat16, torch.float32))
def test_norm_of_a_row_of_zeros(dtype):
    """With eps > 0 everything is 0; without it the row is 0 / 0, and says so."""
    from post_weight_quantization_22_b200 import gq as G
    n = 300
    x = torch.zeros(3, n, dtype=dtype, device="cuda")
    x[1] = 1
    gamma = torch.ones(n, dtype=dtype, device="cuda")
    for eps in (1e-6, 0.0):
        r = G.gq_rmsnorm_quantize(x, gamma, eps, y=torch.empty_like(x),
                                  q=torch.full((3, n), 9, dtype=torch.int8, device="cuda"),
                                  qscale=torch.empty(3, device="cuda"))
        assert not r["q"][::2].any() and bool((r["q"][1] == 127).all())
        want = 0.0 if eps else float("nan")
        for t in (r["y"][::2], r["qscale"][::2]):
            assert torch.equal(t.isnan(), torch.full_like(t, want).isnan())
            assert eps == 0 or not t.any()
        assert bool(r["y"][1].isfinite().all()) and bool(r["qscale"][1].isfinite())

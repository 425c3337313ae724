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

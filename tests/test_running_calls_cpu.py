"""How the pipeline's running calls use streams and buffers, with the library's calls replaced by
recorders (no GPU)."""
import types

import pytest
import torch


@pytest.fixture
def calls(monkeypatch):
    """The binding's running calls as recorders: (name, positional arguments, stream)."""
    from post_weight_quantization_22_b200 import gq as G
    seen = []

    def order_codes(codes, n, bits, perm, out=None, stream=None):
        seen.append(("order", (codes, perm), stream))
        return codes.clone()

    def linear(x, codes, scales, zeros, bits, group_size=0, perm=None, y=None, y_dtype=None,
               ws=None, stream=None):
        seen.append(("linear", (x, codes, scales, zeros, perm), stream))
        return torch.zeros(x.shape[0], codes.shape[0])

    monkeypatch.setattr(G, "gq_order_codes", order_codes)
    monkeypatch.setattr(G, "gq_linear", linear)
    return seen


def _ordered_quantizer(order="act", group=64):
    from post_weight_quantization_22_b200 import gq as G
    from post_weight_quantization_22_b200.pipeline import LayerQuantizer
    return LayerQuantizer(8, 128, G.QuantCfg(bits=4, group_size=group), device="cpu", order=order,
                          max_tokens=16)


def test_output_repacks_on_its_stream(calls):
    """An ordered layer's repacking and the product that reads it run on one stream."""
    stream = types.SimpleNamespace(device=torch.device("cpu"))
    lq = _ordered_quantizer()
    lq.output(torch.zeros(3, 128), stream=stream)
    assert [c[0] for c in calls] == ["order", "linear"]
    assert all(c[2] is stream for c in calls)
    del calls[:]
    lq.linear(stream)
    lq.linear()
    assert [(c[0], c[2]) for c in calls] == [("order", stream), ("order", None)]

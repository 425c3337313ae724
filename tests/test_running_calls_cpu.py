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


@pytest.mark.parametrize("quantized", (True, False))
def test_forward_allocates_on_its_stream(monkeypatch, quantized):
    """What BlockQuantizer.forward allocates for itself is allocated on the stream that its calls
    run on."""
    from post_weight_quantization_22_b200 import gq as G
    from post_weight_quantization_22_b200.pipeline import BlockQuantizer
    side = types.SimpleNamespace(device=types.SimpleNamespace(index=-1))  # a CPU tensor's get_device()
    current, seen = [None], []

    class Use:
        def __init__(self, stream):
            self.stream = stream

        def __enter__(self):
            self.before, current[0] = current[0], self.stream

        def __exit__(self, *exc):
            current[0] = self.before

    def norm(x, gamma, eps=1e-6, residual=None, sum=None, y=None, q=None, qscale=None, stream=None):
        seen.append(("norm", current[0] if stream is None else stream))
        return dict(sum=None, y=y, q=x, qscale=gamma)

    def product(*args, stream=None, **kw):
        stream = args[-1] if stream is None and len(args) > 9 else stream
        seen.append(("product", current[0] if stream is None else stream))
        return args[0]

    def empty_like(x, **kw):
        seen.append(("alloc", current[0]))
        return torch.zeros_like(x)

    bq = BlockQuantizer((("q", 8, 64, "attn"), ("k", 8, 64, "attn")), G.QuantCfg(bits=4),
                        device="cpu", max_tokens=16)
    monkeypatch.setattr(torch.cuda, "stream", Use)
    monkeypatch.setattr(torch, "empty_like", empty_like)
    monkeypatch.setattr(G, "gq_rmsnorm_quantize", norm)
    monkeypatch.setattr(G, "gq_linear", product)
    monkeypatch.setattr(G, "gq_linear_quantized", product)
    bq.forward("attn", torch.zeros(3, 64), torch.ones(64), quantized=quantized, stream=side)
    assert [s[0] for s in seen] == ([] if quantized else ["alloc"]) + ["norm", "product", "product"]
    assert all(s[1] is side for s in seen)


def test_a_kept_ordered_layer_is_a_copy(calls):
    """Grids and order of a repacked layer are its own, as its codes are; a layer that is not
    repacked uses the quantizer's buffers."""
    lq = _ordered_quantizer()
    layer = lq.linear()
    for name in ("codes", "scales", "zeros", "perm"):
        a, b = getattr(layer, name), getattr(lq, name)
        assert a.data_ptr() != b.data_ptr() and torch.equal(a, b), name
    plain = _ordered_quantizer(order=None).linear()
    assert plain.perm is None
    lq = _ordered_quantizer(group=0)
    layer = lq.linear()
    assert layer.perm is None and layer.codes is lq.codes and layer.scales is lq.scales


def test_status_of_the_products_is_reachable(monkeypatch):
    """QuantizedLinear.status and BlockQuantizer.status report the device's products."""
    from post_weight_quantization_22_b200 import gq as G
    from post_weight_quantization_22_b200.pipeline import BlockQuantizer
    assert "gq_linear_status" in G.EXPORTED
    asked = []

    def linear_status(device=None, stream=None):
        asked.append((device, stream))
        return 5

    monkeypatch.setattr(G, "gq_linear_status", linear_status)
    monkeypatch.setattr(G, "gq_workspace_status", lambda ws, stream=None: (0, 0))
    stream = object()
    assert _ordered_quantizer(order=None).linear().status(stream) == 5
    assert asked == [(-1, stream)]
    bq = BlockQuantizer((("q", 8, 64, "attn"),), G.QuantCfg(bits=4), device="cpu", max_tokens=16)
    assert bq.status() == 5


def test_a_workspace_of_another_kind_is_refused(monkeypatch):
    """A workspace in host memory, or one whose bytes its length does not say, never reaches the
    library."""
    from post_weight_quantization_22_b200 import gq as G
    x, q = torch.zeros(64, 16), torch.zeros(64, 16, dtype=torch.int8)
    layer = (torch.zeros(4096, 2, dtype=torch.int32), torch.ones(4096, 1),
             torch.zeros(4096, 1, dtype=torch.uint8))
    # tensors that say of themselves that they are on a GPU, and a library that must not be called
    monkeypatch.setattr(G, "_rows", lambda t, name: (t.shape, 0))
    monkeypatch.setattr(G, "_need_on", lambda *a: None)
    monkeypatch.setattr(G, "_elsewhere", lambda *a: False)
    monkeypatch.setattr(G, "_raw_stream", lambda device: 0)

    class Library:
        def __getattr__(self, name):
            def call(*a):
                raise AssertionError(f"{name} was called")
            return call

    monkeypatch.setattr(G, "LIB", Library())
    for ws in (torch.zeros(1 << 20, dtype=torch.uint8), torch.zeros(1 << 20),
               torch.zeros(1, dtype=torch.uint8).expand(1 << 20)):
        with pytest.raises(ValueError, match="ws"):
            G.gq_linear(x, *layer, 4, y=torch.zeros(64, 4096), ws=ws)
        with pytest.raises(ValueError, match="ws"):
            G.gq_linear_quantized(q, torch.ones(64), *layer, 4, y=torch.zeros(64, 4096), ws=ws)

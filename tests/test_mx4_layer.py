"""The 4-bit layer behind an int8 convolution: the int8, 4-bit and group norm calls together."""
import numpy as np
import pytest
import torch

import convolution_int8_implicit_amd as ifx
from convolution_int8_implicit_amd import model, synth
from oracle import lowp


def f64(t):
    return t.detach().to(torch.float64).cpu().numpy()


def layer_and_input(n=2):
    """res3's conv3 (1x1, 128 -> 512) with int32 output and a 4-bit layer 512 -> 96 behind it."""
    wl = synth.workload(1, n=n)
    spec = wl.convs[0]
    params = synth.conv_params(wl.index, spec)
    d = ifx.conv_desc(n, wl.h, wl.w, 128, 512, 1, 1, 1, 0, ifx.OUT_I32)
    x = synth.input_tensor(wl)
    gen = torch.Generator().manual_seed(4)
    weight = torch.randn(96, 512, generator=gen) / 512 ** 0.5
    nw, nb, bias = 1 + 0.2 * torch.randn(512, generator=gen), 0.3 * torch.randn(512, generator=gen), torch.randn(96, generator=gen)
    acc = torch.empty(n, wl.h, wl.w, 512, dtype=torch.int32, device="cuda")
    w_blk = ifx.pack_weights(d, params["w"].cuda())
    ifx.conv_fused(d, ifx.pack_act(x.cuda()), w_blk, params["bias"].cuda(), None, None, None, acc)
    exact = x.numpy().reshape(-1, 128).astype(np.int64) @ params["w"].numpy().reshape(512, 128).astype(np.int64).T
    assert np.array_equal(acc.cpu().numpy().reshape(-1, 512), exact + params["bias"].numpy().astype(np.int64))
    layer = model.NormPointwise4(weight.cuda(), nw.cuda(), nb.cuda(), 32, 2.0 ** -16, bias.cuda())
    return layer, acc, weight, nw, nb, bias


@pytest.mark.gpu
def test_layer_behind_an_int8_convolution():
    layer, acc, weight, nw, nb, bias = layer_and_input()
    n, h, w, c = acc.shape
    y = layer.forward(acc)
    assert y.shape == (n, h, w, 96) and y.dtype == torch.bfloat16
    # from the kernels' own codes: the product's bound (tests/test_mx4.py), then one rounding
    q = ifx.group_norm_mx4(layer.features(acc), 32, layer.norm_weight, layer.norm_bias, 1e-5, ifx.ACT_SILU)
    codes = (q.codes.cpu().numpy(), q.scales.cpu().numpy())
    wq = (layer.weight.codes.cpu().numpy(), layer.weight.scales.cpu().numpy())
    exact, _, s = lowp.mx4_matmul(codes, wq, c, bias.numpy())
    tol = (4 + 18) * 2.0 ** -23 * s
    low, high = (f64(torch.from_numpy(exact + k * tol).to(torch.bfloat16)) for k in (-1, 1))
    got = f64(y).reshape(-1, 96)
    assert (got >= low).all() and (got <= high).all()
    # against the whole chain in 64 bits: a code may differ where a value lies within rounding of the
    # middle of two levels, about one in 10^5 of them, each worth at most a third of its value
    z = lowp.group_norm(f64(acc).reshape(n, h * w, c) * 2.0 ** -16, 32, f64(nw), f64(nb), 1e-5)[0]
    pixels = np.random.default_rng(0).permutation(n * h * w)[:64]
    ref = lowp.mx4_matmul(lowp.mx4_quantize(lowp.act(z, 2).reshape(-1, c)[pixels]), lowp.mx4_quantize(f64(weight)), c, bias.numpy())[0]
    assert np.linalg.norm(got[pixels] - ref) <= 2.0 ** -8 * np.linalg.norm(ref)
    res = torch.randn(n, h, w, 96, device="cuda").to(torch.bfloat16)
    assert torch.allclose(layer.forward(acc, res).float(), y.float() + res.float(), rtol=2.0 ** -6, atol=2.0 ** -6)


@pytest.mark.gpu
def test_layer_in_a_graph_and_its_gradient():
    """The layer replayed from a graph on new features equals its eager calls; a step along the norm's
    gradient lowers the loss it is the gradient of."""
    layer, acc, *_ = layer_and_input(1)
    eager = layer.forward(acc)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        y = layer.forward(acc)
    for i in range(4):
        y.zero_()
        if i > 1:
            acc.add_(1000 * i)
            eager = layer.forward(acc)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, eager)
    x = layer.features(acc)
    target = torch.randn_like(x)
    losses = []
    for _ in range(3):
        out, mean, rstd = layer.norm(x)
        dy = (out - target) * (2.0 / out.numel())
        losses.append(float((out.double() - target).square().mean()))
        _, dw, db = layer.norm_backward(dy, x, mean, rstd)
        layer.norm_weight -= 20.0 * dw
        layer.norm_bias -= 20.0 * db
    assert losses[2] < losses[1] < losses[0]


def test_features_belong_to_the_stream_that_computes_them(monkeypatch):
    """The features that forward() drops while its kernels still run are memory of the given stream: another
    stream's next allocation cannot be given it."""
    made, used = [], []

    def alloc(like, stream, dtype, *shape):
        made.append((stream, dtype, shape))
        return torch.empty(*shape, dtype=dtype)

    def dequantize(q, scale, out=None, stream=None):
        used.append((out, stream))
        return torch.empty(q.shape) if out is None else out
    monkeypatch.setattr(ifx, "_alloc", alloc)
    monkeypatch.setattr(model, "_alloc", alloc, raising=False)
    monkeypatch.setattr(model, "dequantize_i32", dequantize)
    layer = model.NormPointwise4.__new__(model.NormPointwise4)
    layer.scale = 0.5
    acc = torch.zeros(2, 3, 4, 32, dtype=torch.int32)
    x = layer.features(acc, "a stream")
    assert made == [("a stream", torch.float32, (2, 3, 4, 32))]
    assert len(used) == 1 and used[0][0] is x and used[0][1] == "a stream"


@pytest.mark.gpu
def test_layer_on_a_given_stream():
    """The layer on a stream that is still busy, while the current stream allocates and fills memory: the result
    is that of the calls in order."""
    layer, acc, *_ = layer_and_input()
    res = torch.randn(*acc.shape[:-1], 96, device="cuda").to(torch.bfloat16)
    expect = layer.forward(acc, res)
    work = torch.zeros(1 << 28, device="cuda")
    s = torch.cuda.Stream()
    for given in (s, s.cuda_stream):
        torch.cuda.synchronize()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            for _ in range(8):
                work.add_(1.0)
        y = layer.forward(acc, res, stream=given)
        fill = [torch.full(acc.shape, float("nan"), device="cuda") for _ in range(4)]
        torch.cuda.synchronize()
        assert torch.equal(y, expect)
        del fill


@pytest.mark.gpu
def test_layer_of_no_images():
    """A batch of none gives a result of none, with and without a residual and on a given stream."""
    layer, acc, *_ = layer_and_input(1)
    none = acc[:0]
    shape = (0, *acc.shape[1:3], 96)
    y = layer.forward(none)
    assert y.shape == shape and y.dtype == torch.bfloat16
    res = torch.empty(shape, dtype=torch.float32, device="cuda")
    assert layer.forward(none, res, torch.float32, stream=torch.cuda.Stream()).shape == shape
    x = layer.features(none)
    assert x.shape == none.shape and x.dtype == torch.float32
    out, mean, rstd = layer.norm(x)
    assert out.shape == x.shape and mean.shape == (0, 32)

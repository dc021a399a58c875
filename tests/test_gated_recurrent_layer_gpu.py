"""The recurrent layer's operators together, as the example uses them: gradients of two layers through
torch.autograd against float64, serving in pieces and token by token against one prompt pass."""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                    "gated_recurrent_layer.py")


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("gated_recurrent_layer", PATH)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def plain_conv(u, weight, bias, bounds):
    """SiLU of the convolution of packed documents, document by document."""
    k = weight.shape[1]
    out = []
    for a, b in zip(bounds[:-1], bounds[1:]):
        v = torch.cat([u.new_zeros(k - 1, u.shape[1]), u[a:b]])
        c = sum((weight[:, i] * v[i:i + b - a] for i in range(k)), bias)
        out.append(c * torch.sigmoid(c) if b > a else u[a:b])
    return torch.cat(out)


def plain_recurrence(x, i, r, A, bounds):
    log_a = A * torch.sigmoid(r)
    a, b = log_a.exp(), (-torch.expm1(2 * log_a)).sqrt() * torch.sigmoid(i) * x
    out = []
    for p, q in zip(bounds[:-1], bounds[1:]):
        h = x.new_zeros(x.shape[1])
        for t in range(p, q):
            h = a[t] * h + b[t]
            out.append(h)
    return torch.stack(out)


def rms(v, eps=1e-5):
    return v * (v.square().mean(-1, keepdim=True) + eps).rsqrt()


def plain_model(p, layers, ids, bounds):
    u = t = p["embed"][ids]
    for n in range(layers):
        w = lambda name: p[f"layers.{n}.{name}"]
        c = plain_conv(u @ w("w_x"), w("conv"), w("conv_bias"), bounds)
        i, r = (c @ w("w_gates")).chunk(2, dim=-1)
        y = plain_recurrence(c, i, r, -w("log_rate").exp(), bounds) @ w("w_out")
        z = u @ w("w_z")
        t = t + w("scale") * z * torch.sigmoid(z) * rms(y) * w("post")
        u = rms(t) * w("w")
    return u @ p["head"]


@pytest.mark.parametrize("lengths", [[33, 0, 1, 70], [130], [1, 1, 1, 2]])
def test_gradients_of_two_layers(example, lengths):
    """float32 on the GPU against float64 on the CPU.  Some 30 tensors stand between an input and its
    gradient through two layers and back; the largest rounding of each is that of a matrix product or a
    sum of up to 192 terms, about sqrt(192) 2^-24 = 8e-7 of the size of the values: together 30 * 8e-7 =
    2.5e-5 if all agreed, six deviations of it 1.5e-4; the norms and gates have slopes of the order of
    one.  Held to 1e-3 of an element and the tensor's root mean square."""
    torch.manual_seed(3)
    model = example.Model(11, 96, 2, inner=130, taps=4, dtype=torch.float32).cuda()
    bounds = [0]
    for n in lengths:
        bounds.append(bounds[-1] + n)
    ids = torch.randint(11, (bounds[-1],))
    weight = torch.randn(bounds[-1], 11)
    out = model(ids.cuda(), example.offsets_of(lengths))
    (out * weight.cuda()).sum().backward()
    p = {n: v.detach().double().cpu().requires_grad_() for n, v in model.named_parameters()}
    want = plain_model(p, 2, ids, bounds)
    (want * weight.double()).sum().backward()
    close = lambda got, ref: float(((got.double().cpu() - ref).abs() /
                                    (ref.abs() + ref.square().mean().sqrt() + 1e-30)).max())
    assert close(out.detach(), want.detach()) <= 1e-3
    for n, v in model.named_parameters():
        assert torch.isfinite(v.grad).all(), n
        assert close(v.grad, p[n].grad) <= 1e-3, n


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_trains_and_serves(example, dtype):
    """Served logits differ from the prompt pass's where sums in another order round to the
    neighbouring value: eight rounded bfloat16 tensors a layer, at most 2^-7 of an element each and
    half of that on average if every element did so, sqrt(16) 2^-8 = 0.016 of the logits' size, some
    six deviations of it in the largest: 0.1.  In float32 2^-16 of that, but for the longer sums'
    own roundings."""
    diff = example.main(steps=20, dtype=dtype, quiet=True)
    assert diff <= (0.15 if dtype == "bf16" else 1e-3)

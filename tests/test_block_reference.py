"""The block's float64 reference against closed forms and differences (CPU)."""
import math

import pytest
import torch

import block_reference as ref


def _rand(g, *shape):
    return torch.randn(*shape, generator=g, dtype=torch.float64)


def test_conv_is_the_textbook_convolution():
    g = torch.Generator().manual_seed(0)
    x, w, bias = _rand(g, 2, 9, 3), _rand(g, 3, 4), _rand(g, 3)
    y, tail = ref.conv(x, w, bias, activation="identity")
    full = torch.nn.functional.conv1d(x.transpose(1, 2), w[:, None], bias, padding=3, groups=3)
    assert torch.allclose(y, full[..., :9].transpose(1, 2), atol=1e-12)
    assert torch.equal(tail, x[:, 6:])


def test_conv_in_two_parts_is_the_conv():
    g = torch.Generator().manual_seed(1)
    x, w = _rand(g, 2, 11, 3), _rand(g, 3, 3)
    y, tail = ref.conv(x, w)
    y0, mid = ref.conv(x[:, :1], w)
    y1, end = ref.conv(x[:, 1:], w, state=mid)
    assert torch.allclose(torch.cat([y0, y1], 1), y, atol=1e-14)
    assert torch.equal(end, tail)


def test_scan_with_equal_steps_is_a_geometric_sum():
    T, s, a = 12, 0.3, -0.7
    one = torch.ones(1, T, 1, dtype=torch.float64)
    y, h = ref.scan(one, s * one, torch.full((1, 1), a, dtype=torch.float64), one[..., None],
                    one[..., None], softplus=False)
    r = math.exp(s * a)
    want = [s * (1 - r ** (t + 1)) / (1 - r) for t in range(T)]
    assert torch.allclose(y[0, :, 0], torch.tensor(want, dtype=torch.float64), atol=1e-12)
    assert abs(float(h) - want[-1]) < 1e-12


def test_scan_row_of_length_zero_keeps_its_state():
    g = torch.Generator().manual_seed(2)
    args = [_rand(g, 2, 5, 4), _rand(g, 2, 5, 4), -_rand(g, 4, 3).abs(), _rand(g, 2, 5, 2, 3),
            _rand(g, 2, 5, 2, 3)]
    h0 = _rand(g, 2, 4, 3)
    y, h = ref.scan(*args, h0=h0, lengths=[0, 5])
    assert torch.equal(h[0], h0[0]) and float(y[0].abs().max()) == 0.0
    whole = ref.scan(*args, h0=h0)
    assert torch.equal(y[1], whole[0][1]) and torch.equal(h[1], whole[1][1])


def _against_differences(fn, inputs, names, g):
    """Directional derivatives by central differences; their error is O(step^2)
    plus rounding over step: 1e-5 keeps both below 1e-8 of the sums here."""
    outs = fn(**inputs)
    cot = [_rand(g, *o.shape) for o in outs]
    grads = ref.gradients(fn, inputs, cot)
    for name in names:
        d = _rand(g, *inputs[name].shape)
        step = 1e-5

        def total(k):
            moved = {**inputs, name: inputs[name] + k * step * d}
            return sum(float((o * c).sum()) for o, c in zip(fn(**moved), cot))

        num = (total(1) - total(-1)) / (2 * step)
        assert abs(num - float((grads[name] * d).sum())) < 1e-6 * max(1.0, abs(num)), name


@pytest.mark.parametrize("activation", ["silu", "identity"])
def test_conv_gradients(activation):
    g = torch.Generator().manual_seed(3)
    inputs = dict(x=_rand(g, 2, 7, 3), weight=_rand(g, 3, 4), bias=_rand(g, 3),
                  state=_rand(g, 2, 3, 3), lengths=[7, 2])
    _against_differences(lambda **k: ref.conv(**k, activation=activation), inputs,
                         ("x", "weight", "bias", "state"), g)


@pytest.mark.parametrize("softplus", [True, False])
def test_scan_gradients(softplus):
    g = torch.Generator().manual_seed(4)
    inputs = dict(u=_rand(g, 2, 6, 4), delta=0.3 * _rand(g, 2, 6, 4), A=-_rand(g, 4, 3).abs(),
                  Bm=_rand(g, 2, 6, 2, 3), Cm=_rand(g, 2, 6, 2, 3), D=_rand(g, 4),
                  z=_rand(g, 2, 6, 4), delta_bias=_rand(g, 4), h0=_rand(g, 2, 4, 3),
                  lengths=[6, 3])
    _against_differences(lambda **k: ref.scan(**k, softplus=softplus), inputs,
                         ("u", "delta", "A", "Bm", "Cm", "D", "z", "delta_bias", "h0"), g)

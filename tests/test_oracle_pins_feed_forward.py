"""Pins of the gated feed-forward oracle: closed forms, differences, brute force and hand-worked values."""
import math

import numpy as np
import pytest
import torch

from oracle import feed_forward as ff


@pytest.mark.parametrize("name", ["gelu", "silu"])
def test_activations_against_torch_and_differences(name):
    g = np.concatenate([np.linspace(-9, 9, 301), [0.0, -30.0, 30.0]])
    ref = (torch.nn.functional.gelu if name == "gelu" else torch.nn.functional.silu)(torch.from_numpy(g)).numpy()
    # torch forms 1 + erf, which loses GeLU's far tail below 1e-16 of |g|
    assert np.allclose(ff.act(g, name), ref, rtol=1e-9, atol=1e-14)
    d = 1e-5
    num = (ff.act(g + d, name) - ff.act(g - d, name)) / (2 * d)
    assert np.allclose(ff.act_slope(g, name), num, rtol=1e-7, atol=1e-9)
    # the extrema the kernels' error bounds use
    s = ff.act_slope(np.linspace(-20, 20, 400001), name)
    assert 1.09 < np.max(np.abs(s)) < 1.13
    assert np.max(np.abs(np.diff(s))) / 1e-4 < 0.8


@pytest.mark.parametrize("name", ["gelu", "silu"])
def test_backward_against_differences(name):
    rng = np.random.default_rng(5)
    N, D, H = 4, 5, 6
    x, Wg, Wu = rng.normal(size=(N, D)), rng.normal(size=(H, D)), rng.normal(size=(H, D))
    dh = rng.normal(size=(N, H))
    got = ff.glu_backward(x, Wg, Wu, dh, name)
    assert np.array_equal(got["h"], ff.glu_forward(x, Wg, Wu, name))
    for key, arr in (("dx", x), ("dW_gate", Wg), ("dW_up", Wu)):
        num = np.zeros_like(arr)
        for i in np.ndindex(*arr.shape):
            keep = arr[i]
            loss = []
            for s in (1e-6, -1e-6):
                arr[i] = keep + s
                loss.append(np.sum(dh * ff.glu_forward(x, Wg, Wu, name)))
            arr[i] = keep
            num[i] = (loss[0] - loss[1]) / 2e-6
        assert np.allclose(got[key], num, rtol=1e-6, atol=1e-7), key


def test_act8_hand_worked():
    # m = 1: e = −6 (1 / 2^-6 = 64); 127.5/128 rounds to 128 there, which takes one exponent more
    x = np.zeros((1, 40))
    x[0, 0], x[0, 1], x[0, 2] = 1.0, -0.5, 1.5 / 64
    x[0, 32], x[0, 33] = 127.5 / 128, 0.75 / 64
    codes, scales = ff.act8_pack(x)
    assert scales.tolist() == [[127 - 6, 127 - 6]]
    assert codes[0, :3].tolist() == [64, -32, 2]           # 1.5 rounds to the even 2
    assert codes[0, 32:34].tolist() == [64, 1]             # at e = −7 the largest would be 128
    x[0, 32] = 127.25 / 128
    codes, scales = ff.act8_pack(x)
    assert scales[0, 1] == 127 - 7 and codes[0, 32] == 127
    # zeros, the smallest numbers, an infinity
    x[:] = 0.0
    x[0, 32] = np.inf
    codes, scales = ff.act8_pack(x)
    assert scales.tolist() == [[0, 255]] and not codes.any()
    back = ff.act8_unpack(codes, scales)
    assert np.array_equal(back[0, :32], np.zeros(32)) and np.isnan(back[0, 32:]).all()


def test_act8_error_and_type():
    rng = np.random.default_rng(6)
    x = rng.normal(size=(20, 96)) * np.exp(rng.normal(size=(20, 96)) * 3)
    codes, scales = ff.act8_pack(x)
    back = ff.act8_unpack(codes, scales)
    assert np.abs(codes).max() <= 127 and np.abs(codes).reshape(20, 3, 32).max(2).min() >= 64
    step = np.ldexp(1.0, (scales - 127).astype(int))
    assert (np.abs(back - x).reshape(20, 3, 32).max(2) <= step / 2).all()
    # x̂ is a bfloat16 number
    assert torch.equal(torch.from_numpy(back).to(torch.bfloat16).double(), torch.from_numpy(back))


def test_w4_order_and_scales():
    codes = np.array([[0x8F, 0x10] + [0x88] * 14], dtype=np.uint8)
    w = ff.w4_dequantize(codes, np.array([[0.5]]), 32)
    assert w[0, :4].tolist() == [0.5 * 7, 0.0, 0.5 * -8, 0.5 * -7] and not w[0, 4:].any()


def test_act8_largest_numbers():
    """127.5 · 2^121 and more would round up to 2^128: the exponent stays 121, the codes within ±127."""
    top = 2.0 ** 121
    x = np.zeros((1, 96))
    x[0, 0], x[0, 1], x[0, 2] = 127.25 * top, -126.5 * top, 1.5 * top      # the last that need no care; 126 is even
    x[0, 32], x[0, 33], x[0, 34] = -127.5 * top, 127.0 * top, 0.5 * top    # finfo(bfloat16).min
    x[0, 64], x[0, 65] = float(torch.finfo(torch.float32).max), float(torch.finfo(torch.float32).min)
    codes, scales = ff.act8_pack(x)
    assert scales.tolist() == [[248, 248, 248]]
    assert codes[0, :3].tolist() == [127, -126, 2]
    assert codes[0, 32:35].tolist() == [-127, 127, 0]
    assert codes[0, 64:66].tolist() == [127, -127]
    back = ff.act8_unpack(codes, scales)
    m = np.abs(x).reshape(1, 3, 32).max(2).repeat(32, axis=1)
    assert (np.abs(back - x) <= m / 127).all()
    assert torch.equal(torch.from_numpy(back).to(torch.bfloat16).double(), torch.from_numpy(back))
    assert torch.isfinite(torch.from_numpy(back).to(torch.bfloat16)).all()


def test_gelu_slope_in_the_far_tail():
    """Φ + gφ keeps its digits where Φ is far below one: against Φ's asymptotic series, whose terms alternate, so that
    the error is below the first one left out."""
    g = np.array([-8.0, -8.6875, -10.0, -13.0])
    z = -g
    phi = np.exp(-0.5 * g * g) / math.sqrt(2.0 * math.pi)
    terms = [1.0]
    for k in range(1, 12):
        terms.append(-terms[-1] * (2 * k - 1) / z ** 2)
    tail = phi / z * np.sum(np.broadcast_arrays(*terms[:-1]), axis=0)
    want = tail + g * phi
    assert (np.abs(ff.act_slope(g, "gelu") - want) <= phi / z * np.abs(terms[-1]) + 1e-12 * np.abs(want)).all()

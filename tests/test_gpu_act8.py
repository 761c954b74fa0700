"""8-bit activation checkpoints on the GPU: codes and scale bytes equal to the float64 oracle's, x̂ exactly
what they stand for, and the backward pass from a checkpoint equal to the backward at x̂."""
import numpy as np
import pytest
import torch

from gated_linear_rnn_conv1d_b200 import rglru
from oracle import feed_forward as ff

from _util import f64

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF = torch.bfloat16


def _draw(N, C, dtype, seed=0):
    g = torch.Generator("cpu").manual_seed(seed)
    x = torch.randn(N, C, generator=g) * torch.exp(3 * torch.randn(N, 1, generator=g))
    x[:, ::37] *= 30
    return x.to(dtype)


def _check(x, a):
    codes, scales = ff.act8_pack(f64(x))
    assert torch.equal(a.codes.cpu().long(), torch.from_numpy(codes))
    assert torch.equal(a.scales.cpu().long(), torch.from_numpy(scales))
    back = rglru.act8_unpack(a)
    assert back.dtype == x.dtype
    assert np.array_equal(f64(back), ff.act8_unpack(codes, scales), equal_nan=True)


@pytest.mark.parametrize("dtype", [BF, torch.float32])
@pytest.mark.parametrize("N,C", [(1, 8), (1, 32), (3, 40), (7, 264), (64, 64), (33, 1032), (5, 24)])
def test_codes_and_values(N, C, dtype):
    x = _draw(N, C, dtype, seed=N * C)
    _check(x, rglru.act8_pack(x.to(DEV)))


@pytest.mark.parametrize("dtype", [BF, torch.float32])
def test_borders(dtype):
    """Largest magnitudes just below, at and above the places where the exponent changes; ties; the ends of
    the type's range; zeros of both signs; groups that are not finite."""
    x = torch.zeros(40, 72)
    tops = [1.0, 127.0 / 128, 127.25 / 128, 127.5 / 128, 255.0 / 256, 2.0, 1.9921875, 1.984375, 3.0e38, 1e-30,
            2.0 ** -120, 2.0 ** -121, 2.0 ** -122, 1.5 * 2.0 ** -126, 2.0 ** -127, 2.0 ** -133, 2.0 ** -149]
    for i, t in enumerate(tops):
        x[i, 0], x[i, 40] = t, -t
        x[i, 1:32] = t * torch.arange(-15, 16) / 128 * 1.5
        x[i, 64:72] = t / 3
    x[20] = -0.0
    x[21, 3], x[22, 33], x[23, 71] = float("inf"), float("-inf"), float("nan")
    x[24, 0], x[24, 32] = float("nan"), 1.0
    x = x.to(dtype)
    _check(x, rglru.act8_pack(x.to(DEV)))


@pytest.mark.parametrize("dtype", [BF, torch.float32])
@pytest.mark.parametrize("C", [64, 40])
def test_neighbours_untouched_and_rank(dtype, C):
    x = _draw(6, C, dtype, seed=2).to(DEV)
    a = rglru.act8_pack(x.view(2, 3, C))
    assert a.codes.shape == (2, 3, C) and a.scales.shape == (2, 3, -(-C // 32))
    buf = torch.full((6 * C + 64,), -7.0, dtype=dtype, device=DEV)
    rglru.act8_unpack(a, x=buf[32:32 + 6 * C].view(2, 3, C))
    assert (buf[:32] == -7).all() and (buf[32 + 6 * C:] == -7).all()
    assert torch.equal(buf[32:32 + 6 * C].view(6, C), rglru.act8_unpack(rglru.act8_pack(x)))


def test_many_rows():
    """More than one block's items, against the same rows packed a few at a time."""
    x = _draw(3001, 104, BF, seed=3).to(DEV)
    a = rglru.act8_pack(x)
    b = rglru.act8_unpack(a)
    for lo in range(0, 3001, 500):
        part = rglru.act8_pack(x[lo:lo + 500].contiguous())
        assert torch.equal(part.codes, a.codes[lo:lo + 500]) and torch.equal(part.scales, a.scales[lo:lo + 500])
        assert torch.equal(rglru.act8_unpack(part), b[lo:lo + 500])


@pytest.mark.parametrize("C", [65536, 65528])  # whole groups in a row, and a short one
def test_offsets_past_32_bits(C):
    few = _draw(8, C, BF, seed=4).to(DEV)
    want = rglru.act8_pack(few)
    a = rglru.act8_pack(few.repeat(5000, 1))
    assert torch.equal(a.codes[-8:], want.codes) and torch.equal(a.scales[-8:], want.scales)
    assert torch.equal(a.codes[:8], want.codes) and torch.equal(a.scales[:8], want.scales)
    back = rglru.act8_unpack(a)
    assert torch.equal(back[-8:], rglru.act8_unpack(want)) and torch.equal(back[:8], back[-8:])


@pytest.mark.parametrize("N,D,H", [(1, 40, 72), (30, 264, 136), (300, 136, 520)])
def test_training_step_through_a_checkpoint(N, D, H):
    """The operators as a layer uses them: forward, the checkpoint in the place of x, backward from it; bit for
    bit the backward at x̂, and h again from x̂."""
    g = torch.Generator("cpu").manual_seed(N)
    x = _draw(N, D, BF, seed=N)
    x = (x / x.float().abs().amax(1, keepdim=True).clamp(min=1e-3)).to(BF).to(DEV)
    Wg, Wu = ((torch.randn(H, D, generator=g) / D ** 0.5).to(BF).to(DEV) for _ in range(2))
    dh = torch.randn(N, H, generator=g).to(BF).to(DEV)
    h = rglru.glu_forward(Wg, Wu, x)
    kept = rglru.act8_pack(x)
    xhat = rglru.act8_unpack(kept)
    # one rounding of at most 1/127 of a group's largest magnitude
    pad = torch.nn.functional.pad(f64t(x), (0, -D % 32)).view(N, -1, 32).abs().amax(2)
    assert ((f64t(xhat) - f64t(x)).abs() <= pad.repeat_interleave(32, 1)[:, :D] / 127).all()
    ws = torch.full((rglru.glu_backward_workspace_bytes(N, D, H, True),), 0xFF, dtype=torch.uint8, device=DEV)
    got = rglru.glu_backward(Wg, Wu, kept, dh, want_h=True, workspace=ws)
    want = rglru.glu_backward(Wg, Wu, xhat, dh, want_h=True)
    assert all(torch.equal(got[k], want[k]) for k in want)
    assert torch.equal(got["h"], rglru.glu_forward(Wg, Wu, xhat))
    assert h.shape == got["h"].shape
    assert rglru.workspace_status(None) == 0


def f64t(t):
    return t.double().cpu()


def test_rglru_backward_from_a_checkpoint():
    """Any operator's input can be kept this way: the RG-LRU's own backward at x̂."""
    from gated_linear_rnn_conv1d_b200 import inputs
    w = inputs.make_forward(2, 70, 136, BF, seed=5)
    p = rglru.Params.from_host(w.params)
    x = w.x.to(DEV)
    kept = rglru.act8_pack(x)
    xhat = rglru.act8_unpack(kept)
    y, _, _ = rglru.forward(p, xhat)
    dy = torch.ones_like(y)
    a = rglru.backward(p, rglru.act8_unpack(kept), y, dy)
    b = rglru.backward(p, xhat, y, dy)
    assert torch.equal(a["dx"], b["dx"]) and torch.equal(a["dW_a"], b["dW_a"])


def test_captured_and_replayed():
    xin = _draw(9, 72, BF, seed=6).to(DEV)
    graph = torch.cuda.CUDAGraph()
    rglru.act8_unpack(rglru.act8_pack(xin))
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        out = rglru.act8_unpack(rglru.act8_pack(xin))
    x2 = _draw(9, 72, BF, seed=7).to(DEV)
    xin.copy_(x2)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, rglru.act8_unpack(rglru.act8_pack(x2)))


def test_binding_refusals():
    x = _draw(4, 64, BF).to(DEV)
    a = rglru.act8_pack(x)
    cases = [
        (TypeError, lambda: rglru.act8_pack(x.half())),
        (ValueError, lambda: rglru.act8_pack(x.t())),
        (rglru._abi.RGLRUError, lambda: rglru.act8_pack(x[:, :60].contiguous())),
        (rglru._abi.RGLRUError, lambda: rglru.act8_pack(x[:0])),
        (ValueError, lambda: rglru.act8_unpack(rglru.Act8(a.codes, a.scales[:, :1].contiguous(), BF))),
        (TypeError, lambda: rglru.act8_unpack(rglru.Act8(a.codes.float(), a.scales, BF))),
        (TypeError, lambda: rglru.act8_unpack(a, x=torch.empty(4, 64, device=DEV))),
        (ValueError, lambda: rglru.glu_backward(torch.zeros(8, 72, dtype=BF, device=DEV),
                                                torch.zeros(8, 72, dtype=BF, device=DEV), a,
                                                torch.zeros(4, 8, dtype=BF, device=DEV))),
    ]
    for i, (err, call) in enumerate(cases):
        with pytest.raises(err):
            call()
            raise AssertionError(f"case {i} was taken")


@pytest.mark.parametrize("dtype", [BF, torch.float32])
@pytest.mark.parametrize("C", [64, 72])
def test_largest_numbers(C, dtype):
    """The end of the type's range, where the next power of two is no finite number: every top from 126 · 2^121 on,
    both signs, with smaller neighbours; codes, scales and x̂ as the oracle's, x̂ finite and within 1/127 of the top."""
    info = torch.finfo(dtype)
    tops = [126 * 2.0 ** 121, 126.5 * 2.0 ** 121, 127 * 2.0 ** 121, 127.5 * 2.0 ** 121, info.max, info.min]
    if dtype is torch.float32:
        tops += [127.25 * 2.0 ** 121, 127.5 * 2.0 ** 121 * (1 - 2.0 ** -24), 127.75 * 2.0 ** 121]
    x = torch.zeros(2 * len(tops), C, dtype=torch.float64)
    for i, t in enumerate(tops + [-t for t in tops]):
        x[i, 3] = t
        x[i, 32:64] = t * torch.arange(1, 33, dtype=torch.float64) / 32
        x[i, 64:] = t / 2
    x = x.to(dtype)
    a = rglru.act8_pack(x.to(DEV))
    _check(x, a)
    back = rglru.act8_unpack(a)
    assert torch.isfinite(back).all() and (a.codes >= -127).all()
    m = torch.nn.functional.pad(f64t(x), (0, -C % 32)).view(len(x), -1, 32).abs().amax(2)
    assert ((f64t(back) - f64t(x)).abs() <= m.repeat_interleave(32, 1)[:, :C] / 127).all()


def test_backward_with_masked_channels_of_the_lowest_number():
    """finfo.min in channels that no weight reads: the gradients from the checkpoint are finite, as those at x."""
    N, D, H = 40, 72, 136
    g = torch.Generator("cpu").manual_seed(8)
    x = torch.randn(N, D, generator=g).to(BF)
    x[:, 32:64] = torch.finfo(BF).min
    Wg, Wu = ((torch.randn(H, D, generator=g) / D ** 0.5).to(BF) for _ in range(2))
    Wg[:, 32:64], Wu[:, 32:64] = 0, 0
    dh = torch.randn(N, H, generator=g).to(BF)
    r = rglru.glu_backward(Wg.to(DEV), Wu.to(DEV), rglru.act8_pack(x.to(DEV)), dh.to(DEV), want_h=True)
    keep = torch.ones(D, dtype=torch.bool)
    keep[32:64] = False
    assert torch.isfinite(r["dx"]).all() and torch.isfinite(r["h"]).all()
    assert torch.isfinite(r["dW_gate"][:, keep]).all() and torch.isfinite(r["dW_up"][:, keep]).all()


def test_rglru_backward_at_the_values_of_a_checkpoint():
    """The RG-LRU's backward from a checkpoint against the float64 oracle's at x̂, which the oracle forms from x itself;
    tolerances as of the backward's own tests."""
    import oracle
    from gated_linear_rnn_conv1d_b200 import inputs
    from test_gpu_backward import _tol
    w = inputs.make_forward(2, 70, 136, BF, seed=5)
    p = rglru.Params.from_host(w.params)
    codes, scales = ff.act8_pack(f64(w.x).reshape(140, 136))
    xhat = ff.act8_unpack(codes, scales).reshape(2, 70, 136)
    kept = rglru.act8_unpack(rglru.act8_pack(w.x.to(DEV)))
    y, _, _ = rglru.forward(p, kept)
    dy = torch.randn(2, 70, 136, generator=torch.Generator("cpu").manual_seed(6)).to(BF)
    got = rglru.backward(p, kept, y, dy.to(DEV))
    ref = oracle.rglru_backward(xhat, w.params.conv_w, w.params.conv_b, w.params.W_a, w.params.b_a, w.params.W_x,
                                w.params.b_x, w.params.Lambda, dy)
    for k, v in ref.items():
        err = oracle.max_rel_error(f64(got[k]), v)
        print(f"{k}: {err:.2e}")
        assert err <= _tol(k), k

"""The gated feed-forward block on the GPU, forward and backward, against the float64 oracle; the bounds are
derived in _glu.py."""
import subprocess
import sys
from pathlib import Path

import numpy as np
import pytest
import torch

from gated_linear_rnn_conv1d_b200 import rglru
from oracle import feed_forward as ff

from _glu import HALF, TINY, backward_bounds, forward_bound
from _util import f64

pytestmark = pytest.mark.gpu
DEV = "cuda"
ROOT = Path(__file__).resolve().parent.parent
BF = torch.bfloat16


def _draw(N, D, H, seed=0, scale=1.0):
    g = torch.Generator("cpu").manual_seed(1000 + seed)
    x = torch.randn(N, D, generator=g).to(BF)
    Wg = (torch.randn(H, D, generator=g) * (scale / D ** 0.5)).to(BF)
    Wu = (torch.randn(H, D, generator=g) / D ** 0.5).to(BF)
    dh = torch.randn(N, H, generator=g).to(BF)
    return x, Wg, Wu, dh


def _guarded(shape, dtype=BF):
    """A tensor of that shape inside a larger buffer of a known pattern, and a check that the rest of it is
    as it was."""
    n = int(np.prod(shape))
    buf = torch.full((n + 2048,), -7.0, dtype=dtype, device=DEV)
    view = buf[1024:1024 + n].view(shape)

    def untouched():
        return bool((buf[:1024] == -7.0).all() and (buf[1024 + n:] == -7.0).all())

    return view, untouched


def _check_forward(x, Wg, Wu, act, h):
    ref = ff.glu_forward(f64(x), f64(Wg), f64(Wu), act)
    bound = forward_bound(f64(x), f64(Wg), f64(Wu), lambda g: ff.act(g, act), ref)
    err = np.abs(f64(h) - ref)
    print(f"worst error / bound {np.max(err / bound):.3f}")
    assert (err <= bound).all()


def _check_backward(x, Wg, Wu, dh, act, got):
    X, G, U, DH = f64(x), f64(Wg), f64(Wu), f64(dh)
    ref = ff.glu_backward(X, G, U, DH, act)
    bounds = backward_bounds(X, G, U, DH, lambda g: ff.act(g, act), lambda g: ff.act_slope(g, act))
    bounds["h"] = forward_bound(X, G, U, lambda g: ff.act(g, act), ref["h"])
    for k, b in bounds.items():
        if got[k] is None:
            continue
        err = np.abs(f64(got[k]) - ref[k])
        print(f"{k}: worst error / bound {np.max(err / b):.3f}")
        assert (err <= b).all(), k


# one token; one over a vector, a tile and a pair of tiles; widths below, at and past the tiles' 64,
# 128 and 256; several tiles a CTA pair (9 × 21 tiles on 74 pairs)
SHAPES = [(1, 8, 8), (1, 264, 776), (2, 72, 136), (3, 512, 128), (5, 1032, 264), (8, 256, 1000), (9, 136, 72),
          (16, 264, 520), (17, 64, 264), (23, 520, 136), (32, 1032, 392), (33, 520, 136), (64, 128, 256), (65, 264, 264), (129, 72, 520),
          (256, 264, 136), (257, 328, 392), (513, 136, 264), (2100, 72, 2600)]


@pytest.mark.parametrize("N,D,H", SHAPES)
@pytest.mark.parametrize("act", ["gelu", "silu"])
def test_forward(N, D, H, act):
    x, Wg, Wu, _ = _draw(N, D, H, seed=N)
    h, untouched = _guarded((N, H))
    out = rglru.glu_forward(Wg.to(DEV), Wu.to(DEV), x.to(DEV), activation=act, h=h)
    assert rglru.workspace_status(None) == 0
    assert out is h and untouched()
    _check_forward(x, Wg, Wu, act, h)


# one token to 32: the channels of a block of the streaming kernel are two, four and nine granules of eight
@pytest.mark.parametrize("N,D,H", [(1, 72, 4744), (8, 200, 9480), (3, 136, 20008), (9, 72, 4744), (16, 328, 20008), (17, 136, 9480),
                                   (24, 264, 4744), (25, 72, 20008), (27, 136, 5000),
                                   (32, 520, 9480)])
def test_few_tokens_of_many_channels(N, D, H):
    x, Wg, Wu, _ = _draw(N, D, H, seed=N)
    h, untouched = _guarded((N, H))
    rglru.glu_forward(Wg.to(DEV), Wu.to(DEV), x.to(DEV), activation="gelu", h=h)
    assert untouched()
    _check_forward(x, Wg, Wu, "gelu", h)


@pytest.mark.parametrize("N,D,H", SHAPES)
@pytest.mark.parametrize("act", ["gelu", "silu"])
def test_backward(N, D, H, act):
    x, Wg, Wu, dh = _draw(N, D, H, seed=N + 7)
    # the workspace's old contents are NaN in bf16 and must not be read
    ws = torch.full((rglru.glu_backward_workspace_bytes(N, D, H),), 0xFF, dtype=torch.uint8, device=DEV)
    got = rglru.glu_backward(Wg.to(DEV), Wu.to(DEV), x.to(DEV), dh.to(DEV), activation=act, want_h=True, workspace=ws)
    assert rglru.workspace_status(None) == 0
    _check_backward(x, Wg, Wu, dh, act, got)


# sums cut into pieces: dx's over the channels (few tokens, long H), dW's over the tokens (small weights),
# with a last piece that is shorter, and with columns that fill no tile
@pytest.mark.parametrize("N,D,H", [(17, 72, 4104), (1, 264, 3336), (40, 520, 2056), (5000, 40, 72), (2200, 264, 136)])
def test_backward_of_long_sums(N, D, H):
    x, Wg, Wu, dh = _draw(N, D, H, seed=N + 3)
    plain = 2 * -(-2 * N * (-(-H // 64) * 64) // 256) * 256
    need = rglru.glu_backward_workspace_bytes(N, D, H)
    assert need > plain  # room for the pieces
    ws = torch.full((need,), 0xFF, dtype=torch.uint8, device=DEV)
    dev = [t.to(DEV) for t in (Wg, Wu, x, dh)]
    got = rglru.glu_backward(*dev, want_h=True, workspace=ws)
    assert rglru.workspace_status(None) == 0
    _check_backward(x, Wg, Wu, dh, "gelu", got)
    for _ in range(3):  # the pieces are added in order
        again = rglru.glu_backward(*dev, want_h=True)
        assert all(torch.equal(again[k], got[k]) for k in got)


# few tokens and large weights: where D is a multiple of 64 dW leaves in boxes of 32 × 64, which the last rows do not
# fill, nor the last columns their tiles
@pytest.mark.parametrize("N,D,H", [(40, 1088, 2600), (300, 2048, 1288), (17, 512, 4872), (384, 1344, 1800),
                                   (100, 1032, 2600), (512, 1280, 1800)])
def test_backward_of_large_weights(N, D, H):
    x, Wg, Wu, dh = _draw(N, D, H, seed=N + 5)
    ws = torch.full((rglru.glu_backward_workspace_bytes(N, D, H),), 0xFF, dtype=torch.uint8, device=DEV)
    dev = [t.to(DEV) for t in (Wg, Wu, x, dh)]
    out = {k: _guarded(s) for k, s in (("dx", (N, D)), ("dW_gate", (H, D)), ("dW_up", (H, D)), ("h", (N, H)))}
    code = rglru._abi.load().rglru_glu_backward(
        *(t.data_ptr() for t in dev), *(out[k][0].data_ptr() for k in out), N, D, H, 0, ws.data_ptr(), ws.numel(),
        torch.cuda.current_stream().cuda_stream)
    assert code == 0 and rglru.workspace_status(None) == 0
    assert all(untouched() for _, untouched in out.values())
    _check_backward(x, Wg, Wu, dh, "gelu", {k: v[0] for k, v in out.items()})
    again = rglru.glu_backward(*dev, want_h=True)
    assert all(torch.equal(again[k], out[k][0]) for k in out)


def test_shapes_of_any_rank():
    x, Wg, Wu, dh = _draw(6, 40, 72)
    w = (Wg.to(DEV), Wu.to(DEV))
    flat = rglru.glu_forward(*w, x.to(DEV))
    back = rglru.glu_backward(*w, x.to(DEV), dh.to(DEV))
    for lead in ((2, 3), (1, 6, 1)):
        h = rglru.glu_forward(*w, x.to(DEV).view(*lead, 40))
        assert h.shape == (*lead, 72) and torch.equal(h.view(6, 72), flat)
        r = rglru.glu_backward(*w, x.to(DEV).view(*lead, 40), dh.to(DEV).view(*lead, 72))
        assert r["dx"].shape == (*lead, 40) and r["h"] is None
        assert all(torch.equal(r[k].view_as(back[k]), back[k]) for k in ("dx", "dW_gate", "dW_up"))
    one = rglru.glu_forward(*w, x[0].to(DEV))
    assert one.shape == (72,)


@pytest.mark.parametrize("act", ["gelu", "silu"])
def test_far_pre_activations(act):
    """Pre-activations of tens and hundreds: both tails of the activation and its slope."""
    x, Wg, Wu, dh = _draw(130, 64, 136, seed=3, scale=60.0)
    w = (Wg.to(DEV), Wu.to(DEV))
    _check_forward(x, Wg, Wu, act, rglru.glu_forward(*w, x.to(DEV), activation=act))
    _check_backward(x, Wg, Wu, dh, act, rglru.glu_backward(*w, x.to(DEV), dh.to(DEV), activation=act, want_h=True))


@pytest.mark.parametrize("N", [1, 3, 12, 300])
def test_non_finite_rows_stay_in_their_rows(N):
    x, Wg, Wu, dh = _draw(N, 72, 136, seed=4)
    w = (Wg.to(DEV), Wu.to(DEV))
    clean = rglru.glu_forward(*w, x.to(DEV))
    r0 = rglru.glu_backward(*w, x.to(DEV), dh.to(DEV))
    bad = x.clone()
    bad[N // 2, 5] = float("nan")
    h = rglru.glu_forward(*w, bad.to(DEV))
    r = rglru.glu_backward(*w, bad.to(DEV), dh.to(DEV))
    keep = torch.arange(N) != N // 2
    assert torch.isnan(h[N // 2]).all() and torch.equal(h[keep], clean[keep])
    assert torch.isnan(r["dx"][N // 2]).all() and torch.equal(r["dx"][keep], r0["dx"][keep])
    assert torch.isnan(r["dW_gate"]).all()


def test_zero_rows_and_zero_gradients():
    x, Wg, Wu, dh = _draw(140, 64, 72, seed=5)
    x[::2] = 0
    dh[1::2] = 0
    w = (Wg.to(DEV), Wu.to(DEV))
    h = rglru.glu_forward(*w, x.to(DEV))
    assert not h[::2].any()
    r = rglru.glu_backward(*w, x.to(DEV), dh.to(DEV))
    assert not r["dx"][1::2].any()
    # x = 0 gives u = 0 and act(0) = 0: nothing reaches the weights or x
    assert not r["dx"][::2].any() and not r["dW_gate"].any() and not r["dW_up"].any()


def test_gradient_against_differences_of_the_kernel():
    """Along one direction of x, at float32-sized steps of a bf16 input the loss cannot be differenced
    finely; a step of 2^-4 of unit inputs with the second-order term cancelled leaves a third-order one."""
    x, Wg, Wu, dh = _draw(64, 128, 256, seed=6)
    w = (Wg.to(DEV), Wu.to(DEV))
    v = torch.randn(64, 128, generator=torch.Generator().manual_seed(9)).sign().to(BF) * 2 ** -4
    xb = (x * 8).round().clamp(-24, 24) / 8  # so that x ± v are bf16 numbers
    r = rglru.glu_backward(*w, xb.to(DEV), dh.to(DEV), activation="silu")
    want = float((f64(r["dx"]) * f64(v)).sum())
    loss = [float((f64(dh) * f64(rglru.glu_forward(*w, (xb + s * v).to(DEV), activation="silu"))).sum())
            for s in (1, -1)]
    num = (loss[0] - loss[1]) / 2
    # each h is rounded to bf16: N·H independent errors of at most 2^-8 |h|, about 2^-8/√3 each; five of
    # their standard deviations, and the third-order term, which the float64 oracle gives exactly
    exact = [float((f64(dh) * ff.glu_forward(f64(xb + s * v), f64(Wg), f64(Wu), "silu")).sum()) for s in (1, -1)]
    third = abs((exact[0] - exact[1]) / 2 - float((ff.glu_backward(f64(xb), f64(Wg), f64(Wu), f64(dh), "silu")["dx"]
                                                    * f64(v)).sum()))
    h = ff.glu_forward(f64(xb), f64(Wg), f64(Wu), "silu")
    noise = 5 * 2 ** -8 / 3 ** 0.5 * np.sqrt(np.sum((f64(dh) * h) ** 2))
    slack = 5 * 2 ** -7 / 3 ** 0.5 * np.sqrt(np.sum((f64(r["dx"]) * f64(v)) ** 2))
    print(num, want, third, noise, slack)
    assert abs(num - want) <= third + noise + slack


@pytest.mark.parametrize("N", [1, 7, 200])
def test_streams_and_two_calls_at_once(N):
    x, Wg, Wu, dh = (t.to(DEV) for t in _draw(N, 264, 520, seed=8))
    want = rglru.glu_forward(Wg, Wu, x), rglru.glu_backward(Wg, Wu, x, dh, want_h=True)
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    got = []
    for _ in range(3):
        for s in (a, b):
            got.append((rglru.glu_forward(Wg, Wu, x, stream=s), rglru.glu_backward(Wg, Wu, x, dh, want_h=True, stream=s)))
    torch.cuda.synchronize()
    for h, r in got:
        assert torch.equal(h, want[0])
        assert all(torch.equal(r[k], want[1][k]) for k in want[1])


@pytest.mark.parametrize("N", [1, 40, 300])
def test_captured_and_replayed(N):
    x, Wg, Wu, dh = (t.to(DEV) for t in _draw(N, 136, 264, seed=10))
    rglru.glu_backward(Wg, Wu, x, dh), rglru.glu_forward(Wg, Wu, x)  # first calls outside the capture
    torch.cuda.synchronize()
    xin, din = x.clone(), dh.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        h = rglru.glu_forward(Wg, Wu, xin)
        r = rglru.glu_backward(Wg, Wu, xin, din)
    for seed in (11, 12):
        x2, _, _, d2 = (t.to(DEV) for t in _draw(N, 136, 264, seed=seed))
        xin.copy_(x2)
        din.copy_(d2)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(h, rglru.glu_forward(Wg, Wu, x2))
        want = rglru.glu_backward(Wg, Wu, x2, d2)
        assert all(torch.equal(r[k], want[k]) for k in ("dx", "dW_gate", "dW_up"))
    assert rglru.workspace_status(None) == 0


def test_binding_refusals():
    x, Wg, Wu, dh = (t.to(DEV) for t in _draw(6, 64, 72))
    cases = [
        (TypeError, lambda: rglru.glu_forward(Wg, Wu, x.float())),
        (TypeError, lambda: rglru.glu_forward(Wg.float(), Wu, x)),
        (ValueError, lambda: rglru.glu_forward(Wg, Wu[:64].contiguous(), x)),
        (ValueError, lambda: rglru.glu_forward(Wg, Wu, x[:, :56].contiguous())),
        (ValueError, lambda: rglru.glu_forward(Wg, Wu, x.t().contiguous().t())),
        (ValueError, lambda: rglru.glu_forward(Wg, Wu, x, activation="relu")),
        (ValueError, lambda: rglru.glu_forward(Wg, Wu, x, h=torch.empty(6, 64, dtype=BF, device=DEV))),
        (ValueError, lambda: rglru.glu_forward(Wg, Wu.cpu(), x)),
        (ValueError, lambda: rglru.glu_backward(Wg, Wu, x, dh[:5].contiguous())),
        (ValueError, lambda: rglru.glu_backward(Wg, Wu, x, dh, workspace=torch.empty(256, dtype=torch.uint8, device=DEV))),
        (rglru._abi.RGLRUError, lambda: rglru.glu_forward(Wg, Wu, x[:0])),
        (rglru._abi.RGLRUError, lambda: rglru.glu_forward(x, x, x, h=x.view(-1)[:36].view(6, 6))),
        (rglru._abi.RGLRUError, lambda: rglru.glu_forward(Wg[:64], Wu[:64], x, h=x)),
        (rglru._abi.RGLRUError, lambda: rglru.glu_forward(Wg[:, :60].contiguous(), Wu[:, :60].contiguous(),
                                                          x[:, :60].contiguous())),
    ]
    for i, (err, call) in enumerate(cases):
        with pytest.raises(err):
            call()
            raise AssertionError(f"case {i} was taken")


def test_weights_from_the_call_before():
    """A call's weights are the output of the call before, in the same memory every time: what the kernel may fetch
    before that call has ended must not be what it reads."""
    x, Wg, Wu, _ = (t.to(DEV) for t in _draw(16, 264, 1032, seed=2))
    z = [_draw(n, 1032, 8, seed=n)[0].to(DEV) for n in (4, 40)]
    W = torch.empty(16, 1032, dtype=BF, device=DEV)
    xs = [(x * (1 + i / 8)).to(BF) for i in range(12)]
    want = []
    for t in xs:
        rglru.glu_forward(Wg, Wu, t, h=W)
        torch.cuda.synchronize()
        want.append([rglru.glu_forward(W, W, v) for v in z])
        torch.cuda.synchronize()
    for _ in range(4):
        got = []
        for t in xs:
            rglru.glu_forward(Wg, Wu, t, h=W)
            got.append([rglru.glu_forward(W, W, v) for v in z])
        assert all(torch.equal(g, w) for a, b in zip(got, want) for g, w in zip(a, b))


def test_offsets_past_32_bits():
    """More than 2^31 elements in h, and bytes in a weight: the last rows are what the same rows give alone."""
    N, D, H = 40000, 16, 65536
    x, Wg, Wu, _ = (t.to(DEV) for t in _draw(8, D, H))
    tokens = x.repeat(N // 8, 1)
    h = rglru.glu_forward(Wg, Wu, tokens)
    small = rglru.glu_forward(Wg, Wu, tokens[:256].contiguous())
    assert torch.equal(h[-256:], small)
    _check_forward(x, Wg, Wu, "gelu", h[-8:])
    # gradients reach the first and the last tokens only: dW is theirs
    dh = torch.zeros(N, H, dtype=BF, device=DEV)
    g = torch.randn(8, H, generator=torch.Generator("cpu").manual_seed(5)).to(BF).to(DEV)
    dh[:4], dh[-4:] = g[:4], g[4:]
    got = rglru.glu_backward(Wg, Wu, tokens, dh)
    assert rglru.workspace_status(None) == 0
    assert (got["dx"][4:-4] == 0).all()
    got = {"dx": torch.cat([got["dx"][:4], got["dx"][-4:]]), "dW_gate": got["dW_gate"], "dW_up": got["dW_up"], "h": None}
    _check_backward(x, Wg, Wu, g, "gelu", got)
    del h, dh, tokens
    # the streaming kernel: 65536 rows of 32776 inputs, 4.3 GB a matrix
    D = 32776
    W = torch.randn(64, D, generator=torch.Generator("cpu").manual_seed(6)).div(D ** 0.5).to(BF).to(DEV)
    Wg, Wu = W.repeat(1024, 1), W.roll(1, 0).repeat(1024, 1)
    z = torch.randn(3, D, generator=torch.Generator("cpu").manual_seed(7)).to(BF).to(DEV)
    h = rglru.glu_forward(Wg, Wu, z).view(3, 1024, 64)
    assert torch.equal(h, rglru.glu_forward(W, W.roll(1, 0), z).unsqueeze(1).expand_as(h))


def test_outputs_as_torch_makes_them():
    """On the inputs' device, outside autograd, inference tensors where torch's own would be."""
    x, Wg, Wu, dh = (t.to(DEV) for t in _draw(5, 64, 72))
    calls = lambda: [rglru.glu_forward(Wg, Wu, x), *rglru.glu_backward(Wg, Wu, x, dh, want_h=True).values(),
                     rglru.act8_pack(x).codes, rglru.act8_unpack(rglru.act8_pack(x))]
    want = calls()
    Wg.requires_grad_(), x.requires_grad_()
    plain = calls()
    with torch.inference_mode():
        inside = calls()
    for a, b, c in zip(want, plain, inside):
        assert torch.equal(a, b) and torch.equal(a, c) and a.device == x.device
        assert not (a.requires_grad or b.requires_grad or a.is_inference()) and c.is_inference()


FIRST = """
import sys, torch
from gated_linear_rnn_conv1d_b200 import rglru
BF = torch.bfloat16
r = lambda *s: torch.randn(*s, device="cuda", dtype=BF)
Wg, Wu, x, few, dh = r(136, 64), r(136, 64), r(70, 64), r(3, 64), r(70, 136)
w = rglru.W4Weight(torch.zeros(136, 32, dtype=torch.uint8, device="cuda"), r(136, 2), 32)
torch.cuda.synchronize()
def work():
    a = rglru.act8_pack(x)
    return [rglru.glu_forward(Wg, Wu, few), rglru.glu_forward(Wg, Wu, x), *rglru.glu_backward(Wg, Wu, x, dh).values(),
            a.codes, rglru.act8_unpack(a), rglru.glu_backward(Wg, Wu, a, dh)["dx"], rglru.w4_linear(w, few),
            rglru.w4_glu(w, w, few), rglru.w4_quantize(Wg, 32).codes]
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    got = work()
graph.replay()
torch.cuda.synchronize()
want = work()
torch.cuda.synchronize()
assert all(g is None or torch.equal(g, v) for g, v in zip(got, want))
print("captured")
"""


def test_first_calls_may_be_captured():
    """Nothing that a first call sets up stands in the way of a capture."""
    out = subprocess.run([sys.executable, "-c", FIRST], capture_output=True, text=True, timeout=300, cwd=ROOT)
    assert out.returncode == 0 and "captured" in out.stdout, out.stdout + out.stderr


TRANSFORMS = """
import torch
from gated_linear_rnn_conv1d_b200 import rglru
BF = torch.bfloat16
r = lambda *s: torch.randn(*s, device="cuda", dtype=BF)
W, x, dh = r(72, 64), r(3, 64), r(3, 72)
w4 = rglru.W4Weight(torch.zeros(72, 32, dtype=torch.uint8, device="cuda"), r(72, 1), 64)
calls = {
    "glu_forward": lambda v: rglru.glu_forward(W, W, v),
    "glu_forward's weights": lambda v: rglru.glu_forward(v.expand(72, 64).contiguous() if v.dim() == 1 else v, W, x),
    "glu_backward": lambda v: rglru.glu_backward(W, W, v, dh if v.dim() == 2 else dh[0]),
    "act8_pack": rglru.act8_pack,
    "act8_unpack": lambda v: rglru.act8_unpack(rglru.Act8(v.to(torch.int8), v[..., :2].to(torch.uint8), BF)),
    "w4_quantize": lambda v: rglru.w4_quantize(v if v.dim() == 2 else v.expand(8, 64).contiguous(), 64),
    "w4_linear": lambda v: rglru.w4_linear(w4, v),
    "w4_glu": lambda v: rglru.w4_glu(w4, w4, v),
}
for name, call in calls.items():
    def inside(v):
        try:
            call(v)
        except (RuntimeError, ValueError, TypeError) as e:
            seen.append(str(e))
        return v.float().sum()
    for run in (lambda: torch.vmap(inside)(x), lambda: torch.func.grad(inside)(x),
                lambda: torch.func.jvp(inside, (x,), (x,))):
        seen = []
        run()
        assert len(seen) == 1, name
want = rglru.glu_forward(W, W, x)
torch.cuda.synchronize()
assert torch.isfinite(want).all()
print("refused")
"""


def test_transforms_of_torch_func_are_refused():
    """Inside vmap, grad and jvp a tensor has no memory to hand over: every operator raises an ordinary error."""
    out = subprocess.run([sys.executable, "-c", TRANSFORMS], capture_output=True, text=True, timeout=300, cwd=ROOT)
    assert out.returncode == 0 and "refused" in out.stdout, out.stdout + out.stderr


# What the kernels' activations may be off by, relative to their own size, for −13 ≤ g: GeLU's Φ(−|g|) is fitted to
# 7.3e-5 of its value; z = g²/2·log₂e (g·log₂e for SiLU) is rounded twice, 2^-23 of up to 122, which is 1e-5 in the
# exponential; the hardware's exponential and reciprocal add 2^-22 each and ten float32 operations 2^-24 each: 2e-4 with
# room. The same holds for the two terms of the slope, whose sum may cancel. Below −13 the exponential is flushed.
TAIL = 2e-4


@pytest.mark.parametrize("act", ["gelu", "silu"])
@pytest.mark.parametrize("N", [7, 32, 209])
def test_tails_of_the_activation(N, act):
    """g = x₀ and u = x₁ = 1 exactly, so that h is act(g) rounded once, dx₀ its slope and dx₁ act(g): each to half a step
    of bf16 relative to its own value, however small that is."""
    x = torch.zeros(N, 8)
    x[:, 0] = torch.linspace(-13, 13, N)
    x[:, 1] = 1
    x = x.to(BF)
    Wg, Wu = torch.zeros(8, 8, dtype=BF), torch.zeros(8, 8, dtype=BF)
    Wg[0, 0], Wu[0, 1] = 1, 1
    dh = torch.ones(N, 8, dtype=BF)
    w = (Wg.to(DEV), Wu.to(DEV))
    h = rglru.glu_forward(*w, x.to(DEV), activation=act)
    r = rglru.glu_backward(*w, x.to(DEV), dh.to(DEV), activation=act, want_h=True)
    g = f64(x)[:, 0]
    a, s = ff.act(g, act), ff.act_slope(g, act)
    gate = np.where(g == 0, 0.5, a / np.where(g == 0, 1.0, g))  # Φ or σ
    terms = gate + np.abs(s - gate)

    def check(what, got, ref, size):
        e = TAIL * size
        err, bound = np.abs(f64(got) - ref), e + HALF * (np.abs(ref) + e) + TINY
        print(f"{what}: worst error / bound {np.max(err / bound):.3f} at g = {g[np.argmax(err / bound)]}")
        assert (err <= bound).all(), what

    check("h", h[:, 0], a, np.abs(a))
    check("h again", r["h"][:, 0], a, np.abs(a))
    check("du", r["dx"][:, 1], a, np.abs(a))
    check("dg", r["dx"][:, 0], s, terms)


def _at16(t=None, shape=None, dtype=BF):
    """A tensor (a copy of t, or one to be filled) that starts 16 bytes past a 32-byte border, and a check that what lies
    around it is as it was."""
    shape = tuple(shape if t is None else t.shape)
    n, off = int(np.prod(shape)), 16 // torch.empty(0, dtype=dtype).element_size()
    buf = torch.full((n + 2048,), -7.0, dtype=dtype, device=DEV)
    off += 1024
    view = buf[off:off + n].view(shape)
    assert view.data_ptr() % 32 == 16
    if t is not None:
        view.copy_(t)
    return view, lambda: bool((buf[:off] == -7.0).all() and (buf[off + n:] == -7.0).all())


# widths that are multiples of 16, whose rows start in the middle of a sector only because the buffer does; few tokens,
# tiles, several tiles a pair, and one width that is no multiple of 16, whose rows change sides
@pytest.mark.parametrize("N,D,H", [(5, 64, 272), (40, 136, 272), (300, 80, 528), (2100, 48, 2608), (130, 72, 264)])
def test_forward_off_the_sectors(N, D, H):
    x, Wg, Wu, _ = _draw(N, D, H, seed=N + 1)
    want = rglru.glu_forward(Wg.to(DEV), Wu.to(DEV), x.to(DEV))
    h, untouched = _at16(shape=(N, H))
    rglru.glu_forward(*(_at16(t)[0] for t in (Wg, Wu, x)), h=h)
    assert untouched() and torch.equal(h, want)
    _check_forward(x, Wg, Wu, "gelu", h)


# staged dW, rows stored by threads, sums in pieces, few tokens
@pytest.mark.parametrize("N,D,H", [(40, 1088, 2608), (300, 144, 272), (5000, 48, 80), (40, 528, 2064), (7, 272, 528)])
def test_backward_off_the_sectors(N, D, H):
    x, Wg, Wu, dh = _draw(N, D, H, seed=N + 2)
    dev = [t.to(DEV) for t in (Wg, Wu, x, dh)]
    want = rglru.glu_backward(*dev, want_h=True)
    _check_backward(x, Wg, Wu, dh, "gelu", want)
    ws = torch.empty(rglru.glu_backward_workspace_bytes(N, D, H), dtype=torch.uint8, device=DEV)
    shapes = {"dx": (N, D), "dW_gate": (H, D), "dW_up": (H, D), "h": (N, H)}
    for moved in (*shapes, "all", "inputs too"):
        out = {k: (_at16 if moved in (k, "all", "inputs too") else _guarded)(shape=s) for k, s in shapes.items()}
        inputs = [_at16(t)[0] for t in dev] if moved == "inputs too" else dev
        code = rglru._abi.load().rglru_glu_backward(
            *(t.data_ptr() for t in inputs), *(out[k][0].data_ptr() for k in shapes), N, D, H, 0, ws.data_ptr(),
            ws.numel(), torch.cuda.current_stream().cuda_stream)
        assert code == 0 and rglru.workspace_status(None) == 0
        assert all(untouched() for _, untouched in out.values()), moved
        assert all(torch.equal(out[k][0], want[k]) for k in shapes), moved


def test_others_off_the_sectors():
    """The checkpoint and the 4-bit calls, their inputs and outputs 16 bytes past a 32-byte border."""
    g = torch.Generator("cpu").manual_seed(3)
    W = torch.randn(272, 128, generator=g).to(BF).to(DEV)
    q = rglru.w4_quantize(W, 64)
    again = rglru.w4_quantize(_at16(W)[0], 64)
    assert torch.equal(q.codes, again.codes) and torch.equal(q.scales, again.scales)
    moved = rglru.W4Weight(_at16_bytes(q.codes), _at16(q.scales)[0], 64)
    for M in (1, 9, 40):
        x = torch.randn(M, 128, generator=g).to(BF).to(DEV)
        y, untouched = _at16(shape=(M, 272))
        rglru.w4_linear(moved, _at16(x)[0], y=y)
        assert untouched() and torch.equal(y, rglru.w4_linear(q, x))
        h, untouched = _at16(shape=(M, 272))
        rglru.w4_glu(moved, moved, _at16(x)[0], h=h)
        assert untouched() and torch.equal(h, rglru.w4_glu(q, q, x))
    for dtype in (BF, torch.float32):
        for C in (64, 72):
            x = torch.randn(9, C, generator=g).to(dtype).to(DEV)
            want = rglru.act8_pack(x)
            a = rglru.act8_pack(_at16(x, dtype=dtype)[0])
            assert torch.equal(a.codes, want.codes) and torch.equal(a.scales, want.scales)
            back, untouched = _at16(shape=(9, C), dtype=dtype)
            rglru.act8_unpack(rglru.Act8(_at16_bytes(a.codes), _at16_bytes(a.scales), dtype), x=back)
            assert untouched() and torch.equal(back, rglru.act8_unpack(want))


def _at16_bytes(t):
    buf = torch.empty(t.numel() + 64, dtype=t.dtype, device=DEV)
    view = buf[16:16 + t.numel()].view(t.shape)
    assert view.data_ptr() % 32 == 16
    return view.copy_(t)

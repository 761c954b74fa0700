"""Linears with 4-bit weights on the GPU against the float64 oracle; the bounds are derived in _glu.py."""
import numpy as np
import pytest
import torch

from gated_linear_rnn_conv1d_b200 import rglru
from oracle import feed_forward as ff

from _glu import ACT, HALF, SUM, TINY, w4_bound
from _util import f64

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF = torch.bfloat16


def _weight(N, K, group, seed):
    """Every code, scales over several powers of two."""
    g = torch.Generator("cpu").manual_seed(seed)
    codes = torch.randint(0, 256, (N, K // 2), generator=g, dtype=torch.uint8)
    scales = torch.exp(torch.randn(N, K // group, generator=g)).to(BF) / (8 * K ** 0.5)
    return rglru.W4Weight(codes.to(DEV), scales.to(BF).to(DEV), group)


def _dense(w):
    return ff.w4_dequantize(w.codes.cpu().numpy(), f64(w.scales), w.group)


def _x(M, K, seed):
    return torch.randn(M, K, generator=torch.Generator("cpu").manual_seed(seed)).to(BF)


# group, K: one group (most warps idle), fewer groups than warps, more, an odd number of them
WIDTHS = [(32, 32), (32, 320), (32, 1056), (64, 64), (64, 576), (64, 1088), (128, 128), (128, 1152), (128, 2176)]


@pytest.mark.parametrize("group,K", WIDTHS)
@pytest.mark.parametrize("M,N", [(1, 8), (1, 200), (2, 16), (5, 24), (8, 264), (9, 40), (16, 72), (17, 136), (33, 16),
                                 (64, 104)])
def test_linear(M, N, group, K):
    w, x = _weight(N, K, group, seed=N + K), _x(M, K, seed=M)
    buf = torch.full((M * N + 64,), -7.0, dtype=BF, device=DEV)
    y = rglru.w4_linear(w, x.to(DEV), y=buf[32:32 + M * N].view(M, N))
    assert (buf[:32] == -7).all() and (buf[32 + M * N:] == -7).all()
    W = _dense(w)
    ref = f64(x) @ W.T
    _, bound = w4_bound(f64(x), W, ref)
    err = np.abs(f64(y) - ref)
    print(f"worst error / bound {np.max(err / bound):.3f}")
    assert (err <= bound).all()


@pytest.mark.parametrize("act", ["gelu", "silu"])
@pytest.mark.parametrize("group,K", WIDTHS[1::2])
@pytest.mark.parametrize("M,H", [(1, 8), (3, 72), (8, 136), (12, 24), (40, 40)])
def test_glu(M, H, group, K, act):
    wg, wu, x = _weight(H, K, group, seed=K), _weight(H, K, group, seed=K + 1), _x(M, K, seed=M)
    h = rglru.w4_glu(wg, wu, x.to(DEV), activation=act)
    Wg, Wu = _dense(wg), _dense(wu)
    g, u = f64(x) @ Wg.T, f64(x) @ Wu.T
    eg, eu = w4_bound(f64(x), Wg, g)[0], w4_bound(f64(x), Wu, u)[0]
    a = ff.act(g, act)
    ea = 1.13 * eg + ACT * (np.abs(g) + eg)
    e = ea * np.abs(u) + (np.abs(a) + ea) * eu
    bound = (e + HALF * (np.abs(a * u) + e)) * (1 + 1e-6) + TINY
    err = np.abs(f64(h) - a * u)
    print(f"worst error / bound {np.max(err / bound):.3f}")
    assert (err <= bound).all()


def _dense_here(w):
    """Ŵ in float64 on the GPU: the codes and scales are exact in it."""
    q = torch.stack([w.codes & 15, w.codes >> 4], 2).view(w.codes.shape[0], -1).double() - 8
    return q * w.scales.double().repeat_interleave(w.group, 1)


# With more rows than the SMs take at once a block has two, three and more granules of 16 rows, in one chunk and in
# several; the last has eight rows. K: one panel of scales and several, the last of them short.
@pytest.mark.parametrize("M", [1, 8, 13, 31, 47])
@pytest.mark.parametrize("N,K,group", [(4744, 288, 32), (9480, 2176, 32), (14216, 4224, 64), (14216, 8320, 128),
                                       (38008, 192, 64), (38008, 2080, 32)])
def test_linear_of_many_rows(M, N, K, group):
    g = torch.Generator(DEV).manual_seed(N + K)
    codes = torch.randint(0, 256, (N, K // 2), generator=g, dtype=torch.uint8, device=DEV)
    scales = (torch.exp(torch.randn(N, K // group, generator=g, device=DEV)) / (8 * K ** 0.5)).to(BF)
    w, x = rglru.W4Weight(codes, scales, group), _x(M, K, seed=M).to(DEV)
    buf = torch.full((M * N + 64,), -7.0, dtype=BF, device=DEV)
    y = rglru.w4_linear(w, x, y=buf[32:32 + M * N].view(M, N))
    assert (buf[:32] == -7).all() and (buf[32 + M * N:] == -7).all()
    W = _dense_here(w)
    ref = x.double() @ W.T
    ref, e = f64(ref), (K + 16) * SUM * f64(x.double().abs() @ W.abs().T)  # (as w4_bound)
    bound = (e + HALF * (np.abs(ref) + e)) * (1 + 1e-6) + TINY
    err = np.abs(f64(y) - ref)
    print(f"worst error / bound {np.max(err / bound):.3f}")
    assert (err <= bound).all()
    # the gated form on the same rows as both matrices' halves
    H = N // 2 // 8 * 8
    wg = rglru.W4Weight(codes[:H], scales[:H], group)
    wu = rglru.W4Weight(codes[N - H:], scales[N - H:], group)
    h = rglru.w4_glu(wg, wu, x)
    gg, uu, eg, eu = ref[:, :H], ref[:, N - H:], e[:, :H], e[:, N - H:]
    a = ff.act(gg, "gelu")
    ea = 1.13 * eg + ACT * (np.abs(gg) + eg)
    e = ea * np.abs(uu) + (np.abs(a) + ea) * eu
    assert (np.abs(f64(h) - a * uu) <= (e + HALF * (np.abs(a * uu) + e)) * (1 + 1e-6) + TINY).all()


@pytest.mark.parametrize("group", [32, 64, 128])
def test_quantize(group):
    """Codes and scales from their definition: the same IEEE float32 divisions."""
    g = torch.Generator("cpu").manual_seed(group)
    W = torch.randn(24, 3 * group, generator=g)
    W[0, :group] = 0
    W[1] *= 1e-37
    W[2] *= 1e36
    W[3, :group] = W[3, 0]
    W = W.to(BF)
    W[4, 1], W[5, group + 2] = float("inf"), float("nan")
    q = rglru.w4_quantize(W.to(DEV), group)
    v = W.float().view(24, 3, group)
    s = (v.abs().amax(2) / 7).to(BF)
    bad = ~torch.isfinite(v).all(2)
    assert torch.isnan(q.scales.cpu()[bad]).all() and torch.equal(q.scales.cpu()[~bad], s[~bad])
    c = torch.where((bad | (s == 0)).unsqueeze(2), torch.zeros_like(v),
                    torch.round(v / s.float().unsqueeze(2)).clamp(-7, 7))
    c = (c + 8).to(torch.uint8).view(24, -1, 2)
    assert torch.equal(q.codes.cpu(), c[:, :, 0] | (c[:, :, 1] << 4))
    # the weight is within half a step of its code, where nothing is out of the ordinary
    ok = slice(6, 24)
    dense = torch.from_numpy(_dense(q))[ok].view(18, 3, group)
    assert ((dense - v[ok].double()).abs() <= s[ok].double().unsqueeze(2) * 0.5 * (1 + 2 ** -22)).all()


def test_quantized_weight_serves_the_block():
    """The operators together: a gated block's weights in 4 bits, its two linears and the projection down,
    against the block on the weights those codes stand for."""
    g = torch.Generator("cpu").manual_seed(1)
    D, H, M = 256, 520, 4
    Wg, Wu = ((torch.randn(H, D, generator=g) / D ** 0.5).to(BF).to(DEV) for _ in range(2))
    x = _x(M, D, seed=2).to(DEV)
    qg, qu = rglru.w4_quantize(Wg, 64), rglru.w4_quantize(Wu, 64)
    h = rglru.w4_glu(qg, qu, x)
    g_, u_ = rglru.w4_linear(qg, x), rglru.w4_linear(qu, x)
    # the linears' outputs are rounded to bf16 before the product: 2^-8 each on g (slope ≤ 1.13, |g| ≤ …) and u
    a = ff.act(f64(g_), "gelu")
    ref = a * f64(u_)
    tol = 1.13 * HALF * np.abs(f64(g_)) * np.abs(f64(u_)) * 1.02 + 2.05 * HALF * np.abs(ref) + 1e-5
    assert (np.abs(f64(h) - ref) <= tol).all()


def test_scales_and_non_finite_stay_where_they_are():
    w, x = _weight(40, 256, 64, seed=3), _x(3, 256, seed=4).to(DEV)
    clean = rglru.w4_linear(w, x)
    s = w.scales.clone()
    s[7, 1], s[39, 3] = float("nan"), float("inf")
    y = rglru.w4_linear(rglru.W4Weight(w.codes, s, 64), x)
    keep = torch.ones(40, dtype=torch.bool)
    keep[[7, 39]] = False
    assert torch.equal(y[:, keep], clean[:, keep]) and not torch.isfinite(y[:, ~keep]).any()
    bad = x.clone()
    bad[1, 100] = float("nan")
    y = rglru.w4_linear(w, bad)
    assert torch.isnan(y[1]).all() and torch.equal(y[::2], clean[::2])


def test_more_tokens_give_the_same_rows():
    """A token's result does not depend on how many others are with it."""
    w, x = _weight(72, 640, 128, seed=5), _x(64, 640, seed=6).to(DEV)
    want = rglru.w4_linear(w, x)
    for M in (1, 8, 9, 16, 20, 32, 50):
        assert torch.equal(rglru.w4_linear(w, x[:M].contiguous()), want[:M]), M


def test_streams_and_graphs():
    w, x = _weight(72, 640, 128, seed=5), _x(6, 640, seed=6).to(DEV)
    want = rglru.w4_linear(w, x), rglru.w4_glu(w, w, x)
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    got = [(rglru.w4_linear(w, x, stream=s), rglru.w4_glu(w, w, x, stream=s)) for s in (a, b, a, b)]
    torch.cuda.synchronize()
    assert all(torch.equal(p, want[0]) and torch.equal(q, want[1]) for p, q in got)
    xin = x.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, h = rglru.w4_linear(w, xin), rglru.w4_glu(w, w, xin)
    x2 = _x(6, 640, seed=8).to(DEV)
    xin.copy_(x2)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, rglru.w4_linear(w, x2)) and torch.equal(h, rglru.w4_glu(w, w, x2))


def test_binding_refusals():
    w, x = _weight(16, 128, 64, seed=1), _x(2, 128, seed=1).to(DEV)
    cases = [
        (ValueError, lambda: rglru.w4_linear(w, x[:, :64].contiguous())),
        (TypeError, lambda: rglru.w4_linear(w, x.float())),
        (rglru._abi.RGLRUError, lambda: rglru.w4_linear(w, _x(65, 128, seed=1).to(DEV))),
        (rglru._abi.RGLRUError, lambda: rglru.w4_linear(w, x[:0])),
        (ValueError, lambda: rglru.w4_linear(rglru.W4Weight(w.codes, w.scales, 128), x)),
        (ValueError, lambda: rglru.w4_linear(rglru.W4Weight(w.codes, w.scales, 16), x)),
        (ValueError, lambda: rglru.w4_quantize(x, 256)),
        (rglru._abi.RGLRUError, lambda: rglru.w4_quantize(x, 64)),  # two rows
        (ValueError, lambda: rglru.w4_glu(w, _weight(24, 128, 64, seed=1), x)),
    ]
    for i, (err, call) in enumerate(cases):
        with pytest.raises(err):
            call()
            raise AssertionError(f"case {i} was taken")


@pytest.mark.parametrize("M", [1, 8, 13, 32, 47])
def test_inputs_from_the_call_before(M):
    """The serving chain h = w4_glu(…), y = w4_linear(down, h): x is what the kernel ahead writes, in the same memory
    every time, and so are scales and gradients; the results are those of calls that wait for each other."""
    D, H, K = 640, 4744, 4736
    wg, wu, down = _weight(H, D, 64, seed=1), _weight(H, D, 64, seed=2), _weight(D, K, 64, seed=3)
    W = torch.randn(H, D, generator=torch.Generator("cpu").manual_seed(5)).to(BF).to(DEV)
    xs = [(_x(M, D, seed=4) * (1 + i / 8)).to(BF).to(DEV) for i in range(12)]
    h, y = torch.empty(M, H, dtype=BF, device=DEV), torch.empty(M, D, dtype=BF, device=DEV)

    def chain(x, sync):
        rglru.w4_glu(wg, wu, x, h=h)
        sync()
        rglru.w4_linear(down, h.view(-1)[:M * K].view(M, K), y=y)
        sync()
        few = rglru.glu_forward(W[:72], W[72:144], y)
        sync()
        dx = rglru.glu_backward(W[:72], W[72:144], y, few)["dx"]
        sync()
        q = rglru.w4_quantize((W * x.view(-1)[0]).contiguous(), 64)
        sync()
        last = rglru.w4_linear(q, dx)
        sync()
        return y.clone(), few, dx, last

    want = [chain(x, torch.cuda.synchronize) for x in xs]
    for _ in range(4):
        got = [chain(x, lambda: None) for x in xs]
        assert all(torch.equal(g, w) for a, b in zip(got, want) for g, w in zip(a, b))

"""Refusals of the gated feed-forward block, the 8-bit checkpoints and the 4-bit linears: the library's
argument checks (nothing is launched, so no GPU is needed) and the binding's."""
import ctypes

import pytest
import torch

from gated_linear_rnn_conv1d_b200 import _abi, rglru

OK = ctypes.c_void_p(0x100000)
WS = ctypes.c_void_p(0x200000)
ODD = ctypes.c_void_p(0x100008)


def test_glu_forward_refusals():
    f = _abi.load().rglru_glu_forward
    call = lambda wg=OK, wu=OK, x=OK, h=OK, N=4, D=64, H=72, act=0: f(wg, wu, x, h, N, D, H, act, None)
    for bad in (dict(N=0), dict(N=-1), dict(N=(1 << 30) + 1), dict(D=0), dict(D=12), dict(D=65544), dict(H=4),
                dict(H=100), dict(act=2), dict(act=-1), dict(N=1 << 30, H=65536)):
        assert call(**bad) == -2, bad
    for k in ("wg", "wu", "x", "h"):
        assert call(**{k: None}) == -1, k
        assert call(**{k: ODD}) == -3, k


@pytest.mark.parametrize("packed", [False, True])
def test_glu_backward_refusals(packed):
    lib = _abi.load()
    need = lib.rglru_glu_backward_workspace_bytes(4, 64, 72, int(packed))
    # dg and du with rows of 128 columns, and x̂ for the packed form, each rounded up to 256 bytes
    assert need == 2 * 1024 + (512 if packed else 0)
    assert lib.rglru_glu_backward_workspace_bytes(0, 64, 72, 0) == 0
    assert lib.rglru_glu_backward_workspace_bytes(4, 60, 72, 0) == 0

    def call(wg=OK, wu=OK, x=OK, scales=OK, dh=OK, dx=OK, dwg=OK, dwu=OK, h=None, N=4, D=64, H=72, act=1, ws=WS,
             wsb=need):
        if packed:
            return lib.rglru_glu_backward_act8(wg, wu, x, scales, dh, dx, dwg, dwu, h, N, D, H, act, ws, wsb, None)
        return lib.rglru_glu_backward(wg, wu, x, dh, dx, dwg, dwu, h, N, D, H, act, ws, wsb, None)

    for bad in (dict(N=0), dict(D=20), dict(H=0), dict(act=3)):
        assert call(**bad) == -2, bad
    names = ["wg", "wu", "x", "dh", "dx", "dwg", "dwu"] + (["scales"] if packed else [])
    for k in names:
        assert call(**{k: None}) == -1, k
        assert call(**{k: ODD}) == -3, k
    assert call(h=ODD) == -3
    assert call(ws=None) == -5
    assert call(wsb=need - 1) == -5
    assert call(ws=ctypes.c_void_p(0x200010)) == -3


def test_act8_refusals():
    lib = _abi.load()
    for f in (lib.rglru_act8_pack, lib.rglru_act8_unpack):
        call = lambda a=OK, b=OK, c=OK, N=3, C=40, io=1: f(a, b, c, N, C, io, None)
        assert call(io=2) == -4
        for bad in (dict(N=0), dict(C=0), dict(C=36), dict(C=65544), dict(N=(1 << 30) + 1), dict(N=1 << 30, C=65536)):
            assert call(**bad) == -2, bad
        for k in ("a", "b", "c"):
            assert call(**{k: None}) == -1, k
            assert call(**{k: ODD}) == -3, k


def test_w4_refusals():
    lib = _abi.load()
    q = lambda a=OK, b=OK, c=OK, N=16, K=256, group=64: lib.rglru_w4_quantize(a, b, c, N, K, group, None)
    lin = lambda a=OK, b=OK, x=OK, y=OK, M=1, N=16, K=256, group=64: lib.rglru_w4_linear(a, b, x, y, M, N, K, group, None)
    glu = lambda a=OK, b=OK, c=OK, d=OK, x=OK, h=OK, M=1, N=16, K=256, group=64, act=0: lib.rglru_w4_glu(
        a, b, c, d, x, h, M, N, K, group, act, None)
    for f, ptrs in ((q, "abc"), (lin, "abxy"), (glu, "abcdxh")):
        for bad in (dict(N=0), dict(N=12), dict(K=0), dict(K=96), dict(group=16), dict(group=256), dict(group=0),
                    dict(K=160, group=128)):
            assert f(**bad) == -2, bad
        for k in ptrs:
            assert f(**{k: None}) == -1, k
            assert f(**{k: ODD}) == -3, k
        if f is not q:
            assert f(M=0) == -2 and f(M=65) == -2
    assert glu(act=2) == -2


def test_binding_takes_cuda_tensors_only():
    b = torch.bfloat16
    w, x, dh = torch.zeros(72, 64, dtype=b), torch.zeros(3, 64, dtype=b), torch.zeros(3, 72, dtype=b)
    a8 = rglru.Act8(torch.zeros(3, 64, dtype=torch.int8), torch.zeros(3, 2, dtype=torch.uint8), b)
    w4 = rglru.W4Weight(torch.zeros(72, 32, dtype=torch.uint8), torch.zeros(72, 1, dtype=b), 64)
    for call in (lambda: rglru.glu_forward(w, w, x), lambda: rglru.glu_backward(w, w, x, dh),
                 lambda: rglru.glu_backward(w, w, a8, dh), lambda: rglru.act8_pack(x), lambda: rglru.act8_unpack(a8),
                 lambda: rglru.w4_quantize(w, 64), lambda: rglru.w4_linear(w4, x),
                 lambda: rglru.w4_glu(w4, w4, x)):
        with pytest.raises(ValueError, match="CUDA"):
            call()


def test_outputs_apart_from_inputs():
    """A call whose output overlaps an input, another output or the workspace is refused; the last byte of one
    and the first of the next are apart (the call then ends at the device check where there is no B200)."""
    lib = _abi.load()
    base = 1 << 32

    def at(i):  # 4096 bytes each, room for any buffer of these shapes but the weights' 9216
        return base + 16384 * i

    refused = lambda code: code == -2
    N, D, H = 4, 64, 72
    sizes = {"wg": H * D * 2, "wu": H * D * 2, "x": N * D * 2, "h": N * H * 2}

    def fwd(**over):
        p = {k: at(i) for i, k in enumerate(("wg", "wu", "x", "h"))} | over
        return lib.rglru_glu_forward(p["wg"], p["wu"], p["x"], p["h"], N, D, H, 0, None)

    for i, k in enumerate(("wg", "wu", "x")):
        assert refused(fwd(h=at(i))) and refused(fwd(h=at(i) + sizes[k] - 16)), k
        assert refused(fwd(h=at(i) - sizes["h"] + 16)), k
    if not torch.cuda.is_available():
        assert not refused(fwd()) and not refused(fwd(wu=at(0)))
        assert not refused(fwd(h=at(2) + sizes["x"])) and not refused(fwd(h=at(2) - sizes["h"]))

    names = ("wg", "wu", "x", "dh", "dx", "dwg", "dwu", "h", "ws")
    need = lib.rglru_glu_backward_workspace_bytes(N, D, H, 0)

    def bwd(**over):
        p = {k: at(i) for i, k in enumerate(names)} | over
        return lib.rglru_glu_backward(*(p[k] for k in names[:8]), N, D, H, 0, p["ws"], need, None)

    for out in ("dx", "dwg", "dwu", "h", "ws"):
        for other in range(len(names)):
            if names[other] != out:
                assert refused(bwd(**{out: at(other)})), (out, names[other])
    if not torch.cuda.is_available():
        assert not refused(bwd()) and not refused(bwd(wu=at(0))) and not refused(bwd(h=None))

    assert refused(lib.rglru_act8_pack(at(0), at(0), at(1), 3, 40, 0, None))
    assert refused(lib.rglru_act8_pack(at(0), at(1), at(1) + 112, 3, 40, 0, None))
    assert refused(lib.rglru_act8_unpack(at(0), at(1), at(1) - 224, 3, 40, 0, None))
    assert refused(lib.rglru_w4_quantize(at(0), at(0) + 32, at(1), 8, 64, 32, None))
    assert refused(lib.rglru_w4_linear(at(0), at(1), at(2), at(2), 2, 64, 64, 32, None))
    assert refused(lib.rglru_w4_linear(at(0), at(1), at(2), at(1), 2, 64, 64, 32, None))
    assert refused(lib.rglru_w4_glu(at(0), at(1), at(2), at(3), at(4), at(4), 2, 64, 64, 32, 0, None))
    assert refused(lib.rglru_w4_glu(at(0), at(1), at(2), at(3), at(4), at(3), 2, 64, 64, 32, 0, None))


def _without_calls(monkeypatch):
    import sys

    import gated_linear_rnn_conv1d_b200 as package
    monkeypatch.delattr(package, "_calls", raising=False)
    monkeypatch.setitem(sys.modules, package.__name__ + "._calls", None)  # its import fails
    monkeypatch.setattr(_abi, "_calls", None)


def test_binding_without_its_short_way(monkeypatch):
    """A _calls.so that cannot be loaded costs a warning and time: the calls go the long way, which here finds CPU tensors."""
    _without_calls(monkeypatch)
    b = torch.bfloat16
    w, x = torch.zeros(72, 64, dtype=b), torch.zeros(3, 64, dtype=b)
    with pytest.warns(RuntimeWarning, match="_calls.so"):
        with pytest.raises(ValueError, match="CUDA"):
            rglru.glu_forward(w, w, x)
    with pytest.raises(ValueError, match="CUDA"):
        rglru.act8_pack(x)


@pytest.mark.gpu
def test_long_way_gives_the_same(monkeypatch):
    g = torch.Generator("cpu").manual_seed(1)
    b = torch.bfloat16
    W, x, dh = (torch.randn(*s, generator=g).to(b).to("cuda") for s in ((72, 64), (40, 64), (40, 72)))
    q = rglru.w4_quantize(W, 64)

    def work():
        a = rglru.act8_pack(x)
        r = rglru.glu_backward(W, W, x, dh, want_h=True)
        return [rglru.glu_forward(W, W, x), *r.values(), rglru.glu_backward(W, W, a, dh)["dx"], a.codes, a.scales,
                rglru.act8_unpack(a), rglru.w4_linear(q, x), rglru.w4_glu(q, q, x)]

    want = work()
    _without_calls(monkeypatch)
    with pytest.warns(RuntimeWarning, match="_calls.so"):
        got = work()
    assert all(torch.equal(a, c) for a, c in zip(got, want))


def test_build_without_pytorch(monkeypatch, tmp_path, capsys):
    """librglru.so needs nvcc alone; without PyTorch or g++ the short way is left out, with a line that says so."""
    import builtins
    import shutil

    from gated_linear_rnn_conv1d_b200 import build
    monkeypatch.setattr(build, "CALLS", str(tmp_path / "_calls.so"))
    real = builtins.__import__

    def without_torch(name, *args, **kwargs):
        if name == "torch":
            raise ImportError(name)
        return real(name, *args, **kwargs)

    with monkeypatch.context() as m:
        m.setattr(builtins, "__import__", without_torch)
        build._build_calls(True)
    assert "PyTorch" in capsys.readouterr().err
    monkeypatch.setattr(shutil, "which", lambda name: None)
    build._build_calls(True)
    assert "g++" in capsys.readouterr().err
    assert not (tmp_path / "_calls.so").exists()

"""The token operators without a GPU: bad arguments are refused before any
device is touched, and valid calls fail with BV_ERR_CUDA (no CPU fallback)."""

import pytest
import torch

ARG, SHAPE, WORKSPACE, CUDA = 1, 2, 3, 4
F32, BF16, F16 = 0, 1, 2


@pytest.fixture(scope="module")
def L():
    from bigvgan_waveform_decoder_alias_b200 import build_native, native
    build_native.build()
    return native.lib()


# never dereferenced: the calls fail first.  64 MB apart.
P = [0x100000000 + i * (64 << 20) for i in range(10)]


def norm(L, int8=False, **kw):
    d = dict(x=P[0], xs=64, r=P[1], rs=64, sum=P[2], ss=64, gain=P[3], gdt=BF16, eps=1e-6,
             rows=8, cols=64, dt=BF16, out=P[4], os=64, scale=P[5])
    d.update(kw)
    args = [d["x"], d["xs"], d["r"], d["rs"], d["sum"], d["ss"], d["gain"], d["gdt"], d["eps"],
            d["rows"], d["cols"], d["dt"], d["out"], d["os"]]
    return L.bv_rms_norm_int8(*args, d["scale"], None) if int8 else L.bv_rms_norm(*args, None)


@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("kw,want", [
    (dict(x=None), ARG), (dict(out=None), ARG), (dict(dt=3), ARG), (dict(dt=-1), ARG),
    (dict(gdt=F16), ARG), (dict(gdt=7), ARG), (dict(eps=0.0), ARG), (dict(eps=-1e-6), ARG),
    (dict(eps=float("nan")), ARG), (dict(eps=float("inf")), ARG),
    (dict(x=P[0] + 1), ARG), (dict(r=P[1] + 1), ARG), (dict(sum=P[2] + 1), ARG),
    (dict(gain=P[3] + 1), ARG), (dict(gain=P[3] + 2, gdt=F32), ARG),
    (dict(rows=-1), SHAPE), (dict(cols=0), SHAPE), (dict(xs=-64), SHAPE), (dict(rs=-1), SHAPE),
    (dict(ss=63), SHAPE), (dict(os=63), SHAPE), (dict(os=-1), SHAPE),
    (dict(rows=1 << 40, xs=1 << 40), SHAPE), (dict(rows=1 << 62), SHAPE),
    (dict(sum=P[0] + 2), ARG),              # over x, shifted
    (dict(sum=P[0], ss=65), ARG),           # over x, another stride
    (dict(sum=P[1], rs=0), ARG),            # over a broadcast residual
    (dict(out=P[0]), ARG), (dict(out=P[1]), ARG), (dict(out=P[2]), ARG), (dict(out=P[3]), ARG),
    (dict(sum=P[3]), ARG),
])
def test_norm_refusals(L, int8, kw, want):
    assert norm(L, int8, **kw) == want


@pytest.mark.parametrize("kw,want", [
    (dict(scale=None), ARG), (dict(scale=P[5] + 2), ARG), (dict(scale=P[4]), ARG),
    (dict(scale=P[0]), ARG), (dict(scale=P[2]), ARG)])
def test_norm_int8_scale_refusals(L, kw, want):
    assert norm(L, True, **kw) == want


@pytest.mark.parametrize("kw", [
    dict(), dict(sum=P[0]), dict(sum=P[1]), dict(sum=None), dict(r=None), dict(gain=None),
    dict(xs=0, rs=0), dict(gdt=F32), dict(rows=1, xs=3, os=1),
    # columns of one matrix: spans cross, rows do not
    dict(x=P[0], xs=128, out=P[0] + 128, os=128, dt=BF16)])
def test_valid_norm_needs_a_device(L, kw):
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    assert norm(L, **kw) == CUDA


def quantize(L, **kw):
    d = dict(x=P[0], xs=64, rows=8, cols=64, dt=F32, q=P[1], qs=64, scale=P[2])
    d.update(kw)
    return L.bv_quantize_rows(d["x"], d["xs"], d["rows"], d["cols"], d["dt"], d["q"], d["qs"],
                              d["scale"], None)


@pytest.mark.parametrize("kw,want", [
    (dict(x=None), ARG), (dict(q=None), ARG), (dict(scale=None), ARG), (dict(dt=9), ARG),
    (dict(x=P[0] + 2), ARG), (dict(scale=P[2] + 1), ARG), (dict(rows=-2), SHAPE),
    (dict(cols=0), SHAPE), (dict(qs=63), SHAPE), (dict(qs=-64), SHAPE), (dict(xs=-1), SHAPE),
    (dict(q=P[0]), ARG), (dict(scale=P[0]), ARG), (dict(scale=P[1]), ARG)])
def test_quantize_refusals(L, kw, want):
    assert quantize(L, **kw) == want


def matmul(L, **kw):
    d = dict(a=P[0], as_=64, sa=P[1], w=P[2], ws=64, sw=P[3], bias=P[4], M=8, N=16, K=64, r=P[5],
             rs=16, y=P[6], ys=16, dt=F32, cf=0)
    d.update(kw)
    return L.bv_int8_matmul(d["a"], d["as_"], d["sa"], d["w"], d["ws"], d["sw"], d["bias"], d["M"],
                            d["N"], d["K"], d["r"], d["rs"], d["y"], d["ys"], d["dt"], d["cf"],
                            None)


@pytest.mark.parametrize("kw,want", [
    (dict(a=None), ARG), (dict(sa=None), ARG), (dict(w=None), ARG), (dict(sw=None), ARG),
    (dict(y=None), ARG), (dict(dt=3), ARG), (dict(M=-1), SHAPE), (dict(N=0), SHAPE),
    (dict(K=0), SHAPE), (dict(K=131072), SHAPE), (dict(as_=-1), SHAPE), (dict(ws=-1), SHAPE),
    (dict(as_=1 << 40), SHAPE), (dict(rs=-1), SHAPE), (dict(ys=15), SHAPE),
    (dict(cf=1, ys=7, rs=8), SHAPE), (dict(sa=P[1] + 2), ARG), (dict(sw=P[3] + 1), ARG),
    (dict(bias=P[4] + 2), ARG), (dict(y=P[6] + 2), ARG), (dict(r=P[5] + 1), ARG),
    (dict(y=P[0]), ARG), (dict(y=P[2]), ARG), (dict(y=P[1]), ARG), (dict(y=P[3]), ARG),
    (dict(y=P[4]), ARG), (dict(y=P[5] + 4), ARG), (dict(y=P[5], ys=17), ARG)])
def test_matmul_refusals(L, kw, want):
    assert matmul(L, **kw) == want


@pytest.mark.parametrize("kw", [dict(), dict(y=P[5]), dict(r=None), dict(bias=None),
                                dict(cf=1, ys=8, rs=8), dict(K=63, as_=63, ws=77), dict(as_=0)])
def test_valid_matmul_needs_a_device(L, kw):
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    assert matmul(L, **kw) == CUDA


def front(L, **kw):
    d = dict(x=P[0], xs=64, r=None, rs=0, gain=P[1], gdt=F32, eps=1e-6, S=2, T=10, cols=64,
             dt=BF16, w=P[2], ws=64, sw=P[3], bias=P[4], Cout=32, by_side=1, z=P[5], wsp=P[6],
             bytes=1 << 20)
    d.update(kw)
    return L.bv_token_front_end(d["x"], d["xs"], d["r"], d["rs"], d["gain"], d["gdt"], d["eps"],
                                d["S"], d["T"], d["cols"], d["dt"], d["w"], d["ws"], d["sw"],
                                d["bias"], d["Cout"], d["by_side"], d["z"], d["wsp"], d["bytes"],
                                None)


def test_front_end_workspace_size(L):
    # 20 rows of 65 bytes padded to 80, to 256; then 20 scales
    assert L.bv_token_front_end_workspace_size(2, 10, 65) == 1792 + 80
    for bad in ((0, 10, 64), (2, 0, 64), (2, 10, 0), (2, 10, 131072), (1 << 20, 1 << 20, 64)):
        assert L.bv_token_front_end_workspace_size(*bad) == 0


@pytest.mark.parametrize("kw,want", [
    (dict(x=None), ARG), (dict(w=None), ARG), (dict(sw=None), ARG), (dict(z=None), ARG),
    (dict(S=0), SHAPE), (dict(T=0), SHAPE), (dict(cols=0), SHAPE), (dict(Cout=0), SHAPE),
    (dict(dt=5), ARG), (dict(eps=0.0), ARG), (dict(gdt=F16), ARG), (dict(xs=-1), SHAPE),
    (dict(ws=-1), SHAPE), (dict(xs=1 << 60), SHAPE), (dict(wsp=None), WORKSPACE),
    (dict(bytes=100), WORKSPACE), (dict(wsp=P[6] + 128), ARG), (dict(wsp=P[0]), ARG),
    (dict(wsp=P[5]), ARG), (dict(z=P[0]), ARG), (dict(z=P[2]), ARG), (dict(z=P[5] + 2), ARG),
    (dict(sw=P[3] + 2), ARG), (dict(bias=P[4] + 1), ARG)])
def test_front_end_refusals(L, kw, want):
    assert front(L, **kw) == want


def test_valid_front_end_needs_a_device(L):
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    assert front(L) == CUDA
    assert front(L, by_side=0, r=P[7], rs=64) == CUDA


def test_python_wrappers_refuse_host_tensors(L):
    from bigvgan_waveform_decoder_alias_b200 import native
    x = torch.zeros(4, 64)
    q = torch.zeros(4, 64, dtype=torch.int8)
    s = torch.ones(4)
    with pytest.raises(native.BVError):
        native.bv_rms_norm(x)
    with pytest.raises(native.BVError):
        native.bv_rms_norm_int8(x)
    with pytest.raises(native.BVError):
        native.bv_quantize_rows(x)
    with pytest.raises(native.BVError):
        native.bv_int8_matmul(q, s, q, s)
    with pytest.raises(native.BVError):
        native.bv_int8_matmul(x, s, q, s)


@pytest.mark.parametrize("name", ["rows.cu", "int8_mm.cu"])
def test_overlapped_kernels_read_by_plain_loads(name):
    """Kernels that begin before the one ahead of them has ended may not read
    through the read-only path, whose data no one may write meanwhile: a product
    reads the 8-bit rows and scales that the norm ahead of it writes."""
    import os
    import re

    from bigvgan_waveform_decoder_alias_b200 import build_native
    text = open(os.path.join(build_native.CSRC, name)).read()
    assert "after_previous()" in text  # launched ahead of time
    code = re.sub(r"//[^\n]*", "", text)
    assert not re.search(r"__ldg\s*\(|ld\.global\.nc|__restrict__", code)


@pytest.mark.parametrize("capturing", [False, True])
def test_front_end_waits_for_its_weight(L, monkeypatch, capturing):
    """A front end quantises its weight on the stream it is made on and may then
    be called on any other: its constructor waits for that stream (but not in a
    capture, where a wait is an error)."""
    from contextlib import nullcontext
    from types import SimpleNamespace

    from bigvgan_waveform_decoder_alias_b200 import native
    steps = []
    q = SimpleNamespace(is_cuda=True, device="cuda:0")

    def quantise(x):
        steps.append("quantise")
        return q, q
    monkeypatch.setattr(native, "bv_quantize_rows", quantise)
    monkeypatch.setattr(torch.cuda, "device", lambda d: nullcontext())
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: capturing)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: SimpleNamespace(
        synchronize=lambda: steps.append("wait")))
    native.TokenFrontEnd(None, torch.zeros(4, 8), device="cpu")
    assert steps == (["quantise"] if capturing else ["quantise", "wait"])


@pytest.mark.parametrize("cf", [0, 1])
def test_matmul_extents_stay_inside_64_bits(L, cf):
    """Outputs and residuals of 2^62 values: their byte offsets would wrap, and
    with them the overlap checks."""
    far = dict(M=0x7fffff00, N=0x7fffff00, as_=0, ws=0, cf=cf, rs=0x7fffff00, ys=0x7fffff00,
               a=1 << 20, w=1 << 21, sa=1 << 40, sw=1 << 42, bias=None, r=None)
    assert matmul(L, **far) == SHAPE
    assert matmul(L, **far | dict(M=64, N=64, ys=1 << 31, r=1 << 45, rs=1 << 32)) == SHAPE
    # a broadcast residual has no extent of its own
    if not torch.cuda.is_available():
        assert matmul(L, rs=0) == CUDA


@pytest.mark.parametrize("kw", [
    dict(S=1, T=0x7fffff80, Cout=1, by_side=0), dict(S=1, T=0x7fffff80, Cout=1, by_side=1),
    dict(S=1, T=8, Cout=0x7fffff80), dict(S=1, T=0x7fffff00, Cout=0x7fffff00, ws=0)])
def test_front_end_refuses_the_product_before_the_norm_runs(L, kw):
    """Sizes that the product would refuse are refused before any launch (a call
    that reached the norm would report the missing device here)."""
    far = dict(xs=0, x=1 << 20, gain=None, w=1 << 21, sw=1 << 22, bias=None, z=1 << 40, wsp=1 << 50,
               bytes=1 << 62, cols=16, ws=16)
    assert front(L, **far | kw) == SHAPE

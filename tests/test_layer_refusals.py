"""What the layer operators (convolution, selective scan, gated norm) refuse, through the C ABI with addresses that
are never used: every call here returns from validation (CPU only)."""
import ctypes

import pytest

from chunked_state_space_b200 import build as ssd_build
from chunked_state_space_b200 import ssd

BASE, GB = 1 << 40, 1 << 30


@pytest.fixture(scope="module")
def lib():
    ssd_build.build()
    return ssd.lib()


def at(k, off=0):
    return ctypes.c_void_p(BASE + k * GB + off)


def conv(lib, d=None, **o):
    """A call that would be taken, but for what `o` changes."""
    dims = ssd.ConvDims(*(o.get(k, v) for k, v in dict(batch=2, seqlen=100, channels=64, width=4, io=1, flags=1).items()))
    g = lambda k, v: o.get(k, v)  # noqa: E731
    return lib.ssd_conv_fwd(None if d == "null" else ctypes.byref(dims), g("x", at(0)), g("xb", 6400), g("xt", 64), g("w", at(1)),
                            g("bias", at(2)), g("init", at(3)), g("lengths", at(4)), g("y", at(5)), g("yb", 6400),
                            g("yt", 64), g("final", at(6)), None)


@pytest.mark.parametrize("o,status", [
    (dict(batch=0), 2), (dict(seqlen=0), 2), (dict(channels=0), 2), (dict(width=0), 2), (dict(width=1), 5),
    (dict(width=5), 5), (dict(io=2), 3), (dict(flags=2), 1), (dict(channels=1 << 25), 5),
    (dict(batch=1 << 20, channels=1 << 14), 5), (dict(seqlen=1 << 33), 5),
    (dict(x=None), 1), (dict(w=None), 1), (dict(y=None), 1), (dict(x=at(0, 1)), 4), (dict(w=at(1, 2)), 4),
    (dict(init=at(3, 1)), 4), (dict(lengths=at(4, 2)), 4), (dict(xt=-64), 2), (dict(yt=63), 2), (dict(yt=0), 2),
    (dict(yb=6399), 2), (dict(y=at(0, 128)), 1), (dict(y=at(3, -64)), 1), (dict(final=at(3, 2)), 1),
    (dict(final=at(5)), 1), (dict(final=at(0)), 1), (dict(y=at(1, 16)), 1), (dict(y=at(4)), 1),
])
def test_conv_refuses(lib, o, status):
    assert conv(lib, **o) == status, ssd.status_string(conv(lib, **o))


def test_conv_step_refuses(lib):
    d = ssd.ConvDims(2, 0, 64, 4, 1, 1)  # the length is not looked at
    f = lambda **o: lib.ssd_conv_step(ctypes.byref(o.get("d", d)), o.get("x", at(0)), 64, o.get("w", at(1)), None,  # noqa: E731
                                      o.get("state", at(2)), o.get("y", at(3)), o.get("yb", 64), None)
    assert f(x=None) == 1 and f(w=None) == 1 and f(state=None) == 1 and f(y=None) == 1
    assert f(yb=63) == 2 and f(y=at(0)) == 1 and f(state=at(0)) == 1 and f(y=at(2)) == 1
    assert f(state=at(2, 1)) == 4 and f(d=ssd.ConvDims(2, 0, 64, 6, 1, 1)) == 5
    assert lib.ssd_conv_step(None, at(0), 64, at(1), None, at(2), at(3), 64, None) == 1
    assert conv(lib, d="null") == 1


def scan(lib, **o):
    names = dict(batch=2, seqlen=100, channels=64, dstate=16, ngroups=1, io=1, flags=1)
    dims = ssd.SelectiveDims(*(o.get(k, v) for k, v in names.items()))
    g = lambda k, v: o.get(k, v)  # noqa: E731
    return lib.ssd_selective_fwd(ctypes.byref(dims), g("x", at(0)), 6400, g("xt", 64), g("dt", at(1)), 6400, 64,
                                 g("A", at(2)), g("B", at(3)), g("C", at(4)), 1600, g("bct", 16), g("D", at(5)),
                                 g("z", at(6)), 6400, 64, g("bias", at(7)), g("init", at(8)), g("lengths", at(9)),
                                 g("y", at(10)), 6400, g("yt", 64), g("final", at(11)),
                                 g("ws", None), g("wsb", 0), None)


@pytest.mark.parametrize("o,status", [
    (dict(batch=0), 2), (dict(seqlen=0), 2), (dict(channels=0), 2), (dict(dstate=0), 2), (dict(ngroups=0), 2),
    (dict(ngroups=3), 2), (dict(dstate=129), 5), (dict(io=5), 3), (dict(flags=4), 1), (dict(channels=1 << 25), 5),
    (dict(batch=1 << 14, channels=1 << 13), 5), (dict(seqlen=1 << 31), 5),
    (dict(x=None), 1), (dict(dt=None), 1), (dict(A=None), 1), (dict(B=None), 1), (dict(C=None), 1), (dict(y=None), 1),
    (dict(dt=at(1, 1)), 4), (dict(A=at(2, 2)), 4), (dict(final=at(11, 2)), 4), (dict(xt=-1), 2), (dict(bct=-16), 2),
    (dict(yt=60), 2), (dict(y=at(0)), 1), (dict(y=at(6, 64)), 1), (dict(y=at(3)), 1), (dict(final=at(8, 64)), 1),
    (dict(final=at(2)), 1), (dict(final=at(10)), 1), (dict(y=at(8)), 1), (dict(ws=at(12, 8)), 4),
    (dict(batch=1, seqlen=4096, ws=at(12), wsb=1024), 6),
    (dict(batch=1, seqlen=4096, ws=at(0), wsb=1 << 20), 1),
    (dict(batch=1, seqlen=4096, ws=at(2), wsb=1 << 20), 1),
    (dict(batch=1, seqlen=4096, ws=at(9), wsb=1 << 20), 1),
    (dict(batch=1, seqlen=4096, ws=at(8), wsb=1 << 20), 1),
    (dict(batch=1, seqlen=4096, ws=at(10), wsb=1 << 20), 1),
    (dict(batch=1, seqlen=4096, ws=at(11), wsb=1 << 20), 1),
])
def test_selective_refuses(lib, o, status):
    assert scan(lib, **o) == status, ssd.status_string(scan(lib, **o))


def test_selective_step_refuses(lib):
    d = ssd.SelectiveDims(2, 0, 64, 16, 1, 1, 1)
    f = lambda **o: lib.ssd_selective_step(ctypes.byref(d), o.get("x", at(0)), 64, at(1), 64, at(2), at(3), at(4), 16,  # noqa: E731
                                           None, None, 0, None, o.get("state", at(5)), o.get("y", at(6)), 64, None)
    assert f(x=None) == 1 and f(state=None) == 1 and f(y=None) == 1
    assert f(y=at(0)) == 1 and f(y=at(5)) == 1 and f(state=at(2)) == 1 and f(state=at(5, 2)) == 4
    assert lib.ssd_selective_step(None, *[None] * 1, 0, None, 0, None, None, None, 0, None, None, 0, None, None, None, 0, None) == 1


@pytest.mark.parametrize("o,status", [
    (dict(batch=0), 2), (dict(features=0), 2), (dict(ngroups=3), 2), (dict(io=3), 3), (dict(flags=1), 1),
    (dict(batch=1 << 20, seqlen=1 << 20), 5), (dict(x=None), 1), (dict(out=None), 1), (dict(eps=-1.0), 1),
    (dict(eps=float("nan")), 1), (dict(x=at(0, 1)), 4), (dict(z=at(1, 1)), 4), (dict(w=at(2, 1)), 4), (dict(ot=63), 2),
    (dict(zt=-64), 2), (dict(out=at(0, 128)), 1), (dict(out=at(1)), 1), (dict(out=at(2)), 1),
    (dict(out=at(0), ot=128, ob=12800), 1),  # x itself, but other strides
])
def test_gated_norm_refuses(lib, o, status):
    names = dict(batch=2, seqlen=100, features=64, ngroups=1, io=1, flags=0)
    dims = ssd.NormDims(*(o.get(k, v) for k, v in names.items()))
    g = lambda k, v: o.get(k, v)  # noqa: E731
    s = lib.ssd_rmsnorm_gated(ctypes.byref(dims), g("x", at(0)), 6400, 64, g("z", at(1)), 6400, g("zt", 64),
                              g("w", at(2)), g("eps", 1e-5), g("out", at(3)), g("ob", 6400), g("ot", 64), None)
    assert s == status, ssd.status_string(s)


def test_the_binding_takes_no_host_tensors():
    import torch
    x, w = torch.zeros(2, 9, 32), torch.zeros(32, 4)
    for call in (lambda: ssd.ssd_conv_fwd(x, w), lambda: ssd.ssd_conv_step(x[:, 0], w, torch.zeros(2, 3, 32)),
                 lambda: ssd.ssd_rmsnorm_gated(x)):
        with pytest.raises(ssd.SSDError) as e:
            call()
        assert e.value.status == 1


def test_selective_workspace(lib):
    """Segments where they pay: long sequences that would not fill the GPU."""
    def size(**o):
        names = dict(batch=1, seqlen=4096, channels=64, dstate=16, ngroups=1, io=1, flags=1)
        n = ctypes.c_size_t(7)
        d = ssd.SelectiveDims(*(o.get(k, v) for k, v in names.items()))
        return lib.ssd_selective_workspace_size(ctypes.byref(d), ctypes.byref(n)), n.value

    def bytes_of(n, channels, N=16):
        return -(-(n - 1) * channels * N * 4 // 256) * 256 + (n - 1) * channels * 4

    # whole tiles of 32 tokens to a segment
    assert size() == (0, bytes_of(32, 64)) and size(channels=1536, seqlen=16384) == (0, bytes_of(16, 1536))
    assert size(channels=1, dstate=1, seqlen=1 << 30)[1] == bytes_of(128, 1, 1)
    assert all(size(dstate=n)[1] > 0 for n in (1, 8, 17, 33, 64, 128))
    assert size(channels=20480) == (0, 0) and size(batch=512) == (0, 0)   # the SMs are taken already
    assert all(size(seqlen=n, channels=c) == (0, 0) for n in (1, 200, 256) for c in (1, 64, 1536, 5120))
    assert size(dstate=0)[0] == 2 and size(dstate=129)[0] == 5
    assert lib.ssd_selective_workspace_size(None, ctypes.byref(ctypes.c_size_t())) == 1
    assert lib.ssd_selective_workspace_size(ctypes.byref(ssd.SelectiveDims(1, 1, 1, 1, 1, 1, 0)), None) == 1

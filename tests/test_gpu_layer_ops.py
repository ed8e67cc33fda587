"""The operators around and beside the scan (convolution, selective scan with its step, gated norm) against their
64-bit forms: every element within the bound that tests/layer_ref.py derives for an f32 evaluation, rounded once."""
import numpy as np
import pytest
import torch

import layer_ref as ref
from chunked_state_space_b200 import ssd

pytestmark = pytest.mark.gpu

IO = {"f32": torch.float32, "bf16": torch.bfloat16}


def rnd(seed, *shape, io="f32", scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (scale * torch.randn(shape, generator=g, device="cuda")).to(IO[io])


def wide(t, before, after):
    """t as a slice of wider rows (its neighbours hold NaN, which nothing may use)."""
    buf = torch.full(t.shape[:-1] + (before + t.shape[-1] + after,), float("nan"), dtype=t.dtype, device=t.device)
    buf[..., before:before + t.shape[-1]] = t
    return buf[..., before:before + t.shape[-1]]


def np64(t):
    return None if t is None else t.detach().to(torch.float64).cpu().numpy()


def close(got, want, bound, io):
    got = np64(got)
    assert np.all(np.isfinite(got))
    over = np.abs(got - want) - ref.stored(want, bound, io)
    assert np.all(over <= 0), (float(np.max(over)), np.unravel_index(np.argmax(over), over.shape))


def lens(values):
    return None if values is None else torch.tensor(values, dtype=torch.int32, device="cuda")


# ---------------------------------------------------------------- convolution

@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("width,B,L,C,pad,silu,init,lengths", [
    (4, 1, 1, 1, (0, 0), True, False, None),              # one token of one channel
    (4, 2, 2, 24, (8, 8), True, True, None),              # shorter than the taps, 16-byte rows in a wider buffer
    (3, 2, 7, 13, (1, 2), True, True, None),              # odd everything
    (2, 3, 9, 64, (0, 0), False, False, None),
    (4, 2, 64, 40, (0, 5), True, True, None),             # rows off 16 bytes
    (4, 1, 131, 72, (8, 0), True, False, None),
    (4, 7, 65, 48, (8, 8), True, True, [65, 0, 1, 2, 3, 64, 40]),
    (2, 3, 5, 3, (0, 0), False, False, [5, 0, 1]),
    (3, 3, 33, 16, (0, 0), True, True, [40, -3, 17]),     # lengths outside [0, L] are taken into it
    (4, 2, 700, 1800, (0, 0), True, True, [700, 333]),    # longer runs of tokens per thread
    (4, 3, 70, 1802, (2, 4), True, True, [70, 69, 1]),    # pairs of elements
    (3, 2, 67, 1801, (1, 4), True, True, None),           # single ones
    (2, 2, 66, 14, (6, 0), False, True, None),
])
def test_conv_matches_64_bits(io, width, B, L, C, pad, silu, init, lengths):
    x, w, b = rnd(1, B, L, C, io=io), rnd(2, C, width), rnd(3, C)
    st = rnd(4, B, width - 1, C, io=io) if init else None
    if lengths is not None:
        for k, n in enumerate(lengths):  # what lies behind a sequence must not matter
            x[k, max(n, 0):] = float("nan")
    n = lens(lengths)
    y = torch.full((B, L, C), 7.0, dtype=IO[io], device="cuda")
    got, fin = ssd.ssd_conv_fwd(wide(x, *pad), w, b, init_state=st, lengths=n, silu=silu, y=y)
    assert got is y
    zeros = np.zeros((B, width - 1, C))
    want, bound, state = ref.conv(np.nan_to_num(np64(x)), np64(w), np64(b), zeros if st is None else np64(st), lengths, silu)
    for k in range(B):
        m = L if lengths is None else min(max(lengths[k], 0), L)
        close(got[k, :m], want[k, :m], bound[k, :m], io)
        assert torch.all(got[k, m:] == 7.0)  # left as they were
    assert np.array_equal(np64(fin), state)
    fresh, none = ssd.ssd_conv_fwd(wide(x, *pad), w, b, init_state=st, lengths=n, silu=silu, want_final=False)
    assert none is None
    for k in range(B):
        m = L if lengths is None else min(max(lengths[k], 0), L)
        assert torch.equal(fresh[k, :m], got[k, :m]) and not fresh[k, m:].any()


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("width,C", [(4, 48), (3, 7), (2, 16), (4, 50)])
def test_conv_in_pieces_and_by_tokens_is_the_whole(io, width, C):
    """A prompt in pieces, its cache updated in place, then token by token: bitwise one call over all tokens."""
    x, w, b = rnd(5, 2, 40, C, io=io), rnd(6, C, width), rnd(7, C)
    whole, last = ssd.ssd_conv_fwd(x, w, b)
    cache = torch.zeros(2, width - 1, C, dtype=IO[io], device="cuda")
    out = []
    for lo, hi in ((0, 1), (1, 3), (3, 30), (30, 31)):
        y, same = ssd.ssd_conv_fwd(x[:, lo:hi], w, b, init_state=cache, final_state=cache)
        assert same is cache
        out.append(y)
    for t in range(31, 40):
        out.append(ssd.ssd_conv_step(x[:, t], w, cache, b)[:, None])
    assert torch.equal(torch.cat(out, 1), whole)
    assert torch.equal(cache, last)


def test_conv_writes_only_its_slice_and_takes_any_row_order():
    x, w = rnd(8, 3, 21, 24, io="bf16"), rnd(9, 24, 4)
    plain, _ = ssd.ssd_conv_fwd(x, w, silu=False)
    buf = torch.full((3, 21, 40), 5.0, dtype=torch.bfloat16, device="cuda")
    ssd.ssd_conv_fwd(x, w, silu=False, y=buf[..., 8:32])
    assert torch.equal(buf[..., 8:32], plain)
    assert torch.all(buf[..., :8] == 5.0) and torch.all(buf[..., 32:] == 5.0)
    turned = torch.empty(21, 3, 24, dtype=torch.bfloat16, device="cuda").transpose(0, 1)
    ssd.ssd_conv_fwd(x.transpose(0, 1).contiguous().transpose(0, 1), w, silu=False, y=turned)
    assert torch.equal(turned, plain)
    one = x[:1].expand(3, 21, 24)  # a broadcast input
    y, _ = ssd.ssd_conv_fwd(one, w, silu=False)
    assert torch.equal(y, plain[:1].expand(3, 21, 24))


def test_conv_offsets_past_32_bits():
    step = 2 ** 28 + 8
    buf = torch.empty(10 * step, dtype=torch.bfloat16, device="cuda")
    x = torch.as_strided(buf, (1, 10, 32), (10 * step, step, 1))
    x.copy_(rnd(10, 1, 10, 32, io="bf16"))
    w = rnd(11, 32, 4)
    y, fin = ssd.ssd_conv_fwd(x, w)
    want, same = ssd.ssd_conv_fwd(x.contiguous(), w)
    assert torch.equal(y, want) and torch.equal(fin, same)
    far = torch.as_strided(buf, (1, 10, 32), (10 * step, step, 1), 64)
    ssd.ssd_conv_fwd(x.contiguous(), w, y=far)
    assert torch.equal(far, want)


# ---------------------------------------------------------------- selective scan

def scan_inputs(io, B, L, C, N, G, seed=20, bias=-2.0, gate=True, pad=(0, 0)):
    d = dict(x=wide(rnd(seed, B, L, C, io=io), *pad), dt=wide(rnd(seed + 1, B, L, C, io=io), *pad),
             A=-torch.exp(rnd(seed + 2, C, N).abs()), D=rnd(seed + 5, C),
             z=wide(rnd(seed + 6, B, L, C, io=io), *pad) if gate else None,
             dt_bias=0.2 * rnd(seed + 7, C) + bias)
    bc = wide(rnd(seed + 3, B, L, 2 * G * N, io=io, scale=N ** -0.5), *pad)
    d["Bm"], d["Cm"] = bc[..., :G * N].unflatten(-1, (G, N)), bc[..., G * N:].unflatten(-1, (G, N))
    return d


def scan_want(d, init, lengths=None, softplus=True):
    f = {k: np64(v) for k, v in d.items()}
    C, N = f["A"].shape
    zero = np.zeros(C)
    return ref.selective(np.nan_to_num(f["x"]), np.nan_to_num(f["dt"]), f["A"], np.nan_to_num(f["Bm"]),
                         np.nan_to_num(f["Cm"]), zero if f["D"] is None else f["D"],
                         None if f["z"] is None else np.nan_to_num(f["z"]),
                         zero if f["dt_bias"] is None else f["dt_bias"],
                         np.zeros((f["x"].shape[0], C, N)) if init is None else np64(init), lengths, softplus)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("B,L,C,N,G,pad,gate,init,lengths", [
    (1, 1, 1, 1, 1, (0, 0), False, False, None),
    (2, 3, 5, 2, 1, (0, 0), True, True, None),
    (1, 40, 64, 16, 1, (0, 0), True, True, None),
    (2, 33, 40, 3, 2, (3, 1), True, False, None),
    (3, 70, 77, 13, 7, (1, 0), True, True, None),
    (2, 31, 36, 16, 2, (8, 8), False, True, None),
    (1, 100, 24, 17, 1, (0, 0), True, True, None),
    (2, 65, 16, 32, 4, (8, 0), True, False, None),
    (1, 37, 10, 64, 2, (0, 0), True, True, None),
    (1, 20, 9, 100, 3, (0, 0), False, True, None),
    (2, 50, 8, 128, 1, (0, 0), True, True, None),
    (7, 130, 96, 16, 1, (8, 8), True, True, [130, 0, 1, 2, 64, 65, 33]),
    (4, 32, 20, 5, 1, (0, 0), True, False, [40, -1, 31, 0]),
    (2, 300, 1300, 16, 1, (0, 0), True, True, [300, 177]),
    (20, 66, 2048, 16, 1, (0, 0), True, False, None),
    (3, 64, 24576, 4, 1, (0, 0), True, False, None),
    # each kernel of the prompt, and each way of loading for it: by the number of channels, aligned and not
    (5, 70, 1024, 16, 1, (8, 8), True, True, None),
    (5, 67, 1025, 15, 1, (1, 0), True, True, None),
    (5, 130, 1024, 16, 2, (8, 1), True, True, [130, 0, 1, 63, 129]),
    (9, 40, 2048, 12, 4, (0, 0), True, True, None),
    (9, 33, 1700, 16, 1, (0, 0), False, False, [33, 32, 31, 0, 1, 17, 8, 9, 40]),
    (5, 70, 1024, 32, 1, (0, 0), True, True, None),
    (5, 35, 1026, 21, 2, (1, 0), True, True, [35, 0, 8, 16, 34]),
    (2, 96, 2000, 8, 1, (0, 0), True, True, None),
    (1, 40, 30, 7, 3, (1, 1), True, True, None),
])
def test_selective_matches_64_bits(io, B, L, C, N, G, pad, gate, init, lengths):
    d = scan_inputs(io, B, L, C, N, G, gate=gate, pad=pad)
    st = rnd(30, B, C, N) if init else None
    if lengths is not None:
        for k, n in enumerate(lengths):
            for name in ("x", "dt", "z", "Bm", "Cm"):
                if d[name] is not None:
                    d[name][k, max(n, 0):] = float("nan")
    y = torch.full((B, L, C), 7.0, dtype=IO[io], device="cuda")
    got, fin = ssd.ssd_selective_fwd(**d, init_state=st, lengths=lens(lengths), y=y)
    want, bound, state, sbound = scan_want(d, st, lengths)
    for k in range(B):
        m = L if lengths is None else min(max(lengths[k], 0), L)
        close(got[k, :m], want[k, :m], bound[k, :m], io)
        assert torch.all(got[k, m:] == 7.0)
    close(fin, state, sbound, "f32")


@pytest.mark.parametrize("name", ["D", "z", "dt_bias", "softplus", "growing"])
def test_selective_without_its_options(name):
    d = scan_inputs("f32", 2, 45, 24, 16, 1, seed=40)
    st = rnd(41, 2, 24, 16)
    softplus = name != "softplus"
    if name in ("D", "z", "dt_bias"):
        d[name] = None
    if name == "softplus":
        d["dt"] = d["dt"].abs() * 0.1
        d["dt_bias"] = None
    if name == "growing":
        d["A"] = 0.02 * d["A"].abs()  # rates above zero: a growing state
    got, fin = ssd.ssd_selective_fwd(**d, init_state=st, softplus=softplus)
    want, bound, state, sbound = scan_want(d, st, softplus=softplus)
    close(got, want, bound, "f32")
    close(fin, state, sbound, "f32")


@pytest.mark.parametrize("value", [-200.0, -60.0, -17.0, -5.0, 0.0, 19.0, 21.0, 88.0, 200.0, 3e4])
def test_selective_steps_of_every_size(value):
    """softplus from where it is e^v (and nothing) to where it is v, and rates down to where the state is forgotten."""
    d = scan_inputs("f32", 1, 9, 32, 16, 1, seed=50)
    d["dt_bias"] = torch.full((32,), value, device="cuda")
    st = rnd(51, 1, 32, 16)
    got, fin = ssd.ssd_selective_fwd(**d, init_state=st)
    want, bound, state, sbound = scan_want(d, st)
    close(got, want, bound, "f32")
    close(fin, state, sbound, "f32")


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("B,C,pad", [(2, 48, (0, 0)), (2, 47, (1, 0)), (5, 1024, (0, 0)), (8, 2048, (0, 0))])
def test_selective_passes_over_masked_steps(io, B, C, pad):
    """A step of -inf or of the type's lowest value is 0: the tokens around it see the state as if it were not there
    (bitwise), in the scan and token by token."""
    d = scan_inputs(io, B, 40, C, 16, 1, seed=57, pad=pad)
    masked = [0, 7, 8, 20, 39]
    d["dt"][:, masked] = torch.tensor([float("-inf"), torch.finfo(IO[io]).min, -3e30, -200.0, float("-inf")],
                                      device="cuda").to(IO[io])[None, :, None]
    kept = [t for t in range(40) if t not in masked]
    part = {k: v[:, kept] if k in ("x", "dt", "z", "Bm", "Cm") else v for k, v in d.items()}
    bc = torch.cat([part["Bm"], part["Cm"]], 2)  # B and C of the kept tokens with one pair of strides
    part["Bm"], part["Cm"] = bc[:, :, :1], bc[:, :, 1:]
    st = rnd(58, B, C, 16)
    y, fin = ssd.ssd_selective_fwd(**d, init_state=st)
    want, same = ssd.ssd_selective_fwd(**part, init_state=st)
    assert torch.isfinite(y).all()
    assert torch.equal(y[:, kept], want) and torch.equal(fin, same)
    cache = st.clone()
    for t in (0, 7, 8):
        ssd.ssd_selective_step(d["x"][:, t], d["dt"][:, t], d["A"], d["Bm"][:, t], d["Cm"][:, t], cache, d["D"],
                               dt_bias=d["dt_bias"])
    assert torch.equal(cache, st)


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_selective_keeps_what_is_not_finite_to_its_channel(bad):
    d = scan_inputs("f32", 1, 70, 48, 16, 1, seed=55)
    clean, last = ssd.ssd_selective_fwd(**d)
    d["x"][0, 40, 5] = bad
    y, fin = ssd.ssd_selective_fwd(**d)
    other = torch.arange(48, device="cuda") != 5
    assert torch.equal(y[:, :, other], clean[:, :, other]) and torch.equal(fin[:, other], last[:, other])
    assert torch.equal(y[:, :40], clean[:, :40]) and not torch.isfinite(y[0, 40:, 5]).any()
    assert not torch.isfinite(fin[0, 5]).any()


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("B,C,N,G", [(2, 48, 16, 1), (1, 21, 13, 3), (3, 8, 1, 2), (2, 10, 128, 1), (2, 33, 6, 1),
                                     (1, 24, 64, 2), (40, 520, 16, 1)])
def test_selective_by_tokens_matches_64_bits(io, B, C, N, G):
    L = 6
    d = scan_inputs(io, B, L, C, N, G, seed=60, pad=(3, 2))
    st = rnd(61, B, C, N)
    want, bound, state, sbound = scan_want(d, st)
    cache = st.clone()
    for t in range(L):
        y = ssd.ssd_selective_step(d["x"][:, t], d["dt"][:, t], d["A"], d["Bm"][:, t], d["Cm"][:, t], cache, d["D"],
                                   z=d["z"][:, t], dt_bias=d["dt_bias"])
        close(y, want[:, t], bound[:, t], io)
    close(cache, state, sbound, "f32")


def test_selective_in_pieces_is_the_whole():
    d = scan_inputs("bf16", 2, 150, 48, 16, 1, seed=70)
    st = rnd(71, 2, 48, 16)
    want, bound, state, sbound = scan_want(d, st)
    cache, out = st.clone(), []
    for lo, hi in ((0, 1), (1, 64), (64, 150)):
        part = {k: v[:, lo:hi] if k in ("x", "dt", "z", "Bm", "Cm") else v for k, v in d.items()}
        out.append(ssd.ssd_selective_fwd(**part, init_state=cache, final_state=cache)[0])
    close(torch.cat(out, 1), want, bound, "bf16")
    close(cache, state, sbound, "f32")


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("B,L,C,N,G,pad,lengths", [
    (1, 2000, 64, 16, 1, (8, 0), None),
    (1, 1500, 30, 13, 3, (1, 0), None),
    (3, 1301, 65, 16, 1, (0, 0), [1301, 0, 640]),
    (2, 1024, 40, 3, 1, (0, 2), [1, 1024]),
    (4, 900, 32, 16, 1, (0, 0), None),
    (1, 600, 64, 8, 1, (0, 0), None), (1, 1500, 400, 8, 2, (0, 0), None), (1, 1500, 401, 5, 1, (1, 0), None),
    (1, 1500, 400, 16, 1, (0, 0), None), (1, 1500, 401, 14, 1, (1, 0), None), (2, 1400, 400, 16, 1, (0, 0), [1400, 33]),
    (1, 1000, 64, 32, 1, (0, 0), None), (1, 1500, 400, 32, 1, (0, 0), None), (1, 1500, 400, 29, 2, (0, 0), None),
    (1, 1000, 64, 64, 2, (0, 0), None), (1, 1000, 63, 50, 1, (1, 0), None), (1, 1000, 64, 128, 1, (0, 0), None),
    (1, 1000, 33, 70, 1, (0, 0), None), (1, 3000, 1536, 16, 1, (0, 0), None), (1, 1500, 1001, 13, 1, (1, 0), None),
    (1, 1500, 1601, 5, 1, (1, 0), None), (1, 1500, 1401, 29, 1, (1, 0), None), (1, 1500, 1400, 32, 1, (0, 0), None),
])
def test_selective_in_segments(io, B, L, C, N, G, pad, lengths):
    """Long sequences of few channels: cut into segments, as one, and in place."""
    d = scan_inputs(io, B, L, C, N, G, seed=75, bias=-4.0, pad=pad)
    dims = ssd.SelectiveDims(B, L, C, N, G, int(io == "bf16"), 1)
    size = ssd.ssd_selective_workspace_size(dims)
    assert size > 0
    st = rnd(76, B, C, N)
    if lengths is not None:
        for k, n in enumerate(lengths):
            for name in ("x", "dt", "z", "Bm", "Cm"):
                d[name][k, n:] = float("nan")
    want, bound, state, sbound = scan_want(d, st, lengths)
    ws = torch.full((size,), 255, dtype=torch.uint8, device="cuda")  # NaN: nothing is read before it is written
    y = torch.full((B, L, C), 7.0, dtype=IO[io], device="cuda")
    cache = st.clone()
    got, fin = ssd.ssd_selective_fwd(**d, init_state=cache, final_state=cache, lengths=lens(lengths), y=y, workspace=ws)
    assert fin is cache
    for k in range(B):
        m = L if lengths is None else lengths[k]
        close(got[k, :m], want[k, :m], bound[k, :m], io)
        assert torch.all(got[k, m:] == 7.0)
    close(cache, state, sbound, "f32")
    again, last = ssd.ssd_selective_fwd(**d, init_state=st, lengths=lens(lengths))
    for k in range(B):
        m = L if lengths is None else lengths[k]
        assert torch.equal(again[k, :m], got[k, :m])
    assert torch.equal(last, cache)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    there = [ssd.ssd_selective_fwd(**d, init_state=st, lengths=lens(lengths), stream=s)
             for s in (side, side.cuda_stream)]
    side.synchronize()
    assert all(torch.equal(f, cache) for _, f in there)
    zero, _ = ssd.ssd_selective_fwd(**d, lengths=lens(lengths), want_final=False)
    want, bound, _, _ = scan_want(d, None, lengths)
    for k in range(B):
        m = L if lengths is None else lengths[k]
        close(zero[k, :m], want[k, :m], bound[k, :m], io)


def test_selective_in_segments_with_growing_states():
    """Rates above 0: a segment's factor is infinite while the state is still 0, which it then stays."""
    d = scan_inputs("f32", 1, 2000, 16, 16, 1, seed=78)
    d["A"] = torch.full_like(d["A"], 4.0)
    d["dt_bias"] = torch.zeros_like(d["dt_bias"])
    d["dt"][:, :1000], d["dt"][:, 1000:] = 1.0, -12.0
    d["x"][:, :1000] = 0.0
    assert ssd.ssd_selective_workspace_size(ssd.SelectiveDims(1, 2000, 16, 16, 1, 0, 1)) > 0
    want, bound, state, sbound = scan_want(d, None, None)
    got, fin = ssd.ssd_selective_fwd(**d)
    close(got, want, bound, "f32")
    close(fin, state, sbound, "f32")


def test_zeros_behind_sequences_on_another_stream():
    """A y made for a padded batch is filled on the stream that then writes it, not behind it on the current one."""
    d = scan_inputs("bf16", 2, 300, 64, 16, 1, seed=79)
    ln = lens([300, 120])
    w, b = rnd(81, 64, 4), rnd(82, 64)
    want = ssd.ssd_selective_fwd(**d, lengths=ln)[0], ssd.ssd_conv_fwd(d["x"], w, b, lengths=ln)[0]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for s in (side, side.cuda_stream):
        torch.cuda._sleep(200_000_000)  # about a tenth of a second of the current stream
        got = [ssd.ssd_selective_fwd(**d, lengths=ln, stream=s)[0], ssd.ssd_conv_fwd(d["x"], w, b, lengths=ln, stream=s)[0]]
        torch.cuda.synchronize()
        for g, y in zip(got, want):
            assert torch.equal(g, y)


def test_selective_refuses_workspaces():
    d = scan_inputs("bf16", 1, 2000, 64, 16, 1, seed=83)
    size = ssd.ssd_selective_workspace_size(ssd.SelectiveDims(1, 2000, 64, 16, 1, 1, 1))
    byte = torch.zeros(1, dtype=torch.uint8, device="cuda")
    for ws in (byte.expand(size), byte, torch.zeros(size), torch.zeros(size + 8, dtype=torch.uint8, device="cuda")[8:]):
        with pytest.raises(ssd.SSDError):
            ssd.ssd_selective_fwd(**d, workspace=ws)


def test_selective_in_segments_captured():
    """Its launches and workspace inside a graph: two graphs, replayed in turn, keep to their own."""
    graphs, held, ins, outs = [], [], [], []
    for seed in (77, 87):
        d = scan_inputs("bf16", 1, 1200, 48, 16, 1, seed=seed)
        ssd.ssd_selective_fwd(**d)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            held.append(ssd.ssd_selective_fwd(**d))
        graphs.append(g)
        ins.append(d)
    for k in range(2):
        for i in range(2):
            ins[i]["x"].copy_(rnd(97 + 2 * k + i, *ins[i]["x"].shape, io="bf16"))
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        for d, (y, fin) in zip(ins, held):
            want, last = ssd.ssd_selective_fwd(**d)
            assert torch.equal(y, want) and torch.equal(fin, last)
    del graphs


def test_selective_with_one_rate_is_the_vector_decay_scan():
    """With x scaled by the step, one channel per head and N rates: ssd_scan_fwd_vdecay at head dim 1."""
    d = scan_inputs("f32", 2, 50, 12, 16, 2, seed=80, gate=False)
    y, fin = ssd.ssd_selective_fwd(**d)
    step = torch.nn.functional.softplus(d["dt"] + d["dt_bias"])
    v, vf = ssd.ssd_scan_fwd_vdecay((step * d["x"])[..., None].contiguous(), step, d["A"], d["Bm"].contiguous(),
                                    d["Cm"].contiguous())
    torch.testing.assert_close(v[..., 0] + d["D"] * d["x"], y, rtol=1e-5, atol=1e-5)
    torch.testing.assert_close(vf[..., 0], fin, rtol=1e-5, atol=1e-5)


def test_selective_offsets_past_32_bits():
    step = 2 ** 28 + 8
    buf = torch.empty(10 * step, dtype=torch.bfloat16, device="cuda")
    d = scan_inputs("bf16", 1, 10, 32, 16, 1, seed=90)
    want, fin = ssd.ssd_selective_fwd(**d)
    far = {k: torch.as_strided(buf, (1, 10, 32), (10 * step, step, 1), 64 * i) for i, k in enumerate(("x", "dt", "z"))}
    for k, v in far.items():
        v.copy_(d[k])
    y = torch.as_strided(buf, (1, 10, 32), (10 * step, step, 1), 10 * 64)
    with pytest.raises(ssd.SSDError):  # their extents meet: refused, as for every other scan
        ssd.ssd_selective_fwd(**{**d, **far}, y=y)
    got, same = ssd.ssd_selective_fwd(**{**d, **far})
    assert torch.equal(got, want) and torch.equal(same, fin)
    ssd.ssd_selective_fwd(**d, y=y)
    assert torch.equal(y, want)


# ---------------------------------------------------------------- gated norm

@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("B,L,F,G,pad,gate,weighted", [
    (1, 1, 1, 1, (0, 0), True, True), (2, 3, 7, 1, (1, 1), True, True), (2, 5, 64, 2, (8, 8), True, False),
    (3, 4, 1530, 2, (0, 0), True, True), (2, 9, 1024, 1, (0, 8), False, True), (1, 6, 1040, 1, (8, 0), True, True),
    (2, 3, 5120, 1, (0, 0), True, True), (1, 2, 5121, 1, (0, 0), True, True), (1, 2, 32768 + 8, 1, (0, 0), True, True),
    (2, 2, 9000, 2, (1, 0), True, True), (1, 2, 48, 48, (0, 0), False, False),
    # parts of a warp, and each number of pieces that a warp holds
    (3, 67, 64, 8, (0, 0), True, True), (2, 33, 192, 3, (8, 0), False, True), (2, 5, 130, 10, (1, 0), True, True),
    (5, 41, 256, 1, (0, 0), True, True), (2, 700, 512, 1, (0, 0), True, True), (2, 9, 760, 1, (0, 0), True, False),
    (700, 3, 1160, 1, (0, 0), True, True), (3, 3, 1288, 1, (0, 0), True, True), (1500, 2, 2568, 1, (8, 8), True, True),
    # pairs of elements
    (3, 4, 1530, 1, (2, 2), True, True), (2, 3, 130, 5, (4, 2), True, True), (1, 2, 13002, 1, (2, 0), True, True),
])
def test_gated_norm_matches_64_bits(io, B, L, F, G, pad, gate, weighted):
    x, z = rnd(100, B, L, F, io=io), rnd(101, B, L, F, io=io) if gate else None
    w = rnd(102, F) if weighted else None
    x[0, 0] = 0  # a row of zeros: eps alone
    got = ssd.ssd_rmsnorm_gated(wide(x, *pad), None if z is None else wide(z, *pad), w, eps=1e-5, ngroups=G)
    want, bound = ref.gated_norm(np64(x), np64(z), np.ones(F) if w is None else np64(w), 1e-5, G)
    close(got, want, bound, io)
    again = ssd.ssd_rmsnorm_gated(x[:, 0], None if z is None else z[:, 0], w, eps=1e-5, ngroups=G)
    close(again, want[:, 0], bound[:, 0], io)
    same = x.clone()
    assert ssd.ssd_rmsnorm_gated(same, z, w, eps=1e-5, ngroups=G, out=same) is same
    close(same, want, bound, io)


def test_gated_norm_without_gate_is_the_norm():
    x = rnd(110, 2, 3, 4, 64, io="bf16")
    assert torch.equal(ssd.ssd_rmsnorm_gated(x.flatten(2), eps=1e-6), ssd.ssd_rmsnorm(x, 1e-6).flatten(2))


# ---------------------------------------------------------------- all of them: streams, graphs, refusals

def calls():
    """One call of each operator on tensors of its own: a function that runs it and returns its outputs, the input
    that a later replay changes, and what it updates in place."""
    x, w = rnd(120, 2, 50, 48, io="bf16"), rnd(121, 48, 4)
    d = scan_inputs("bf16", 2, 50, 48, 16, 1, seed=122)
    cache, state = rnd(130, 2, 3, 48, io="bf16"), rnd(131, 2, 48, 16)
    tok = {k: (v[:, 0].contiguous() if k in ("x", "dt", "z", "Bm", "Cm") else v) for k, v in d.items()}
    g, norm_w = rnd(132, 2, 50, 48, io="bf16"), rnd(133, 48)
    return {
        "conv": (lambda: ssd.ssd_conv_fwd(x, w), x, None),
        "conv_step": (lambda: ssd.ssd_conv_step(x[:, 0], w, cache), x, cache),
        "selective": (lambda: ssd.ssd_selective_fwd(**d), d["x"], None),
        "selective_step": (lambda: ssd.ssd_selective_step(**tok, state=state), tok["x"], state),
        "norm": (lambda: ssd.ssd_rmsnorm_gated(x, g, norm_w), x, None),
    }


def flat(r):
    return [t.clone() for t in (r if isinstance(r, tuple) else (r,))]


@pytest.mark.parametrize("name", ["conv", "conv_step", "selective", "selective_step", "norm"])
def test_captured_replayed_and_on_another_stream(name):
    fn, x, inplace = calls()[name]
    saved = None if inplace is None else inplace.clone()

    def eager():
        if inplace is not None:
            inplace.copy_(saved)
        out = flat(fn())
        return out + ([] if inplace is None else [inplace.clone()])

    want = eager()
    other = torch.cuda.Stream()
    other.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(other):
        got = eager()
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(want, got))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        held = fn()
    for k in range(2):
        x.copy_(rnd(140 + k, *x.shape, io="bf16"))
        want = eager()
        if inplace is not None:
            inplace.copy_(saved)
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(want, flat(held)))
        assert inplace is None or torch.equal(inplace, want[-1])
    del g


def test_the_binding_refuses_what_the_kernels_do_not_take():
    x, w = rnd(150, 2, 9, 32, io="bf16"), rnd(151, 32, 4)
    d = scan_inputs("bf16", 2, 9, 32, 16, 1, seed=152)

    def refused(status, fn, *a, **k):
        with pytest.raises(ssd.SSDError) as e:
            fn(*a, **k)
        assert e.value.status == status

    conv, scan, norm = ssd.ssd_conv_fwd, ssd.ssd_selective_fwd, ssd.ssd_rmsnorm_gated
    refused(1, conv, x.cpu(), w)
    refused(3, conv, x.half(), w)
    refused(3, conv, x, w.bfloat16())
    refused(2, conv, x, w[:31])
    refused(2, conv, x[0], w)
    refused(5, conv, x, rnd(153, 32, 5))
    refused(5, conv, x, rnd(153, 32, 1))
    refused(1, conv, x, rnd(154, 4, 32).t())
    refused(2, conv, x.transpose(1, 2).contiguous().transpose(1, 2), w)
    refused(3, conv, x, w, lengths=torch.ones(2, dtype=torch.int64, device="cuda"))
    refused(1, conv, x, w, y=x)
    refused(2, conv, x, w, y=torch.empty(1, 9, 32, dtype=x.dtype, device="cuda").expand(2, 9, 32))
    refused(2, conv, x[:0], w)
    refused(2, conv, x, w, init_state=torch.zeros(2, 4, 32, dtype=x.dtype, device="cuda"))
    refused(3, scan, **{**d, "dt": d["dt"].float()})
    refused(2, scan, **{**d, "A": d["A"][:, :8]})
    refused(2, scan, **{**d, "Cm": d["Cm"].contiguous()})       # other strides than Bm
    refused(2, scan, **{**d, "Bm": d["Bm"][:, :8], "Cm": d["Cm"][:, :8]})
    refused(1, scan, **d, y=d["z"])
    refused(1, scan, **{**d, "A": d["A"].cpu()})
    refused(2, norm, x, z=x[:, :8])
    refused(2, norm, x, ngroups=5)
    refused(1, norm, x, eps=float("nan"))
    refused(1, norm, x, z=rnd(155, 2, 9, 32, io="bf16"), weight=rnd(156, 32).cpu())
    z = rnd(157, 2, 9, 32, io="bf16")
    refused(1, norm, x, z=z, out=z)


# ---------------------------------------------------------------- as they are used

@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_a_layer_with_the_selective_scan_prompt_then_tokens(io):
    """A padded batch of prompts through convolution and gated scan, then tokens through their single-token forms,
    against the 64-bit forms run over each sequence's own tokens."""
    B, L, C, N, R, K = 3, 40, 64, 16, 4, 3
    lengths = [40, 17, 2]
    rows = rnd(160, B, L + K, 2 * C, io=io)               # [x | z] of a projection
    w, bias = rnd(161, C, 4, scale=0.5), rnd(162, C)
    Wx, Wdt = rnd(163, C, R + 2 * N, scale=C ** -0.5).to(IO[io]), rnd(164, R, C, scale=R ** -0.5).to(IO[io])
    A, D, dtb = -torch.exp(rnd(165, C, N).abs()), rnd(166, C), rnd(167, C) * 0.2 - 2

    def parts(u):
        p = u @ Wx
        return p[..., :R] @ Wdt, p[..., R:R + N].unflatten(-1, (1, N)), p[..., R + N:].unflatten(-1, (1, N))

    n = lens(lengths)
    u, cache = ssd.ssd_conv_fwd(rows[:, :L, :C], w, bias, lengths=n)
    dt, Bm, Cm = parts(u)
    y, state = ssd.ssd_selective_fwd(u, dt, A, Bm, Cm, D, z=rows[:, :L, C:], dt_bias=dtb, lengths=n)
    zeros = np.zeros((B, 3, C))
    cw, cb, cs = ref.conv(np64(rows[:, :L, :C]), np64(w), np64(bias), zeros, lengths, True)
    sw, sb, ss, sse = ref.selective(np64(u), np64(dt), np64(A), np64(Bm), np64(Cm), np64(D), np64(rows[:, :L, C:]),
                                    np64(dtb), np.zeros((B, C, N)), lengths, True)
    for k, m in enumerate(lengths):
        close(u[k, :m], cw[k, :m], cb[k, :m], io)
        close(y[k, :m], sw[k, :m], sb[k, :m], io)
    close(state, ss, sse, "f32")
    for j in range(K):
        before, h = np64(cache), np64(state)
        row = rows[:, L + j]
        u1 = ssd.ssd_conv_step(row[:, :C], w, cache, bias)
        dt1, B1, C1 = parts(u1)
        y1 = ssd.ssd_selective_step(u1, dt1, A, B1, C1, state, D, z=row[:, C:], dt_bias=dtb)
        cw, cb, cs = ref.conv(np64(row[:, None, :C]), np64(w), np64(bias), before, None, True)
        close(u1, cw[:, 0], cb[:, 0], io)
        assert np.array_equal(np64(cache), cs)
        sw, sb, ss, sse = ref.selective(*(np64(t)[:, None] for t in (u1, dt1)), np64(A), np64(B1)[:, None],
                                        np64(C1)[:, None], np64(D), np64(row[:, None, C:]), np64(dtb), h, None, True)
        close(y1, sw[:, 0], sb[:, 0], io)
        close(state, ss, sse, "f32")


def test_a_layer_with_the_chunked_scan_prompt_then_tokens():
    """Convolution over x, B and C in one projection row, the chunked scan on slices of its output, the gated norm;
    then tokens: conv step, scan step, norm.  Each operator against its 64-bit form on what it was given."""
    import oracle
    B, L, H, P, N = 2, 300, 4, 64, 128
    HP, K = H * P, 2
    rows = rnd(170, B, L + K, 2 * HP + 2 * N, io="bf16")  # [z | x | B | C]
    w, bias, weight = rnd(171, HP + 2 * N, 4, scale=0.5), rnd(172, HP + 2 * N), 1 + 0.1 * rnd(173, HP)
    dt = torch.nn.functional.softplus(rnd(174, B, L + K, H) - 2)
    A, D = -torch.exp(rnd(175, H).abs()), rnd(176, H)
    u, cache = ssd.ssd_conv_fwd(rows[:, :L, HP:], w, bias)
    cut = lambda t: (t[..., :HP].unflatten(-1, (H, P)), t[..., HP:HP + N].unflatten(-1, (1, N)),  # noqa: E731
                     t[..., HP + N:].unflatten(-1, (1, N)))
    xs, Bm, Cm = cut(u)
    y, state = ssd.ssd_scan_fwd_strided(xs, dt[:, :L], A, Bm, Cm, D)
    out = ssd.ssd_rmsnorm_gated(y.flatten(2), rows[:, :L, :HP], weight)
    cw, cb, cs = ref.conv(np64(rows[:, :L, HP:]), np64(w), np64(bias), np.zeros((B, 3, HP + 2 * N)), None, True)
    close(u, cw, cb, "bf16")
    yr, sr = oracle.scan_recurrence(np64(xs), np64(dt[:, :L]), np64(A), np64(Bm), np64(Cm), np64(D),
                                    np.zeros((B, H, N, P)))
    assert np.max(np.abs(np64(y) - yr)) <= 5e-3 * np.max(np.abs(yr))
    nw, nb = ref.gated_norm(np64(y.flatten(2)), np64(rows[:, :L, :HP]), np64(weight), 1e-5, 1)
    close(out, nw, nb, "bf16")
    for j in range(K):
        row, h, before = rows[:, L + j], np64(state), np64(cache)
        u1 = ssd.ssd_conv_step(row[:, HP:], w, cache, bias)
        x1, B1, C1 = (t.contiguous() for t in cut(u1))
        y1 = ssd.ssd_step(x1, dt[:, L + j].contiguous(), A, B1, C1, state, D=D)
        out1 = ssd.ssd_rmsnorm_gated(y1.flatten(1), row[:, :HP], weight)
        cw, cb, cs = ref.conv(np64(row[:, None, HP:]), np64(w), np64(bias), before, None, True)
        close(u1, cw[:, 0], cb[:, 0], "bf16")
        yr, sr = oracle.scan_recurrence(*(np64(t)[:, None] for t in (x1, dt[:, L + j])), np64(A), np64(B1)[:, None],
                                        np64(C1)[:, None], np64(D), h)
        assert np.max(np.abs(np64(y1) - yr[:, 0])) <= 5e-3 * np.max(np.abs(yr))
        nw, nb = ref.gated_norm(np64(y1.flatten(1)), np64(row[:, :HP]), np64(weight), 1e-5, 1)
        close(out1, nw, nb, "bf16")

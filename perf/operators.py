"""The operators of a selective state-space layer around and beside the chunked scan, as work to time and check.

Five operators: the short causal convolution before a scan (a prompt, one token), the selective scan with a step per
channel (a prompt, one token), and the gated RMS norm behind a scan.  ``run`` computes them in their plain form, in
32 bits with elementary torch operations, or, where ``own`` is set, by this package's kernels.
"""
import math

import torch

own = False

WIDTH = 4     # taps of the convolution where a case names none
DEV = "cuda"


# ---------------------------------------------------------------- cases

def listed():
    return [
        # the convolution over x, B and C of the 2.7B-shaped layer's whole workload, a slice of its projection
        dict(name="conv_prompt_2p7b_bf16", op="conv", dtype="bf16", batch=8, seqlen=16384, channels=5376, before=5120,
             after=80, init=False, ragged=False),
        # a padded batch of prompts of different lengths, continuing from a cache, 32-bit 130M-shaped layer
        dict(name="conv_ragged_f32", op="conv", dtype="f32", batch=5, seqlen=1111, channels=1792, before=1536, after=24,
             init=True, ragged=True),
        # one token of one sequence: latency
        dict(name="conv_token_1_bf16", op="conv_step", dtype="bf16", batch=1, channels=1792, before=1536, after=24),
        # one token of many sequences
        dict(name="conv_token_256_bf16", op="conv_step", dtype="bf16", batch=256, channels=5376, before=5120, after=80),
        # prompts of a batch at the 2.7B layer's inner width, gated, z a slice of the projection
        dict(name="scan_prompt_8_bf16", op="scan", dtype="bf16", batch=8, seqlen=2048, channels=5120, dstate=16,
             ngroups=1, gate=True, init=False, ragged=False, slow=False, sliced=True),
        # one long prompt at the 130M layer's inner width, slow decay, continuing from a state
        dict(name="scan_long_1_bf16", op="scan", dtype="bf16", batch=1, seqlen=16384, channels=1536, dstate=16,
             ngroups=1, gate=True, init=True, ragged=False, slow=True, sliced=False),
        # a padded batch, odd sizes (rows that are no multiple of 16 bytes), two groups
        dict(name="scan_ragged_odd_bf16", op="scan", dtype="bf16", batch=5, seqlen=777, channels=1530, dstate=13,
             ngroups=2, gate=True, init=True, ragged=True, slow=False, sliced=True),
        # a small 32-bit layer without a gate: latency
        dict(name="scan_small_f32", op="scan", dtype="f32", batch=2, seqlen=256, channels=64, dstate=16, ngroups=1,
             gate=False, init=True, ragged=False, slow=False, sliced=False),
        # one token of one sequence: latency
        dict(name="scan_token_1_bf16", op="scan_step", dtype="bf16", batch=1, channels=5120, dstate=16, ngroups=1,
             gate=True),
        # one token of many sequences: the state's traffic
        dict(name="scan_token_256_bf16", op="scan_step", dtype="bf16", batch=256, channels=5120, dstate=16, ngroups=1,
             gate=True),
        # the norm behind the 2.7B-shaped layer's scan
        dict(name="norm_prompt_bf16", op="norm", dtype="bf16", batch=8, seqlen=2048, features=5120, ngroups=1,
             gate=True, after=5456),
        # the norm of one token of 64 sequences, two groups of features
        dict(name="norm_token_64_bf16", op="norm", dtype="bf16", batch=64, seqlen=1, features=1536, ngroups=2,
             gate=True, after=1816),
    ]


def draw(rng):
    def size(lo, hi):  # spread over the logarithm, both ends included
        return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))

    def channels(lo, hi):  # half of them whole 16-byte rows, half of them any
        c = size(lo, hi)
        return max(lo, c // 64 * 64) if rng.random() < 0.5 else c

    op = rng.choice(["conv", "conv_step", "scan", "scan", "scan_step", "norm"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    c = dict(op=op, dtype=dtype)
    if op in ("conv", "conv_step"):
        n = channels(32, 7168)
        c.update(channels=n, before=rng.choice([0, n, size(1, 5120)]), after=rng.choice([0, 80, size(1, 200)]),
                 width=rng.choice([2, 3, 4, 4]))
        if op == "conv":
            batch = size(1, 16)
            most = 8 * 16384 * 5376 // (batch * n * (2 if dtype == "f32" else 1)) // 2
            c.update(batch=batch, seqlen=size(1, min(16384, max(1, most))), init=rng.random() < 0.5,
                     ragged=batch > 1 and rng.random() < 0.5)
        else:
            c.update(batch=size(1, min(256, 256 * 5376 // n)))
    elif op in ("scan", "scan_step"):
        g = rng.choice([1, 1, 1, 2, 4])
        n = max(1, channels(32, 5120) // g) * g
        # 16 state entries are the common case; others from one to the largest that the scan takes
        c.update(channels=n, ngroups=g, dstate=rng.choice([16, 16, 16, size(1, 128)]), gate=rng.random() < 0.7)
        if op == "scan":
            batch = size(1, 8)
            most = 8 * 2048 * 5120 * 16 // (batch * n * c["dstate"]) // 2
            c.update(batch=batch, seqlen=size(1, min(16384, max(1, most))), init=rng.random() < 0.5,
                     ragged=batch > 1 and rng.random() < 0.5, slow=rng.random() < 0.5, sliced=rng.random() < 0.5)
        else:
            c.update(batch=size(1, max(1, min(256, 256 * 16 * 5120 // (n * c["dstate"])))))
    else:
        g = rng.choice([1, 1, 2, 8])
        n = max(1, channels(32, 7168) // g) * g
        rows = size(1, 8 * 2048 * 5120 // 2 // n)
        batch = rng.choice([1, size(1, 8)])
        c.update(features=n, ngroups=g, batch=batch, seqlen=max(1, min(16384, rows // batch)), gate=rng.random() < 0.8,
                 after=rng.choice([0, n, size(1, 5456)]))
    return c


def _lengths(case):
    """The tokens of each sequence of a padded batch: the first full, the third empty, the second a single token."""
    L, B = case["seqlen"], case["batch"]
    if not case["ragged"]:
        return [L] * B
    some = [L, 1, 0]
    return [some[b] if b < 3 else 1 + (b * 7919) % L for b in range(B)]


def work(case):
    es = 2 if case["dtype"] == "bf16" else 4
    op, B = case["op"], case["batch"]
    if op == "conv":
        t, c, w = sum(_lengths(case)), case["channels"], case.get("width", WIDTH)
        states = (2 if case["init"] else 1) * B * (w - 1) * c * es
        return {"bytes": 2 * t * c * es + states + 4 * c * (w + 1), "flops": t * c * (2 * w + 4)}
    if op == "conv_step":
        c, w = case["channels"], case.get("width", WIDTH)
        return {"bytes": B * c * es * (2 * (w - 1) + 2) + 4 * c * (w + 1), "flops": B * c * (2 * w + 4)}
    if op in ("scan", "scan_step"):
        t = sum(_lengths(case)) if op == "scan" else B
        c, n, g = case["channels"], case["dstate"], case["ngroups"]
        states = (2 if op == "scan_step" or case["init"] else 1) * B * c * n * 4
        return {"bytes": t * c * es * (4 if case["gate"] else 3) + 2 * t * g * n * es + states + 4 * c * (n + 2),
                "flops": t * c * (7 * n + 10)}
    t, f = B * case["seqlen"], case["features"]
    return {"bytes": t * f * es * (3 if case["gate"] else 2) + 4 * f, "flops": t * f * 9}


# ---------------------------------------------------------------- inputs

def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    io = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
    op, B = case["op"], case["batch"]

    def randn(*shape, dtype=torch.float32):
        return torch.randn(shape, generator=gen, device=DEV, dtype=dtype)

    def rand(*shape):
        return torch.rand(shape, generator=gen, device=DEV)

    s = {"op": op}
    if case.get("ragged"):
        s["lengths"] = torch.tensor(_lengths(case), dtype=torch.int32, device=DEV)
    if op in ("conv", "conv_step"):
        c, w, lo = case["channels"], case.get("width", WIDTH), case["before"]
        rows = (B, case["seqlen"]) if op == "conv" else (B,)
        s["x"] = randn(*rows, lo + c + case["after"], dtype=io)[..., lo:lo + c]  # a slice of a projection's output
        s["weight"] = randn(c, w) / math.sqrt(w)
        s["bias"] = 0.1 * randn(c)
        state = randn(B, w - 1, c, dtype=io)
        if op == "conv_step":
            s["state"] = state
        else:
            s["init"] = state if case["init"] else None
            s["y"] = torch.zeros(B, case["seqlen"], c, dtype=io, device=DEV) if case["ragged"] else None
    elif op in ("scan", "scan_step"):
        c, n, g = case["channels"], case["dstate"], case["ngroups"]
        rows = (B, case["seqlen"]) if op == "scan" else (B,)
        rank = -(-c // 32)  # B and C are the last columns of a projection to (rank, B, C)
        bc = randn(*rows, rank + 2 * g * n, dtype=io) / math.sqrt(n)
        s["B"] = bc[..., rank:rank + g * n].unflatten(-1, (g, n))
        s["C"] = bc[..., rank + g * n:].unflatten(-1, (g, n))
        s["x"], s["dt"] = randn(*rows, c, dtype=io), randn(*rows, c, dtype=io)
        s["z"] = None
        if case["gate"]:
            s["z"] = randn(*rows, 2 * c, dtype=io)[..., c:] if case.get("sliced") else randn(*rows, c, dtype=io)
        s["dt_bias"] = 0.2 * randn(c) - (4.0 if case.get("slow") else 2.0)
        s["A"] = -torch.exp(rand(c, n) * math.log(16.0))
        s["D"] = randn(c)
        state = math.sqrt(0.1) * randn(B, c, n)
        if op == "scan_step":
            s["state"] = state
        else:
            s["init"] = state if case["init"] else None
            s["y"] = torch.zeros(B, case["seqlen"], c, dtype=io, device=DEV) if case["ragged"] else None
    else:
        f, rows = case["features"], (B, case["seqlen"])
        s["x"] = randn(*rows, f, dtype=io)
        s["z"] = randn(*rows, f + case["after"], dtype=io)[..., :f] if case["gate"] else None
        s["weight"] = 1.0 + 0.1 * randn(f)
        s["groups"] = case["ngroups"]
    return s


# ---------------------------------------------------------------- one pass

def run(s):
    if own:
        return _kernels(s)
    return {"conv": _conv, "conv_step": _conv_step, "scan": _scan, "scan_step": _scan_step, "norm": _norm}[s["op"]](s)


def _kernels(s):
    from chunked_state_space_b200 import ssd
    if s["op"] == "conv":
        y, state = ssd.ssd_conv_fwd(s["x"], s["weight"], s["bias"], init_state=s["init"], lengths=s.get("lengths"),
                                    silu=True, y=s["y"])
    elif s["op"] == "conv_step":
        state = s["state"]
        y = ssd.ssd_conv_step(s["x"], s["weight"], state, s["bias"], silu=True)
    elif s["op"] == "scan":
        y, state = ssd.ssd_selective_fwd(s["x"], s["dt"], s["A"], s["B"], s["C"], s["D"], z=s["z"],
                                         dt_bias=s["dt_bias"], init_state=s["init"], lengths=s.get("lengths"),
                                         softplus=True, y=s["y"])
    elif s["op"] == "scan_step":
        state = s["state"]
        y = ssd.ssd_selective_step(s["x"], s["dt"], s["A"], s["B"], s["C"], state, s["D"], z=s["z"],
                                   dt_bias=s["dt_bias"], softplus=True)
    else:
        return {"y": ssd.ssd_rmsnorm_gated(s["x"], s["z"], s["weight"], eps=1e-5, ngroups=s["groups"])}
    return {"y": y, "state": state}


def _silu(v):
    return v / (1.0 + torch.exp(-v))


def _softplus(v):
    return torch.clamp(v, min=0.0) + torch.log1p(torch.exp(-torch.abs(v)))


def _conv(s):
    x, w = s["x"].float(), s["weight"]
    B, L, c = x.shape
    taps = w.shape[1]
    first = s["init"].float() if s["init"] is not None else x.new_zeros(B, taps - 1, c)
    seen = torch.cat([first, x], dim=1)
    y = _silu(sum(seen[:, k:k + L] * w[:, k] for k in range(taps)) + s["bias"]).to(s["x"].dtype)
    if "lengths" not in s:
        return {"y": y, "state": seen[:, L:].to(s["x"].dtype)}
    n = s["lengths"].long()
    inside = torch.arange(L, device=x.device) < n[:, None]
    last = n[:, None] + torch.arange(taps - 1, device=x.device)
    state = seen.gather(1, last[:, :, None].expand(B, taps - 1, c)).to(s["x"].dtype)
    return {"y": torch.where(inside[:, :, None], y, s["y"]), "state": state}


def _conv_step(s):
    seen = torch.cat([s["state"].float(), s["x"].float()[:, None]], dim=1)
    y = _silu((seen * s["weight"].t()).sum(1) + s["bias"]).to(s["x"].dtype)
    s["state"].copy_(seen[:, 1:])
    return {"y": y, "state": s["state"]}


def _scan(s):
    x, dt = s["x"].float(), _softplus(s["dt"].float() + s["dt_bias"])
    L, per = x.shape[1], x.shape[2] // s["B"].shape[2]
    if "lengths" in s:
        inside = (torch.arange(L, device=x.device) < s["lengths"].long()[:, None])[:, :, None]
        x, dt = torch.where(inside, x, 0.0), torch.where(inside, dt, 0.0)  # behind a sequence the state stands still
    a = torch.exp(dt[..., None] * s["A"])                                                # [B, L, C, N]
    h = (dt * x)[..., None] * s["B"].float().repeat_interleave(per, dim=2)
    if s["init"] is not None:
        h[:, 0] += a[:, 0] * s["init"]
    d = 1
    while d < L:  # after each turn, token t has what the 2 d tokens up to it put into the state
        h = torch.cat([h[:, :d], h[:, d:] + a[:, d:] * h[:, :-d]], dim=1)
        a = torch.cat([a[:, :d], a[:, d:] * a[:, :-d]], dim=1)
        d *= 2
    del a
    state = h[:, -1].clone()
    y = (h * s["C"].float().repeat_interleave(per, dim=2)).sum(-1) + s["D"] * x
    if s["z"] is not None:
        y = y * _silu(s["z"].float())
    y = y.to(s["x"].dtype)
    return {"y": torch.where(inside, y, s["y"]) if "lengths" in s else y, "state": state}


def _scan_step(s):
    x, dt = s["x"].float(), _softplus(s["dt"].float() + s["dt_bias"])
    per = x.shape[1] // s["B"].shape[1]
    h = torch.exp(dt[..., None] * s["A"]) * s["state"]
    h = h + (dt * x)[..., None] * s["B"].float().repeat_interleave(per, dim=1)
    y = (h * s["C"].float().repeat_interleave(per, dim=1)).sum(-1) + s["D"] * x
    if s["z"] is not None:
        y = y * _silu(s["z"].float())
    s["state"].copy_(h)
    return {"y": y.to(s["x"].dtype), "state": s["state"]}


def _norm(s):
    u = s["x"].float()
    if s["z"] is not None:
        u = u * _silu(s["z"].float())
    v = u.unflatten(-1, (s["groups"], -1))
    v = v / torch.sqrt((v * v).mean(-1, keepdim=True) + 1e-5)
    return {"y": (v.flatten(-2) * s["weight"]).to(s["x"].dtype)}


# ---------------------------------------------------------------- in 64 bits

def exact(case, seed):
    """The definitions token by token (the convolution: tap by tap) in 64 bits."""
    s = {k: v.double() if torch.is_tensor(v) and v.is_floating_point() else v for k, v in prepare(case, seed).items()}
    op, x = case["op"], s["x"]
    if op == "norm":
        g = x * torch.sigmoid(s["z"]) * s["z"] if s["z"] is not None else x
        out, n = torch.empty_like(x), case["features"] // case["ngroups"]
        for k in range(case["ngroups"]):
            part = g[..., k * n:(k + 1) * n]
            out[..., k * n:(k + 1) * n] = part * (part.pow(2).sum(-1, keepdim=True) / n + 1e-5).rsqrt()
        return {"y": out * s["weight"]}
    lens = _lengths(case) if op in ("conv", "scan") else None
    if op == "conv":
        w, (B, L, c) = case.get("width", WIDTH), x.shape
        y, state = torch.zeros(B, L, c, dtype=x.dtype, device=x.device), torch.zeros(B, w - 1, c, dtype=x.dtype, device=x.device)
        for b in range(B):
            old = s["init"][b] if s["init"] is not None else state[b].clone()
            seq = x[b, :lens[b]]
            acc = s["bias"].repeat(lens[b], 1)
            for back in range(w):  # the input `back` tokens ago, from the cache where that is before the sequence
                acc[back:] += seq[:max(0, lens[b] - back)] * s["weight"][:, w - 1 - back]
                for t in range(min(back, lens[b])):
                    acc[t] += old[w - 1 - back + t] * s["weight"][:, w - 1 - back]
            y[b, :lens[b]] = acc * torch.sigmoid(acc)
            keep = min(w - 1, lens[b])
            state[b] = torch.cat([old[keep:], seq[lens[b] - keep:]])
        return {"y": y, "state": state}
    if op == "conv_step":
        acc = s["bias"] + x * s["weight"][:, -1]
        for k in range(s["state"].shape[1]):
            acc = acc + s["state"][:, k] * s["weight"][:, k]
        return {"y": acc * torch.sigmoid(acc), "state": torch.cat([s["state"][:, 1:], x[:, None]], 1)}
    per, n = case["channels"] // case["ngroups"], case["dstate"]
    B, c = case["batch"], case["channels"]

    def token(h, x, dt, Bt, Ct, z):
        d = torch.logaddexp(dt + s["dt_bias"], torch.zeros_like(dt))
        h = torch.exp(d[:, :, None] * s["A"]) * h
        h = h + (d * x)[:, :, None] * Bt[:, :, None, :].expand(B, -1, per, n).reshape(B, c, n)
        y = torch.einsum("bcn,bcn->bc", h, Ct[:, :, None, :].expand(B, -1, per, n).reshape(B, c, n)) + s["D"] * x
        return h, y if z is None else y * z * torch.sigmoid(z)

    if op == "scan_step":
        h, y = token(s["state"], x, s["dt"], s["B"], s["C"], s["z"])
        return {"y": y, "state": h}
    h = s["init"] if s["init"] is not None else torch.zeros(B, c, n, dtype=x.dtype, device=x.device)
    out = torch.zeros_like(x)
    ends = torch.tensor(lens, device=x.device)
    for t in range(case["seqlen"]):
        new, y = token(h, x[:, t], s["dt"][:, t], s["B"][:, t], s["C"][:, t], s["z"][:, t] if s["z"] is not None else None)
        live = t < ends
        h = torch.where(live[:, None, None], new, h)
        out[:, t] = torch.where(live[:, None], y, 0.0)
    return {"y": out, "state": h}

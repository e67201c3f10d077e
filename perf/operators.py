"""Cases for the operators around the attention call: rotary positions on q
and k, the backward's finalize step with the rotary adjoint, layer norm, and
dropout with a residual, alone and together with the layer norm behind it.

``listed()`` and ``draw()`` give cases, ``prepare`` makes a case's inputs on
the GPU from a seed, ``run`` computes one pass (elementary torch operations,
or with ``own`` set the library's calls), ``exact`` the same in 64 bits and
``work`` the bytes and operations that one pass cannot do without.

Sizes are those of this repository's attention workloads (q heads x head
dimension = 32 x 128 = 4096 columns for the grouped-query one) or generic.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
CODES = {"bf16": 0, "fp16": 1, "fp32": 2}
SIZE = {"bf16": 2, "fp16": 2, "fp32": 4}


# ----------------------------------------------------------------- the cases
def _rotary(name, B, N, H, H_kv, d, rot, style, packed, adjoint, dtype, far, scaling="none",
            factor=1.0):
    c = dict(op="rotary", B=B, N=N, H=H, H_kv=H_kv, d=d, rot=rot, style=style, packed=packed,
             adjoint=adjoint, dtype=dtype, far=far, scaling=scaling, factor=factor)
    return dict(c, name=name) if name else c


def _finalize(name, B, N, H, H_kv, d, rot, style, packed, far):
    c = dict(op="finalize", B=B, N=N, H=H, H_kv=H_kv, d=d, rot=rot, style=style, packed=packed,
             dtype="bf16", far=far, scaling="none", factor=1.0)
    return dict(c, name=name) if name else c


def _norm(name, direction, rows, C, dtype, wdtype):
    c = dict(op="norm", direction=direction, rows=rows, C=C, dtype=dtype, wdtype=wdtype)
    return dict(c, name=name) if name else c


def _dropout(name, rows, C, p, residual, dtype):
    c = dict(op="dropout", rows=rows, C=C, p=p, residual=residual, dtype=dtype)
    return dict(c, name=name) if name else c


def _add_norm(name, direction, rows, C, p, dtype, wdtype):
    c = dict(op="add_norm", direction=direction, rows=rows, C=C, p=p, dtype=dtype, wdtype=wdtype)
    return dict(c, name=name) if name else c


def listed():
    return [
        # one new token for each of 64 requests, far into their contexts, read
        # from the packed q/k/v projection: the call's latency counts
        _rotary("rotary, one token a request", 64, 1, 32, 8, 128, 128, "half", True, False,
                "bf16", 131072, "ramp", 8.0),
        # the grouped-query training workload: packed projection in, the
        # attention call's [B, H, N, d] out
        _rotary("rotary, training", 2, 4096, 32, 8, 128, 128, "half", True, False, "bf16", 0),
        # gradients taken back through a partial, interleaved rotation at an
        # odd length
        _rotary("rotary adjoint, odd length", 8, 1021, 16, 16, 64, 32, "interleaved", False, True,
                "bf16", 0, "base", 4.0),
        # the end of a backward pass: smallest workload, and the grouped-query
        # one with gradients going back into the packed layout
        _finalize("finalize, small", 1, 256, 2, 2, 64, 64, "half", False, 0),
        _finalize("finalize, training", 2, 4096, 32, 8, 128, 128, "half", True, 0),
        # each head's queries normed over the head dimension
        _norm("norm of heads", "fwd", 2 * 32 * 4096, 128, "bf16", "fp32"),
        # ragged tokens, odd width
        _norm("norm backward, odd", "bwd", 2047, 1001, "fp16", "fp32"),
        # residual dropout behind the attention's output projection
        _dropout("dropout add, training", 8192, 4096, 0.1, True, "bf16"),
        # its adjoint (no residual), odd sizes, a high rate
        _dropout("dropout, odd", 4095, 2047, 0.5, False, "bf16"),
        # a decoding step's add + norm of 64 tokens (no dropout when serving)
        _add_norm("add norm, one token a request", "fwd", 64, 4096, 0.0, "bf16", "bf16"),
        # a training step's, forward and backward
        _add_norm("add norm, training", "fwd", 8192, 4096, 0.1, "bf16", "bf16"),
        _add_norm("add norm backward, training", "bwd", 8192, 4096, 0.1, "bf16", "bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    most = max(work(c)["bytes"] for c in listed())
    while True:
        op = rng.choice(["rotary", "rotary", "finalize", "norm", "norm", "dropout", "add_norm",
                         "add_norm"])
        dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
        wdtype = rng.choice([dtype, "fp32"])
        if op in ("rotary", "finalize"):
            d = rng.choice([64, 128, 256])
            rot = rng.choice([d, d, d // 2, d // 4])
            H_kv = rng.choice([1, 2, 4, 8, 16])
            H = H_kv * rng.choice([1, 2, 4, 8])
            B, N = _log(rng, 1, 16), _log(rng, 1, 16384)
            style, packed = rng.choice(["half", "interleaved"]), rng.random() < 0.5
            far = rng.choice([0, 0, 32768, 1000000])
            if op == "rotary":
                scaling = rng.choice(["none", "linear", "base", "ramp"])
                c = _rotary("", B, N, H, H_kv, d, rot, style, packed, rng.random() < 0.4, dtype,
                            far, scaling, 1.0 if scaling == "none" else rng.choice([2.0, 4.0, 8.0]))
            else:
                c = _finalize("", B, N, H, H_kv, d, rot, style, packed, far)
        else:
            C = _log(rng, 32, 16384)
            C = C if rng.random() < 0.3 else max(32, C // 64 * 64)
            rows = _log(rng, 1, 65536)
            direction = rng.choice(["fwd", "bwd"])
            if op == "norm":
                c = _norm("", direction, rows, C, dtype, wdtype)
            elif op == "dropout":
                c = _dropout("", rows, C, rng.choice([0.05, 0.1, 0.5]), rng.random() < 0.6, dtype)
            else:
                c = _add_norm("", direction, rows, C, rng.choice([0.0, 0.1, 0.2]), dtype, wdtype)
        if work(c)["bytes"] <= most and _measurable(c):
            return c


def _measurable(c):
    """Cases below some kilobytes are all the same launch: one in the list
    stands for them, and the drawn ones go from there up."""
    return work(c)["bytes"] >= 1 << 14


def work(c):
    s = SIZE[c["dtype"]]
    if c["op"] in ("rotary", "finalize"):
        q, k = c["B"] * c["N"] * c["H"] * c["d"], c["B"] * c["N"] * c["H_kv"] * c["d"]
        rotated = (q + k) * c["rot"] // c["d"]
        extra = 8 * c["B"] * c["N"] + 4 * c["rot"]
        if c["op"] == "rotary":
            return {"bytes": 2 * s * (q + k) + extra, "flops": 3 * rotated}
        return {"bytes": (4 + s) * q + 2 * s * k + extra, "flops": 3 * rotated + q}
    n = c["rows"] * c["C"]
    if c["op"] == "dropout":
        return {"bytes": s * n * (3 if c["residual"] else 2), "flops": 2 * n}
    w, stats = SIZE[c["wdtype"]] * c["C"], 8 * c["rows"]
    if c["op"] == "norm":
        if c["direction"] == "fwd":
            return {"bytes": 2 * s * n + 2 * w + stats, "flops": 7 * n}
        return {"bytes": 3 * s * n + 3 * w + stats, "flops": 14 * n}
    masked = 1 if c["p"] > 0 else 0
    if c["direction"] == "fwd":
        return {"bytes": 4 * s * n + 2 * w + stats, "flops": (8 + masked) * n}
    return {"bytes": (4 + masked) * s * n + 3 * w + stats, "flops": (15 + masked) * n}


# ---------------------------------------------------------------- the inputs
def _frequencies(c):
    """Angles per position (radians, 64 bits) of the rot / 2 pairs and the
    factor on cosine and sine: base 10000; "linear" divides every frequency by
    the factor, "base" raises the base to 10000 factor^(rot / (rot - 2)),
    "ramp" divides the frequencies with less than 1 turn over 4096 positions,
    keeps those with more than 32 and goes over linearly in the number of
    turns between, with the factor 1 + 0.1 ln(factor) on cosine and sine."""
    rot, factor = c["rot"], c["factor"]
    i = np.arange(rot // 2, dtype=np.float64)
    base, magnitude = 10000.0, 1.0
    if c["scaling"] == "base" and rot > 2:
        base *= factor ** (rot / (rot - 2.0))
    freq = base ** (-2.0 * i / rot)
    if c["scaling"] == "linear":
        freq = freq / factor
    if c["scaling"] == "ramp":
        turns = 4096.0 * freq / (2 * math.pi)
        keep = np.clip((turns - 1.0) / (32.0 - 1.0), 0.0, 1.0)
        freq = freq * keep + freq / factor * (1.0 - keep)
        magnitude = 1.0 + 0.1 * math.log(factor)
    return freq, magnitude


def prepare(case, seed):
    c, dev = case, torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    dtype = DTYPES[c["dtype"]]

    def normal(*shape, scale=1.0, shift=0.0, dt=None):
        x = torch.randn(shape, generator=g, device=dev, dtype=torch.float32)
        return (x * scale + shift).to(dt or dtype)

    s = dict(case=c, stream=torch.cuda.current_stream())
    if c["op"] in ("rotary", "finalize"):
        B, N, H, H_kv, d = c["B"], c["N"], c["H"], c["H_kv"], c["d"]
        freq, s["magnitude"] = _frequencies(c)
        # turns per position as 64-bit fractions: position times them, modulo
        # 2^64, is the angle, exactly, however far the position
        turns = [int(round(f / (2 * math.pi) * 2.0 ** 64)) for f in freq]
        s["turns"] = torch.tensor([t - (1 << 64) if t >> 63 else t for t in turns],
                                  dtype=torch.int64, device=dev)
        if c["far"]:  # each request somewhere else in its context
            start = torch.randint(0, c["far"], (B, 1), generator=g, device=dev)
            s["positions"] = (start + torch.arange(N, device=dev)[None, :]).contiguous()
        else:
            s["positions"] = torch.arange(N, device=dev)[None, :].repeat(B, 1)

        def heads(make):  # q's and k's, [B, heads, N, d]; packed: parts of [B, N, H + 2 H_kv, d]
            if not c["packed"]:
                return make(B, H, N, d), make(B, H_kv, N, d)
            whole = make(B, N, H + 2 * H_kv, d)
            return (whole[:, :, :H].transpose(1, 2), whole[:, :, H:H + H_kv].transpose(1, 2))

        def empty(*shape):
            return torch.empty(shape, dtype=dtype, device=dev)

        if c["op"] == "rotary":
            s["q"], s["k"] = heads(normal)
            s["q_out"], s["k_out"] = empty(B, H, N, d), empty(B, H_kv, N, d)
        else:
            s["scale"] = 1.0 / math.sqrt(d)
            s["dq_accum"] = normal(B, H, N, d, dt=torch.float32)
            s["dk"] = normal(B, H_kv, N, d)
            s["dq"], s["dk_out"] = heads(empty)
        strides = [t.stride()[:3] for t in ([s["q"], s["k"], s["q_out"], s["k_out"]]
                                            if c["op"] == "rotary" else [s["dq"], s["dk_out"]])]
        s["strides"] = [v for t in strides for v in t]
        return s
    rows, C = c["rows"], c["C"]
    s["seed"] = (seed * 0x9E3779B97F4A7C15 + 12345) % (1 << 64)
    if c["op"] == "dropout":
        s["x"] = normal(rows, C)
        s["residual"] = normal(rows, C) if c["residual"] else None
        s["y"] = torch.empty_like(s["x"])
        return s
    wd = DTYPES[c["wdtype"]]
    s["eps"] = 1e-5
    s["gamma"] = normal(C, scale=0.2, shift=1.0, dt=wd)
    if c["direction"] == "fwd":
        s["beta"] = normal(C, scale=0.2, dt=wd)
        s["x"] = normal(rows, C, scale=1.5, shift=0.25)
        if c["op"] == "add_norm":
            s["residual"] = normal(rows, C)
            s["z"] = torch.empty_like(s["x"])
        s["y"] = torch.empty_like(s["x"])
        s["mean"] = torch.empty(rows, dtype=torch.float32, device=dev)
        s["rstd"] = torch.empty(rows, dtype=torch.float32, device=dev)
        return s
    s["z"] = normal(rows, C, scale=1.5, shift=0.25)
    z = s["z"].double()
    s["mean"] = z.mean(1).float()
    s["rstd"] = (z.var(1, unbiased=False) + s["eps"]).rsqrt().float()
    del z
    s["dy"] = normal(rows, C)
    if c["op"] == "add_norm":
        s["dz"] = normal(rows, C)
        s["dres"] = torch.empty_like(s["z"])
    s["dx"] = torch.empty_like(s["z"])
    s["dgamma"], s["dbeta"] = torch.empty_like(s["gamma"]), torch.empty_like(s["gamma"])
    # the backward's scratch: two fp32 sums a column for each of at most 1024 blocks
    s["workspace"] = torch.empty(1024 * 2 * C, dtype=torch.float32, device=dev)
    return s


# ---------------------------------------------------------------- the passes
def run(s):
    return _run_own(s) if own else _run_plain(s)


def _run_own(s):
    import flashattention_attention_backward_gb300 as attn

    c, stream = s["case"], s["stream"]
    code = CODES[c["dtype"]]
    if c["op"] == "rotary":
        attn.check(attn.attn_rotary(
            s["q"], s["k"], s["q_out"], s["k_out"], s["turns"], s["positions"], c["N"], c["B"],
            c["H"], c["H_kv"], c["N"], c["d"], c["rot"], s["magnitude"],
            c["style"] == "interleaved", c["adjoint"], code, s["strides"], stream))
        return s["q_out"], s["k_out"]
    if c["op"] == "finalize":
        attn.check(attn.attn_bwd_finalize_rotary(
            s["dq_accum"], s["dq"], s["dk"], s["dk_out"], s["scale"], s["turns"], s["positions"],
            c["N"], c["B"], c["H"], c["H_kv"], c["N"], c["d"], c["rot"], s["magnitude"],
            c["style"] == "interleaved", s["strides"], stream))
        return s["dq"], s["dk_out"]
    if c["op"] == "dropout":
        attn.check(attn.attn_dropout_add(s["x"], s["residual"], s["y"], c["rows"] * c["C"], c["p"],
                                         s["seed"], code, stream))
        return s["y"]
    wcode = CODES[c["wdtype"]]
    if c["direction"] == "fwd":
        if c["op"] == "norm":
            attn.check(attn.attn_layer_norm(s["x"], s["gamma"], s["beta"], s["y"], s["mean"],
                                            s["rstd"], c["rows"], c["C"], s["eps"], code, wcode,
                                            stream))
            return s["y"], s["mean"], s["rstd"]
        attn.check(attn.attn_dropout_add_norm(
            s["x"], s["residual"], s["gamma"], s["beta"], s["z"], s["y"], s["mean"], s["rstd"],
            c["rows"], c["C"], s["eps"], c["p"], s["seed"], code, wcode, stream))
        return s["z"], s["y"], s["mean"], s["rstd"]
    if c["op"] == "norm":
        attn.check(attn.attn_layer_norm_bwd(
            s["dy"], s["z"], s["gamma"], s["mean"], s["rstd"], s["dx"], s["dgamma"], s["dbeta"],
            s["workspace"], c["rows"], c["C"], code, wcode, stream))
        return s["dx"], s["dgamma"], s["dbeta"]
    # without dropout the two gradients are one tensor
    dx = s["dx"] if c["p"] > 0 else None
    attn.check(attn.attn_dropout_add_norm_bwd(
        s["dy"], s["dz"], s["z"], s["gamma"], s["mean"], s["rstd"], dx, s["dres"], s["dgamma"],
        s["dbeta"], s["workspace"], c["rows"], c["C"], c["p"], s["seed"], code, wcode, stream))
    return (s["dx"] if c["p"] > 0 else s["dres"]), s["dres"], s["dgamma"], s["dbeta"]


def _keep(n, p, seed, device):
    """Truth values [n]: element e is kept iff word e mod 4 of the Philox4x32-10
    output of counter (e / 4 mod 2^32, e / 2^34, 0, 1) under the seed's two
    halves is at least round(p 2^32)."""
    low = 0xFFFFFFFF
    ctr = torch.arange((n + 3) // 4, dtype=torch.int64, device=device)
    w = (ctr & low, ctr >> 32, torch.zeros_like(ctr), torch.ones_like(ctr))
    k0, k1 = seed & low, seed >> 32

    def mixed(w, k0, k1):
        a, b = w[0] * 0xD2511F53, w[2] * 0xCD9E8D57
        return (((b >> 32) & low) ^ w[1] ^ k0, b & low, ((a >> 32) & low) ^ w[3] ^ k1, a & low)

    def rounds(w, k0, k1, left):
        w = mixed(w, k0, k1)
        if left == 1:
            return w
        return rounds(w, (k0 + 0x9E3779B9) & low, (k1 + 0xBB67AE85) & low, left - 1)

    words = torch.stack(rounds(w, k0, k1, 10), 1).reshape(-1)[:n]
    return words >= int(math.floor(float(np.float32(p)) * 2.0 ** 32 + 0.5))


def _dropped(x, p, seed):
    """x with its elements dropped at rate p, the kept ones over 1 - p."""
    if p <= 0:
        return x
    keep = _keep(x.numel(), p, seed, x.device).reshape(x.shape)
    return torch.where(keep, x * (1.0 / (1.0 - p)), torch.zeros_like(x))


def _rotated(x, s, sign):
    """x [B, heads, N, d] (32 bits) with its first `rot` columns rotated."""
    c = s["case"]
    half = c["rot"] // 2
    # the product wraps modulo 2^64; angle and its functions in 64 bits
    turn = (s["positions"][:, :, None] * s["turns"]).double() * 2.0 ** -64
    cos = (s["magnitude"] * torch.cos(2 * math.pi * turn)).float()[:, None]
    sin = (sign * s["magnitude"] * torch.sin(2 * math.pi * turn)).float()[:, None]
    if c["style"] == "half":
        a, b = x[..., :half], x[..., half:2 * half]
        parts = [a * cos - b * sin, a * sin + b * cos]
    else:
        a, b = x[..., 0:2 * half:2], x[..., 1:2 * half:2]
        parts = [torch.stack((a * cos - b * sin, a * sin + b * cos), -1).flatten(-2)]
    return torch.cat(parts + [x[..., 2 * half:]], -1)


def _run_plain(s):
    c = s["case"]
    dt = DTYPES[c["dtype"]]
    if c["op"] == "rotary":
        sign = -1.0 if c["adjoint"] else 1.0
        return (_rotated(s["q"].float(), s, sign).to(dt), _rotated(s["k"].float(), s, sign).to(dt))
    if c["op"] == "finalize":
        return (_rotated(s["dq_accum"] * s["scale"], s, -1.0).to(dt),
                _rotated(s["dk"].float(), s, -1.0).to(dt))
    if c["op"] == "dropout":
        y = _dropped(s["x"].float(), c["p"], s["seed"])
        return (y if s["residual"] is None else y + s["residual"].float()).to(dt)
    wd, gamma = DTYPES[c["wdtype"]], s["gamma"].float()
    if c["direction"] == "fwd":
        x = s["x"].float()
        if c["op"] == "add_norm":
            x = _dropped(x, c["p"], s["seed"]) + s["residual"].float()
        mean = x.mean(1, keepdim=True)
        off = x - mean
        rstd = 1.0 / torch.sqrt((off * off).mean(1, keepdim=True) + s["eps"])
        y = (off * rstd * gamma + s["beta"].float()).to(dt)
        stats = mean[:, 0], rstd[:, 0]
        return (y,) + stats if c["op"] == "norm" else (x.to(dt), y) + stats
    dy, rstd = s["dy"].float(), s["rstd"][:, None]
    xh = (s["z"].float() - s["mean"][:, None]) * rstd
    g = dy * gamma
    dz = rstd * (g - g.mean(1, keepdim=True) - xh * (g * xh).mean(1, keepdim=True))
    dgamma, dbeta = (dy * xh).sum(0).to(wd), dy.sum(0).to(wd)
    if c["op"] == "norm":
        return dz.to(dt), dgamma, dbeta
    dz = dz + s["dz"].float()
    return _dropped(dz, c["p"], s["seed"]).to(dt), dz.to(dt), dgamma, dbeta


# --------------------------------------------------- the definition, 64 bits
def _philox_words(first, count, key):
    """uint32 [count, 4]: Philox4x32-10 of the counters first, first + 1, ...
    (low and high word), 0, 1."""
    m = np.uint64(0xFFFFFFFF)
    i = np.arange(first, first + count, dtype=np.uint64)
    x = [i & m, i >> np.uint64(32), np.zeros_like(i), np.ones_like(i)]
    for r in range(10):
        k0 = np.uint64((key + r * 0x9E3779B9) & 0xFFFFFFFF)
        k1 = np.uint64(((key >> 32) + r * 0xBB67AE85) & 0xFFFFFFFF)
        p, q = x[0] * np.uint64(0xD2511F53), x[2] * np.uint64(0xCD9E8D57)
        x = [(q >> np.uint64(32)) ^ x[1] ^ k0, q & m, (p >> np.uint64(32)) ^ x[3] ^ k1, p & m]
    return np.stack(x, 1).astype(np.uint32)


def _mask(shape, p, key):
    """1 / (1 - p) where an element is kept, 0 elsewhere, in 64 bits."""
    n = shape[0] * shape[1]
    edge = np.uint32(min(int(float(np.float32(p)) * 2.0 ** 32 + 0.5), 0xFFFFFFFF))
    step = 1 << 21
    kept = np.concatenate([(_philox_words(a, min(step, (n + 3) // 4 - a), key) >= edge).reshape(-1)
                           for a in range(0, (n + 3) // 4, step)])[:n]
    kept = torch.from_numpy(kept).cuda().reshape(shape)
    return kept.double() / (1.0 - float(np.float32(p)))


def _turned(x, c, positions, direction):
    """The rotation as a product of complex numbers, in 64 bits."""
    freq, magnitude = _frequencies(c)
    angle = positions.double()[:, None, :, None] * torch.from_numpy(freq).to(x.device)
    unit = torch.polar(torch.full_like(angle, magnitude), direction * angle)
    y, r = x.double().clone(), c["rot"]
    if c["style"] == "half":
        w = torch.complex(y[..., :r // 2], y[..., r // 2:r]) * unit
        y[..., :r // 2], y[..., r // 2:r] = w.real, w.imag
    else:
        w = torch.complex(y[..., :r:2], y[..., 1:r:2]) * unit
        y[..., :r:2], y[..., 1:r:2] = w.real, w.imag
    return y


def exact(case, seed):
    s, c = prepare(case, seed), case
    if c["op"] == "rotary":
        way = -1.0 if c["adjoint"] else 1.0
        return tuple(_turned(s[n], c, s["positions"], way) for n in ("q", "k"))
    if c["op"] == "finalize":
        return (_turned(s["dq_accum"].double() * s["scale"], c, s["positions"], -1.0),
                _turned(s["dk"], c, s["positions"], -1.0))
    first = s["x"] if "x" in s else s["z"]
    mask = _mask(tuple(first.shape), c["p"], s["seed"]) if c.get("p", 0) > 0 else 1.0
    if c["op"] == "dropout":
        y = first.double() * mask
        return y if s["residual"] is None else y + s["residual"].double()
    gamma = s["gamma"].double()
    if c["direction"] == "fwd":
        z = first.double()
        if c["op"] == "add_norm":
            z = z * mask + s["residual"].double()
        mean = z.mean(1)
        rstd = torch.rsqrt(z.var(1, unbiased=False) + s["eps"])
        y = (z - mean[:, None]) * (rstd[:, None] * gamma) + s["beta"].double()
        return (y, mean, rstd) if c["op"] == "norm" else (z, y, mean, rstd)
    dy, r = s["dy"].double(), s["rstd"].double()[:, None]
    hat = (s["z"].double() - s["mean"].double()[:, None]) * r
    g = dy * gamma
    # g without its parts along the ones and along hat, over the row's C
    # columns (the stored statistics are the row's own)
    along = torch.stack((g.sum(1), (g * hat).sum(1)), 1) / c["C"]
    dz = (g - along[:, :1] - hat * along[:, 1:]) * r
    dgamma, dbeta = (dy * hat).sum(0), dy.sum(0)
    if c["op"] == "norm":
        return dz, dgamma, dbeta
    dz = dz + s["dz"].double()
    return dz * mask, dz, dgamma, dbeta

"""Cases for attention with a sliding window and first tokens that stay visible
(forward and backward), for appending rotated keys and values to a paged cache,
and for the attention of new tokens over such a cache.

``listed()`` and ``draw()`` give cases, ``prepare`` makes a case's inputs on
the GPU from a seed, ``run`` computes one pass (elementary torch operations,
or with ``own`` set the library's calls), ``exact`` the same in 64 bits and
``work`` the bytes and operations that one pass cannot do without.

Sizes are those of this repository's attention workloads (32 query heads over 8
key/value heads of 128 columns for the grouped-query one) or generic.
"""
import math
import random

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
CODES = {"bf16": 0, "fp16": 1}


# ----------------------------------------------------------------- the cases
def _sinks(name, direction, B, H, H_kv, N, d, causal, left, right, sinks, softcap=0.0):
    c = dict(op="sinks", direction=direction, B=B, H=H, H_kv=H_kv, N=N, d=d, causal=causal,
             left=left, right=right, sinks=sinks, softcap=softcap)
    return dict(c, name=name) if name else c


def _append(name, B, new, ctx, ragged, H, H_kv, d, rot, style, page, dtype, mix=1):
    c = dict(op="append", B=B, new=new, ctx=ctx, ragged=ragged, H=H, H_kv=H_kv, d=d, rot=rot,
             style=style, page=page, dtype=dtype, mix=mix)
    return dict(c, name=name) if name else c


def _cache(name, B, new, ctx, ragged, H, H_kv, d, page, dtype, causal=True, left=-1, sinks=0,
           softcap=0.0, mix=1):
    c = dict(op="cache", B=B, new=new, ctx=ctx, ragged=ragged, H=H, H_kv=H_kv, d=d, page=page,
             dtype=dtype, causal=causal, left=left, sinks=sinks, softcap=softcap, mix=mix)
    return dict(c, name=name) if name else c


def listed():
    return [
        # the grouped-query training workload under a window of 1024 keys with
        # four first tokens that every later one still sees
        _sinks("window and sinks, training", "fwd", 2, 32, 8, 4096, 128, True, 1023, -1, 4),
        _sinks("window and sinks backward, training", "bwd", 2, 32, 8, 4096, 128, True, 1023, -1,
               4),
        # one long document
        _sinks("window and sinks backward, long", "bwd", 1, 16, 16, 16384, 128, True, 2047, -1,
               64),
        # a two-sided band at an odd length, sinks that end inside a key block
        _sinks("band and sinks backward, odd", "bwd", 3, 6, 3, 1999, 64, False, 255, 100, 130,
               30.0),
        # one new token for each of 64 requests: the call's latency counts
        _append("append, one token a request", 64, 1, 4096, True, 32, 8, 128, 128, "half", 64,
                "bf16"),
        # the prompts of four requests, out of the packed projection
        _append("append, prompts", 4, 4096, 0, False, 32, 8, 128, 128, "half", 64, "bf16"),
        # ragged chunks, a partial interleaved rotation, small pages
        _append("append, odd", 23, 301, 2000, True, 15, 5, 64, 32, "interleaved", 16, "fp16"),
        # one token of one short request: the smallest call, all latency
        _cache("one token, one short request", 1, 1, 499, False, 32, 8, 128, 64, "bf16"),
        # a decoding step of 64 requests somewhere in their contexts
        _cache("one token a request", 64, 1, 8192, True, 32, 8, 128, 64, "bf16"),
        # two requests far into long contexts
        _cache("one token, long contexts", 2, 1, 131072, False, 32, 8, 128, 128, "bf16"),
        # a chunk of a prompt behind what the cache holds of it
        _cache("chunk of a prompt", 1, 2048, 16384, False, 32, 8, 128, 64, "bf16"),
        # decoding and prompt chunks in one batch under a window with sinks,
        # odd sizes
        _cache("mixed, window and sinks, odd", 29, 203, 5001, True, 21, 7, 64, 16, "fp16",
               left=1023, sinks=5, softcap=50.0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    works = [work(c) for c in listed()]
    bytes_, flops = (max(w[n] for w in works) for n in ("bytes", "flops"))
    while True:
        op = rng.choice(["sinks", "append", "cache", "cache"])
        d = rng.choice([64, 128, 128, 256])
        H_kv = rng.choice([1, 2, 4, 5, 8, 16])
        H = H_kv * rng.choice([1, 2, 3, 4, 8])
        left = rng.choice([_log(rng, 1, 4096), 1023, -1])
        sinks = rng.choice([0, 1, 4, _log(rng, 1, 300)])
        softcap = rng.choice([0.0, 0.0, 30.0])
        if op == "sinks":
            N = _log(rng, 64, 16384)
            causal = rng.random() < 0.7
            c = _sinks("", rng.choice(["fwd", "bwd"]), _log(rng, 1, 8), H, H_kv, N, d, causal,
                       left, -1 if causal else rng.choice([-1, _log(rng, 1, 1000)]), sinks,
                       softcap)
        else:
            B = _log(rng, 1, 256)
            new = rng.choice([1, rng.randint(2, 8), _log(rng, 9, 4096)])
            ctx = _log(rng, 1, 131072)
            page = rng.choice([16, 32, 64, 128, 256])
            dtype = rng.choice(["bf16", "bf16", "fp16"])
            mix, ragged = rng.randint(1, 1 << 20), rng.random() < 0.7
            if op == "append":
                c = _append("", B, new, min(ctx, 8192), ragged, H, H_kv, d,
                            rng.choice([d, d // 2, d // 4, 0]), rng.choice(["half", "interleaved"]),
                            page, dtype, mix)
            else:
                c = _cache("", B, new, ctx, ragged, H, H_kv, d, page, dtype,
                           rng.random() < 0.9, left, sinks, softcap, mix)
        w = work(c)
        if w["bytes"] <= bytes_ and w["flops"] <= flops and w["bytes"] >= 1 << 14 and _fits(c):
            return c


def _fits(c):
    """The cache's slots, all of them (a window reads few of many), stay within
    some gigabytes, and the plain forms, which compute hidden scores too, within
    the time and memory of the listed cases."""
    if c["op"] == "sinks":
        return c["B"] * c["H"] * c["N"] ** 2 * c["d"] <= 6e11
    seqs = _sequences(c)
    if sum(L for _, L in seqs) * c["H_kv"] * c["d"] > 1 << 29:
        return False
    return c["op"] == "append" or (max(n * L for n, L in seqs) * c["H"] <= 1 << 31 and
                                   sum(n * L for n, L in seqs) * c["H"] * c["d"] <= 6e11)


def _sequences(c):
    """(new tokens, length with them) of each sequence; the same for every
    seed, so that a case's work is one number."""
    if not c["ragged"]:
        return [(c["new"], c["ctx"] + c["new"])] * c["B"]
    rng = random.Random(c["mix"])
    out = []
    for b in range(c["B"]):
        n = c["new"] if c["new"] == 1 else rng.choice([1, rng.randint(0, c["new"])])
        out.append((n, n + rng.randint(0, c["ctx"])))
    out[0] = (c["new"], out[0][1] - out[0][0] + c["new"])  # no batch is without a new token
    return out


def _visible(c, pos, length):
    """How many keys the queries at `pos` see (an array)."""
    last = np.full_like(pos, length - 1)
    if c["causal"]:
        last = np.minimum(last, pos)
    elif c.get("right", -1) >= 0:
        last = np.minimum(last, pos + c["right"])
    first = np.maximum(pos - c["left"], 0) if c["left"] >= 0 else np.zeros_like(pos)
    return last - first + 1 + np.minimum(c["sinks"], first)


def work(c):
    if c["op"] == "sinks":
        q, k = c["B"] * c["H"] * c["N"] * c["d"], c["B"] * c["H_kv"] * c["N"] * c["d"]
        pairs = int(_visible(c, np.arange(c["N"]), c["N"]).sum()) * c["B"] * c["H"]
        stats = 4 * c["B"] * c["H"] * c["N"]
        if c["direction"] == "fwd":
            return {"bytes": 2 * (2 * q + 2 * k) + stats, "flops": 4 * c["d"] * pairs}
        return {"bytes": 2 * (4 * q + 4 * k) + stats, "flops": 10 * c["d"] * pairs}
    seqs = _sequences(c)
    T = sum(n for n, _ in seqs)
    q, k = T * c["H"] * c["d"], T * c["H_kv"] * c["d"]
    if c["op"] == "append":
        return {"bytes": 2 * (2 * q + 4 * k) + 16 * c["B"], "flops": 3 * (q + k) * c["rot"] // c["d"]}
    pairs = slots = 0
    for n, L in seqs:
        if n == 0:
            continue
        pairs += int(_visible(c, np.arange(L - n, L), L).sum())
        first = max(0, L - n - c["left"]) if c["left"] >= 0 else 0
        slots += L - first + min(c["sinks"], first)
    return {"bytes": 2 * (2 * q + 2 * slots * c["H_kv"] * c["d"]) + 4 * T * c["H"] + 16 * c["B"],
            "flops": 4 * c["d"] * c["H"] * pairs}


# ---------------------------------------------------------------- the inputs
def prepare(case, seed):
    c, dev = case, torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)

    def normal(*shape, dtype=torch.bfloat16):
        return torch.randn(shape, generator=g, device=dev, dtype=torch.float32).to(dtype)

    s = dict(case=c, stream=torch.cuda.current_stream(), scale=1.0 / math.sqrt(c["d"]))
    H, H_kv, d = c["H"], c["H_kv"], c["d"]
    if c["op"] == "sinks":
        B, N = c["B"], c["N"]
        s["q"], s["k"], s["v"] = normal(B, H, N, d), normal(B, H_kv, N, d), normal(B, H_kv, N, d)
        if c["direction"] == "fwd":
            s["o"] = torch.empty_like(s["q"])
            s["lse"] = torch.empty(B, H, N, device=dev)
            return s
        s["o"], s["lse"] = _band_forward(s)
        s["do"] = normal(B, H, N, d)
        s["dq"], s["dk"], s["dv"] = (torch.empty_like(s[n]) for n in ("q", "k", "v"))
        s["dq_accum"] = torch.empty(B, H, N, d, device=dev)
        s["dpsum"] = torch.empty(B, H, N, device=dev)
        return s
    dt, page, seqs = DTYPES[c["dtype"]], c["page"], _sequences(c)
    T = sum(n for n, _ in seqs)
    need = [(L + page - 1) // page for _, L in seqs]
    s["max_pages"], s["n_pages"] = max(need) + 1, sum(need) + 3
    order = torch.randperm(s["n_pages"], generator=g, device=dev).to(torch.int32)
    s["pages"] = torch.full((c["B"], s["max_pages"]), -1, dtype=torch.int32, device=dev)
    at = 0
    for b, n in enumerate(need):
        s["pages"][b, :n] = order[at:at + n]
        at += n
    s["seqs"], s["T"] = seqs, T
    s["starts"] = torch.tensor(np.cumsum([0] + [n for n, _ in seqs]), dtype=torch.int32, device=dev)
    s["lengths"] = torch.tensor([L for _, L in seqs], dtype=torch.int32, device=dev)
    s["k_cache"] = normal(s["n_pages"], page, H_kv, d, dtype=dt)
    s["v_cache"] = normal(s["n_pages"], page, H_kv, d, dtype=dt)
    if c["op"] == "append":
        # q, k and v are parts of one projection's output
        whole = normal(T, H + 2 * H_kv, d, dtype=dt)
        s["q"], s["k"], s["v"] = whole[:, :H], whole[:, H:H + H_kv], whole[:, H + H_kv:]
        s["q_out"] = torch.empty(T, H, d, dtype=dt, device=dev)
        # turns per position as 64-bit fractions: position times them, modulo
        # 2^64, is the angle, exactly, however far the position
        turns = [int(round(f / (2 * math.pi) * 2.0 ** 64)) for f in _frequencies(c)]
        s["turns"] = torch.tensor([t - (1 << 64) if t >> 63 else t for t in turns] or [0],
                                  dtype=torch.int64, device=dev)
        s["strides"] = [v for t in ("q", "k", "v", "q_out") for v in s[t].stride()[:2]] + \
            [v for t in ("k_cache", "v_cache") for v in s[t].stride()[:3]]
        return s
    s["q"] = normal(T, H, d, dtype=dt)
    s["o"] = torch.empty_like(s["q"])
    s["lse"] = torch.empty(T, H, device=dev)
    if own:
        import flashattention_attention_backward_gb300 as attn
        size = attn.attn_cache_fwd_workspace_bytes(T, c["B"], H, H_kv, d)
        s["workspace"] = torch.empty(max(size, 16), dtype=torch.uint8, device=dev)
    return s


def _frequencies(c):
    """Radians per position of the rot / 2 pairs, 64 bits."""
    return 10000.0 ** (-2.0 * np.arange(c["rot"] // 2, dtype=np.float64) / max(c["rot"], 1))


# ---------------------------------------------------------------- the passes
def run(s):
    return _run_own(s) if own else _run_plain(s)


def _run_own(s):
    import flashattention_attention_backward_gb300 as attn

    c, stream = s["case"], s["stream"]
    H, H_kv, d, cap = c["H"], c["H_kv"], c["d"], c.get("softcap", 0.0)
    if c["op"] == "sinks":
        B, N = c["B"], c["N"]
        if c["direction"] == "fwd":
            attn.check(attn.attn_fwd_sinks(s["q"], s["k"], s["v"], s["o"], s["lse"], B, H, H_kv, N,
                                           d, s["scale"], c["causal"], cap, c["left"], c["right"],
                                           c["sinks"], stream))
            return s["o"], s["lse"]
        attn.check(attn.attn_bwd_preprocess(s["o"], s["do"], s["dpsum"], s["dq_accum"], B, H, N, d,
                                            stream))
        attn.check(attn.attn_bwd_sinks(s["q"], s["k"], s["v"], s["o"], s["do"], s["lse"],
                                       s["dq_accum"], s["dk"], s["dv"], B, H, H_kv, N, d,
                                       s["scale"], c["causal"], cap, s["dpsum"], c["left"],
                                       c["right"], c["sinks"], stream))
        attn.check(attn.attn_bwd_finalize(s["dq_accum"], s["dq"], s["scale"], B, H, N, d, stream))
        return s["dq"], s["dk"], s["dv"]
    code = CODES[c["dtype"]]
    if c["op"] == "append":
        attn.check(attn.attn_cache_append(
            s["q"], s["k"], s["v"], s["q_out"], s["k_cache"], s["v_cache"], s["turns"],
            s["starts"], s["lengths"], s["pages"], s["T"], c["B"], H, H_kv, d, c["rot"], 1.0,
            c["style"] == "interleaved", c["page"], s["max_pages"], s["n_pages"], code,
            s["strides"], stream))
        return s["q_out"], s["k_cache"], s["v_cache"]
    attn.check(attn.attn_cache_fwd(
        s["q"], s["k_cache"], s["v_cache"], s["o"], s["lse"], s["starts"], s["lengths"],
        s["pages"], s["workspace"], s["T"], c["B"], H, H_kv, d, c["page"], s["max_pages"],
        s["n_pages"], s["scale"], c["causal"], cap, c["left"], c["sinks"], code, None, stream))
    return s["o"], s["lse"]


def _hidden(c, pos, count):
    """[len(pos), count] truth values: key j is not visible to the query at pos."""
    j = torch.arange(count, device=pos.device)[None, :]
    i = pos[:, None]
    hidden = torch.zeros((pos.numel(), count), dtype=torch.bool, device=pos.device)
    if c["causal"]:
        hidden |= j > i
    elif c.get("right", -1) >= 0:
        hidden |= j > i + c["right"]
    if c["left"] >= 0:
        hidden |= (j < i - c["left"]) & (j >= c["sinks"])
    return hidden


def _logits(q, k, scale, softcap):
    z = (q @ k.transpose(-1, -2)) * scale
    return softcap * torch.tanh(z / softcap) if softcap > 0 else z


def _softmax(x):
    """(weights, log of the sum) of rows that see something."""
    m = x.amax(-1, keepdim=True)
    p = torch.exp(x - m)
    total = p.sum(-1, keepdim=True)
    return p / total, (m + torch.log(total))[..., 0]


def _band_forward(s):
    c = s["case"]
    B, H, N, G = c["B"], c["H"], c["N"], c["H"] // c["H_kv"]
    hidden = _hidden(c, torch.arange(N, device=s["q"].device), N)
    o, lse = torch.empty_like(s["q"]), torch.empty(B, H, N, device=s["q"].device)
    for b in range(B):
        for h in range(H):
            k, v = s["k"][b, h // G].float(), s["v"][b, h // G].float()
            x = _logits(s["q"][b, h].float(), k, s["scale"], c["softcap"])
            p, lse[b, h] = _softmax(x.masked_fill_(hidden, -math.inf))
            o[b, h] = (p @ v).to(o.dtype)
    return o, lse


def _band_backward(s):
    c = s["case"]
    B, H, N, G, cap = c["B"], c["H"], c["N"], c["H"] // c["H_kv"], c["softcap"]
    hidden = _hidden(c, torch.arange(N, device=s["q"].device), N)
    dq, dk, dv = (torch.empty_like(s[n]) for n in ("q", "k", "v"))
    for b in range(B):
        for g in range(c["H_kv"]):
            k, v = s["k"][b, g].float(), s["v"][b, g].float()
            sum_k, sum_v = torch.zeros_like(k), torch.zeros_like(v)
            for h in range(g * G, (g + 1) * G):
                q, do = s["q"][b, h].float(), s["do"][b, h].float()
                x = _logits(q, k, s["scale"], cap)
                p = torch.exp(x - s["lse"][b, h][:, None]).masked_fill_(hidden, 0.0)
                sum_v += p.T @ do
                rows = (do * s["o"][b, h].float()).sum(1, keepdim=True)
                ds = p * (do @ v.T - rows) * s["scale"]
                if cap > 0:
                    ds = ds * (1.0 - (x / cap) ** 2)
                dq[b, h] = (ds @ k).to(dq.dtype)
                sum_k += ds.T @ q
            dk[b, g], dv[b, g] = sum_k.to(dk.dtype), sum_v.to(dv.dtype)
    return dq, dk, dv


def _tokens(s):
    """(sequence, position) of every new token, 64 bits."""
    starts, t = s["starts"].long(), torch.arange(s["T"], device=s["q"].device)
    b = torch.searchsorted(starts, t, right=True) - 1
    return b, s["lengths"].long()[b] - starts[b + 1] + t


def _rotated(x, s, pos):
    c = s["case"]
    half, x = c["rot"] // 2, x.float()
    # the product wraps modulo 2^64; angle and its functions in 64 bits
    turn = (pos[:, None] * s["turns"][:half]).double() * 2.0 ** -64
    cos, sin = (f(2 * math.pi * turn).float()[:, None] for f in (torch.cos, torch.sin))
    if c["style"] == "half":
        a, b = x[..., :half], x[..., half:2 * half]
        parts = [a * cos - b * sin, a * sin + b * cos]
    else:
        a, b = x[..., 0:2 * half:2], x[..., 1:2 * half:2]
        parts = [torch.stack((a * cos - b * sin, a * sin + b * cos), -1).flatten(-2)]
    return torch.cat(parts + [x[..., 2 * half:]], -1)


def _run_plain(s):
    c = s["case"]
    if c["op"] == "sinks":
        return _band_forward(s) if c["direction"] == "fwd" else _band_backward(s)
    if c["op"] == "append":
        dt, (b, pos) = s["q"].dtype, _tokens(s)
        where = s["pages"][b, pos // c["page"]].long(), pos % c["page"]
        s["k_cache"][where] = _rotated(s["k"], s, pos).to(dt)
        s["v_cache"][where] = s["v"]
        return _rotated(s["q"], s, pos).to(dt), s["k_cache"], s["v_cache"]
    o, lse = torch.empty_like(s["q"]), torch.empty_like(s["lse"])
    G, at = c["H"] // c["H_kv"], 0
    for b, (n, L) in enumerate(s["seqs"]):
        if n == 0:
            continue
        used = s["pages"][b, :(L + c["page"] - 1) // c["page"]].long()
        k, v = (s[name][used].flatten(0, 1)[:L].transpose(0, 1).float()
                for name in ("k_cache", "v_cache"))  # [H_kv, L, d]
        hidden = _hidden(c, torch.arange(L - n, L, device=k.device), L)
        q = s["q"][at:at + n].float().reshape(n, c["H_kv"], G, c["d"]).permute(1, 2, 0, 3)
        x = _logits(q, k[:, None], s["scale"], c["softcap"])  # [H_kv, G, n, L]
        p, total = _softmax(x.masked_fill_(hidden, -math.inf))
        o[at:at + n] = (p @ v[:, None]).permute(2, 0, 1, 3).reshape(n, c["H"], -1).to(o.dtype)
        lse[at:at + n] = total.permute(2, 0, 1).reshape(n, c["H"])
        at += n
    return o, lse


# --------------------------------------------------- the definition, 64 bits
def _seen(c, pos, count):
    """0 where the query at pos sees key j, -infinity elsewhere, from the
    distance of the two."""
    j = torch.arange(count, device=pos.device, dtype=torch.float64)
    ahead = j - pos.double()[:, None]
    reach = 0 if c["causal"] else (c.get("right", -1) if c.get("right", -1) >= 0 else math.inf)
    near = ahead >= (-c["left"] if c["left"] >= 0 else -math.inf)
    seen = (ahead <= reach) & (near | (j < c["sinks"]))
    return torch.where(seen, 0.0, -math.inf)


def _exact_band(s, c):
    B, H_kv, G = c["B"], c["H_kv"], c["H"] // c["H_kv"]
    seen = _seen(c, torch.arange(c["N"], device="cuda"), c["N"])
    out = {n: torch.zeros(s[n].shape, dtype=torch.float64, device="cuda")
           for n in (("q", "lse") if c["direction"] == "fwd" else ("q", "k", "v"))}
    for b in range(B):
        for h in range(c["H"]):
            q, k, v = (s[n][b, i].double() for n, i in (("q", h), ("k", h // G), ("v", h // G)))
            z = torch.mul(torch.matmul(k, q.T).T, s["scale"])
            slope = None
            if c["softcap"] > 0:
                t = torch.tanh(z / c["softcap"])
                z, slope = c["softcap"] * t, 1.0 - t * t
            z = z + seen
            if c["direction"] == "fwd":
                out["lse"][b, h] = torch.logsumexp(z, 1)
                out["q"][b, h] = torch.matmul(torch.exp(z - out["lse"][b, h][:, None]), v)
                continue
            w = torch.exp(z - s["lse"][b, h].double()[:, None])
            do, o = s["do"][b, h].double(), s["o"][b, h].double()
            grad = w * (torch.matmul(do, v.T) - (do * o).sum(1)[:, None])
            if slope is not None:
                grad = grad * slope
            out["q"][b, h] = s["scale"] * torch.matmul(grad, k)
            out["k"][b, h // G] += s["scale"] * torch.matmul(grad.T, q)
            out["v"][b, h // G] += torch.matmul(w.T, do)
    return tuple(out.values())


def _exact_append(s, c):
    freq = torch.from_numpy(_frequencies(c)).cuda()
    q_out = s["q"].double()
    caches = s["k_cache"].double(), s["v_cache"].double()
    pages, at, half = s["pages"].tolist(), 0, c["rot"] // 2
    for b, (n, L) in enumerate(s["seqs"]):
        pos = torch.arange(L - n, L, device="cuda")
        unit = torch.polar(torch.ones(n, 1, half, dtype=torch.float64, device="cuda"),
                           pos.double()[:, None, None] * freq)

        def turned(x):
            y = x.double().clone()
            if c["style"] == "half":
                w = torch.complex(y[..., :half], y[..., half:2 * half]) * unit
                y[..., :half], y[..., half:2 * half] = w.real, w.imag
            else:
                w = torch.complex(y[..., 0:2 * half:2], y[..., 1:2 * half:2]) * unit
                y[..., 0:2 * half:2], y[..., 1:2 * half:2] = w.real, w.imag
            return y

        q_out[at:at + n] = turned(s["q"][at:at + n])
        for cache, rows in ((caches[0], turned(s["k"][at:at + n])),
                            (caches[1], s["v"][at:at + n].double())):
            p = L - n
            while p < L:  # page by page
                end = min(L, (p // c["page"] + 1) * c["page"])
                first = p % c["page"]
                cache[pages[b][p // c["page"]], first:first + end - p] = \
                    rows[p - L + n:end - L + n]
                p = end
        at += n
    return (q_out,) + caches


def _exact_cache(s, c):
    o = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.zeros(s["lse"].shape, dtype=torch.float64, device="cuda")
    G, at = c["H"] // c["H_kv"], 0
    for b, (n, L) in enumerate(s["seqs"]):
        if n == 0:
            continue
        slot = torch.arange(L, device="cuda")
        page = s["pages"][b].long()[torch.div(slot, c["page"], rounding_mode="floor")]
        seen = _seen(c, torch.arange(L - n, L, device="cuda"), L)
        for g in range(c["H_kv"]):
            k, v = (s[name][page, slot % c["page"], g].double() for name in ("k_cache", "v_cache"))
            for h in range(g * G, (g + 1) * G):
                z = s["scale"] * torch.matmul(s["q"][at:at + n, h].double(), k.T)
                if c["softcap"] > 0:
                    z = c["softcap"] * torch.tanh(z / c["softcap"])
                z = z + seen
                lse[at:at + n, h] = torch.logsumexp(z, 1)
                o[at:at + n, h] = torch.matmul(torch.exp(z - lse[at:at + n, h][:, None]), v)
        at += n
    return o, lse


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "sinks":
        return _exact_band(s, case)
    return _exact_append(s, case) if case["op"] == "append" else _exact_cache(s, case)

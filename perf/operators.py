"""The operators around the recurrence, as cases to be measured: the short causal convolution, the
norm of queries and keys with the position rotation, and the selective state space scan, each for
prompts and (convolution, scan) for one token of every beam.

`run` computes an operator either in its plain form (torch operations in 32 bits, 64 where sums of
exponents or angles need them) or, with `own`, by the library's call on the same tensors.
"""
import math

import torch

own = False

BF16, F32 = "bf16", "f32"


def _dtype(case):
    return torch.bfloat16 if case["dtype"] == BF16 else torch.float32


# ---------------------------------------------------------------------------------- cases

def listed():
    return [
        # the q, k and v channels of a GDN layer (16 heads of 128 x 128), one 1K prompt
        {"name": "conv_prompt_1k", "op": "conv", "dtype": BF16, "R": 1, "P": 1024, "C": 6144,
         "W": 4, "silu": True, "bias": False, "state": False, "lens": False, "wide": 6144},
        # eight 5K prompts; the channels are a slice of a wider projection's rows
        {"name": "conv_prompt_5k_sliced", "op": "conv", "dtype": BF16, "R": 8, "P": 5120,
         "C": 6144, "W": 4, "silu": True, "bias": True, "state": False, "lens": False,
         "wide": 8192},
        # a padded batch that continues earlier prompt pieces, fp32, odd sizes
        {"name": "conv_ragged_f32", "op": "conv", "dtype": F32, "R": 7, "P": 777, "C": 1001,
         "W": 3, "silu": True, "bias": True, "state": True, "lens": True, "wide": 1001},
        # one decode step of 512 beams for 16 requests, windows taken from the parents
        {"name": "conv_step_beams", "op": "conv_step", "dtype": BF16, "R": 16, "B": 512,
         "Bp": 512, "C": 6144, "W": 4, "silu": True, "bias": True, "parents": True},
        # one token of one sequence: latency
        {"name": "conv_step_token", "op": "conv_step", "dtype": BF16, "R": 1, "B": 1, "Bp": 1,
         "C": 6144, "W": 4, "silu": True, "bias": False, "parents": False},
        # what the GDN recurrence takes: unit queries and keys of eight 5K prompts, no rotation
        {"name": "qk_norm_unit_prompt", "op": "qk_norm", "dtype": BF16, "R": 8, "P": 5120,
         "Hq": 16, "Hk": 16, "d": 128, "l2": True, "weights": False, "rot": 0, "pair": False},
        # weighted RMS norm, a quarter of 256 dims rotated, few key heads, far positions
        {"name": "qk_norm_rotated_prompt", "op": "qk_norm", "dtype": BF16, "R": 4, "P": 5120,
         "Hq": 16, "Hk": 2, "d": 256, "l2": False, "weights": True, "rot": 64, "pair": False},
        # one token: latency
        {"name": "qk_norm_token", "op": "qk_norm", "dtype": BF16, "R": 1, "P": 1, "Hq": 16,
         "Hk": 4, "d": 128, "l2": False, "weights": True, "rot": 128, "pair": False},
        # one 1K prompt, one key group for all 32 heads, gated output
        {"name": "scan_prompt_1k", "op": "scan", "dtype": BF16, "R": 1, "P": 1024, "H": 32,
         "G": 1, "d_k": 128, "d_v": 64, "z": True, "D": True, "state": False, "lens": False},
        # 64 requests of 5K tokens, 16 heads of 128 x 128 with their own keys
        {"name": "scan_prompt_5k_64", "op": "scan", "dtype": BF16, "R": 64, "P": 5120, "H": 16,
         "G": 16, "d_k": 128, "d_v": 128, "z": False, "D": False, "state": False,
         "lens": False},
        # a padded fp32 batch that continues earlier states, odd sizes
        {"name": "scan_ragged_f32", "op": "scan", "dtype": F32, "R": 3, "P": 777, "H": 6,
         "G": 2, "d_k": 64, "d_v": 32, "z": True, "D": True, "state": True, "lens": True},
        # one decode step of 64 beams for 8 requests, states taken from the parents
        {"name": "scan_step_beams", "op": "scan_step", "dtype": BF16, "R": 8, "B": 64, "Bp": 64,
         "H": 16, "G": 16, "d_k": 128, "d_v": 128, "z": False, "D": True, "parents": True},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["conv", "conv_step", "qk_norm", "scan", "scan", "scan_step"])
    dtype = rng.choice([BF16, BF16, F32])
    flip = lambda: rng.random() < 0.5  # noqa: E731
    if op == "conv":
        C = _log_int(rng, 64, 8192)
        if rng.random() < 0.8:
            C = C // 8 * 8
        R = _log_int(rng, 1, 16)
        P = _log_int(rng, 1, max(1, min(5120, 250_000_000 // (R * C))))
        return {"op": op, "dtype": dtype, "R": R, "P": P, "C": C, "W": rng.randint(2, 4),
                "silu": flip(), "bias": flip(), "state": flip(), "lens": flip(),
                "wide": C + rng.choice([0, 0, 64, 1024])}
    if op == "conv_step":
        C = _log_int(rng, 64, 8192)
        if rng.random() < 0.8:
            C = C // 8 * 8
        R = _log_int(rng, 1, 32)
        B = _log_int(rng, 1, min(512, max(1, 50_000_000 // (R * C))))
        par = flip()
        return {"op": op, "dtype": dtype, "R": R, "B": B, "Bp": rng.choice([1, B]) if par else B,
                "C": C, "W": rng.randint(2, 4), "silu": flip(), "bias": flip(), "parents": par}
    if op == "qk_norm":
        d = rng.choice([64, 80, 96, 128, 256])
        Hk = rng.choice([1, 2, 4, 8, 16])
        Hq = Hk * rng.choice([1, 2, 4])
        R = _log_int(rng, 1, 16)
        P = _log_int(rng, 1, max(1, min(5120, 170_000_000 // (R * (Hq + Hk) * d))))
        rot = rng.choice([0, d // 16 * 16, 32])
        return {"op": op, "dtype": dtype, "R": R, "P": P, "Hq": Hq, "Hk": Hk, "d": d,
                "l2": flip(), "weights": flip(), "rot": rot, "pair": flip()}
    d_k, d_v = rng.choice([64, 128]), rng.choice([32, 64, 128, 128])
    if rng.random() < 0.15:
        d_k, d_v = rng.choice([16, 32, 256]), rng.choice([16, 64, 256])
    G = rng.choice([1, 1, 2, 4, 16])
    H = max(G, rng.choice([8, 16, 32]))
    if op == "scan":
        most = 80_000_000 if dtype == BF16 else 20_000_000
        R = _log_int(rng, 1, 16)
        P = _log_int(rng, 1, max(1, min(5120, most // (R * H * max(d_k, d_v)))))
        return {"op": op, "dtype": dtype, "R": R, "P": P, "H": H, "G": G, "d_k": d_k, "d_v": d_v,
                "z": flip(), "D": flip(), "state": flip(), "lens": flip()}
    R = _log_int(rng, 1, 16)
    B = _log_int(rng, 1, max(1, min(512, 150_000_000 // (R * H * d_k * d_v))))
    par = flip()
    return {"op": op, "dtype": dtype, "R": R, "B": B, "Bp": rng.choice([1, B]) if par else B,
            "H": H, "G": G, "d_k": d_k, "d_v": d_v, "z": flip(), "D": flip(), "parents": par}


# ---------------------------------------------------------------------------------- inputs

def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    dt = _dtype(case)

    def randn(*shape, dtype=None, scale=1.0):
        x = torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32)
        return (x if scale == 1.0 else x * scale).to(dtype or dt)

    def lens(R, P):
        return torch.randint(0, P + 1, (R,), generator=gen, device="cuda", dtype=torch.int32)

    def parents(R, B, Bp):
        # beams near the top of the order have most of the children
        u = torch.rand((R, B), generator=gen, device="cuda")
        return (u * u * Bp).to(torch.int32).clamp_(max=Bp - 1)

    s = {"case": case}
    op = case["op"]
    if op in ("conv", "conv_step"):
        R, C, W = case["R"], case["C"], case["W"]
        s["w"] = randn(C, W, dtype=torch.float32, scale=1.0 / math.sqrt(W))
        s["bias"] = randn(C, dtype=torch.float32, scale=0.5) if case["bias"] else None
        if op == "conv":
            P = case["P"]
            s["x"] = randn(R, P, case["wide"])[:, :, :C]
            s["state"] = randn(R, W - 1, C) if case["state"] else None
            s["lens"] = lens(R, P) if case["lens"] else None
            s["y"] = torch.zeros((R, P, C), device="cuda", dtype=dt)
            s["state_out"] = torch.zeros((R, W - 1, C), device="cuda", dtype=dt)
        else:
            B, Bp = case["B"], case["Bp"]
            s["x"] = randn(R, B, C)
            s["state"] = randn(R, Bp, W - 1, C)
            s["parents"] = parents(R, B, Bp) if case["parents"] else None
            s["y"] = torch.zeros((R, B, C), device="cuda", dtype=dt)
            s["state_out"] = torch.zeros((R, B, W - 1, C), device="cuda", dtype=dt)
    elif op == "qk_norm":
        R, P, Hq, Hk, d, rot = (case[x] for x in ("R", "P", "Hq", "Hk", "d", "rot"))
        s["q"], s["k"] = randn(R, P, Hq, d), randn(R, P, Hk, d)
        s["wq"], s["wk"] = ((1.0 + randn(d, dtype=torch.float32, scale=0.2),
                             1.0 + randn(d, dtype=torch.float32, scale=0.2))
                            if case["weights"] else (None, None))
        s["positions"] = s["inv_freq"] = None
        if rot:
            # each sequence starts somewhere in a long context
            start = torch.randint(0, 200_000, (R, 1), generator=gen, device="cuda")
            s["positions"] = (start + torch.arange(P, device="cuda")).to(torch.int32)
            i = torch.arange(rot // 2, device="cuda", dtype=torch.float64)
            s["inv_freq"] = (1e6 ** (-2.0 * i / rot)).float()
        s["q_out"], s["k_out"] = torch.empty_like(s["q"]), torch.empty_like(s["k"])
    else:
        R, H, G, d_k, d_v = (case[x] for x in ("R", "H", "G", "d_k", "d_v"))
        n = case["P"] if op == "scan" else case["B"]
        s["v"] = randn(R, n, H, d_v)
        s["k"] = randn(R, n, G, d_k, scale=d_k ** -0.5)
        s["q"] = randn(R, n, G, d_k)
        # steps of about 0.001 to 0.1 after the softplus, decay rates of 1 to 16
        u = torch.rand((H,), generator=gen, device="cuda")
        step = torch.exp(u * math.log(100.0) + math.log(1e-3))
        s["dt_bias"] = torch.log(torch.expm1(step))
        s["dt"] = randn(R, n, H, dtype=torch.float32)
        s["A"] = -(1.0 + 15.0 * torch.rand((H,), generator=gen, device="cuda"))
        s["D"] = (1.0 + randn(H, dtype=torch.float32, scale=0.2)) if case["D"] else None
        s["z"] = randn(R, n, H, d_v) if case["z"] else None
        s["y"] = torch.zeros((R, n, H, d_v), device="cuda", dtype=dt)
        if op == "scan":
            s["state"] = (randn(R, H, d_v, d_k, dtype=torch.float32, scale=0.3)
                          if case["state"] else None)
            s["lens"] = lens(R, n) if case["lens"] else None
            s["state_out"] = torch.zeros((R, H, d_v, d_k), device="cuda")
        else:
            Bp = case["Bp"]
            s["state"] = randn(R, Bp, H, d_v, d_k, dtype=torch.float32, scale=0.3)
            s["parents"] = parents(R, n, Bp) if case["parents"] else None
            s["state_out"] = torch.zeros((R, n, H, d_v, d_k), device="cuda")
    return s


# ---------------------------------------------------------------------------------- one pass

def run(s):
    if own:
        return _run_own(s)
    op = s["case"]["op"]
    if op == "conv":
        return _conv(s)
    if op == "conv_step":
        return _conv_step(s)
    if op == "qk_norm":
        return _qk_norm(s)
    if op == "scan":
        return _scan(s)
    return _scan_step(s)


def _run_own(s):
    import linear_attention_beam_gdn_b200 as ola
    op, c = s["case"]["op"], s["case"]
    if op == "conv":
        return ola.conv(s["x"], s["w"], s["bias"], state=s["state"], lens=s["lens"],
                        silu=c["silu"], out=s["y"], state_out=s["state_out"])
    if op == "conv_step":
        return ola.conv_step(s["x"], s["w"], s["bias"], state=s["state"],
                             parent_idx=s["parents"], silu=c["silu"], out=s["y"],
                             state_out=s["state_out"])
    if op == "qk_norm":
        return ola.qk_norm(s["q"], s["k"], wq=s["wq"], wk=s["wk"], eps=1e-6, l2=c["l2"],
                           positions=s["positions"], inv_freq=s["inv_freq"], pair=c["pair"],
                           q_out=s["q_out"], k_out=s["k_out"])
    if op == "scan":
        return ola.scan(s["v"], s["dt"], s["A"], s["k"], s["q"], D=s["D"],
                        dt_bias=s["dt_bias"], z=s["z"], S_in=s["state"], lens=s["lens"],
                        softplus=True, out=s["y"], S_out=s["state_out"])
    return ola.scan_step(s["v"], s["dt"], s["A"], s["k"], s["q"], state=s["state"], D=s["D"],
                         dt_bias=s["dt_bias"], z=s["z"], parent_idx=s["parents"], softplus=True,
                         out=s["y"], state_out=s["state_out"])


def _silu(u):
    return u / (1.0 + torch.exp(-u))


def _softplus(x):
    return torch.where(x > 20.0, x, torch.log1p(torch.exp(torch.clamp(x, max=20.0))))


def _taps(s, full, n):
    """bias + sum over the taps of w[:, i] * full[:, i : i + n]."""
    c = s["case"]
    u = sum(s["w"][:, i] * full[:, i:i + n] for i in range(c["W"]))
    if s["bias"] is not None:
        u = u + s["bias"]
    return _silu(u) if c["silu"] else u


def _conv(s):
    c = s["case"]
    R, P, C, W = c["R"], c["P"], c["C"], c["W"]
    x = s["x"]
    old = s["state"] if s["state"] is not None else torch.zeros(
        (R, W - 1, C), device=x.device, dtype=x.dtype)
    full = torch.cat([old, x], 1)
    y = _taps(s, full.float(), P).to(x.dtype)
    n = s["lens"] if s["lens"] is not None else torch.full((R,), P, device=x.device)
    valid = torch.arange(P, device=x.device) < n[:, None]
    y = torch.where(valid[:, :, None], y, s["y"])
    at = n[:, None].long() + torch.arange(W - 1, device=x.device)
    state = torch.gather(full, 1, at[:, :, None].expand(R, W - 1, C))
    return y, state


def _conv_step(s):
    c = s["case"]
    R, B, C, W = c["R"], c["B"], c["C"], c["W"]
    x, old = s["x"], s["state"]
    if s["parents"] is not None:
        old = old[torch.arange(R, device=x.device)[:, None], s["parents"].long()]
    full = torch.cat([old, x[:, :, None]], 2)                       # [R, B, W, C]
    y = _taps(s, full.float().reshape(R * B, W, C), 1).reshape(R, B, C).to(x.dtype)
    return y, full[:, :, 1:].contiguous()


def _rotate(x, cos, sin, rot, pair):
    if pair:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([turned, x[..., rot:]], -1)


def _qk_norm(s):
    c = s["case"]
    rot = c["rot"]
    cos = sin = None
    if rot:
        angle = s["positions"].double()[..., None] * s["inv_freq"].double()
        cos, sin = torch.cos(angle).float()[:, :, None], torch.sin(angle).float()[:, :, None]

    def one(x, w):
        f = x.float()
        sq = (f * f).sum(-1, keepdim=True)
        f = f * torch.rsqrt((sq if c["l2"] else sq / c["d"]) + 1e-6)
        if w is not None:
            f = f * w
        return (_rotate(f, cos, sin, rot, c["pair"]) if rot else f).to(x.dtype)

    return one(s["q"], s["wq"]), one(s["k"], s["wk"])


def _gated(s, o, v):
    if s["D"] is not None:
        o = o + s["D"][:, None] * v
    if s["z"] is not None:
        o = o * _silu(s["z"].float())
    return o


def _scan(s):
    """Chunks of 128 tokens: inside a chunk a masked product of queries and keys, between chunks
    the states, joined by their decays (sums of exponents in 64 bits)."""
    c, Q = s["case"], 128
    R, P, H, G, d_k, d_v = (c[x] for x in ("R", "P", "H", "G", "d_k", "d_v"))
    dev, n = s["v"].device, -(-P // Q)
    length = s["lens"] if s["lens"] is not None else torch.full((R,), P, device=dev)
    valid = torch.arange(P, device=dev) < length[:, None]            # [R, P]
    dt = torch.where(valid[:, :, None], _softplus(s["dt"] + s["dt_bias"]),
                     torch.zeros((), device=dev))

    def chunks(x):
        x = torch.cat([x, x.new_zeros((R, n * Q - P) + x.shape[2:])], 1) if n * Q > P else x
        return x.reshape((R, n, Q) + x.shape[2:]).transpose(2, 3)    # [R, n, heads, Q, ...]

    v = s["v"].float()
    vc, kc, qc, dc = chunks(v), chunks(s["k"].float()), chunks(s["q"].float()), chunks(dt)
    cum = torch.cumsum((dc.double() * s["A"].double()[:, None]), -1)  # [R, n, H, Q]
    gap = cum[..., :, None] - cum[..., None, :]
    lower = torch.ones((Q, Q), device=dev, dtype=torch.bool).tril()
    decay = torch.where(lower, gap, torch.full((), -math.inf, device=dev,
                                               dtype=torch.float64)).exp_().float()
    del gap
    qk = torch.matmul(qc, kc.transpose(-1, -2))                      # [R, n, G, Q, Q]
    m = (decay.reshape(R, n, G, H // G, Q, Q) * qk[:, :, :, None]).reshape(R, n, H, Q, Q)
    del decay, qk
    vd = vc * dc[..., None]
    o = torch.matmul(m, vd)
    del m
    end = cum[..., -1]                                               # [R, n, H]
    vw = vd * torch.exp(end[..., None] - cum).float()[..., None]
    per = H // G
    vw = vw.reshape(R, n, G, per, Q, d_v)
    grow = torch.matmul(vw.transpose(-1, -2), kc[:, :, :, None])     # [R, n, G, per, d_v, d_k]
    grow = grow.reshape(R, n, H, d_v * d_k)
    tot = torch.cumsum(end, 1).transpose(1, 2)                       # [R, H, n], through chunk j
    before = torch.cat([torch.zeros((R, H, 1), device=dev, dtype=torch.float64), tot], -1)
    gap = before[..., :, None] - tot[..., None, :]                   # [R, H, n + 1, n]
    earlier = torch.arange(n, device=dev) < torch.arange(n + 1, device=dev)[:, None]
    join = torch.where(earlier, gap, torch.full((), -math.inf, device=dev,
                                                dtype=torch.float64)).exp_().float()
    states = torch.matmul(join, grow.transpose(1, 2))                # [R, H, n + 1, d_v * d_k]
    if s["state"] is not None:
        states = states + torch.exp(before).float()[..., None] * s["state"].reshape(
            R, H, 1, d_v * d_k)
    last = states[:, :, n].reshape(R, H, d_v, d_k).clone()
    states = states[:, :, :n].reshape(R, G, per, n, d_v, d_k)
    o2 = torch.matmul(states, qc.permute(0, 2, 1, 4, 3)[:, :, None])  # [R, G, per, n, d_v, Q]
    del states
    o2 = o2.reshape(R, H, n, d_v, Q).permute(0, 2, 1, 4, 3)
    o = o + torch.exp(cum).float()[..., None] * o2
    o = o.transpose(2, 3).reshape(R, n * Q, H, d_v)[:, :P]
    y = _gated(s, o, v).to(s["v"].dtype)
    return torch.where(valid[:, :, None, None], y, s["y"]), last


def _scan_step(s):
    c = s["case"]
    R, B, H, G = c["R"], c["B"], c["H"], c["G"]
    old = s["state"]
    if s["parents"] is not None:
        old = old[torch.arange(R, device=old.device)[:, None], s["parents"].long()]
    dt = _softplus(s["dt"] + s["dt_bias"])
    a = torch.exp(dt.double() * s["A"].double()).float()
    v = s["v"].float()
    k = s["k"].float().repeat_interleave(H // G, 2)
    q = s["q"].float().repeat_interleave(H // G, 2)
    new = a[..., None, None] * old + (dt[..., None] * v)[..., None] * k[..., None, :]
    o = (new * q[..., None, :]).sum(-1)
    return _gated(s, o, v).to(s["v"].dtype), new


# ---------------------------------------------------------------------------------- work

def _sources(case):
    """How many distinct parents the beams of one request have, on average."""
    B, n = case["B"], case["Bp"]
    if not case["parents"]:
        return B
    return sum(1.0 - (1.0 - (math.sqrt((j + 1) / n) - math.sqrt(j / n))) ** B for j in range(n))


def work(case):
    """Inputs once (of the states, those that are some beam's parent), outputs once; the
    operations of the definition."""
    e = 2 if case["dtype"] == BF16 else 4
    op = case["op"]
    if op in ("conv", "conv_step"):
        R, C, W = case["R"], case["C"], case["W"]
        n = R * (case["P"] if op == "conv" else case["B"])
        b = 2 * n * C * e + C * W * 4 + (C * 4 if case["bias"] else 0)
        if op == "conv":
            b += R * (W - 1) * C * e * (2 if case["state"] else 1)
        else:
            b += (R * _sources(case) + n) * (W - 1) * C * e + (4 * n if case["parents"] else 0)
        return {"bytes": b, "flops": n * C * (2 * W + (4 if case["silu"] else 0))}
    if op == "qk_norm":
        n, d = case["R"] * case["P"], case["d"]
        heads = case["Hq"] + case["Hk"]
        b = 2 * n * heads * d * e + (8 * d if case["weights"] else 0)
        b += 4 * n + 2 * case["rot"] if case["rot"] else 0
        return {"bytes": b, "flops": n * heads * (4 * d + 3 * case["rot"])}
    R, H, G, d_k, d_v = (case[x] for x in ("R", "H", "G", "d_k", "d_v"))
    n = R * (case["P"] if op == "scan" else case["B"])
    rows = n * H * d_v * e * (3 if case["z"] else 2) + 2 * n * G * d_k * e + 4 * n * H + 12 * H
    one = H * d_v * d_k * 4
    if op == "scan":
        states = R * one * (2 if case["state"] else 1)
    else:
        states = (R * _sources(case) + n) * one + (4 * n if case["parents"] else 0)
    return {"bytes": rows + states, "flops": n * H * (5 * d_k * d_v + 6 * d_v)}


# ---------------------------------------------------------------------------------- 64 bits

def exact(case, seed):
    """The definitions in 64 bits, token by token where the operator is a recurrence."""
    s = prepare(case, seed)
    op = case["op"]
    f = lambda t: None if t is None else t.double()  # noqa: E731
    if op == "conv":
        R, P, W = case["R"], case["P"], case["W"]
        y = s["y"].double()
        state = s["state_out"].double()
        for r in range(R):
            n = P if s["lens"] is None else int(s["lens"][r])
            old = torch.zeros((W - 1, case["C"]), device="cuda", dtype=torch.float64) \
                if s["state"] is None else f(s["state"][r])
            full = torch.cat([old, f(s["x"][r, :n])])
            if n:
                u = torch.zeros_like(full[:n])
                for i in range(W):
                    u.addcmul_(full[i:i + n], f(s["w"])[:, i])
                if s["bias"] is not None:
                    u += f(s["bias"])
                y[r, :n] = u * torch.sigmoid(u) if case["silu"] else u
            state[r] = full[n:n + W - 1]
        return y, state
    if op == "conv_step":
        R, B, W = case["R"], case["B"], case["W"]
        y = s["y"].double()
        state = s["state_out"].double()
        for r in range(R):
            src = s["state"][r] if s["parents"] is None else s["state"][r][s["parents"][r].long()]
            state[r, :, :W - 2] = f(src[:, 1:])
            state[r, :, W - 2] = f(s["x"][r])
            u = f(s["x"][r]) * f(s["w"])[:, W - 1] + torch.einsum(
                "bic,ci->bc", f(src), f(s["w"])[:, :W - 1])
            if s["bias"] is not None:
                u = u + f(s["bias"])
            y[r] = u * torch.sigmoid(u) if case["silu"] else u
        return y, state
    if op == "qk_norm":
        out = []
        rot, half = case["rot"], case["rot"] // 2
        for x, w in ((s["q"], s["wq"]), (s["k"], s["wk"])):
            o = torch.empty(x.shape, device="cuda", dtype=torch.float64)
            for r in range(case["R"]):
                t = f(x[r])
                norm = t.square().sum(-1, keepdim=True) if case["l2"] else \
                    t.square().mean(-1, keepdim=True)
                t = t / torch.sqrt(norm + 1e-6)
                if w is not None:
                    t = t * f(w)
                if rot:
                    ang = torch.outer(f(s["positions"][r]), f(s["inv_freq"]))
                    turn = torch.polar(torch.ones_like(ang), ang)[:, None]
                    if case["pair"]:
                        zc = torch.view_as_complex(
                            t[..., :rot].reshape(t.shape[:-1] + (half, 2)).contiguous()) * turn
                        head = torch.view_as_real(zc).flatten(-2)
                    else:
                        zc = torch.complex(t[..., :half], t[..., half:rot]) * turn
                        head = torch.cat([zc.real, zc.imag], -1)
                    t = torch.cat([head, t[..., rot:]], -1)
                o[r] = t
            out.append(o)
        return tuple(out)
    R, H, G, d_k, d_v = (case[x] for x in ("R", "H", "G", "d_k", "d_v"))
    n = case["P"] if op == "scan" else case["B"]
    A = f(s["A"])
    y = s["y"].double()

    def parts(r, at):
        """(dt, v, k, q) of rows `at` of sequence or request r, heads first."""
        step = torch.nn.functional.softplus(f(s["dt"][r, at]) + f(s["dt_bias"]), threshold=60.0)
        rep = lambda t: f(t[r, at]).repeat_interleave(H // G, -2)  # noqa: E731
        return step, f(s["v"][r, at]), rep(s["k"]), rep(s["q"])

    def finish(o, r, at):
        if s["D"] is not None:
            o = o + f(s["D"])[:, None] * f(s["v"][r, at])
        if s["z"] is not None:
            z = f(s["z"][r, at])
            o = o * z * torch.sigmoid(z)
        return o

    if op == "scan_step":
        new = torch.empty(s["state_out"].shape, device="cuda", dtype=torch.float64)
        for r in range(R):
            src = s["state"][r] if s["parents"] is None else s["state"][r][s["parents"][r].long()]
            step, v, k, q = parts(r, slice(None))
            new[r] = f(src) * torch.exp(step * A)[..., None, None]
            new[r] += torch.einsum("bhv,bhk->bhvk", v * step[..., None], k)
            y[r] = finish(torch.einsum("bhvk,bhk->bhv", new[r], q), r, slice(None))
        return y, new
    # all sequences together, one token after the other; a sequence that has ended keeps its state
    S = torch.zeros((R, H, d_v, d_k), device="cuda", dtype=torch.float64)
    if s["state"] is not None:
        S += s["state"]
    rows = slice(None)
    if n * (2e-4 + R * H * d_v * d_k * 40 / 4e12) > 15.0:
        return None
    length = None if s["lens"] is None else s["lens"]
    block = max(1, min(n, 30_000_000 // (R * H * max(d_k, d_v))))
    for p0 in range(0, n, block):
        at = slice(p0, min(n, p0 + block))
        step, v, k, q = parts(rows, at)
        a = torch.exp(step * A)
        v = v * step[..., None]
        o = torch.empty((R, at.stop - p0, H, d_v), device="cuda", dtype=torch.float64)
        for i in range(at.stop - p0):
            new = S * a[:, i, :, None, None]
            new += v[:, i, :, :, None] * k[:, i, :, None, :]
            if length is not None:
                new = torch.where((length > p0 + i)[:, None, None, None], new, S)
            S = new
            o[:, i] = torch.matmul(S, q[:, i, :, :, None])[..., 0]
        o = finish(o, rows, at)
        if length is not None:
            keep = (torch.arange(p0, at.stop, device="cuda") < length[:, None])[:, :, None, None]
            o = torch.where(keep, o, y[:, at])
        y[:, at] = o
    return y, S

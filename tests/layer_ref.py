"""The operators around the recurrence in 64 bits, straight from their definitions (CPU, torch
double), with running bounds of what fp32 arithmetic may lose. Shares nothing with the kernels."""
import torch

U = 2.0 ** -24                      # half a step of fp32, relative
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}   # of the result's own rounding


def d(x):
    return None if x is None else x.detach().cpu().double()


def silu(u):
    return u * torch.sigmoid(u)


def conv(x, w, bias, state, lens, act, out0):
    """(y, state_out, tol of y). y rows behind a sequence's end are out0's."""
    dt = x.dtype
    R, P, C = x.shape
    W = w.shape[1]
    x, w64, y = d(x), d(w), d(out0).clone()
    tol = torch.zeros_like(y)
    st = torch.zeros(R, W - 1, C, dtype=torch.float64) if state is None else d(state)
    st_out = torch.empty_like(st)
    for r in range(R):
        n = P if lens is None else max(0, min(P, int(lens[r])))
        u = torch.cat([st[r], x[r, :n]])
        st_out[r] = u[n:n + W - 1]
        for p in range(n):
            terms = u[p:p + W].t() * w64
            s, a = terms.sum(-1), terms.abs().sum(-1)
            if bias is not None:
                s, a = s + d(bias), a + d(bias).abs()
            y[r, p] = silu(s) if act else s
            # W fused steps of the sum; SiLU's slope is below 1.1 and its own steps (exponential,
            # sum, quotient) lose a few units (the fast ones a few units of 2^-22)
            fast = 2.0 ** -20 if dt == torch.bfloat16 else 8 * U
            tol[r, p] = 1.1 * (W + 1) * U * a + fast * y[r, p].abs() + HALF[dt] * y[r, p].abs()
    return y, st_out, tol + 1e-30


def qk_norm(x, w, eps, l2, positions, inv_freq, pair):
    """(out, tol)"""
    dt = x.dtype
    x64 = d(x)
    dim = x.shape[-1]
    s = x64.square().sum(-1, keepdim=True)
    n = x64 / torch.sqrt((s if l2 else s / dim) + eps)
    if w is not None:
        n = n * d(w)
    mag = n.abs()
    if inv_freq is not None and inv_freq.numel():
        half = inv_freq.numel()
        ang = (d(positions)[..., None] * d(inv_freq))[:, :, None]     # [R, P, 1, half]
        c, sn = torch.cos(ang), torch.sin(ang)
        a, b = (n[..., 0:2 * half:2], n[..., 1:2 * half:2]) if pair else \
            (n[..., :half], n[..., half:2 * half])
        ta, tb = a * c - b * sn, b * c + a * sn
        both = a.abs() + b.abs()
        n, mag = n.clone(), mag.clone()
        if pair:
            n[..., 0:2 * half:2], n[..., 1:2 * half:2] = ta, tb
            mag[..., 0:2 * half:2], mag[..., 1:2 * half:2] = both, both
        else:
            n[..., :half], n[..., half:2 * half] = ta, tb
            mag[..., :half], mag[..., half:2 * half] = both, both
    # the sum of dim squares (half of its relative error after the root), the root, the weight,
    # the rotation's cosine, products and sum
    tol = (dim / 2 + 24) * U * mag + HALF[dt] * n.abs()
    return n, tol + 1e-30


def softplus(x):
    return torch.where(x > 40, x, torch.log1p(torch.exp(torch.clamp(x, max=40.0))))


def scan(v, dt, A, k, q, D, dt_bias, z, S_in, lens, use_softplus, out0, chunked=False):
    """(y, S, tol of y, tol of S). `chunked`: y's token-to-token weights and the state's copy are
    rounded to bf16 on the way."""
    t = v.dtype
    R, P, H, dv = v.shape
    G, dk = k.shape[2], k.shape[3]
    y = d(out0).clone()
    toly = torch.zeros_like(y)
    S = torch.zeros(R, H, dv, dk, dtype=torch.float64) if S_in is None else d(S_in).clone()
    tolS = torch.zeros_like(S)
    v64, dt64, k64, q64, z64 = d(v), d(dt), d(k), d(q), d(z)
    if dt_bias is not None:
        dt64 = dt64 + d(dt_bias)
    raw = dt64
    if use_softplus:
        dt64 = softplus(dt64)
    # what fp32 makes of the step: its own rounding and that of raw + bias, then softplus
    for r in range(R):
        n = P if lens is None else max(0, min(P, int(lens[r])))
        M, E = S[r].abs(), torch.zeros_like(S[r])      # sum of |contributions|, bound of the error
        T = S[r].clone()
        for p in range(n):
            kk = k64[r, p].repeat_interleave(H // G, 0)
            qq = q64[r, p].repeat_interleave(H // G, 0)
            g = dt64[r, p] * d(A)
            a = torch.exp(g)[:, None, None]
            step_rel = 8 * U * (1 + raw[r, p].abs() / dt64[r, p].abs().clamp(min=1e-30)).clamp(
                max=1e6) if use_softplus else (8 * U * (1 + raw[r, p].abs() /
                                                        dt64[r, p].abs().clamp(min=1e-30))).clamp(max=1.0)
            w = (dt64[r, p][:, None] * v64[r, p])[:, :, None] * kk[:, None, :]
            # decay: exp's own error, and that of its argument
            dec = (8 * U + g.abs() * step_rel)[:, None, None]
            E = a * (E + (dec + 2 * U) * M) + (step_rel[:, None, None] + 4 * U) * w.abs()
            M = a * M + w.abs()
            T = a * T + w
            E = E + 2 * U * M
            o = (T * qq[:, None, :]).sum(-1)
            oa = (M * qq.abs()[:, None, :]).sum(-1)
            eo = (E * qq.abs()[:, None, :]).sum(-1) + (dk + 4) * U * oa
            if chunked:
                # each contribution is rounded to bf16 once (its weight or the state holding it);
                # a state's copy is two bf16 numbers at best, one at worst
                eo = eo + 2.0 ** -8 * oa * 1.01
            if D is not None:
                o = o + d(D)[:, None] * v64[r, p]
                eo = eo + 2 * U * (o.abs() + (d(D)[:, None] * v64[r, p]).abs())
            if z is not None:
                gate = silu(z64[r, p])
                o, eo = o * gate, eo * gate.abs() + 2.0 ** -20 * (o * gate).abs() \
                    if t == torch.bfloat16 else eo * gate.abs() + 12 * U * (o * gate).abs()
            y[r, p] = o
            toly[r, p] = eo + HALF[t] * o.abs()
        if chunked:
            # A chunk's own contributions are summed by 8 accumulation steps of 16 products. A step
            # aligns its addends to the largest and cuts them at 24 bits or more: up to 2 U of it
            # for the accumulator and for each of the 16 products, so 8 * 2 U + 16 * 2 U of the
            # sum of |contributions| at most (the second and third bf16 part of a weight add
            # 2^-8 of that). These errors decay with the contributions, so over all chunks they
            # stay below 50 U of M. (The weights' exponents are covered above: a sum of at most 8
            # additions of terms off by 3 U is off by 11 U of itself, below step_rel's 16 U.)
            E = E + 50 * U * M
        S[r], tolS[r] = T, E
    return y, S, toly + 1e-30, tolS + 1e-30

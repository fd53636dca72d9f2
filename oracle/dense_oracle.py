"""The dense side's operators in 64 bits, from their definitions, and how far a 16-bit product with
fp32 sums may be from them.  Test infrastructure: the kernels' results are compared with these.

Tensors are torch tensors on any device.  Attention takes lists of sequences' tokens by offsets and
works one sequence and head at a time.
"""
from __future__ import annotations

import math

import torch

U = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
TINY = {torch.float32: 2.0 ** -150, torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -134}
F32 = 2.0 ** -24


def visible(n: int, window: int, sinks: int, device="cpu"):
    i = torch.arange(n, device=device)[:, None]
    j = torch.arange(n, device=device)[None]
    return (j <= i) & ((i - j < window) | (j < sinks))


def _softmax(s, see):
    s = s.masked_fill(~see, -math.inf)
    lse = torch.logsumexp(s, -1)
    return torch.exp(s - lse[:, None]), lse


def _head(q, k, scale):
    """Scores, and the relative error of exp(score) when products and sums are fp32 and the
    exponential is good to a few units in the last place."""
    s = q @ k.T * scale
    worst = (q.abs() @ k.abs().T * abs(scale)).max().item() if s.numel() else 0.0
    return s, 2 * (q.shape[1] + 8) * F32 * worst + 16 * F32


def attn_fwd(q, k, v, offsets, window, sinks, scale):
    """out, lse, and the bounds of a kernel's error at them."""
    dt = q.dtype
    u, tiny = U.get(dt, 0.0), TINY.get(dt, 0.0)
    g = q.shape[1] // k.shape[1]
    out = torch.zeros(q.shape, dtype=torch.float64, device=q.device)
    lse = torch.zeros((q.shape[1], q.shape[0]), dtype=torch.float64, device=q.device)
    b_out, b_lse = torch.zeros_like(out), torch.zeros_like(lse)
    off = offsets.tolist()
    for a, z in zip(off[:-1], off[1:]):
        n = z - a
        see = visible(n, window, sinks, q.device)
        for h in range(q.shape[1] if n else 0):
            qq, kk, vv = q[a:z, h].double(), k[a:z, h // g].double(), v[a:z, h // g].double()
            s, rel = _head(qq, kk, scale)
            p, l = _softmax(s, see)
            o = p @ vv
            # each probability is rounded to 16 bits (u of itself, or half the smallest subnormal:
            # the largest stands at 1 or more) and sums of n terms to fp32
            rel += n * F32
            out[a:z, h], lse[h, a:z] = o, l
            b_out[a:z, h] = u * o.abs() + (u + 2 * rel) * (1 + u) * (p @ vv.abs()) + \
                tiny * see.double() @ vv.abs() + tiny
            b_lse[h, a:z] = 2 * rel + 4 * F32 * l.abs()
    return out, lse, b_out, b_lse


def attn_bwd(q, k, v, offsets, window, sinks, scale, out, lse, dout):
    """dq, dk, dv from the forward's results as given, and the bounds of a kernel's error."""
    dt = q.dtype
    u, tiny = U.get(dt, 0.0), TINY.get(dt, 0.0)
    g = q.shape[1] // k.shape[1]
    zero = lambda x: torch.zeros(x.shape, dtype=torch.float64, device=x.device)  # noqa: E731
    dq, dk, dv, bq, bk, bv = zero(q), zero(k), zero(k), zero(q), zero(k), zero(k)
    off = offsets.tolist()
    for a, z in zip(off[:-1], off[1:]):
        n = z - a
        see = visible(n, window, sinks, q.device)
        for h in range(q.shape[1] if n else 0):
            x = h // g
            qq, kk, vv = q[a:z, h].double(), k[a:z, x].double(), v[a:z, x].double()
            do, oo = dout[a:z, h].double(), out[a:z, h].double()
            s, rel = _head(qq, kk, scale)
            rel += 8 * F32 * lse[h, a:z].abs().max().item()
            p = torch.exp(s - lse[h, a:z].double()[:, None]).masked_fill(~see, 0.0)
            dp = do @ vv.T
            delta = (do * oo).sum(1, keepdim=True)
            ds = p * (dp - delta)
            # dp and delta are fp32 sums over the head's dimensions
            e = (q.shape[2] + 8) * F32 * (do.abs() @ vv.abs().T + (do * oo).abs().sum(1, keepdim=True))
            eds = p * e + ((u + 2 * rel + n * F32) * ds.abs() + tiny) * see * (1 + u)
            ep = ((u + 2 * rel + n * F32) * p + tiny) * see
            dq[a:z, h] = ds @ kk * scale
            bq[a:z, h] = eds @ kk.abs() * abs(scale)
            dk[a:z, x] += ds.T @ qq * scale
            bk[a:z, x] += eds.T @ qq.abs() * abs(scale)
            dv[a:z, x] += p.T @ do
            bv[a:z, x] += ep.T @ do.abs()
    fin = lambda x, b: b * (1 + u) + u * x.abs() + tiny  # noqa: E731
    return dq, dk, dv, fin(dq, bq), fin(dk, bk), fin(dv, bv)


def shared_sees(n_hist: int, first, window: int, sinks: int, device="cpu"):
    """Which of the history's events, then of its own tokens, each token of a request sees.  first: of each token, by
    its place in the request."""
    i = torch.arange(len(first), device=device)[:, None]
    j = torch.arange(n_hist, device=device)
    hist = ((n_hist - j < window) | (j < sinks)).expand(len(first), -1)
    j = torch.arange(len(first), device=device)
    return torch.cat([hist, (j <= i) & (j >= first[:, None])], 1)


def _requests(q, k, v, hk, hv, offsets, first, hist_offsets, window, sinks):
    """Of each request with tokens and each query head: tokens, history events, heads, what they see, and q, k, v."""
    g = q.shape[1] // k.shape[1]
    for a, z, ha, hz in zip(offsets.tolist()[:-1], offsets.tolist()[1:], hist_offsets.tolist()[:-1], hist_offsets.tolist()[1:]):
        f = torch.arange(z - a, device=q.device) if first is None else first[a:z].long() - a
        see = shared_sees(hz - ha, f, window, sinks, q.device)
        for h in range(q.shape[1] if z > a else 0):
            x = h // g
            yield (slice(a, z), slice(ha, hz), h, x, see, q[a:z, h].double(),
                   torch.cat([hk[ha:hz, x], k[a:z, x]]).double(), torch.cat([hv[ha:hz, x], v[a:z, x]]).double())


def attn_shared_fwd(q, k, v, hk, hv, offsets, first, hist_offsets, window, sinks, scale):
    """out, lse, and the bounds of a kernel's error at them, as attn_fwd's."""
    dt = q.dtype
    u, tiny = U.get(dt, 0.0), TINY.get(dt, 0.0)
    out = torch.zeros(q.shape, dtype=torch.float64, device=q.device)
    lse = torch.zeros((q.shape[1], q.shape[0]), dtype=torch.float64, device=q.device)
    b_out, b_lse = torch.zeros_like(out), torch.zeros_like(lse)
    for t, _, h, _, see, qq, kk, vv in _requests(q, k, v, hk, hv, offsets, first, hist_offsets, window, sinks):
        s, rel = _head(qq, kk, scale)
        p, l = _softmax(s, see)
        o = p @ vv
        # parts of a request's keys have maxima of their own, as in attn_decode
        rel += len(kk) * F32
        out[t, h], lse[h, t] = o, l
        b_out[t, h] = u * o.abs() + (u + 2 * rel) * (1 + u) * (p @ vv.abs()) + tiny * see.double() @ vv.abs() + tiny
        b_lse[h, t] = 2 * rel + 4 * F32 * l.abs()
    return out, lse, b_out, b_lse


def attn_shared_bwd(q, k, v, hk, hv, offsets, first, hist_offsets, window, sinks, scale, out, lse, dout):
    """dq, dk, dv and the history's dk and dv, then the bounds of a kernel's error at each, as attn_bwd's."""
    dt = q.dtype
    u, tiny = U.get(dt, 0.0), TINY.get(dt, 0.0)
    got = [torch.zeros(x.shape, dtype=torch.float64, device=q.device) for x in (q, k, v, hk, hv)]
    bound = [torch.zeros_like(x) for x in got]
    for t, j, h, x, see, qq, kk, vv in _requests(q, k, v, hk, hv, offsets, first, hist_offsets, window, sinks):
        n = j.stop - j.start
        do, oo = dout[t, h].double(), out[t, h].double()
        s, rel = _head(qq, kk, scale)
        rel += 8 * F32 * lse[h, t].abs().max().item()
        p = torch.exp(s - lse[h, t].double()[:, None]).masked_fill(~see, 0.0)
        dp = do @ vv.T
        delta = (do * oo).sum(1, keepdim=True)
        ds = p * (dp - delta)
        e = (q.shape[2] + 8) * F32 * (do.abs() @ vv.abs().T + (do * oo).abs().sum(1, keepdim=True))
        eds = p * e + ((u + 2 * rel + len(kk) * F32) * ds.abs() + tiny) * see * (1 + u)
        ep = ((u + 2 * rel + len(kk) * F32) * p + tiny) * see
        got[0][t, h] = ds @ kk * scale
        bound[0][t, h] = eds @ kk.abs() * abs(scale)
        dk, dv, bk, bv = ds.T @ qq * scale, p.T @ do, eds.T @ qq.abs() * abs(scale), ep.T @ do.abs()
        for to, own, hist, y in ((got, 1, 3, dk), (got, 2, 4, dv), (bound, 1, 3, bk), (bound, 2, 4, bv)):
            to[hist][j, x] += y[:n]
            to[own][t, x] += y[n:]
    return got, [b * (1 + u) + u * x.abs() + tiny for x, b in zip(got, bound)]


def power(exp):
    """2^(exp - 127) in 64 bits."""
    return (exp.long() - 127 + 1023 << 52).view(torch.float64)


def quantise(x):
    """e4m3 codes (uint8) and the exponent of each row of x [..., dim], by search: the nearest of all codes, halfway
    the even one."""
    dt, x = x.dtype, x.double()
    fine = x.isfinite()
    top = torch.where(fine, x.abs(), 0.0).amax(-1)
    k = torch.where(top > 0, torch.frexp(top)[1] - 8, -127).clamp(min=-127)
    y = x / power(k + 127)[..., None]
    most = {torch.float16: 8}.get(dt, 120)
    values = torch.arange(127, dtype=torch.uint8, device=x.device).view(torch.float8_e4m3fn).double()  # ascending
    at = torch.searchsorted(values, y.abs().contiguous()).clamp(1, 126)  # the first not below
    up, down = values[at] - y.abs(), y.abs() - values[at - 1]
    code = torch.where((up < down) | ((up == down) & (at % 2 == 0)), at, at - 1)
    code = torch.where((k == most)[..., None], code.clamp(max=int((values <= 240).sum()) - 1), code)
    code = torch.where(torch.signbit(x), code + 128, code)
    return torch.where(fine, code, 127).to(torch.uint8), (k + 127).to(torch.uint8)


def values_of(codes, exp):
    """What codes and their rows' exponents stand for; an exponent of 255 is NaN."""
    return codes.view(torch.float8_e4m3fn).double() * torch.where(exp == 255, math.nan, power(exp))[..., None]


def attn_decode(q, k, v, lens, window, sinks, scale):
    dt = q.dtype
    u, tiny = U[dt], TINY[dt]
    g = q.shape[1] // k.shape[2]
    out = torch.zeros(q.shape, dtype=torch.float64, device=q.device)
    bound = torch.zeros_like(out)
    for b, n in enumerate(lens.tolist()):
        j = torch.arange(n, device=q.device)
        j = j[(j >= n - window) | (j < sinks)]
        for h in range(q.shape[1] if n else 0):
            kk, vv = k[b, j, h // g].double(), v[b, j, h // g].double()
            s, rel = _head(q[b, h:h + 1].double(), kk, scale)
            p = torch.softmax(s, 1)
            o = (p @ vv)[0]
            rel += len(j) * F32
            out[b, h] = o
            # each part of split keys has a maximum of its own, so a probability is rounded to a
            # multiple of `tiny` of its part's largest, which is at most the whole's
            bound[b, h] = u * o.abs() + (u + 2 * rel) * (1 + u) * (p @ vv.abs())[0] + \
                tiny * vv.abs().sum(0) + tiny
    return out, bound


# ---------------------------------------------------------------------------------- norms
def rms(x, eps):
    return x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)


def norm_fwd(x, y, gate, w_post, w_pre, alpha, eps):
    r = alpha * x.double()
    if y is not None:
        n = y.double()
        if w_post is not None:
            n = rms(n, eps) * w_post.double()
        r = r + (n if gate is None else n * gate.double())
    h = None if w_pre is None else rms(r, eps) * w_pre.double()
    return r, h


def norm_bwd(r, y, gate, w_post, w_pre, alpha, eps, dr, dh):
    """dx, dy, dgate (of rows: by row), dw_post, dw_pre; None where an input is."""
    def back(z, g):  # of rms at z
        q = torch.sqrt((z * z).mean(-1, keepdim=True) + eps)
        return g / q - z * (g * z).mean(-1, keepdim=True) / q ** 3
    dR = torch.zeros((1,), dtype=torch.float64, device=(dr if dr is not None else dh).device)
    if dr is not None:
        dR = dr.double()
    dw_pre = None
    if w_pre is not None:
        rr = r.double()
        dR = dR + back(rr, dh.double() * w_pre.double())
        dw_pre = (dh.double() * rms(rr, eps)).sum(0)
    dy = dgate = dw_post = None
    if y is not None:
        yy = y.double()
        unit = yy if w_post is None else rms(yy, eps)
        n = unit if w_post is None else unit * w_post.double()
        dn = dR if gate is None else dR * gate.double()
        if gate is not None:
            dgate = dR * n
            if gate.dim() == 1:
                dgate = dgate.sum(0)
        dy = dn if w_post is None else back(yy, dn * w_post.double())
        if w_post is not None:
            dw_post = (dn * unit).sum(0)
    return alpha * dR, dy, dgate, dw_post, dw_pre


# ---------------------------------------------------------------------------------- AdamW
BLOCK = 128


def adamw(w, g, m, v, step, lr, b1, b2, eps, wd):
    """New weight, m and v of one tensor, in the inputs' precision (pass 64 bits for the exact)."""
    m = b1 * m + (1 - b1) * g
    v = b2 * v + (1 - b2) * g * g
    return w - lr * (m / (1 - b1 ** step) / (torch.sqrt(v / (1 - b2 ** step)) + eps) + wd * w), m, v


def hash_bits(seed: int, index):
    """32 bits for each element index: two rounds of MurmurHash3's finaliser."""
    def mix(x):
        x = ((x ^ (x >> 16)) * 0x85EBCA6B) & 0xFFFFFFFF
        x = ((x ^ (x >> 13)) * 0xC2B2AE35) & 0xFFFFFFFF
        return x ^ (x >> 16)
    low = mix(torch.tensor(seed & 0xFFFFFFFF)).to(index.device)
    base = mix(low ^ ((seed >> 32) & 0xFFFFFFFF) ^ (((index >> 32) * 0x9E3779B1) & 0xFFFFFFFF))
    return mix((index + base) & 0xFFFFFFFF)


def pow2(k):
    """2^k for whole k, exact (a library's power need not be)."""
    return ((k.long() + 1023) << 52).view(torch.float64)


def values(codes, exp):
    """What e4m3 codes with block exponents (plus 127) stand for."""
    return (codes.view(torch.float8_e4m3fn).double().reshape(-1, BLOCK) * pow2(exp.int() - 127)[:, None]).reshape(-1)


def e4m3_neighbours(x):
    """The e4m3-like codes below and above |x| (values), with four significant bits down to 2^-9."""
    step = pow2(torch.frexp(x.abs().clamp(min=2.0 ** -6))[1] - 4)
    low = torch.floor(x.abs() / step) * step
    return low, low + step, step


def block_exponents(x):
    """floor(log2(largest)) - 7 of each block of 128, -127 where all are zero."""
    top = x.reshape(-1, BLOCK).abs().amax(1)
    return torch.where(top > 0, torch.frexp(top)[1] - 8, -127).clamp(min=-127)


def to_codes(x, bits, keep):
    """Values of codes and block exponents of fp32 x with 16 random bits an element."""
    k = block_exponents(x)
    y = x.double().reshape(-1, BLOCK) * pow2(-k)[:, None]
    low, high, step = e4m3_neighbours(y)
    up = (bits.reshape(-1, BLOCK).double() + 0.5) / 65536
    # the upper where the place between two codes and `up` are over one; 64 bits hold that sum
    c = (torch.ceil(y.abs() / step + up) - 1) * step
    if keep:
        c = torch.where((y != 0) & (c == 0), 2.0 ** -9, c)
    return (c * torch.sign(y) * pow2(k)[:, None]).reshape(-1), k

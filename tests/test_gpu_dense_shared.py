"""Attention of candidates that share a history against the 64-bit oracle: training and serving forms, histories
in 16 and 8 bits, and the newest event against a cache in 8 bits, at lengths, head layouts, widths and strides where
the kernels' tiles end; within bounds that count the 16-bit roundings of results, probabilities and their gradients."""
import pytest

torch = pytest.importorskip("torch")

from ad_recommendation_amd import dense, emb  # noqa: E402
from oracle import dense_oracle as O  # noqa: E402

pytestmark = pytest.mark.gpu
F16, BF16 = torch.float16, torch.bfloat16
U8 = torch.uint8
BIG = 2 ** 31 - 1


def offsets(lens):
    return torch.tensor([0] + torch.tensor(lens).cumsum(0).tolist(), dtype=torch.int32, device="cuda")


def rand(*shape, dtype, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(*shape, generator=g, device="cuda").to(dtype)


def within(got, want, bound, what):
    err = (got.double() - want).abs()
    assert torch.isfinite(got).all(), what
    worst = (err - bound).max().item() if err.numel() else -1.0
    assert worst <= 0, f"{what}: {worst:.3g} over its bound, largest error {err.max().item():.3g}"


def candidates(lens, tokens):
    """first: candidates of 1 to 2 * tokens - 1 tokens, in turn; None for one token each."""
    if tokens == 1:
        return None
    first, at = [], 0
    for n in lens:
        i, size = 0, 1
        while i < n:
            m = min(size, n - i)
            first += [at + i] * m
            i += m
            size = size % (2 * tokens - 1) + 1
        at += n
    return torch.tensor(first, dtype=torch.int32, device="cuda")


def workspace(n):
    """Bytes that are NaN where they are not written, and some behind them that are to stay."""
    return torch.full((n + 64,), 0xFF, dtype=U8, device="cuda")


def inputs(c, h, hq, hk, d, dtype, seed=0):
    n, m = sum(c), sum(h)
    x = rand(n, hq + 2 * hk, d, dtype=dtype, seed=seed + n + d)
    y = rand(m, 2 * hk, d, dtype=dtype, seed=seed + m + d + 1)
    return x[:, :hq], x[:, hq:hq + hk], x[:, hq + hk:], y[:, :hk], y[:, hk:]


def fwd(q, k, v, hk, hv, off, first, hoff, window, sinks, scale, lse=True):
    n, hq, d = q.shape
    out = torch.full((n, hq, d), 7, dtype=q.dtype, device="cuda")
    l = torch.full((hq, n), 7.0, device="cuda") if lse else None
    nb = dense.attn_shared_fwd_workspace_bytes(n, off.numel() - 1, hk.shape[0], hq, k.shape[1], d)
    ws = workspace(nb)
    dense.attn_shared_fwd(q, k, v, hk, hv, off, first, hoff, window, sinks, scale, out, l, ws[:nb])
    assert (ws[nb:] == 0xFF).all()
    return (out, l) if lse else out


def cached(x, h, cap):
    """Packed histories in caches, with what must not be read behind them."""
    y = torch.full((len(h), cap, *x.shape[1:]), float("nan"), dtype=x.dtype, device="cuda")
    at = 0
    for s, n in enumerate(h):
        y[s, :n] = x[at:at + n]
        at += n
    return y


def in_8_bits(x):
    """Codes and exponents of a cache, and the values."""
    c, e = O.quantise(x)
    return c, e.transpose(1, 2).contiguous(), O.values_of(c, e).to(x.dtype)


# candidates' tokens, histories, q heads, kv heads, dim, window, sinks, tokens of a candidate
SHAPES = [
    ([1], [0], 1, 1, 8, BIG, 0, 1),
    ([1], [1], 1, 1, 16, BIG, 0, 1),
    ([0, 3, 2, 0, 1], [4, 0, 1, 0, 33], 2, 1, 16, BIG, 0, 2),
    ([5, 8], [31, 32], 4, 4, 32, BIG, 0, 1),
    ([6, 1, 9], [33, 63, 64], 4, 2, 64, 20, 3, 1),
    ([6, 1, 9], [65, 127, 300], 6, 2, 40, 1, 5, 3),
    ([10], [1000], 8, 1, 128, BIG, 0, 1),
    ([30], [1500], 8, 2, 64, 700, 4, 4),
    ([16, 0, 17, 15], [500, 3, 129, 0], 2, 2, 24, 128, 0, 1),
    ([127, 128, 129], [64, 0, 65], 2, 1, 64, BIG, 0, 1),
    ([200, 3, 0, 257], [128, 500, 9, 31], 6, 2, 40, 100, 32, 5),
    ([300], [777], 4, 1, 128, BIG, 0, 1),
    ([70, 400], [1029, 450], 4, 4, 128, 300, 2, 70),
    ([513], [2000], 1, 1, 80, 1999, 1, 1),
    ([90, 33], [400, 600], 3, 1, 104, 256, 0, 2),
    ([64] * 40, [70] * 40, 2, 2, 32, 65, 7, 1),
    ([3] * 150, [5] * 150, 3, 3, 48, BIG, 0, 2),
    ([40], [50], 40, 1, 32, BIG, 0, 1),
    ([0, 0], [3, 0], 2, 2, 32, 4, 2, 1),
]


@pytest.mark.parametrize("dtype", [F16, BF16], ids=str)
@pytest.mark.parametrize("c,h,hq,hk,d,window,sinks,tokens", SHAPES)
def test_forward_forms(c, h, hq, hk, d, window, sinks, tokens, dtype):
    print(f"[shared] {c[:6]} {h[:6]} heads {hq}/{hk} dim {d} window {window} sinks {sinks} tokens {tokens} {dtype}",
          flush=True)
    q, k, v, kh, vh = inputs(c, h, hq, hk, d, dtype)
    off, hoff, first, scale = offsets(c), offsets(h), candidates(c, tokens), 1.3 * d ** -0.5
    out, lse = fwd(q, k, v, kh, vh, off, first, hoff, window, sinks, scale)
    o, l, bo, bl = O.attn_shared_fwd(q, k, v, kh, vh, off, first, hoff, window, sinks, scale)
    within(out, o, bo, "out")
    within(lse, l, bl, "lse")
    again = fwd(q, k, v, kh, vh, off, first, hoff, window, sinks, scale)
    assert torch.equal(out, again[0]) and torch.equal(lse, again[1])  # the same bits again
    assert torch.equal(out, fwd(q, k, v, kh, vh, off, first, hoff, window, sinks, scale, lse=False))
    # against caches
    cap, lens = max(h) + 3, torch.tensor(h, dtype=torch.int32, device="cuda")
    kc, vc = cached(kh, h, cap), cached(vh, h, cap)
    n = sum(c)
    nb = dense.attn_shared_cache_workspace_bytes(n, len(c), cap, hq, hk, d)
    ws, got = workspace(nb), torch.full((n, hq, d), 7, dtype=dtype, device="cuda")
    dense.attn_shared_cache(q, k, v, kc, vc, off, first, lens, window, sinks, scale, got, ws[:nb])
    assert (ws[nb:] == 0xFF).all()
    within(got, o, bo, "out from caches")
    # in 8 bits
    kq, ke, kv_ = in_8_bits(kh.unsqueeze(0).float().to(dtype))
    vq, ve, vv_ = in_8_bits(vh.unsqueeze(0).float().to(dtype))
    o, _, bo, _ = O.attn_shared_fwd(q, k, v, kv_[0], vv_[0], off, first, hoff, window, sinks, scale)
    codes = [torch.full((len(c), cap, hk, d), 0x7F, dtype=U8, device="cuda") for _ in range(2)]
    exps = [torch.full((len(c), hk, cap), 0xFF, dtype=U8, device="cuda") for _ in range(2)]
    at = 0
    for s, m in enumerate(h):
        for x, y, a, b in ((codes[0], exps[0], kq, ke), (codes[1], exps[1], vq, ve)):
            x[s, :m], y[s, :, :m] = a[0, at:at + m], b[0, :, at:at + m]
        at += m
    ws, got = workspace(nb), torch.full((n, hq, d), 7, dtype=dtype, device="cuda")
    dense.attn_shared_cache_q8(q, k, v, codes[0], exps[0], codes[1], exps[1], off, first, lens, window, sinks, scale,
                               got, ws[:nb])
    assert (ws[nb:] == 0xFF).all()
    within(got, o, bo, "out from 8 bits")


def bwd(q, k, v, hk, hv, off, first, hoff, window, sinks, scale, out, lse, dout):
    n, hq, d = q.shape
    got = [torch.full(x.shape, 7, dtype=x.dtype, device="cuda") for x in (q, k, v, hk, hv)]
    nb = dense.attn_shared_bwd_workspace_bytes(n, off.numel() - 1, hk.shape[0], hq, k.shape[1], d)
    ws = workspace(nb)
    dense.attn_shared_bwd(q, k, v, hk, hv, off, first, hoff, window, sinks, scale, out, lse, dout, *got, ws[:nb])
    assert (ws[nb:] == 0xFF).all()
    return got


NAMES = ("dq", "dk", "dv", "dhist_k", "dhist_v")


@pytest.mark.parametrize("dtype", [F16, BF16], ids=str)
@pytest.mark.parametrize("c,h,hq,hk,d,window,sinks,tokens", SHAPES)
def test_backward(c, h, hq, hk, d, window, sinks, tokens, dtype):
    print(f"[shared bwd] {c[:6]} {h[:6]} heads {hq}/{hk} dim {d} window {window} sinks {sinks} tokens {tokens} {dtype}",
          flush=True)
    q, k, v, kh, vh = inputs(c, h, hq, hk, d, dtype)
    off, hoff, first, scale = offsets(c), offsets(h), candidates(c, tokens), 1.3 * d ** -0.5
    args = q, k, v, kh, vh, off, first, hoff, window, sinks, scale
    out, lse = fwd(*args)
    dout = rand(sum(c), hq, d, dtype=dtype, seed=9)
    got = bwd(*args, out, lse, dout)
    want, bound = O.attn_shared_bwd(*args, out, lse, dout)
    for name, g, w, b in zip(NAMES, got, want, bound):
        within(g, w, b, name)
    for g, again in zip(got, bwd(*args, out, lse, dout)):
        assert torch.equal(g, again)


# sequences' lengths, q heads, kv heads, dim, window, sinks
DECODE = [
    ([0, 1, 2, 31, 32, 33], 2, 1, 8, BIG, 0),
    ([5, 700, 64], 8, 2, 64, 100, 4),
    ([4000], 4, 1, 128, BIG, 0),
    ([1500, 0, 37], 3, 3, 40, 64, 32),
    ([300] * 70, 8, 8, 32, 129, 1),
    ([90, 2000], 66, 2, 80, 1000, 2),
]


@pytest.mark.parametrize("dtype", [F16, BF16], ids=str)
@pytest.mark.parametrize("lens,hq,hk,d,window,sinks", DECODE)
def test_newest_event_in_8_bits(lens, hq, hk, d, window, sinks, dtype):
    print(f"[decode q8] {lens[:6]} heads {hq}/{hk} dim {d} window {window} sinks {sinks} {dtype}", flush=True)
    n, cap, scale = len(lens), max(lens) + 5, 1.3 * d ** -0.5
    q = rand(n, hq, d, dtype=dtype, seed=1)
    kq, ke, kv = in_8_bits(rand(n, cap, hk, d, dtype=dtype, seed=2))
    vq, ve, vv = in_8_bits(rand(n, cap, hk, d, dtype=dtype, seed=3))
    for s, m in enumerate(lens):  # not to be read
        kq[s, m:], vq[s, m:], ke[s, :, m:], ve[s, :, m:] = 0x7F, 0x7F, 0xFF, 0xFF
    l = torch.tensor(lens, dtype=torch.int32, device="cuda")
    nb = dense.attn_window_decode_q8_workspace_bytes(n, cap, hq, hk, d, window, sinks)
    ws, out = workspace(nb), torch.full_like(q, 7)
    dense.attn_window_decode_q8(q, kq, ke, vq, ve, l, window, sinks, scale, out, ws[:nb])
    assert (ws[nb:] == 0xFF).all()
    o, bo = O.attn_decode(q, kv, vv, l, window, sinks, scale)
    within(out, o, bo, "out")
    again = torch.full_like(q, 7)
    dense.attn_window_decode_q8(q, kq, ke, vq, ve, l, window, sinks, scale, again, ws[:nb])
    assert torch.equal(out, again)


# ---------------------------------------------------------------------------------- with the operators beside it
@pytest.mark.parametrize("window,sinks", [(1, 0), (50, 3), (BIG, 0)])
def test_a_candidate_is_the_next_event(window, sinks):
    """Forward, gradients of the candidate and the cache's forms agree with windowed attention at the next event."""
    n, hq, hk, d, scale = 301, 4, 2, 64, 0.125
    q, k, v = (rand(n, h, d, dtype=F16, seed=s) for s, h in ((1, hq), (2, hk), (3, hk)))
    off, one, hoff = offsets([n]), offsets([1]), offsets([n - 1])
    want, lse = torch.empty_like(q), torch.empty(hq, n, device="cuda")
    dense.attn_window_fwd(q, k, v, off, window, sinks, scale, want, lse)
    _, _, bo, bl = O.attn_fwd(q, k, v, off, window, sinks, scale)
    out, l = fwd(q[-1:], k[-1:], v[-1:], k[:-1], v[:-1], one, None, hoff, window, sinks, scale)
    within(out[0], want[-1].double(), 2 * bo[-1], "out")
    within(l[:, 0], lse[:, -1].double(), 2 * bl[:, -1], "lse")
    # the same event, cached, as the newest
    kq, ke, kv = in_8_bits(k[None])
    vq, ve, vv = in_8_bits(v[None])
    lens = torch.tensor([n], dtype=torch.int32, device="cuda")
    got = torch.empty(1, hq, d, dtype=F16, device="cuda")
    nb = dense.attn_window_decode_q8_workspace_bytes(1, n, hq, hk, d, window, sinks)
    dense.attn_window_decode_q8(q[-1:], kq, ke, vq, ve, lens, window, sinks, scale, got, workspace(nb)[:nb])
    o, bo = O.attn_decode(q[-1:], kv, vv, lens, window, sinks, scale)
    within(got, o, bo, "newest from 8 bits")
    nb = dense.attn_shared_cache_workspace_bytes(1, 1, n, hq, hk, d)
    dense.attn_shared_cache_q8(q[-1:], kv[0, -1:], vv[0, -1:], kq, ke, vq, ve, one, None, lens - 1, window, sinks, scale, got,
                               workspace(nb)[:nb])
    within(got, o, bo, "candidate against 8 bits")


def test_one_candidate_of_many_tokens_is_causal_attention():
    lens, hq, hk, d = [130, 1, 0, 300], 4, 2, 32
    n, off = sum(lens), offsets(lens)
    first = torch.repeat_interleave(off[:-1], off[1:] - off[:-1]).int()
    q, k, v = (rand(n, h, d, dtype=BF16, seed=s) for s, h in ((1, hq), (2, hk), (3, hk)))
    none = torch.empty(0, hk, d, dtype=BF16, device="cuda")
    args = q, k, v, none, none, off, first, torch.zeros_like(off), 5, 1, 0.2
    out, lse = fwd(*args)
    o, l, bo, bl = O.attn_fwd(q, k, v, off, BIG, 0, 0.2)
    within(out, o, bo, "out")
    within(lse, l, bl, "lse")
    dout = rand(n, hq, d, dtype=BF16, seed=4)
    got = bwd(*args, out, lse, dout)
    want = O.attn_bwd(q, k, v, off, BIG, 0, 0.2, out, lse, dout)
    for g, w, b in zip(got, want[:3], want[3:]):
        within(g, w, b, "gradient")


def test_write_decode_rank_and_read_together():
    """A serving step: new events written in 8 bits, the newest answered, candidates ranked, the history read back."""
    users, cap, hq, hk, d, scale = 5, 90, 4, 2, 64, 0.125
    lens = torch.tensor([0, 3, 60, 89, 31], dtype=torch.int32, device="cuda")
    codes = [torch.zeros(users, cap, hk, d, dtype=U8, device="cuda") for _ in range(2)]
    exps = [torch.zeros(users, hk, cap, dtype=U8, device="cuda") for _ in range(2)]
    cache = codes[0], exps[0], codes[1], exps[1]
    old = [rand(int(lens.sum()), hk, d, dtype=BF16, seed=s) for s in (1, 2)]
    off = offsets(lens.tolist())
    dense.cache_q8_write(*old, off, None, *cache)
    new = [rand(users, hk, d, dtype=BF16, seed=s) for s in (3, 4)]
    dense.cache_q8_write(*new, None, lens, *cache)
    lens = lens + 1
    off = offsets(lens.tolist())
    back = [torch.empty(int(off[-1]), hk, d, dtype=BF16, device="cuda") for _ in range(2)]
    dense.cache_q8_read(*cache, off, None, *back)
    for x, (a, b) in enumerate(zip(old, new)):
        whole = []
        for u, (s, e) in enumerate(zip(off.tolist(), off.tolist()[1:])):
            whole += [a[s - u:e - u - 1], b[u:u + 1]]
        assert torch.equal(back[x], O.values_of(*O.quantise(torch.cat(whole))).to(BF16))
    packed = [torch.zeros(users, cap, hk, d, dtype=BF16, device="cuda") for _ in range(2)]
    for x in range(2):
        for u, (s, e) in enumerate(zip(off.tolist(), off.tolist()[1:])):
            packed[x][u, :e - s] = back[x][s:e]
    q, out = rand(users, hq, d, dtype=BF16, seed=5), torch.empty(users, hq, d, dtype=BF16, device="cuda")
    nb = dense.attn_window_decode_q8_workspace_bytes(users, cap, hq, hk, d, 40, 2)
    dense.attn_window_decode_q8(q, *cache, lens, 40, 2, scale, out, workspace(nb)[:nb])
    o, bo = O.attn_decode(q, *packed, lens, 40, 2, scale)
    within(out, o, bo, "newest")
    c = [4, 0, 70, 9, 33]
    q, k, v, _, _ = inputs(c, [1], hq, hk, d, BF16, seed=6)
    got = torch.empty(sum(c), hq, d, dtype=BF16, device="cuda")
    nb = dense.attn_shared_cache_workspace_bytes(sum(c), users, cap, hq, hk, d)
    dense.attn_shared_cache_q8(q, k, v, *cache, offsets(c), None, lens, 40, 2, scale, got, workspace(nb)[:nb])
    o, _, bo, _ = O.attn_shared_fwd(q, k, v, *back, offsets(c), None, off, 40, 2, scale)
    within(got, o, bo, "candidates")


# ---------------------------------------------------------------------------------- values
@pytest.mark.parametrize("c,h", [([9, 3], [40, 300]), ([150, 200], [90, 700])])
@pytest.mark.parametrize("scale", [0.0, -0.2])
def test_scale_of_any_sign(scale, c, h):
    q, k, v, kh, vh = inputs(c, h, 2, 1, 32, F16)
    args = q, k, v, kh, vh, offsets(c), candidates(c, 2), offsets(h), 60, 2, scale
    out, lse = fwd(*args)
    o, l, bo, bl = O.attn_shared_fwd(*args)
    within(out, o, bo, "out")
    within(lse, l, bl, "lse")
    dout = rand(*out.shape, dtype=F16, seed=5)
    want, bound = O.attn_shared_bwd(*args, out, lse, dout)
    for name, g, w, b in zip(NAMES, bwd(*args, out, lse, dout), want, bound):
        within(g, w, b, name)


@pytest.mark.parametrize("c", [[12], [400]])
def test_scores_that_grow_and_dwarf_one_another(c):
    """The running maximum moves many times, and far, also between parts that several workgroups have."""
    h = [3000]
    q, k, v, kh, vh = inputs(c, h, 2, 2, 64, F16)
    kh = kh * torch.linspace(0.01, 12, h[0], device="cuda")[:, None, None].half()
    for order in (slice(None), torch.arange(h[0] - 1, -1, -1, device="cuda")):
        args = q, k, v, kh[order], vh[order], offsets(c), None, offsets(h), BIG, 0, 0.125
        out, lse = fwd(*args)
        o, l, bo, bl = O.attn_shared_fwd(*args)
        within(out, o, bo, "out")
        within(lse, l, bl, "lse")
        dout = rand(*out.shape, dtype=F16, seed=5)
        want, bound = O.attn_shared_bwd(*args, out, lse, dout)
        for name, g, w, b in zip(NAMES, bwd(*args, out, lse, dout), want, bound):
            within(g, w, b, name)


@pytest.mark.parametrize("tokens", [1, 4])
@pytest.mark.parametrize("c", [[6, 11, 4], [150, 210, 90]])
@pytest.mark.parametrize("d,hq,dtype", [(32, 2, BF16), (128, 2, BF16), (64, 4, F16), (128, 6, F16)])
def test_what_is_not_finite_reaches_only_what_sees_it(d, hq, dtype, c, tokens):
    h, window, sinks = [60, 130, 40], 100, 2
    q, k, v, kh, vh = (x.contiguous() for x in inputs(c, h, hq, 2, d, dtype))
    off, hoff, first = offsets(c), offsets(h), candidates(c, tokens)
    n = sum(c)
    rest = off, first, hoff, window, sinks, 0.2
    out, lse = fwd(q, k, v, kh, vh, *rest)
    o, l, bo, bl = O.attn_shared_fwd(q, k, v, kh, vh, *rest)
    dout = rand(n, hq, d, dtype=dtype, seed=7)
    want, bound = O.attn_shared_bwd(q, k, v, kh, vh, *rest, out, lse, dout)
    rows = torch.arange(n, device="cuda")
    request = torch.repeat_interleave(torch.arange(3, device="cuda"), torch.tensor(c, device="cuda"))
    start = rows if first is None else first.long()
    at = c[0] + c[1] // 2  # a token of the second request
    seeing = (start == start[at]) & (rows >= at)  # tokens that see it
    seen = (start == start[at]) & (rows <= at)    # tokens that it sees
    for x, bad in ((k, float("nan")), (v, float("inf")), (v, float("nan"))):
        keep = x[at].clone()
        x[at] = bad
        got, _ = fwd(q, k, v, kh, vh, *rest)
        within(got[~seeing], o[~seeing], bo[~seeing], "out")
        assert not got[seeing].isfinite().all(-1).any()
        grads = bwd(q, k, v, kh, vh, *rest, out, lse, dout)
        within(grads[0][~seeing], want[0][~seeing], bound[0][~seeing], "dq")
        assert not grads[0][seeing].isfinite().all(-1).any()
        others = rows != at
        for i in (1, 2):
            within(grads[i][others], want[i][others], bound[i][others], NAMES[i])
        for i in (3, 4):
            within(grads[i], want[i], bound[i], NAMES[i])
        x[at] = keep
    # an event of the second history: its window begins at 31, sinks are 0 and 1
    for j, visible in ((h[0] + 1, True), (h[0] + 90, True), (h[0] + 10, False)):
        for x, bad in ((kh, float("nan")), (vh, float("inf"))):
            keep = x[j].clone()
            x[j] = bad
            got, _ = fwd(q, k, v, kh, vh, *rest)
            hit = (request == 1) & visible
            within(got[~hit], o[~hit], bo[~hit], "out")
            assert not got[hit].isfinite().all(-1).any()
            grads = bwd(q, k, v, kh, vh, *rest, out, lse, dout)
            within(grads[0][~hit], want[0][~hit], bound[0][~hit], "dq")
            events = torch.arange(sum(h), device="cuda") != j
            for i in (3, 4):
                within(grads[i][events], want[i][events], bound[i][events], NAMES[i])
            x[j] = keep
    mine = torch.zeros(sum(h), dtype=torch.bool, device="cuda")
    mine[h[0]:h[0] + h[1]] = True
    mine[h[0] + 2:h[0] + 31] = False
    for x in (q, dout):
        keep = x[at].clone()
        x[at] = float("nan")
        grads = bwd(q, k, v, kh, vh, *rest, out, lse, dout)
        others = rows != at
        within(grads[0][others], want[0][others], bound[0][others], "dq")
        assert not grads[0][at].isfinite().any()
        for i in (1, 2):
            within(grads[i][~seen], want[i][~seen], bound[i][~seen], NAMES[i])
        assert not grads[1][seen].isfinite().all(-1).any()
        for i in (3, 4):
            within(grads[i][~mine], want[i][~mine], bound[i][~mine], NAMES[i])
        assert not grads[3][mine].isfinite().all(-1).any()
        x[at] = keep


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("c,tokens", [([20], 1), ([20], 3), ([300], 1), ([300], 50)])
@pytest.mark.parametrize("h,big,grow", [([150], 1, 16000), ([2], 32, 500)])
def test_gradients_of_scores_past_fp16(h, big, grow, c, tokens, d):
    """Products of dout and v far past 65504, and with two events of history their gradients as well; the sums are not."""
    q, k, v, kh, vh = inputs(c, h, 2, 1, d, F16)
    q, k, kh, v, vh = q * 2.0 ** -6, k * 2.0 ** -6, kh * 2.0 ** -6, v * big, vh * big
    args = q, k, v, kh, vh, offsets(c), candidates(c, tokens), offsets(h), BIG, 0, 2.0 ** -8
    out, lse = fwd(*args)
    dout = (rand(*out.shape, dtype=torch.float32, seed=5) * grow).clamp(-60000, 60000).half()
    want, bound = O.attn_shared_bwd(*args, out, lse, dout)
    assert max(w.abs().max() for w in want) < 60000
    ds = (dout.double() @ vh[:2, 0].double().T - (dout.double() * out).sum(-1, keepdim=True)).abs() / (max(h) + tokens)
    if tokens == 1:
        assert (ds.max() > 65504) == (h == [2])
    for name, g, w, b in zip(NAMES, bwd(*args, out, lse, dout), want, bound):
        # once brought into range a gradient below 2^-24 of the largest may be lost
        within(g, w, 2 * b + 2.0 ** -12 * w.abs().max(), name)


def test_a_score_of_minus_infinity_weighs_nothing():
    c, h = [5, 140], [60, 200]
    q, k, v, kh, vh = (x.contiguous() for x in inputs(c, h, 1, 1, 32, F16))
    q[:, 0, 0] = 1
    gone = torch.tensor([3, 70], device="cuda")
    kh[gone, 0, 0] = -float("inf")
    k[[1, 9], 0, 0] = -float("inf")
    out = fwd(q, k, v, kh, vh, offsets(c), None, offsets(h), BIG, 0, 0.2)[0]
    for r, (a, z, ha, hz) in enumerate(((0, 5, 0, 60), (5, 145, 60, 260))):
        kk = torch.cat([kh[ha:hz, 0], k[a:z, 0]]).double().nan_to_num(0, 0, 0)
        vv = torch.cat([vh[ha:hz, 0], v[a:z, 0]]).double()
        see = torch.cat([torch.ones(z - a, hz - ha, device="cuda"), torch.eye(z - a, device="cuda")], 1).bool()
        see[:, gone[r] - ha] = False
        see[:, (hz - ha) + (1 if r == 0 else 4)] = False
        s = q[a:z, 0].double() @ kk.T * 0.2
        p = torch.softmax(s.masked_fill(~see, -float("inf")), 1)
        rel = 2 * 40 * O.F32 * (q[a:z, 0].abs().double() @ kk.abs().T * 0.2).max() + (16 + len(kk)) * O.F32
        u = O.U[F16]
        within(out[a:z, 0], p @ vv, u * (p @ vv).abs() + (u + 2 * rel) * (1 + u) * (p @ vv.abs()) +
               O.TINY[F16] * (1 + see.double() @ vv.abs()), "out")


# ---------------------------------------------------------------------------------- layouts and sizes
@pytest.mark.parametrize("d", [32, 64, 128])
@pytest.mark.parametrize("c,h", [([20, 5], [90, 130]), ([160, 140], [90, 230])])
def test_tokens_far_apart_and_heads_first(d, c, h):
    """Strides over which a tile of rows spans more than 2^31 bytes, and orders of heads and tokens."""
    n, m = sum(c), sum(h)
    far = torch.empty(max(n, m), (1 << 23) + 8, dtype=F16, device="cuda")
    tensors = list(inputs(c, h, 2, 2, d, F16)) + [rand(n, 2, d, dtype=F16, seed=9)]
    at, views = 0, []
    for x in tensors:
        y = far[:x.shape[0], at:at + 2 * d].unflatten(1, (2, d))
        y.copy_(x)
        views.append(y)
        at += 1024
    rest = offsets(c), candidates(c, 2), offsets(h), 70, 3, 0.1

    def run(q, k, v, kh, vh, dout):
        out, lse = fwd(q, k, v, kh, vh, *rest)
        return [out, lse, *bwd(q, k, v, kh, vh, *rest, out, lse, dout)]
    want, got = run(*tensors), run(*views)
    del far, views
    o, l, bo, bl = O.attn_shared_fwd(*tensors[:5], *rest)
    within(want[0], o, bo, "out")
    within(got[0], o, bo, "out")
    grads, bounds = O.attn_shared_bwd(*tensors[:5], *rest, want[0], want[1], tensors[5])
    for name, g, w, x, b in zip(NAMES, got[2:], want[2:], grads, bounds):
        within(w, x, b, name)
        within(g, x, 3 * b, name)  # from another rounding of out
    heads_first = [x.transpose(0, 1).contiguous().transpose(0, 1) for x in tensors]
    assert heads_first[0].stride() == (d, n * d, 1)
    o2 = run(*heads_first)
    for name, g, x, b in zip(NAMES, o2[2:], grads, bounds):
        within(g, x, 3 * b, name)
    within(o2[0], o, bo, "out")


def test_outputs_into_views_and_rows_behind_the_last_request():
    c, h, hq, hk, d = [30, 140], [200, 70], 4, 2, 64
    n, m = sum(c), sum(h)
    x = rand(n + 9, hq + 2 * hk, d, dtype=BF16, seed=1)
    y = rand(m + 5, 2 * hk, d, dtype=BF16, seed=2)
    q, k, v, kh, vh = x[:, :hq], x[:, hq:hq + hk], x[:, hq + hk:], y[:, :hk], y[:, hk:]
    for tokens in (1, 3):
        first = candidates(c + [9], tokens)
        rest = offsets(c), first, offsets(h), BIG, 0, 0.125
        dx, dy = torch.full_like(x, 7), torch.full_like(y, 7)
        out, lse = fwd(q, k, v, kh, vh, *rest)
        assert (out[n:] == 7).all() and (lse[:, n:] == 7).all()
        dout = rand(n + 9, hq, d, dtype=BF16, seed=3)
        nb = dense.attn_shared_bwd_workspace_bytes(n + 9, 2, m + 5, hq, hk, d)
        dense.attn_shared_bwd(q, k, v, kh, vh, *rest, out, lse, dout, dx[:, :hq], dx[:, hq:hq + hk], dx[:, hq + hk:],
                              dy[:, :hk], dy[:, hk:], workspace(nb)[:nb])
        assert (dx[n:] == 7).all() and (dy[m:] == 7).all()
        cut = q[:n], k[:n], v[:n], kh[:m], vh[:m]
        rest = rest[0], None if first is None else first[:n], *rest[2:]
        o, l, bo, bl = O.attn_shared_fwd(*cut, *rest)
        within(out[:n], o, bo, "out")
        want, bound = O.attn_shared_bwd(*cut, *rest, out[:n], lse[:, :n], dout[:n])
        got = dx[:n, :hq], dx[:n, hq:hq + hk], dx[:n, hq + hk:], dy[:m, :hk], dy[:m, hk:]
        for name, g, w, b in zip(NAMES, got, want, bound):
            within(g, w, b, name)


def test_shared_out_requests_with_rows_behind_the_last():
    """Keys of one request shared out over workgroups, in both shapes, and tokens that no request has."""
    for c, pad in ((20, 3), (600, 40)):
        q, k, v, kh, vh = inputs([c + pad], [9000], 4, 2, 64, F16)
        off, hoff = offsets([c]), offsets([9000])
        assert dense.attn_shared_fwd_workspace_bytes(c + pad, 1, 9000, 4, 2, 64) > 0
        out, lse = fwd(q, k, v, kh, vh, off, None, hoff, BIG, 0, 0.125)
        assert (out[c:] == 7).all() and (lse[:, c:] == 7).all()
        o, l, bo, bl = O.attn_shared_fwd(q[:c], k[:c], v[:c], kh, vh, off, None, hoff, BIG, 0, 0.125)
        within(out[:c], o, bo, "out")
        within(lse[:, :c], l, bl, "lse")


def test_empty_sizes():
    q, k, v, kh, vh = inputs([4], [6], 2, 1, 16, F16)
    none, zero = q[:0], offsets([])
    assert dense.attn_shared_fwd(q[:0], k[:0], v[:0], kh, vh, offsets([0]), None, offsets([6]), BIG, 0, 1.0, none) is None
    assert dense.attn_shared_fwd(q[:0], k[:0], v[:0], kh[:0], vh[:0], zero, None, zero, BIG, 0, 1.0, none) is None
    # no tokens: the history's gradients are zeros
    got = bwd(q[:0], k[:0], v[:0], kh, vh, offsets([0, 0]), None, offsets([4, 2]), BIG, 0, 1.0, none,
              torch.empty(2, 0, device="cuda"), none)
    assert (got[3] == 0).all() and (got[4] == 0).all()
    # no history, and a cache without room
    out, _ = fwd(q, k, v, kh[:0], vh[:0], offsets([4]), None, offsets([0]), BIG, 0, 1.0)
    assert torch.equal(out, v.expand(-1, 2, -1))
    cache = torch.empty(1, 0, 1, 16, dtype=F16, device="cuda")
    lens = torch.tensor([5], dtype=torch.int32, device="cuda")
    got = torch.full_like(out, 7)
    dense.attn_shared_cache(q, k, v, cache, cache, offsets([4]), None, lens, BIG, 0, 1.0, got)
    assert torch.equal(got, out)
    codes, exp = torch.empty(1, 0, 1, 16, dtype=U8, device="cuda"), torch.empty(1, 1, 0, dtype=U8, device="cuda")
    dense.attn_window_decode_q8(q[:1], codes, exp, codes, exp, lens, BIG, 0, 1.0, got[:1], None)
    assert (got[0] == 0).all()


def test_caches_past_32_bits():
    """The last request's keys lie past 2^32 bytes, or 2^31 elements, from the cache's start."""
    users, cap, hk, d, m = 3, 200_000, 64, 128, 600
    codes = [torch.zeros(users, cap, hk, d, dtype=U8, device="cuda") for _ in range(2)]
    exps = [torch.zeros(users, hk, cap, dtype=U8, device="cuda") for _ in range(2)]
    assert codes[0].numel() > 2 ** 32
    k, v = rand(m, hk, d, dtype=F16, seed=1), rand(m, hk, d, dtype=F16, seed=2)
    start = torch.tensor([0, 0, cap - m], dtype=torch.int32, device="cuda")
    dense.cache_q8_write(k, v, offsets([0, 0, m]), start, codes[0], exps[0], codes[1], exps[1])
    kv, vv = (O.values_of(*O.quantise(x)).to(F16) for x in (k, v))
    lens = torch.tensor([0, 5, cap], dtype=torch.int32, device="cuda")
    for c in ([0, 0, 9], [0, 2, 200]):
        n = sum(c)
        q, ko, vo = rand(n, hk, d, dtype=F16, seed=3), rand(n, hk, d, dtype=F16, seed=4), rand(n, hk, d, dtype=F16, seed=5)
        out = torch.full_like(q, 7)
        nb = dense.attn_shared_cache_workspace_bytes(n, users, cap, hk, hk, d)
        ws = torch.empty(nb, dtype=U8, device="cuda")
        dense.attn_shared_cache_q8(q, ko, vo, codes[0], exps[0], codes[1], exps[1], offsets(c), None, lens, 500, 0, 0.1, out,
                                   ws)
        a = c[1]
        o, _, bo, _ = O.attn_shared_fwd(*(x[a:, :4] for x in (q, ko, vo)), kv[:, :4], vv[:, :4], offsets(c[2:]), None,
                                        offsets([m]), 500, 0, 0.1)
        within(out[a:, :4], o, bo, "out")
    q, out = rand(users, hk, d, dtype=F16, seed=6), torch.full((users, hk, d), 7, dtype=F16, device="cuda")
    nb = dense.attn_window_decode_q8_workspace_bytes(users, cap, hk, hk, d, 500, 0)
    dense.attn_window_decode_q8(q, codes[0], exps[0], codes[1], exps[1], lens, 500, 0, 0.1, out, workspace(nb)[:nb] if nb else None)
    o, bo = O.attn_decode(q[2:, :4], kv[None, :, :4], vv[None, :, :4], torch.tensor([m], device="cuda"), 500, 0, 0.1)
    within(out[2:, :4], o, bo, "newest")
    assert (out[0] == 0).all()


# ---------------------------------------------------------------------------------- use
def serve_and_train(c, h, dtype):
    """A step of every call, into buffers of its own; what it reads may be changed from outside."""
    hq, hk, d, cap = 4, 2, 64, max(h) + 4
    t = dict(zip(("q", "k", "v", "kh", "vh"), (x.contiguous() for x in inputs(c, h, hq, hk, d, dtype))))
    n, m = sum(c), sum(h)
    t.update(off=offsets(c), hoff=offsets(h), first=candidates(c, 3), lens=torch.tensor(h, dtype=torch.int32, device="cuda"),
             dout=rand(n, hq, d, dtype=dtype, seed=8), q1=rand(len(h), hq, d, dtype=dtype, seed=9))
    cache = [torch.zeros(len(h), cap, hk, d, dtype=U8, device="cuda") if x % 2 == 0 else
             torch.zeros(len(h), hk, cap, dtype=U8, device="cuda") for x in range(4)]
    new = lambda *s: torch.empty(*s, dtype=dtype, device="cuda")  # noqa: E731
    out, served, newest, back = new(n, hq, d), new(n, hq, d), new(len(h), hq, d), [new(m, hk, d), new(m, hk, d)]
    lse, grads = torch.empty(hq, n, device="cuda"), [torch.empty_like(t[x]) for x in ("q", "k", "v", "kh", "vh")]
    b = lambda nb: torch.empty(max(nb, 16), dtype=U8, device="cuda")  # noqa: E731
    ws = [b(dense.attn_shared_fwd_workspace_bytes(n, len(h), m, hq, hk, d)),
          b(dense.attn_shared_bwd_workspace_bytes(n, len(h), m, hq, hk, d)),
          b(dense.attn_shared_cache_workspace_bytes(n, len(h), cap, hq, hk, d)),
          b(dense.attn_window_decode_q8_workspace_bytes(len(h), cap, hq, hk, d, 300, 2))]

    def step(ws=ws):
        a = t["q"], t["k"], t["v"]
        for first in (t["first"], None):
            dense.attn_shared_fwd(*a, t["kh"], t["vh"], t["off"], first, t["hoff"], 300, 2, 0.125, out, lse, ws[0])
            dense.attn_shared_bwd(*a, t["kh"], t["vh"], t["off"], first, t["hoff"], 300, 2, 0.125, out, lse, t["dout"],
                                  *grads, ws[1])
        dense.cache_q8_write(t["kh"], t["vh"], t["hoff"], None, *cache)
        dense.cache_q8_read(*cache, t["hoff"], None, *back)
        dense.attn_shared_cache_q8(*a, *cache, t["off"], t["first"], t["lens"], 300, 2, 0.125, served, ws[2])
        dense.attn_window_decode_q8(t["q1"], *cache, t["lens"], 300, 2, 0.125, newest, ws[3])
        return [x.clone() for x in (out, lse, *grads, *back, served, newest)]
    return t, step


@pytest.mark.parametrize("c,h", [([20, 3], [700, 90]), ([300, 170], [2500, 900]), ([3] * 80, [30] * 80)])
def test_on_a_side_stream_and_in_a_graph(c, h):
    t, step = serve_and_train(c, h, BF16)
    want = step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = step()
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for turn in range(3):
        for s, name in enumerate(("q", "kh", "vh", "dout")):
            t[name].copy_(rand(*t[name].shape, dtype=BF16, seed=20 + 10 * turn + s))
        graph.replay()
        torch.cuda.synchronize()
        replayed = [x.clone() for x in got]
        assert all(torch.equal(a, b) for a, b in zip(replayed, step()))


def test_two_graphs_that_share_workspaces():
    """What a workspace holds from one call means nothing to the next."""
    (t1, step1), (t2, step2) = serve_and_train([200], [5000], F16), serve_and_train([180], [5100], F16)
    hq, hk, d = 4, 2, 64
    sizes = [max(f(n, 1, m, hq, hk, d) for n, m in ((200, 5000), (180, 5100))) for f in (
        dense.attn_shared_fwd_workspace_bytes, dense.attn_shared_bwd_workspace_bytes, dense.attn_shared_cache_workspace_bytes)]
    sizes[2] = max(dense.attn_shared_cache_workspace_bytes(n, 1, m + 4, hq, hk, d) for n, m in ((200, 5000), (180, 5100)))
    sizes.append(max(dense.attn_window_decode_q8_workspace_bytes(1, m + 4, hq, hk, d, 300, 2) for m in (5000, 5100)))
    one = torch.full((max(sizes + [16]),), 0xFF, dtype=U8, device="cuda")
    ws = [one] * 4
    want = step1(), step2()
    graphs, got = [torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()], []
    for g, step in zip(graphs, (step1, step2)):
        with torch.cuda.graph(g):
            got.append(step(ws))
    for which in (0, 1, 1, 0, 1):
        graphs[which].replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got[which], want[which]))


def test_offsets_lengths_and_first_are_checked_on_request(monkeypatch):
    q, k, v, kh, vh = inputs([20], [9], 1, 1, 32, F16)
    out = torch.empty_like(q)
    i = lambda o: None if o is None else torch.tensor(o, dtype=torch.int32, device="cuda")  # noqa: E731
    good = list(range(0, 5)) + [5] * 5 + [10, 10] + list(range(12, 20))
    run = lambda o, hist, first: dense.attn_shared_fwd(q, k, v, kh, vh, i(o), i(first), i(hist), 4, 0, 1.0, out)  # noqa: E731
    monkeypatch.setenv("EMB_VALIDATE", "1")
    run([0, 5, 20], [0, 9, 9], good)
    run([0, 5, 18], [0, 2, 3], good)  # fewer than there are rows for
    for bad in ([1, 5, 20], [0, 6, 5], [0, 5, 21], [0, -1, 20]):
        with pytest.raises(emb.EmbError, match="offsets"):
            run(bad, [0, 9, 9], None)
    for bad in ([1, 5, 9], [0, 6, 5], [0, 5, 10]):
        with pytest.raises(emb.EmbError, match="offsets"):
            run([0, 5, 20], bad, None)
    for at, x in ((0, 1), (5, 4), (7, 6), (11, 11 - 2), (19, 20), (3, -1)):
        bad = list(good)
        bad[at] = x
        with pytest.raises(emb.EmbError, match="first"):
            run([0, 5, 20], [0, 9, 9], bad)
    cache = kh[None]
    with pytest.raises(emb.EmbError, match="length"):
        dense.attn_shared_cache(q, k, v, cache, cache, i([0, 20]), None, i([10]), 4, 0, 1.0, out)
    codes, exp = torch.zeros(1, 9, 1, 32, dtype=U8, device="cuda"), torch.zeros(1, 1, 9, dtype=U8, device="cuda")
    with pytest.raises(emb.EmbError, match="length"):
        dense.attn_window_decode_q8(q[:1], codes, exp, codes, exp, i([-1]), 4, 0, 1.0, out[:1], None)
    with pytest.raises(emb.EmbError, match="offsets"):
        dense.cache_q8_write(kh, vh, i([0, 10]), None, codes, exp, codes.clone(), exp.clone())


def test_malformed_first_stays_within_the_request():
    """What `first` may hold besides candidates: a token sees itself whatever stands there, and nothing of another
    request."""
    c, h = [40, 200], [30, 100]
    q, k, v, kh, vh = inputs(c, h, 2, 2, 32, F16)
    v2 = v.clone()
    v2[:40] = float("nan")  # of the first request
    for x in (-(2 ** 31), -1, 0, 2 ** 31 - 1):
        first = torch.full((240,), x, dtype=torch.int32, device="cuda")
        a, _ = fwd(q, k, v, kh, vh, offsets(c), first, offsets(h), BIG, 0, 0.2)
        b, _ = fwd(q, k, v2, kh, vh, offsets(c), first, offsets(h), BIG, 0, 0.2)
        assert a.isfinite().all() and torch.equal(a[40:], b[40:])


@pytest.mark.parametrize("name", ["attn_shared_fwd", "attn_shared_bwd", "attn_shared_cache", "attn_shared_cache_q8",
                                  "attn_window_decode_q8", "cache_q8_write", "cache_q8_read"])
def test_tensors_of_another_device_are_refused(name, monkeypatch):
    q, k, v, kh, vh = inputs([4], [6], 2, 1, 16, F16)
    off, hoff, lens = offsets([4]), offsets([6]), torch.tensor([6], dtype=torch.int32, device="cuda")
    out, lse, ws = torch.empty_like(q), torch.empty(2, 4, device="cuda"), torch.empty(1 << 16, dtype=U8, device="cuda")
    c = [torch.zeros(1, 6, 1, 16, dtype=U8, device="cuda") if x % 2 == 0 else torch.zeros(1, 1, 6, dtype=U8, device="cuda")
         for x in range(4)]
    g = [torch.empty_like(x) for x in (q, k, v, kh, vh)]
    calls = {
        "attn_shared_fwd": lambda: dense.attn_shared_fwd(q, k, v, kh, vh, off, None, hoff, 4, 0, 1.0, out, lse, ws),
        "attn_shared_bwd": lambda: dense.attn_shared_bwd(q, k, v, kh, vh, off, None, hoff, 4, 0, 1.0, out, lse, out, *g, ws),
        "attn_shared_cache": lambda: dense.attn_shared_cache(q, k, v, kh[None], vh[None], off, None, lens, 4, 0, 1.0, out, ws),
        "attn_shared_cache_q8": lambda: dense.attn_shared_cache_q8(q, k, v, *c, off, None, lens, 4, 0, 1.0, out, ws),
        "attn_window_decode_q8": lambda: dense.attn_window_decode_q8(q[:1], *c, lens, 4, 0, 1.0, out[:1], ws),
        "cache_q8_write": lambda: dense.cache_q8_write(kh, vh, hoff, None, *c),
        "cache_q8_read": lambda: dense.cache_q8_read(*c, hoff, None, torch.empty_like(kh), torch.empty_like(vh)),
    }
    calls[name]()
    torch.cuda.synchronize()
    monkeypatch.setattr(dense, "_device", lambda: 1)
    monkeypatch.setattr(dense, "_stream", lambda *a: pytest.fail("a tensor of another device was taken"))
    with pytest.raises(TypeError, match="current device"):
        calls[name]()


@pytest.mark.parametrize("n", [22, 30, 44, 64, 65])
def test_hundreds_of_workgroups_of_unlike_work(n):
    """Between one and two workgroups a unit of the GPU and past that, requests sorted by their work and not."""
    gen = torch.Generator().manual_seed(n)
    c = torch.randint(100, 160, (n,), generator=gen).tolist()
    h = torch.randint(0, 900, (n,), generator=gen).tolist()
    for tokens in (1, 3):
        args = *inputs(c, h, 8, 4, 32, BF16), offsets(c), candidates(c, tokens), offsets(h), 600, 1, 0.2
        out, lse = fwd(*args)
        o, l, bo, bl = O.attn_shared_fwd(*args)
        within(out, o, bo, "out")
        within(lse, l, bl, "lse")
        dout = rand(*out.shape, dtype=BF16, seed=5)
        want, bound = O.attn_shared_bwd(*args, out, lse, dout)
        for name, g, w, b in zip(NAMES, bwd(*args, out, lse, dout), want, bound):
            within(g, w, b, name)


def test_two_calls_at_once():
    """Steps on two streams, each with workspaces of its own."""
    steps = [serve_and_train([200, 30], [5000, 80], F16)[1], serve_and_train([3] * 70, [90] * 70, BF16)[1]]
    want = [step() for step in steps]
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in range(2)], []
    for _ in range(4):
        for stream, step in zip(streams, steps):
            with torch.cuda.stream(stream):
                got.append(step())
    torch.cuda.synchronize()
    for i, g in enumerate(got):
        assert all(torch.equal(a, b) for a, b in zip(g, want[i % 2]))


# c, h, dim, whether keys are shared out over workgroups: 32 rows a workgroup and 128, joins of each kind
@pytest.mark.parametrize("c,h,d,shared", [([5, 3], [40, 30], 32, False), ([20], [9000], 64, True), ([400, 200], [90, 60], 64, False),
                                          ([600], [9000], 64, True), ([3000], [9000], 64, True), ([300, 200], [2000, 700], 64, True)])
@pytest.mark.parametrize("tokens", [1, 3])
def test_rows_whose_scores_are_all_minus_infinity(c, h, d, shared, tokens):
    """Their softmax is NaN, and so is out, however many workgroups share the keys; lse is minus infinity."""
    hq, hk, n = 4, 2, sum(c)
    q, k, v, kh, vh = (x.contiguous() for x in inputs(c, h, hq, hk, d, F16))
    k[..., 0] = kh[..., 0] = 1
    gone = torch.zeros(n, hq, dtype=torch.bool, device="cuda")
    gone[n - 2, 1:3] = gone[0, 0] = True
    kept = q.clone()
    q[..., 0].masked_fill_(gone, -float("inf"))
    off, hoff, first, scale = offsets(c), offsets(h), candidates(c, tokens), 0.2
    assert (dense.attn_shared_fwd_workspace_bytes(n, len(c), sum(h), hq, hk, d) > 0) == shared
    o, l, bo, bl = O.attn_shared_fwd(kept, k, v, kh, vh, off, first, hoff, BIG, 0, scale)

    def check(out, o, bo, gone, what):
        assert out[gone].isnan().all(), what
        within(out[~gone], o[~gone], bo[~gone], what)
    out, lse = fwd(q, k, v, kh, vh, off, first, hoff, BIG, 0, scale)
    check(out, o, bo, gone, "out")
    assert (lse.T[gone] == -float("inf")).all()
    within(lse.T[~gone], l.T[~gone], bl.T[~gone], "lse")
    cap, lens = max(h) + 3, torch.tensor(h, dtype=torch.int32, device="cuda")
    kc, vc, got = cached(kh, h, cap), cached(vh, h, cap), torch.full_like(q, 7)
    nb = dense.attn_shared_cache_workspace_bytes(n, len(c), cap, hq, hk, d)
    dense.attn_shared_cache(q, k, v, kc, vc, off, first, lens, BIG, 0, scale, got, workspace(nb)[:nb])
    check(got, o, bo, gone, "out from caches")
    # the newest event against 8 bits, of which a 1 is one
    (kq, ke, kv), (vq, ve, vv) = in_8_bits(kc.nan_to_num(0)), in_8_bits(vc.nan_to_num(0))
    q1, gone1 = kept[:len(c)].clone(), torch.zeros(len(c), hq, dtype=torch.bool, device="cuda")
    gone1[0, 3] = True
    o, bo = O.attn_decode(q1, kv, vv, lens, BIG, 0, scale)
    q1[..., 0].masked_fill_(gone1, -float("inf"))
    nb = dense.attn_window_decode_q8_workspace_bytes(len(c), cap, hq, hk, d, BIG, 0)
    got = torch.full_like(q1, 7)
    dense.attn_window_decode_q8(q1, kq, ke, vq, ve, lens, BIG, 0, scale, got, workspace(nb)[:nb] if nb else None)
    check(got, o, bo, gone1, "newest")


@pytest.mark.parametrize("c,h", [([12, 8], [90, 130]), ([160, 140], [90, 230])])
@pytest.mark.parametrize("d,hq,dtype", [(32, 2, BF16), (128, 4, BF16), (64, 4, F16)])
def test_gradients_beside_an_own_score_of_minus_infinity(d, hq, dtype, c, h):
    """A key of a candidate's own, minus infinity in one column, weighs nothing where its score is that: gradients are as
    without it, but for that column of dq, which is 0 times infinity."""
    window, sinks, scale, hk, n = 100, 2, 0.2, 2, sum(c)
    q, k, v, kh, vh = (x.contiguous() for x in inputs(c, h, hq, hk, d, dtype))
    q[..., 5] = 1
    off, hoff, first = offsets(c), offsets(h), candidates(c, 4)
    gone = torch.zeros(n, dtype=torch.bool, device="cuda")
    gone[torch.tensor([2, c[0] + 6, n - 3], device="cuda")] = True
    k[gone, :, 5] = -float("inf")
    args = q, k, v, kh, vh, off, first, hoff, window, sinks, scale
    out, lse = fwd(*args)
    assert out.isfinite().all() and lse.isfinite().all()
    dout = rand(n, hq, d, dtype=dtype, seed=7)
    got = bwd(*args, out, lse, dout)
    u, tiny, g = O.U[dtype], O.TINY[dtype], hq // hk
    want, bound = ([torch.zeros(x.shape, dtype=torch.float64, device="cuda") for x in (q, k, v, kh, vh)] for _ in range(2))
    odd = torch.zeros(n, dtype=torch.bool, device="cuda")
    for a, z, b, y in zip(off.tolist()[:-1], off.tolist()[1:], hoff.tolist()[:-1], hoff.tolist()[1:]):
        see = O.shared_sees(y - b, first[a:z].long() - a, window, sinks, "cuda")
        odd[a:z] = (see[:, y - b:] & gone[a:z]).any(1)
        see = see & ~torch.cat([torch.zeros(y - b, dtype=torch.bool, device="cuda"), gone[a:z]])
        for i in range(hq):
            x = i // g
            kk = torch.cat([kh[b:y, x], k[a:z, x]]).double().nan_to_num(0, 0, 0)
            vv, qq, do, oo = torch.cat([vh[b:y, x], v[a:z, x]]).double(), q[a:z, i].double(), dout[a:z, i].double(), out[a:z, i].double()
            s, rel = O._head(qq, kk, scale)
            rel += (8 * lse[i, a:z].abs().max().item() + len(kk)) * O.F32
            p = torch.exp(s - lse[i, a:z].double()[:, None]).masked_fill(~see, 0.0)
            delta, both = (do * oo).sum(1, keepdim=True), (do * oo).abs().sum(1, keepdim=True)
            ds = p * (do @ vv.T - delta)
            # as the oracle's: dp and delta are fp32 sums, p and ds are rounded to 16 bits
            e = p * (d + 8) * O.F32 * (do.abs() @ vv.abs().T + both) + ((u + 2 * rel) * ds.abs() + tiny) * see * (1 + u)
            ep = ((u + 2 * rel) * p + tiny) * see
            want[0][a:z, i], bound[0][a:z, i] = ds @ kk * scale, e @ kk.abs() * scale
            for to, y_ in ((want, (ds.T @ qq * scale, p.T @ do)), (bound, (e.T @ qq.abs() * scale, ep.T @ do.abs()))):
                for own, hist, t in ((1, 3, y_[0]), (2, 4, y_[1])):
                    to[hist][b:y, x] += t[:y - b]
                    to[own][a:z, x] += t[y - b:]
    assert got[0][odd][..., 5].isnan().all() and odd.any()
    got[0][..., 5].masked_fill_(odd[:, None], 0)
    want[0][..., 5].masked_fill_(odd[:, None], 0)
    for name, x, w, b in zip(NAMES, got, want, bound):
        within(x, w, b * (1 + u) + u * w.abs() + tiny, name)


@pytest.mark.parametrize("grow", [2.0 ** -10, 2.0 ** -14, 2.0 ** -18])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("c,tokens", [([20], 1), ([20], 3), ([300], 1), ([300], 50)])
def test_small_gradients_of_scores_in_fp16(c, tokens, d, grow):
    """Of thousands of events and a small dout they lie at 2^-19, 2^-23 and 2^-27, where fp16 has few bits left or none, and
    results where it has more."""
    h = [4000]
    q, k, v, kh, vh = inputs(c, h, 2, 1, d, F16)
    q, k, kh, scale = q * 2.0 ** -8, k * 2.0 ** -8, kh * 2.0 ** -8, 2.0 ** 20 / d
    args = q, k, v, kh, vh, offsets(c), candidates(c, tokens), offsets(h), BIG, 0, scale
    out, lse = fwd(*args)
    dout = rand(*out.shape, dtype=F16, seed=5) * grow
    # Gradients are linear in dout, and the bounds of those of one `more` times as large allow for 2^-25 lost of a score's
    # gradient.  Standing at 2^12, one loses 2^-37; where a row's largest, or a key's, is below 2^-6 there all are brought
    # to a largest of 2^8, and lose 2^-33 of one below 2^-18.
    more = 2.0 ** 12
    want, bound = O.attn_shared_bwd(*args, out, lse, dout.double() * more)
    got = bwd(*args, out, lse, dout)
    for i, (name, g, w, b) in enumerate(zip(NAMES, got, want, bound)):
        w, b = w / more, b / more
        if i == 0 or i == 3 and grow > 2.0 ** -18:
            assert w.abs().max() > 2.0 ** -14, name  # past fp16's lower end there is nothing to see
        within(g, w, b + O.TINY[F16], name)


@pytest.mark.parametrize("d", [32, 64, 128])
@pytest.mark.parametrize("c,tokens", [([300], 1), ([40, 30], 3)])
def test_small_probabilities_in_fp16(c, tokens, d):
    """60000 events of equal weight: each probability is rounded the same way, and a sum of them is off by as much."""
    h = [60000] + [40000] * (len(c) - 1)
    q, k, v, kh, vh = inputs(c, h, 1, 1, d, F16)
    q = torch.zeros_like(q)
    args = q, k, v, kh, vh, offsets(c), candidates(c, tokens), offsets(h), BIG, 0, 0.2
    out, lse = fwd(*args)
    dout = torch.full_like(out, 64)
    got = bwd(*args, out, lse, dout)
    for own in (2, 4):
        for s, (n, m) in enumerate(zip(c, h)):
            if own == 4:
                total, at = n / (m + 1), slice(sum(h[:s]), sum(h[:s + 1]))
                if tokens > 1:  # a candidate's tokens see one, two, ... of its own
                    first = candidates(c, tokens)[sum(c[:s]):sum(c[:s + 1])] - sum(c[:s])
                    total = (1 / (m + 1 + torch.arange(n, device="cuda") - first).double()).sum().item()
                # a rounding of each probability, of the result, and fp32's of the exponent, at most about 16 + 15, and sums
                rel = 2.0 ** -11 * 2 + (2 * 32 + 64 + n) * O.F32
                err = (got[4][at].double() / 64 - total).abs().max().item()
                assert err <= rel * total, (d, err / total)
            elif tokens == 1:
                err = (got[2][sum(c[:s]):sum(c[:s + 1])].double() / 64 - 1 / (m + 1)).abs().max().item()
                assert err <= (2.0 ** -11 + 256 * O.F32) / (m + 1), (d, err * (m + 1))


# requests whose keys are shared out, more of them than are sorted: by 128 rows a workgroup, and by 32
@pytest.mark.parametrize("c,h,hq,hk,d,tokens", [(140, 6000, 2, 1, 64, 1), (140, 6000, 1, 1, 128, 5), (3, 4000, 2, 1, 64, 1),
                                                (4, 3000, 3, 1, 32, 2)])
@pytest.mark.parametrize("n", [65, 100])
def test_many_requests_whose_keys_are_shared_out(n, c, h, hq, hk, d, tokens):
    gen = torch.Generator().manual_seed(n + c)
    c, h = (torch.randint(0, x + 1, (n,), generator=gen).tolist() for x in (c, h))
    c[0], c[-1], h[1], window, sinks, scale = 0, 0, 0, 2500, 3, 1.3 * d ** -0.5
    q, k, v, kh, vh = inputs([sum(c) + 5], h, hq, hk, d, BF16)  # tokens of no request behind the last
    off, hoff, first = offsets(c), offsets(h), candidates(c + [5], tokens)
    m = sum(c)
    for f in (dense.attn_shared_fwd_workspace_bytes, dense.attn_shared_cache_workspace_bytes):
        assert f(m + 5, n, sum(h) if f is dense.attn_shared_fwd_workspace_bytes else max(h), hq, hk, d) > 0
    rest = off, first, hoff, window, sinks, scale
    out, lse = fwd(q, k, v, kh, vh, *rest)
    assert (out[m:] == 7).all() and (lse[:, m:] == 7).all()
    cut = q[:m], k[:m], v[:m], kh, vh, off, None if first is None else first[:m], *rest[2:]
    o, l, bo, bl = O.attn_shared_fwd(*cut)
    within(out[:m], o, bo, "out")
    within(lse[:, :m], l, bl, "lse")
    dout = rand(m + 5, hq, d, dtype=BF16, seed=9)
    want, bound = O.attn_shared_bwd(*cut, out[:m], lse[:, :m], dout[:m])
    for name, g, w, b in zip(NAMES, bwd(q, k, v, kh, vh, *rest, out, lse, dout), want, bound):
        assert (g[w.shape[0]:] == 7).all()
        within(g[:w.shape[0]], w, b, name)
    # against caches, in 16 bits and in 8
    cap, lens = max(h), torch.tensor(h, dtype=torch.int32, device="cuda")
    nb, got = dense.attn_shared_cache_workspace_bytes(m + 5, n, cap, hq, hk, d), torch.full_like(out, 7)
    ws = workspace(nb)
    dense.attn_shared_cache(q, k, v, cached(kh, h, cap), cached(vh, h, cap), off, first, lens, window, sinks, scale, got, ws[:nb])
    assert (ws[nb:] == 0xFF).all() and (got[m:] == 7).all()
    within(got[:m], o, bo, "out from caches")
    cache = [torch.full((n, cap, hk, d) if x % 2 == 0 else (n, hk, cap), 0x7F, dtype=U8, device="cuda") for x in range(4)]
    dense.cache_q8_write(kh, vh, hoff, None, *cache)
    kv, vv = (O.values_of(*O.quantise(x)).to(BF16) for x in (kh, vh))
    o, _, bo, _ = O.attn_shared_fwd(*cut[:3], kv, vv, *cut[5:])
    ws = workspace(nb)
    dense.attn_shared_cache_q8(q, k, v, *cache, off, first, lens, window, sinks, scale, got, ws[:nb])
    assert (ws[nb:] == 0xFF).all() and (got[m:] == 7).all()
    within(got[:m], o, bo, "out from 8 bits")


@pytest.mark.parametrize("tokens", [1, 3])
@pytest.mark.parametrize("c,pad", [(20, 3), (600, 40)])
def test_shared_out_backward_with_rows_behind_the_last(c, pad, tokens):
    q, k, v, kh, vh = inputs([c + pad], [9000], 4, 2, 64, F16)
    first = candidates([c, pad], tokens)
    rest = offsets([c]), first, offsets([9000]), BIG, 0, 0.125
    out, lse = fwd(q, k, v, kh, vh, *rest)
    dout = rand(c + pad, 4, 64, dtype=F16, seed=9)
    cut = q[:c], k[:c], v[:c], kh, vh, rest[0], None if first is None else first[:c], *rest[2:]
    want, bound = O.attn_shared_bwd(*cut, out[:c], lse[:, :c], dout[:c])
    for name, g, w, b in zip(NAMES, bwd(q, k, v, kh, vh, *rest, out, lse, dout), want, bound):
        assert (g[w.shape[0]:] == 7).all()
        within(g[:w.shape[0]], w, b, name)


@pytest.mark.parametrize("d,hq,hk", [(32, 2, 2), (64, 2, 1), (128, 4, 2)])
@pytest.mark.parametrize("c,h,tokens", [([20], [900], 1), ([20], [900], 3), ([300, 40], [700, 90], 1), ([300, 40], [700, 90], 3),
                                        ([12, 40, 0, 25], [300, 90, 7, 0], 3), ([150], [64], 50), ([150, 90], [3, 2], 3)])
@pytest.mark.parametrize("few", [False, True])
def test_score_gradients_of_many_magnitudes_in_fp16(c, h, tokens, few, d, hq, hk):
    """Tokens' douts from 2^-3 down to 2^-17, in any order, and weights from one to e^-20: large and small ones come one
    after the other for each query and each key.  few: every 32nd token's alone is small, which other tiles' rows meet
    among large ones."""
    q, k, v, kh, vh = inputs(c, h, hq, hk, d, F16)
    args = q, k, v, kh, vh, offsets(c), candidates(c, tokens), offsets(h), BIG, 0, 4 * d ** -0.5
    out, lse = fwd(*args)
    gen = torch.Generator(device="cuda").manual_seed(d + len(c))
    down = torch.randint(3, 18, (sum(c), 1, 1), generator=gen, device="cuda")
    if few:
        down = torch.where(torch.arange(sum(c), device="cuda") % 32 == 0, 17, 3)[:, None, None]
    dout = (rand(*out.shape, dtype=torch.float32, seed=5) * 0.5 ** down).half()
    # as above: standing at 2^12 at least a score's gradient loses 2^-37, while none is past 16, where they would move down
    more = 2.0 ** 12
    want, bound = O.attn_shared_bwd(*args, out, lse, dout.double() * more)
    for t, _, i, _, see, qq, kk, vv in O._requests(*args[:9], 0):
        p = torch.exp(qq @ kk.T * args[10] - lse[i, t].double()[:, None]).masked_fill(~see, 0.0)
        do = dout[t, i].double()
        assert (p * (do @ vv.T - (do * out[t, i].double()).sum(1, keepdim=True))).abs().max() < 16
    for name, g, w, b in zip(NAMES, bwd(*args, out, lse, dout), want, bound):
        within(g, w / more, b / more + O.TINY[F16], name)


@pytest.mark.parametrize("c,h", [([12, 8], [90, 130]), ([160, 140], [90, 230])])
@pytest.mark.parametrize("tokens", [1, 3])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_a_value_that_is_not_finite_shows_beside_a_score_of_minus_infinity(bad, tokens, c, h):
    """0 times it is NaN, of an own token as of an event of the history; other columns do not change."""
    q, k, v, kh, vh = (x.contiguous() for x in inputs(c, h, 2, 1, 64, F16))
    q[..., 5] = 1
    own, event = c[0] + 4, h[0] + 3
    k[own, 0, 5] = kh[event, 0, 5] = -float("inf")
    off, hoff, first = offsets(c), offsets(h), candidates(c, tokens)
    rest = off, first, hoff, BIG, 0, 0.2
    want, lse = fwd(q, k, v, kh, vh, *rest)
    assert want.isfinite().all() and lse.isfinite().all()
    rows = torch.arange(sum(c), device="cuda")
    start = rows if first is None else first.long()
    for x, at, seeing in ((v, own, (start == start[own]) & (rows >= own)), (vh, event, rows >= c[0])):
        keep = x[at, 0, 7].clone()
        x[at, 0, 7] = bad
        got, l = fwd(q, k, v, kh, vh, *rest)
        assert not got[seeing][..., 7].isfinite().any()
        got[..., 7].masked_fill_(seeing[:, None], 0)
        assert torch.equal(got, torch.where(seeing[:, None, None] & (torch.arange(64, device="cuda") == 7), 0, want))
        assert torch.equal(l, lse)
        x[at, 0, 7] = keep

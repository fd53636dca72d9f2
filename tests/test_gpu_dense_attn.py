"""Windowed attention with sinks against the 64-bit oracle: forward, backward and one new event, at
lengths, head layouts, widths and strides where the kernels' tiles end; within bounds that count the
16-bit roundings of results, probabilities and their gradients."""
import pytest

torch = pytest.importorskip("torch")

from ad_recommendation_amd import dense, emb  # noqa: E402
from oracle import dense_oracle as O  # noqa: E402

pytestmark = pytest.mark.gpu
F16, BF16 = torch.float16, torch.bfloat16
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


def bwd(q, k, v, off, window, sinks, scale, out, lse, dout):
    n, hq, d = q.shape
    dq, dk, dv = torch.full_like(out, 7), torch.full(k.shape, 7, dtype=q.dtype, device="cuda"), None
    dv = torch.full_like(dk, 7)
    nb = dense.attn_window_bwd_workspace_bytes(n, off.numel() - 1, hq, k.shape[1], d, sinks)
    ws = torch.full((nb + 64,), 0xFF, dtype=torch.uint8, device="cuda")  # NaN where it is not written
    dense.attn_window_bwd(q, k, v, off, window, sinks, scale, out, lse, dout, dq, dk, dv, ws[:nb])
    assert (ws[nb:] == 0xFF).all()
    return dq, dk, dv


# lens, q heads, kv heads, dim, window, sinks
SHAPES = [
    ([1], 1, 1, 8, 1, 0),
    ([0, 1, 0, 2, 0], 2, 1, 16, 1, 1),
    ([31, 32, 33, 0, 64, 65, 1], 4, 4, 32, 5, 3),
    ([127, 128, 129], 4, 2, 64, 64, 4),
    ([200, 3, 0, 257], 6, 2, 40, 63, 32),
    ([300], 8, 1, 128, 32, 32),
    ([1000, 17, 500], 4, 2, 64, 100, 4),
    ([1500], 2, 1, 80, 1, 7),
    ([1400, 700], 2, 2, 128, 129, 1),
    ([400, 129, 64], 2, 2, 24, BIG, 5),
    ([513, 640], 3, 1, 104, 512, 0),
    ([700, 300], 4, 2, 32, 300, 3),
    ([1500, 0, 220], 4, 2, 64, 200, 7),
    ([650], 2, 1, 48, 200, 32),
    ([900, 100], 2, 2, 32, 150, 32),
    ([0, 0], 2, 2, 32, 4, 2),
    ([5] * 70 + [0] * 70 + [40] * 70, 2, 1, 32, 7, 2),
]


@pytest.mark.parametrize("dtype", [F16, BF16], ids=str)
@pytest.mark.parametrize("lens,hq,hk,d,window,sinks", SHAPES)
def test_forward_and_backward(lens, hq, hk, d, window, sinks, dtype):
    off = offsets(lens)
    n = int(off[-1])
    print(f"[attn] {lens[:8]} heads {hq}/{hk} dim {d} window {window} sinks {sinks} {dtype}", flush=True)
    x = rand(n, hq + 2 * hk, d, dtype=dtype, seed=n + d)
    q, k, v = x[:, :hq], x[:, hq:hq + hk], x[:, hq + hk:]
    scale = 1.3 * d ** -0.5
    out = torch.full((n, hq, d), 7, dtype=dtype, device="cuda")
    lse = torch.full((hq, n), 7.0, device="cuda")
    dense.attn_window_fwd(q, k, v, off, window, sinks, scale, out, lse)
    o, l, bo, bl = O.attn_fwd(q, k, v, off, window, sinks, scale)
    within(out, o, bo, "out")
    within(lse, l, bl, "lse")
    dout = rand(n, hq, d, dtype=dtype, seed=n + d + 1)
    got = bwd(q, k, v, off, window, sinks, scale, out, lse, dout)
    want = O.attn_bwd(q, k, v, off, window, sinks, scale, out, lse, dout)
    for name, g, w, b in zip(("dq", "dk", "dv"), got, want[:3], want[3:]):
        within(g, w, b, name)
    # the same bits again
    out2, lse2 = torch.empty_like(out), torch.empty_like(lse)
    dense.attn_window_fwd(q, k, v, off, window, sinks, scale, out2, lse2)
    assert torch.equal(out, out2) and torch.equal(lse, lse2)
    for g, again in zip(got, bwd(q, k, v, off, window, sinks, scale, out, lse, dout)):
        assert torch.equal(g, again)


@pytest.mark.parametrize("d,window", [(32, 40), (64, BIG), (128, 2)])
def test_tokens_far_apart(d, window):
    """Strides over which a tile of rows spans more than 2^31 bytes, and orders of heads and tokens."""
    n = 300
    off = offsets([n])
    big = torch.empty(n, (1 << 23) + 8, dtype=F16, device="cuda")
    q, k, v, dout = (big[:, 1024 * x:1024 * x + 2 * d].unflatten(1, (2, d)) for x in range(4))
    dense_of = [rand(n, 2, d, dtype=F16, seed=x) for x in range(4)]
    for t, x in zip((q, k, v, dout), dense_of):
        t.copy_(x)

    def run(q, k, v, dout):
        out, lse = torch.empty(n, 2, d, dtype=F16, device="cuda"), torch.empty(2, n, device="cuda")
        dense.attn_window_fwd(q, k, v, off, window, 3, 0.1, out, lse)
        return [out, lse, *bwd(q, k, v, off, window, 3, 0.1, out, lse, dout)]
    got, want = run(q, k, v, dout), run(*dense_of)
    del big, q, k, v, dout
    o, l, bo, bl = O.attn_fwd(*dense_of[:3], off, window, 3, 0.1)
    within(got[0], o, bo, "out")
    grads = O.attn_bwd(*dense_of[:3], off, window, 3, 0.1, want[0], want[1], dense_of[3])
    for g, w, b in zip(got[2:], grads[:3], grads[3:]):
        within(g, w, 3 * b, "gradient")  # from another rounding of out
    # heads before tokens
    heads_first = [x.transpose(0, 1).contiguous().transpose(0, 1) for x in dense_of]
    assert heads_first[0].stride() == (d, n * d, 1)
    assert all(torch.equal(a, b) for a, b in zip(run(*heads_first), want))


@pytest.mark.parametrize("scale", [0.0, -0.2])
def test_scale_of_any_sign(scale):
    off = offsets([70, 150])
    q, k, v, dout = (rand(220, 2, 32, dtype=F16, seed=s) for s in range(4))
    out, lse = torch.empty_like(q), torch.empty(2, 220, device="cuda")
    dense.attn_window_fwd(q, k, v, off, 40, 2, scale, out, lse)
    o, l, bo, bl = O.attn_fwd(q, k, v, off, 40, 2, scale)
    within(out, o, bo, "out")
    within(lse, l, bl, "lse")
    want = O.attn_bwd(q, k, v, off, 40, 2, scale, out, lse, dout)
    for g, w, b in zip(bwd(q, k, v, off, 40, 2, scale, out, lse, dout), want[:3], want[3:]):
        within(g, w, b, "gradient")
    kc, vc = k[:64].view(1, 64, 2, 32), v[:64].view(1, 64, 2, 32)
    lens = torch.tensor([64], dtype=torch.int32, device="cuda")
    check_decode(q[:1], kc, vc, lens, 40, 2, scale)


def test_scores_that_grow_and_dwarf_one_another():
    """The running maximum moves many times, and far."""
    n = 600
    off = offsets([n])
    q = rand(n, 1, 64, dtype=F16, seed=1)
    k = rand(n, 1, 64, dtype=F16, seed=2) * torch.linspace(0.01, 12, n, device="cuda")[:, None, None].half()
    v, dout = rand(n, 1, 64, dtype=F16, seed=3), rand(n, 1, 64, dtype=F16, seed=4)
    out, lse = torch.empty_like(q), torch.empty(1, n, device="cuda")
    dense.attn_window_fwd(q, k, v, off, BIG, 0, 0.125, out, lse)
    o, l, bo, bl = O.attn_fwd(q, k, v, off, BIG, 0, 0.125)
    within(out, o, bo, "out")
    within(lse, l, bl, "lse")
    want = O.attn_bwd(q, k, v, off, BIG, 0, 0.125, out, lse, dout)
    for g, w, b in zip(bwd(q, k, v, off, BIG, 0, 0.125, out, lse, dout), want[:3], want[3:]):
        within(g, w, b, "gradient")


@pytest.mark.parametrize("at", [100, 101, 150, 399])
@pytest.mark.parametrize("d", [32, 128])
def test_what_is_not_finite_reaches_only_what_sees_it(at, d):
    lens, window, sinks = [100, 300, 100], 30, 2
    off = offsets(lens)
    q, k, v, dout = (rand(500, 2, d, dtype=BF16, seed=s) for s in range(4))

    def run(q, k, v):
        out, lse = torch.empty_like(q), torch.empty(2, 500, device="cuda")
        dense.attn_window_fwd(q, k, v, off, window, sinks, 0.2, out, lse)
        return out, lse
    out, lse = run(q, k, v)
    want = bwd(q, k, v, off, window, sinks, 0.2, out, lse, dout)
    # what is computed once more sums in another order
    o, _, bo, _ = O.attn_fwd(q, k, v, off, window, sinks, 0.2)
    dq, dk, dv, bq, bk, bv = O.attn_bwd(q, k, v, off, window, sinks, 0.2, out, lse, dout)
    j = at - 100
    rows = torch.arange(500, device="cuda")
    others = rows != at
    seeing = (rows >= at) & (rows < 400) & ((rows - at < window) | (j < sinks))  # queries that see key j
    seen = (rows <= at) & (rows >= 100) & ((at - rows < window) | (rows - 100 < sinks))  # keys row j sees
    for x, bad in ((k, float("nan")), (v, float("inf"))):
        keep = x[at].clone()
        x[at] = bad
        out2, _ = run(q, k, v)
        within(out2[~seeing], o[~seeing], bo[~seeing], "out")
        assert not out2[seeing].isfinite().all(-1).any()
        # the backward of what was computed from finite values, but for this one input
        got = bwd(q, k, v, off, window, sinks, 0.2, out, lse, dout)
        within(got[0][~seeing], dq[~seeing], bq[~seeing], "dq")
        assert not got[0][seeing].isfinite().all(-1).any()
        assert torch.equal(want[1][others], got[1][others]) and torch.equal(want[2][others], got[2][others])
        x[at] = keep
    for x in (q, dout):
        keep = x[at].clone()
        x[at] = float("nan")
        got = bwd(q, k, v, off, window, sinks, 0.2, out, lse, dout)
        assert torch.equal(got[0][others], want[0][others])
        assert not got[0][at].isfinite().any()
        within(got[1][~seen], dk[~seen], bk[~seen], "dk")
        within(got[2][~seen], dv[~seen], bv[~seen], "dv")
        assert not got[1][seen].isfinite().all(-1).any()
        x[at] = keep


@pytest.mark.parametrize("d", [32, 128])
def test_a_score_of_minus_infinity_weighs_nothing(d):
    n, window, dtype = 200, 20, F16
    off = offsets([n])
    q, k, v = (rand(n, 1, d, dtype=dtype, seed=s) for s in range(3))
    q[:, 0, 0] = 1
    k[[0, 60], 0, 0] = -float("inf")
    v[150] = float("nan")  # hidden from most, in a tile with many that do not see it
    v[1] = float("inf")
    out, lse = torch.empty_like(q), torch.empty(1, n, device="cuda")
    dense.attn_window_fwd(q, k, v, off, window, 0, 0.2, out, lse)
    with_zeros = k.clone()
    with_zeros[[0, 60]] = 0
    s = q[:, 0].double() @ with_zeros[:, 0].double().T * 0.2
    see = O.visible(n, window, 0, "cuda")
    see[:, [0, 60]] = False
    rel = 2 * (d + 8) * O.F32 * (q[:, 0].abs().double() @ with_zeros[:, 0].abs().double().T * 0.2).max() + \
        (16 + n) * O.F32
    p = torch.softmax(s.masked_fill(~see, -float("inf")), -1)
    fine = torch.ones(n, dtype=torch.bool, device="cuda")
    fine[0] = False  # sees key 0 alone: 0 / 0
    fine[1:1 + window] = False
    fine[150:150 + window] = False
    vv = v[:, 0].double().nan_to_num(0, 0, 0)
    want, u = (p @ vv)[fine], O.U[dtype]
    bound = u * want.abs() + (u + 2 * rel) * (1 + u) * (p @ vv.abs())[fine] + \
        O.TINY[dtype] * (1 + (see.double() @ vv.abs())[fine])
    within(out[fine, 0], want, bound, "out")
    assert not out[~fine].isfinite().all(-1).any()
    assert out[0].isnan().all()
    # key 1's value is +inf and key 0 weighs nothing: the sums are +inf, not NaN
    assert (out[1:1 + window] == float("inf")).all()


# ---------------------------------------------------------------------------------- one new event
def decode(q, kc, vc, lens, window, sinks, scale):
    n, hq, d = q.shape
    nb = dense.attn_window_decode_workspace_bytes(n, kc.shape[1], hq, kc.shape[2], d, window, sinks)
    ws = torch.full((nb + 64,), 0xFF, dtype=torch.uint8, device="cuda")
    out = torch.full((n, hq, d), 7, dtype=q.dtype, device="cuda")
    dense.attn_window_decode(q, kc, vc, lens, window, sinks, scale, out, ws[:nb] if nb else None)
    assert (ws[nb:] == 0xFF).all()
    return out


def check_decode(q, kc, vc, lens, window, sinks, scale):
    got = decode(q, kc, vc, lens, window, sinks, scale)
    want, bound = O.attn_decode(q, kc, vc, lens, window, sinks, scale)
    within(got, want, bound, "out")
    assert torch.equal(got, decode(q, kc, vc, lens, window, sinks, scale))


# lens, capacity, q heads, kv heads, dim, window, sinks
CACHES = [
    ([0, 1], 1, 1, 1, 8, 1, 0),
    ([0, 1, 2, 31, 32, 33, 64], 64, 4, 2, 16, 5, 3),
    ([500, 129, 128, 0], 500, 8, 2, 64, 127, 4),
    ([3100], 3100, 4, 1, 128, 2000, 32),
    ([3100, 7, 3099, 1024], 3101, 40, 1, 32, BIG, 0),
    ([100] * 300, 101, 16, 8, 40, 64, 1),
    ([1000, 400], 1000, 66, 2, 80, 300, 9),
]


@pytest.mark.parametrize("dtype", [F16, BF16], ids=str)
@pytest.mark.parametrize("lens,cap,hq,hk,d,window,sinks", CACHES)
def test_one_new_event(lens, cap, hq, hk, d, window, sinks, dtype):
    print(f"[decode] {lens[:8]} of {cap} heads {hq}/{hk} dim {d} window {window} sinks {sinks}", flush=True)
    n = len(lens)
    c = rand(n, cap, 2 * hk, d, dtype=dtype, seed=cap)
    kc, vc = c[:, :, :hk], c[:, :, hk:]
    for b, m in enumerate(lens):  # places past the length are not read
        c[b, m:] = float("nan")
    q = rand(n, hq, d, dtype=dtype, seed=cap + 1)
    check_decode(q, kc, vc, torch.tensor(lens, dtype=torch.int32, device="cuda"), window, sinks, d ** -0.5)


def test_one_new_event_of_a_cache_past_32_bits():
    """The last sequence's keys lie past 2^31 elements from the cache's start."""
    n, cap, hk, d = 3, 120_000, 64, 128
    kc = torch.zeros(n, cap, hk, d, dtype=F16, device="cuda")
    assert kc.numel() > 2 ** 31
    vc = torch.zeros_like(kc)
    kc[2, -600:], vc[2, -600:] = rand(600, hk, d, dtype=F16, seed=1), rand(600, hk, d, dtype=F16, seed=2)
    kc[2, :2], vc[2, :2] = rand(2, hk, d, dtype=F16, seed=3), rand(2, hk, d, dtype=F16, seed=4)
    q = rand(n, hk, d, dtype=F16, seed=5)
    lens = torch.tensor([0, 5, cap], dtype=torch.int32, device="cuda")
    got = decode(q, kc, vc, lens, 500, 2, 0.1)
    want, bound = O.attn_decode(q[:, :4], kc[:, :, :4], vc[:, :, :4], lens, 500, 2, 0.1)
    within(got[:, :4], want, bound, "out")
    assert (got[0] == 0).all() and (got[1] == 0).all()


def test_forward_and_decode_agree_on_the_newest_event():
    off = offsets([400])
    q, k, v = (rand(400, 4, 64, dtype=BF16, seed=s) for s in range(3))
    out = torch.empty_like(q)
    dense.attn_window_fwd(q, k, v, off, 100, 4, 0.125, out)
    o, _, bo, _ = O.attn_fwd(q, k, v, off, 100, 4, 0.125)
    for n in (1, 50, 104, 105, 400):
        lens = torch.tensor([n], dtype=torch.int32, device="cuda")
        got = decode(q[n - 1:n], k[None], v[None], lens, 100, 4, 0.125)
        within(got[0], out[n - 1].double(), 2 * bo[n - 1], "newest")


# ---------------------------------------------------------------------------------- use
def test_on_a_side_stream_and_in_a_graph():
    off = offsets([300, 0, 450])
    q, k, v, dout = (rand(750, 2, 64, dtype=BF16, seed=s) for s in range(4))
    res = [torch.empty_like(q) for _ in range(4)]
    lse = torch.empty(2, 750, device="cuda")
    ws = torch.empty(dense.attn_window_bwd_workspace_bytes(750, 3, 2, 2, 64, 4), dtype=torch.uint8, device="cuda")
    lens = torch.tensor([40], dtype=torch.int32, device="cuda")
    dws = torch.empty(dense.attn_window_decode_workspace_bytes(1, 750, 2, 2, 64, 700, 4), dtype=torch.uint8,
                      device="cuda")
    new = torch.empty(1, 2, 64, dtype=BF16, device="cuda")

    def step():
        dense.attn_window_fwd(q, k, v, off, 90, 4, 0.125, res[0], lse)
        dense.attn_window_bwd(q, k, v, off, 90, 4, 0.125, res[0], lse, dout, *res[1:], ws)
        dense.attn_window_decode(q[:1], k[None], v[None], lens, 700, 4, 0.125, new, dws)
        return [x.clone() for x in res + [lse, new]]
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
        q.copy_(rand(750, 2, 64, dtype=BF16, seed=20 + turn))
        lens.fill_(100 * turn + 1)
        graph.replay()
        torch.cuda.synchronize()
        replayed = [x.clone() for x in got]
        assert all(torch.equal(a, b) for a, b in zip(replayed, step()))


def test_offsets_are_checked_on_request(monkeypatch):
    q, k, v = (rand(20, 1, 32, dtype=F16, seed=s) for s in range(3))
    out = torch.empty_like(q)
    run = lambda o: dense.attn_window_fwd(q, k, v, torch.tensor(o, dtype=torch.int32, device="cuda"),  # noqa: E731
                                          4, 0, 1.0, out)
    monkeypatch.setenv("EMB_VALIDATE", "1")
    run([0, 5, 20])
    for bad in ([1, 5, 20], [0, 6, 5, 20], [0, 5, 19], [0, 5, 21], [0, -1, 20]):
        with pytest.raises(emb.EmbError) as e:
            run(bad)
        assert e.value.name == "EMB_EINVAL" and "offsets" in str(e.value)
    lens = torch.tensor([21], dtype=torch.int32, device="cuda")
    with pytest.raises(emb.EmbError) as e:
        dense.attn_window_decode(q[:1], k[None], v[None], lens, 4, 0, 1.0, out[:1], None)
    assert e.value.name == "EMB_EINVAL" and "length" in str(e.value)

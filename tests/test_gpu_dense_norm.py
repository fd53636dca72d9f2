"""The norms around a block with its gate and residual against the 64-bit oracle, forward and
backward: every type, gate and left-out part, columns from one to the most, rows of any alignment.
Bounds count the rounding of each result to its type and of fp32 sums of known length."""
import pytest

torch = pytest.importorskip("torch")

from ad_recommendation_amd import dense  # noqa: E402
from oracle import dense_oracle as O  # noqa: E402

pytestmark = pytest.mark.gpu
F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16
E = 2.0 ** -24


def within(got, want, bound, what):
    err = (got.double() - want).abs()
    assert torch.isfinite(got).all(), what
    worst = (err - bound).max().item() if err.numel() else -1.0
    assert worst <= 0, f"{what}: {worst:.3g} over its bound, largest error {err.max().item():.3g}"


def make(rows, dim, dtype, gate, seed, offset=0):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def rand(*shape, t=dtype, by=1.0):
        n = 1
        for s in shape:
            n *= s
        flat = torch.empty(n + offset, dtype=t, device="cuda")
        flat.copy_((by * torch.randn(n + offset, generator=g, device="cuda")).to(t))
        return flat[offset:].view(*shape)  # `offset` elements past an aligned address
    x = dict(x=rand(rows, dim), y=rand(rows, dim, by=3.0), r=rand(rows, dim), dr=rand(rows, dim),
             dh=rand(rows, dim), w_post=1 + 0.2 * rand(dim, t=F32), w_pre=1 + 0.2 * rand(dim, t=F32))
    x["gate"] = {"none": None, "vec": rand(dim), "row": rand(rows, dim)}[gate]
    return x


def check_fwd(t, alpha=0.8, eps=1e-6):
    dtype, dim = t["x"].dtype, t["x"].shape[1]
    u, tiny = O.U[dtype], O.TINY[dtype]
    r = torch.full_like(t["x"], 7)
    h = None if t["w_pre"] is None else torch.full_like(t["x"], 7)
    dense.norm_gate_residual_fwd(t["x"], t["y"], t["gate"], t["w_post"], t["w_pre"], alpha, eps, r, h)
    r0, h0 = O.norm_fwd(t["x"], t["y"], t["gate"], t["w_post"], t["w_pre"], alpha, eps)
    ax = alpha * t["x"].double()
    # sums of dim squares, 64 additions deep at most; a dozen products and sums after them
    f = 80 * E * (ax.abs() + (r0 - ax).abs())
    within(r, r0, u * r0.abs() + f + tiny, "r")
    if h is not None:
        inv = torch.rsqrt((r0 * r0).mean(-1, keepdim=True) + eps)
        fh = f * inv * t["w_pre"].abs() + h0.abs() * inv * f.norm(dim=-1, keepdim=True) / dim ** 0.5
        within(h, h0, (u + 80 * E) * h0.abs() + 2 * fh + tiny, "h")
    return r, h


def run_bwd(t, alpha, eps):
    new = lambda like: None if like is None else torch.full_like(like, 7)  # noqa: E731
    dgate = None
    if t["gate"] is not None:
        dgate = torch.full((t["gate"].shape[0],), 7.0, device="cuda") if t["gate"].dim() == 1 else new(t["gate"])
    res = dict(dx=new(t["x"]), dy=new(t["y"]), dgate=dgate, dw_post=new(t["w_post"]), dw_pre=new(t["w_pre"]))
    n, d = t["x"].shape
    nb = dense.norm_gate_residual_bwd_workspace_bytes(n, d)
    ws = torch.full((nb + 64,), 0xFF, dtype=torch.uint8, device="cuda")
    dense.norm_gate_residual_bwd(t["r"], t["y"], t["gate"], t["w_post"], t["w_pre"], alpha, eps, t["dr"],
                                 t["dh"], res["dx"], res["dy"], res["dgate"], res["dw_post"],
                                 res["dw_pre"], ws[:nb] if nb else None)
    assert (ws[nb:] == 0xFF).all()
    return res


def check_bwd(t, alpha=0.8, eps=1e-6):
    dtype, (n, d) = t["x"].dtype, t["x"].shape
    u, tiny = O.U[dtype], O.TINY[dtype]
    res = run_bwd(t, alpha, eps)
    want = dict(zip(("dx", "dy", "dgate", "dw_post", "dw_pre"), O.norm_bwd(
        t["r"], t["y"], t["gate"], t["w_post"], t["w_pre"], alpha, eps, t["dr"], t["dh"])))
    D = lambda k: 0.0 if t[k] is None else t[k].double()  # noqa: E731
    zero = torch.zeros(n, d, dtype=torch.float64, device="cuda")
    r, dr, dh = D("r") + zero, D("dr") + zero, (D("dh") if t["w_pre"] is not None else 0.0) + zero
    uu = dh * (D("w_pre") if t["w_pre"] is not None else 1.0)
    inv = torch.rsqrt((r * r).mean(-1, keepdim=True) + eps)
    k = 160 * E  # two nested row sums, 64 additions deep each, and the products around them
    m1 = inv ** 3 * (uu * r).abs().mean(-1, keepdim=True)
    f_R = k * (dr.abs() + inv * uu.abs() + r.abs() * m1)
    within(res["dx"], want["dx"] + zero, u * (want["dx"] + zero).abs() + abs(alpha) * f_R + tiny, "dx")
    rows = n / 768 + 128  # additions in a column sum: a block's rows, then the blocks
    if t["w_pre"] is not None:
        within(res["dw_pre"], want["dw_pre"], (k + rows * E) * (dh * r * inv).abs().sum(0) + tiny, "dw_pre")
    if t["y"] is None:
        return res
    y = D("y")
    g = 1.0 if t["gate"] is None else D("gate")
    w = 1.0 if t["w_post"] is None else D("w_post")
    iny = torch.rsqrt((y * y).mean(-1, keepdim=True) + eps) if t["w_post"] is not None else 1.0
    dR = want["dx"] / alpha + zero
    a = (g * w * y).abs()
    f_y = (iny * g * w).abs() * f_R + k * iny * (g * w * dR).abs() if t["w_post"] is not None else \
        (g * w) * 0 + abs(g) * f_R + k * (g * dR).abs() if t["gate"] is not None else f_R + k * dR.abs()
    if t["w_post"] is not None:
        m = ((a * dr.abs()).mean(-1, keepdim=True) + inv * (a * uu.abs()).mean(-1, keepdim=True)
             + m1 * (a * r.abs()).mean(-1, keepdim=True))
        f_y = f_y + 2 * k * y.abs() * iny ** 3 * m
    within(res["dy"], want["dy"], u * want["dy"].abs() + f_y + tiny, "dy")
    unit = y * iny
    if t["w_post"] is not None:
        within(res["dw_post"], want["dw_post"],
               ((g * unit).abs() * f_R + (k + rows * E) * (g * unit * dR).abs()).sum(0) + tiny, "dw_post")
    if t["gate"] is not None:
        each = (w * unit).abs() * f_R + k * (w * unit * dR).abs()
        if t["gate"].dim() == 1:
            within(res["dgate"], want["dgate"], (each + rows * E * (w * unit * dR).abs()).sum(0) + tiny, "dgate")
        else:
            within(res["dgate"], want["dgate"], u * want["dgate"].abs() + each + tiny, "dgate")
    return res


DIMS = [1, 2, 7, 8, 9, 64, 255, 256, 257, 333, 512, 520, 1000, 2048, 2049, 4096, 5000, 8192]


@pytest.mark.parametrize("dtype", [F32, F16, BF16], ids=str)
@pytest.mark.parametrize("dim", DIMS)
def test_every_width(dim, dtype):
    for rows, gate in ((1, "vec"), (9, "row"), (67, "none"), (1300 if dim < 600 else 130, "vec")):
        print(f"[norm] {rows} x {dim} {dtype} gate {gate}", flush=True)
        t = make(rows, dim, dtype, gate, seed=rows + dim)
        check_fwd(t)
        res = check_bwd(t)
        for a, b in zip(res.values(), run_bwd(t, 0.8, 1e-6).values()):  # the same bits again
            assert a is b is None or torch.equal(a, b)


@pytest.mark.parametrize("dtype", [F32, BF16], ids=str)
def test_a_training_batch_of_rows(dtype):
    t = make(5000, 96, dtype, "row", seed=1)
    check_fwd(t)
    check_bwd(t)


def test_more_data_than_the_caches_hold():
    """Over 256 MB the kernels pass the caches by; every row is as in smaller calls, bit by bit."""
    rows, dim, part = 36000, 1001, 9000
    t = make(rows, dim, BF16, "vec", seed=2)
    r, h = torch.empty_like(t["x"]), torch.empty_like(t["x"])
    dense.norm_gate_residual_fwd(t["x"], t["y"], t["gate"], t["w_post"], t["w_pre"], 0.8, 1e-6, r, h)
    res = run_bwd(t, 0.8, 1e-6)
    sums = {k: 0.0 for k in ("dw_post", "dw_pre", "dgate")}
    for a in range(0, rows, part):
        p = {k: v[a:a + part] if v is not None and v.dim() == 2 else v for k, v in t.items()}
        r2, h2 = torch.empty_like(p["x"]), torch.empty_like(p["x"])
        dense.norm_gate_residual_fwd(p["x"], p["y"], p["gate"], p["w_post"], p["w_pre"], 0.8, 1e-6, r2, h2)
        assert torch.equal(r2, r[a:a + part]) and torch.equal(h2, h[a:a + part])
        res2 = run_bwd(p, 0.8, 1e-6)
        assert torch.equal(res2["dx"], res["dx"][a:a + part]) and torch.equal(res2["dy"], res["dy"][a:a + part])
        sums = {k: s + res2[k].double() for k, s in sums.items()}
    # column sums of 36000 terms, each about one: additions in a block and of the blocks
    for k, s in sums.items():
        assert ((res[k].double() - s).abs() <= 2 * (rows / 768 + 128) * E * rows * 4).all()


@pytest.mark.parametrize("dtype", [F32, F16], ids=str)
@pytest.mark.parametrize("offset", [1, 3])
def test_rows_aligned_to_their_elements_alone(offset, dtype):
    for dim in (40, 64, 1001):
        t = make(33, dim, dtype, "row", seed=dim, offset=offset)
        check_fwd(t)
        check_bwd(t)


@pytest.mark.parametrize("gate", ["none", "vec", "row"])
@pytest.mark.parametrize("left_out", [("w_post",), ("w_pre", "dh"), ("w_post", "w_pre", "dh"), ("dr",),
                                      ("y", "w_post", "gate")])
def test_parts_left_out(left_out, gate):
    if "gate" in left_out and gate != "none":
        pytest.skip("no gate without y")
    t = make(70, 100, BF16, gate, seed=3)
    for k in left_out:
        t[k] = None
    check_fwd(t)
    check_bwd(t)


def test_values_far_from_one_and_rows_of_zeros():
    t = make(40, 320, F32, "vec", seed=4)
    t["y"][:10] *= 1e-12  # eps outweighs the mean square
    t["y"][10:20] *= 1e12
    t["y"][20] = 0
    t["x"][21] = 0
    t["r"][22] = 0
    t["r"][23] *= 1e9
    check_fwd(t)
    check_bwd(t)


@pytest.mark.parametrize("dtype", [F32, BF16], ids=str)
@pytest.mark.parametrize("dim", [8, 320, 2048])
@pytest.mark.parametrize("by", [1e13, 1e14, 1e15, 1e16, 1e17])
def test_rows_so_large_that_the_cube_of_their_inverse_is_zero(by, dim, dtype):
    """Without a gradient of r beside it, what the norms subtract is as large as what they subtract it from."""
    t = make(24, dim, dtype, "vec", seed=9)
    t["r"] *= by
    t["dr"] = None
    check_bwd(t)
    t["y"] *= by
    check_bwd(t)


@pytest.mark.parametrize("dtype", [F32, BF16], ids=str)
def test_rows_of_zeros_with_an_eps_whose_inverse_cubed_is_infinite(dtype):
    t = make(24, 320, dtype, "row", seed=10)
    t["r"][3] = 0
    t["y"][5] = 0
    check_fwd(t, eps=1e-30)
    check_bwd(t, eps=1e-30)


def test_what_is_not_finite_stays_in_its_row():
    t = make(40, 320, F32, "row", seed=5)
    r, h = check_fwd(t)
    res = run_bwd(t, 0.8, 1e-6)
    t["y"][7, 3] = float("nan")
    r2, h2 = torch.empty_like(r), torch.empty_like(h)
    dense.norm_gate_residual_fwd(t["x"], t["y"], t["gate"], t["w_post"], t["w_pre"], 0.8, 1e-6, r2, h2)
    res2 = run_bwd(t, 0.8, 1e-6)
    rows = torch.arange(40, device="cuda") != 7
    for a, b in ((r, r2), (h, h2), (res["dx"], res2["dx"]), (res["dy"], res2["dy"]), (res["dgate"], res2["dgate"])):
        assert torch.equal(a[rows], b[rows])
    assert r2[7].isnan().all() and h2[7].isnan().all() and res2["dy"][7].isnan().all()


def test_in_place():
    t = make(50, 512, BF16, "vec", seed=6)
    r, h = check_fwd(t)
    x, y = t["x"].clone(), t["y"].clone()
    dense.norm_gate_residual_fwd(x, y, t["gate"], t["w_post"], t["w_pre"], 0.8, 1e-6, x, y)
    assert torch.equal(x, r) and torch.equal(y, h)
    res = run_bwd(t, 0.8, 1e-6)
    dr, dh = t["dr"].clone(), t["dh"].clone()
    dw = torch.empty(512, device="cuda")
    ws = torch.empty(dense.norm_gate_residual_bwd_workspace_bytes(50, 512), dtype=torch.uint8, device="cuda")
    dense.norm_gate_residual_bwd(t["r"], t["y"], t["gate"], t["w_post"], t["w_pre"], 0.8, 1e-6, dr, dh,
                                 dr, dh, None, dw, None, ws)
    assert torch.equal(dr, res["dx"]) and torch.equal(dh, res["dy"]) and torch.equal(dw, res["dw_post"])


@pytest.mark.parametrize("dtype", [F32, BF16], ids=str)
@pytest.mark.parametrize("dim", [1, 9, 17, 63, 121, 333, 777, 1501, 2051, 4093, 8191])
def test_in_place_where_a_vector_ends_with_the_row(dim, dtype):
    rows = 700
    t = make(rows, dim, dtype, "row", seed=dim)
    r, h = check_fwd(t)
    x, y = t["x"].clone(), t["y"].clone()
    dense.norm_gate_residual_fwd(x, y, t["gate"], t["w_post"], t["w_pre"], 0.8, 1e-6, x, y)
    assert torch.equal(x, r) and torch.equal(y, h)
    # no sum before r is written
    first, x = torch.empty_like(x), t["x"].clone()
    dense.norm_gate_residual_fwd(t["x"], None, None, None, None, 0.8, 1e-6, first, None)
    dense.norm_gate_residual_fwd(x, None, None, None, None, 0.8, 1e-6, x, None)
    assert torch.equal(x, first)
    res = check_bwd(t)
    dr, dh = t["dr"].clone(), t["dh"].clone()
    dw, dw_pre = torch.empty(2, dim, device="cuda")
    ws = torch.empty(dense.norm_gate_residual_bwd_workspace_bytes(rows, dim), dtype=torch.uint8, device="cuda")
    dense.norm_gate_residual_bwd(t["r"], t["y"], t["gate"], t["w_post"], t["w_pre"], 0.8, 1e-6, dr, dh,
                                 dr, dh, None, dw, dw_pre, ws)
    assert torch.equal(dr, res["dx"]) and torch.equal(dh, res["dy"])
    assert torch.equal(dw, res["dw_post"]) and torch.equal(dw_pre, res["dw_pre"])


def test_no_rows_give_no_sums():
    t = make(0, 77, F16, "vec", seed=7)
    res = run_bwd(t, 1.0, 1e-6)
    assert all((res[k] == 0).all() for k in ("dw_post", "dw_pre", "dgate"))


def test_in_a_graph():
    t = make(300, 768, BF16, "vec", seed=8)
    graph = torch.cuda.CUDAGraph()
    r, h = torch.empty_like(t["x"]), torch.empty_like(t["x"])

    def step():
        dense.norm_gate_residual_fwd(t["x"], t["y"], t["gate"], t["w_post"], t["w_pre"], 0.8, 1e-6, r, h)
        ws = torch.empty(dense.norm_gate_residual_bwd_workspace_bytes(300, 768), dtype=torch.uint8, device="cuda")
        out = [torch.empty_like(t["x"]), torch.empty_like(t["x"]), *(torch.empty(768, device="cuda") for _ in range(3))]
        dense.norm_gate_residual_bwd(r, t["y"], t["gate"], t["w_post"], t["w_pre"], 0.8, 1e-6, t["dr"],
                                     t["dh"], *out, ws)
        return [r.clone(), h.clone()] + out
    step()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        got = step()
    for turn in range(3):
        t["y"].copy_(make(300, 768, BF16, "vec", seed=20 + turn)["y"])
        graph.replay()
        torch.cuda.synchronize()
        replayed = [x.clone() for x in got]
        assert all(torch.equal(a, b) for a, b in zip(replayed, step()))

"""Attention of candidates and caches in 8 bits on the CPU: the C ABI and the binding refuse bad arguments before any
device work; workspaces are enough for every window; the oracle against differences, closed forms and torch."""
import ctypes as C
import math
import os
import subprocess
import sys

import pytest

torch = pytest.importorskip("torch")

from ad_recommendation_amd import dense, emb  # noqa: E402
from oracle import dense_oracle as O  # noqa: E402
from tests.test_dense_cpu import BAD_ATTN, BF16, F16, F32, P, attn, heads, refused  # noqa: E402

BIG = 1 << 50
OWN = ("q", "k", "v")
GRADS = ("dq", "dk", "dv", "dhk", "dhv")


def codes(p=P, seq=1 << 20, tok=128, head=64):
    return dense.EmbHeads(p, seq, tok, head)


def exps(p=P, seq=1 << 20, tok=1, head=1 << 12):
    return dense.EmbHeads(p, seq, tok, head)


def pick(t, names, make=heads):
    return [None if t.get(n, 0) is None else C.byref(t.get(n, make())) for n in names]


def fwd(a=None, n_seq=2, n_tok=10, n_hist=50, off=P, first=P, hist=P, lse=P, ws=P, ws_bytes=BIG, **t):
    return dense.lib().attn_shared_fwd(C.byref(a or attn()), *pick(t, OWN + ("hk", "hv")), off, first, hist, n_seq, n_tok,
                                       n_hist, *pick(t, ("out",)), lse, ws, ws_bytes, None)


def bwd(a=None, n_seq=2, n_tok=10, n_hist=50, off=P, first=P, hist=P, lse=P, ws=P, ws_bytes=BIG, **t):
    return dense.lib().attn_shared_bwd(C.byref(a or attn()), *pick(t, OWN + ("hk", "hv")), off, first, hist, n_seq, n_tok,
                                       n_hist, *pick(t, ("out",)), lse, *pick(t, ("dout",) + GRADS), ws, ws_bytes, None)


def cache(a=None, n_seq=2, n_tok=10, cap=4000, off=P, first=P, lens=P, ws=P, ws_bytes=BIG, **t):
    return dense.lib().attn_shared_cache(C.byref(a or attn()), *pick(t, OWN + ("hk", "hv")), off, first, lens, n_seq,
                                         n_tok, cap, *pick(t, ("out",)), ws, ws_bytes, None)


def cache_q8(a=None, n_seq=2, n_tok=10, cap=4000, off=P, first=P, lens=P, ws=P, ws_bytes=BIG, **t):
    kv = pick(t, ("kc",), codes) + pick(t, ("ke",), exps) + pick(t, ("vc",), codes) + pick(t, ("ve",), exps)
    return dense.lib().attn_shared_cache_q8(C.byref(a or attn()), *pick(t, OWN), *kv, off, first, lens, n_seq, n_tok, cap,
                                            *pick(t, ("out",)), ws, ws_bytes, None)


def dec(a=None, n_seq=2, cap=4000, lens=P, ws=P, ws_bytes=BIG, **t):
    kv = pick(t, ("kc",), codes) + pick(t, ("ke",), exps) + pick(t, ("vc",), codes) + pick(t, ("ve",), exps)
    return dense.lib().attn_window_decode_q8(C.byref(a or attn()), *pick(t, ("q",)), *kv, lens, n_seq, cap,
                                             *pick(t, ("out",)), ws, ws_bytes, None)


@pytest.mark.parametrize("bad,text", BAD_ATTN)
@pytest.mark.parametrize("call", [fwd, bwd, cache, cache_q8, dec])
def test_bad_descriptors_are_refused(call, bad, text):
    refused(call(attn(**bad)), "EMB_EINVAL", text)


@pytest.mark.parametrize("call", [fwd, bwd, cache, cache_q8, dec])
def test_bad_arguments_are_refused(call):
    names = {fwd: OWN + ("hk", "hv", "out"), bwd: OWN + ("hk", "hv", "out", "dout") + GRADS,
             cache: OWN + ("hk", "hv", "out"), cache_q8: OWN + ("out",), dec: ("q", "out")}[call]
    for name in names:
        refused(call(**{name: None}), "EMB_EINVAL", "null")
        refused(call(**{name: heads(p=None)}), "EMB_EINVAL", "null")
        refused(call(**{name: heads(p=P + 8)}), "EMB_EINVAL", "aligned")
        refused(call(**{name: heads(tok=100)}), "EMB_EINVAL", "stride")
        refused(call(**{name: heads(head=33)}), "EMB_EINVAL", "stride")
    if call in (cache_q8, dec):
        for name, make in (("kc", codes), ("ke", exps), ("vc", codes), ("ve", exps)):
            refused(call(**{name: None}), "EMB_EINVAL", "null")
            refused(call(**{name: make(p=None)}), "EMB_EINVAL", "null")
        for name in ("kc", "vc"):
            refused(call(**{name: codes(p=P + 4)}), "EMB_EINVAL", "aligned")
            for bad in (dict(tok=100), dict(head=12), dict(seq=4)):
                refused(call(**{name: codes(**bad)}), "EMB_EINVAL", "stride")
    refused(call(n_seq=-1), "EMB_EINVAL", "negative")
    refused(call(n_seq=2 ** 30 + 1), "EMB_ERANGE")
    for name in ("out",) if call is not bwd else GRADS:
        four = name in ("out", "dq")  # the others have two heads
        for bad in (dict(tok=0), dict(head=0), dict(head=56), dict(tok=-8), dict(tok=128 if four else 64, head=64),
                    dict(tok=64, head=320 if call is not dec else 64)):
            refused(call(**{name: heads(**bad)}), "EMB_EINVAL", "overlap")
    if call is not dec:
        refused(call(n_tok=-1), "EMB_EINVAL", "negative")
        refused(call(n_tok=2 ** 30 + 1), "EMB_ERANGE")
        refused(call(off=None), "EMB_EINVAL", "offsets")
        refused(call(off=P + 2), "EMB_EINVAL", "aligned")
        refused(call(first=P + 1), "EMB_EINVAL", "aligned")
        assert call(n_seq=0, n_tok=0) == 0
    if call in (fwd, bwd):
        refused(call(n_hist=-1), "EMB_EINVAL", "negative")
        refused(call(n_hist=2 ** 30 + 1), "EMB_ERANGE")
        refused(call(hist=None), "EMB_EINVAL")
        refused(call(hist=P + 2), "EMB_EINVAL", "aligned")
        refused(call(lse=P + 2), "EMB_EINVAL", "aligned")
    else:
        refused(call(cap=-1), "EMB_EINVAL", "negative")
        refused(call(cap=2 ** 30 + 1), "EMB_ERANGE")
        refused(call(lens=None), "EMB_EINVAL", "lens")
        refused(call(lens=P + 2), "EMB_EINVAL", "aligned")
    if call is bwd:
        refused(call(lse=None), "EMB_EINVAL", "null")
        refused(call(ws=None), "EMB_EINVAL", "null")
        refused(call(ws=P + 4), "EMB_EINVAL", "misaligned")
        refused(call(ws_bytes=100), "EMB_ENOSPACE")
    else:
        assert call(n_seq=0) == 0
        long = dict(a=attn(window=2 ** 31 - 1), **({"cap": 1 << 16} if call is not fwd else {"n_hist": 1 << 16}))
        refused(call(ws=None, **long), "EMB_EINVAL", "workspace")
        refused(call(ws=P + 8, **long), "EMB_EINVAL", "workspace")
        refused(call(ws_bytes=16, **long), "EMB_ENOSPACE")


def test_calls_past_what_a_launch_holds_are_refused():
    wide = attn(q_heads=64, kv_heads=64, dim=64)
    apart = {n: heads(tok=4096, head=64) for n in ("out",) + GRADS}
    for call in (fwd, bwd, cache, cache_q8):
        refused(call(wide, n_seq=2 ** 21, n_tok=2 ** 21, **apart), "EMB_ERANGE", "launch")
    refused(bwd(attn(dim=128), n_seq=2 ** 22, n_tok=4, n_hist=2 ** 22, **{n: heads(tok=512, head=128) for n in GRADS}),
            "EMB_ERANGE", "launch")
    refused(dec(wide, n_seq=2 ** 20, **apart), "EMB_ERANGE", "launch")


def test_workspaces_cover_every_window():
    L, n = dense.lib(), C.c_size_t()
    for n_tok, n_seq, hist in ((1, 1, 1), (72, 1, 16000), (24, 3, 9000), (30, 1, 1100), (500, 8, 33000), (4000, 64, 90000),
                               (2000, 200, 100000), (10 ** 6, 7, 10 ** 6), (3, 3, 0), (0, 5, 1000)):
        for q, kv, d in ((4, 2, 64), (16, 16, 128), (8, 1, 32), (32, 8, 128)):
            a = attn(q_heads=q, kv_heads=kv, dim=d, sinks=32)
            for fn in (L.attn_shared_fwd_workspace_bytes, L.attn_shared_bwd_workspace_bytes, L.attn_shared_cache_workspace_bytes):
                sizes = []
                for w in (2 ** 31 - 1, 1, 2, 33, 100, 500, 1000, 1024, 1025, 2047, 4096, 8000, 12345, 16000, 10 ** 6):
                    a.window = w
                    assert fn(C.byref(a), n_seq, n_tok, hist, C.byref(n)) == 0
                    sizes.append(n.value)
                assert max(sizes) == sizes[0], (n_tok, n_seq, hist, q, kv, d)
    for fn in (L.attn_shared_fwd_workspace_bytes, L.attn_shared_bwd_workspace_bytes, L.attn_shared_cache_workspace_bytes):
        refused(fn(C.byref(attn()), 1, 1, 1, None), "EMB_EINVAL")
        refused(fn(C.byref(attn(dim=7)), 1, 1, 1, C.byref(n)), "EMB_EINVAL")
        refused(fn(C.byref(attn()), 1, -1, 1, C.byref(n)), "EMB_EINVAL")
    refused(L.attn_window_decode_q8_workspace_bytes(C.byref(attn()), 1, 1, None), "EMB_EINVAL")
    assert dense.attn_window_decode_q8_workspace_bytes(1024, 8192, 4, 2, 64, 4096, 4) == 0
    assert dense.attn_shared_cache_workspace_bytes(72, 1, 16000, 8, 2, 64) > 0


# ---------------------------------------------------------------------------------- caches in 8 bits
def write(kv=2, dim=64, dtype=F16, n_seq=2, n_tok=10, cap=16, off=P, start=P, call="cache_q8_write", **t):
    own = pick(t, ("k", "v"))
    kvs = pick(t, ("kc",), codes) + pick(t, ("ke",), exps) + pick(t, ("vc",), codes) + pick(t, ("ve",), exps)
    if call == "cache_q8_write":
        return dense.lib().cache_q8_write(kv, dim, dtype, *own, off, start, n_seq, n_tok, *kvs, cap, None)
    return dense.lib().cache_q8_read(kv, dim, dtype, *kvs, cap, off, start, n_seq, n_tok, *own, None)


@pytest.mark.parametrize("call", ["cache_q8_write", "cache_q8_read"])
def test_bad_cache_arguments_are_refused(call):
    bad = [dict(dtype=3), dict(kv=0), dict(kv=-1), dict(kv=4097), dict(dim=0), dict(dim=4), dict(dim=20), dict(dim=136),
           dict(n_seq=-1), dict(n_tok=-1), dict(cap=-1), dict(off=None), dict(off=P + 2), dict(start=P + 1),
           dict(kc=codes(p=P + 4)), dict(vc=codes(tok=100)), dict(kc=codes(head=4))]
    bad += [{n: None} for n in ("k", "v", "kc", "ke", "vc", "ve")]
    bad += [{n: heads(p=None)} for n in ("k", "v")] + [{n: exps(p=None)} for n in ("ke", "ve")]
    bad += [dict(k=heads(p=P + 8)), dict(v=heads(tok=100))]
    for b in bad:
        refused(write(call=call, **b), "EMB_EINVAL")
    for b in (dict(n_seq=2 ** 30 + 1), dict(n_tok=2 ** 30 + 1), dict(cap=2 ** 30 + 1)):
        refused(write(call=call, **b), "EMB_ERANGE")
    assert write(call=call, n_seq=0, n_tok=0) == 0 and write(call=call, n_tok=0) == 0
    if call == "cache_q8_write":
        assert write(cap=0, kc=codes(p=None)) == 0  # nowhere to write to
        for b in (dict(kc=codes(tok=64)), dict(vc=codes(seq=0)), dict(kc=codes(seq=1024)), dict(vc=codes(head=0)),
                  dict(ke=exps(tok=0)), dict(ve=exps(head=8)), dict(ke=exps(seq=8))):
            refused(write(**b), "EMB_EINVAL", "overlap")
    else:
        for b in (dict(k=heads(tok=0)), dict(v=heads(head=32)), dict(k=heads(tok=64))):
            refused(write(call=call, **b), "EMB_EINVAL", "overlap")


def test_binding_refuses_bad_tensors():
    h = torch.float16
    x, off = torch.zeros(4, 2, 8, dtype=h), torch.zeros(2, dtype=torch.int32)
    c, e = torch.zeros(1, 5, 2, 8, dtype=torch.uint8), torch.zeros(1, 2, 5, dtype=torch.uint8)
    with pytest.raises(TypeError, match="CUDA"):
        dense.attn_shared_fwd(x, x, x, x, x, off, None, off, 1, 0, 1.0, x)
    with pytest.raises(TypeError, match="float16 or bfloat16"):
        dense.attn_shared_fwd(x.float(), x, x, x, x, off, None, off, 1, 0, 1.0, x)
    with pytest.raises(ValueError, match="events, heads, dim"):
        dense.attn_shared_fwd(x, x, x, x[0], x, off, None, off, 1, 0, 1.0, x)
    with pytest.raises(ValueError, match="capacity"):
        dense.attn_shared_cache(x, x, x, x, x, off, None, off[:1], 1, 0, 1.0, x)
    with pytest.raises(ValueError, match="capacity"):
        dense.attn_window_decode_q8(x, x, e, x, e, off, 1, 0, 1.0, x, None)
    with pytest.raises(ValueError, match="capacity"):
        dense.cache_q8_write(x, x, off, None, c[0], e, c, e)
    with pytest.raises(TypeError, match="float32, float16 or bfloat16"):
        dense.cache_q8_write(x.double(), x, off, None, c, e, c, e)
    with pytest.raises(ValueError, match="heads and dim"):
        dense.cache_q8_write(x[:, :1], x, off, None, c, e, c, e)
    with pytest.raises(TypeError, match="CUDA"):
        dense.cache_q8_write(x, x, off, None, c, e, c, e)
    with pytest.raises(TypeError, match="CUDA"):
        dense.cache_q8_read(c, e, c, e, off, None, x, x)
    for window, sinks in ((-2 ** 40, 0), (1, 2 ** 32)):
        with pytest.raises(ValueError, match="32 bits"):
            dense.attn_shared_fwd(x, x, x, x, x, off, None, off, window, sinks, 1.0, x)


# ---------------------------------------------------------------------------------- the oracle
def case(window=4, sinks=2, g=None):
    g = torch.Generator().manual_seed(1) if g is None else g
    rand = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)  # noqa: E731
    off, hoff = torch.tensor([0, 5, 5, 9]), torch.tensor([0, 7, 10, 10])
    first = torch.tensor([0, 0, 2, 3, 3, 5, 5, 5, 8], dtype=torch.int32)
    return (rand(9, 4, 8), rand(9, 2, 8), rand(9, 2, 8), rand(10, 2, 8), rand(10, 2, 8), off, first, hoff, window, sinks, 0.4)


def test_shared_oracle_against_differences():
    args = list(case())
    dout = torch.randn(9, 4, 8, generator=torch.Generator().manual_seed(2), dtype=torch.float64)
    f = lambda: (O.attn_shared_fwd(*args)[0] * dout).sum().item()  # noqa: E731
    out, lse = O.attn_shared_fwd(*args)[:2]
    grads, _ = O.attn_shared_bwd(*args, out, lse, dout)
    g = torch.Generator().manual_seed(3)
    for x, d in zip(args[:5], grads):
        way = torch.randn(x.shape, generator=g, dtype=torch.float64)
        keep, h = x.clone(), 1e-5
        x.copy_(keep + h * way)
        up = f()
        x.copy_(keep - h * way)
        down = f()
        x.copy_(keep)
        assert abs((up - down) / (2 * h) - (d * way).sum().item()) < 1e-8


def test_shared_oracle_is_window_attention_of_the_next_event():
    """A candidate of one token sees what the event after its history would, and itself."""
    g = torch.Generator().manual_seed(4)
    rand = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)  # noqa: E731
    q, k, v, off = rand(12, 4, 8), rand(12, 2, 8), rand(12, 2, 8), torch.tensor([0, 12])
    for window, sinks in ((1, 0), (3, 2), (11, 0), (12, 1), (100, 0)):
        want = O.attn_fwd(q, k, v, off, window, sinks, 0.3)
        got = O.attn_shared_fwd(q[11:], k[11:], v[11:], k[:11], v[:11], torch.tensor([0, 1]), None, torch.tensor([0, 11]),
                                window, sinks, 0.3)
        assert torch.allclose(got[0][0], want[0][11], atol=1e-14) and torch.allclose(got[1][:, 0], want[1][:, 11], atol=1e-13)
    # one candidate of all tokens and no history: plain causal attention
    want = O.attn_fwd(q, k, v, off, 100, 0, 0.3)
    got = O.attn_shared_fwd(q, k, v, k[:0], v[:0], off, torch.zeros(12, dtype=torch.int32), torch.tensor([0, 0]), 5, 1, 0.3)
    assert torch.allclose(got[0], want[0], atol=1e-14)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16, torch.float32], ids=str)
def test_quantising_oracle_is_torchs_cast(dtype):
    g = torch.Generator().manual_seed(5)
    x = (torch.randn(500, 24, generator=g) * torch.exp(2 * torch.randn(500, 1, generator=g))).to(dtype)
    x[3] = 0
    c, e = O.quantise(x)
    y = x.double() / O.power(e.long())[:, None]
    assert torch.equal(c, y.float().to(torch.float8_e4m3fn).view(torch.uint8))
    assert (y.abs().amax(1)[x.abs().amax(1) > 0] >= 128).all() and (y.abs() < 256).all()
    back = O.values_of(c, e)
    # half a step: an e4m3 value has four significant bits
    assert ((back - x.double()).abs() <= 2.0 ** -4 * x.double().abs() + 2.0 ** -10 * O.power(e.long())[:, None]).all()
    again = O.quantise(back.to(torch.float32))
    assert torch.equal(O.values_of(*again), back)


def test_checks_under_asan_and_ubsan():
    from tests.test_sanitized_host_cpu import ROOT, _runtime
    asan = _runtime("libasan.so")
    if asan is None or os.environ.get("MI355EMB_LIB"):
        pytest.skip("no AddressSanitizer runtime for g++ here, or already under it")
    from ad_recommendation_amd import build as B
    env = dict(os.environ, MI355EMB_LIB=B.build_sanitized(), LD_PRELOAD=asan,
               ASAN_OPTIONS="detect_leaks=0:abort_on_error=1", UBSAN_OPTIONS="halt_on_error=1:print_stacktrace=1")
    r = subprocess.run([sys.executable, "-m", "pytest", "-q", "-x", "-p", "no:cacheprovider", "tests/test_dense_shared_cpu.py"],
                       cwd=ROOT, env=env, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True, timeout=600)
    assert r.returncode == 0 and " passed" in r.stdout, "\n".join(r.stdout.splitlines()[-30:])

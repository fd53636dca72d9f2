"""The binding's calls run on the current device and take no tensor of another."""
import pytest

torch = pytest.importorskip("torch")

from ad_recommendation_amd import dense  # noqa: E402

pytestmark = pytest.mark.gpu


def calls():
    """Every call by name, and whether it has a tensor to look at."""
    new = lambda *s, t=torch.float16: torch.zeros(*s, dtype=t, device="cuda")  # noqa: E731
    q, o, lse = new(4, 2, 8), new(4, 2, 8), new(2, 4, t=torch.float32)
    off, ws = torch.tensor([0, 4], dtype=torch.int32, device="cuda"), new(1 << 16, t=torch.uint8)
    x, w, f = new(3, 16), new(16, t=torch.float32), [new(5, t=torch.float32)]
    s, b = new(128, t=torch.float32), new(128, t=torch.uint8)
    e = new(1, t=torch.uint8)
    return {
        "attn_window_fwd": lambda: dense.attn_window_fwd(q, q, q, off, 2, 0, 1.0, o, lse),
        "attn_window_bwd": lambda: dense.attn_window_bwd(q, q, q, off, 2, 0, 1.0, o, lse, o, new(4, 2, 8),
                                                         new(4, 2, 8), new(4, 2, 8), ws),
        "attn_window_decode": lambda: dense.attn_window_decode(q[:1], q[None], q[None], off[1:], 2, 0, 1.0, o[:1], ws),
        "norm_gate_residual_fwd": lambda: dense.norm_gate_residual_fwd(x, x, None, w, w, 1.0, 1e-6, new(3, 16),
                                                                       new(3, 16)),
        "norm_gate_residual_bwd": lambda: dense.norm_gate_residual_bwd(x, x, None, w, w, 1.0, 1e-6, x, x, new(3, 16),
                                                                       new(3, 16), None, None, None, ws),
        "adamw_step": lambda: dense.adamw_step(f, f, s, s.clone(), 1, 1e-3, 0.9, 0.99, 1e-8, 0.0),
        "adamw_step_q8": lambda: dense.adamw_step_q8(f, f, b, e, b.clone(), e.clone(), 1, 1e-3, 0.9, 0.99, 1e-8, 0.0, 1),
        "adamw_q8_values": lambda: dense.adamw_q8_values(b, e, s),
    }


@pytest.mark.parametrize("name", list(dense._SIG))
def test_tensors_of_another_device_are_refused(name, monkeypatch):
    if name not in calls():
        pytest.skip("host only")
    call = calls()[name]
    call()
    torch.cuda.synchronize()
    # as it looks where another device is current: the binding refuses before it asks for that one's stream
    monkeypatch.setattr(dense, "_device", lambda: 1)
    monkeypatch.setattr(dense, "_stream", lambda *a: pytest.fail("a tensor of another device was taken"))
    with pytest.raises(TypeError, match="current device"):
        call()

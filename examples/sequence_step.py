"""One training step of a model over users' event sequences, and its serving form, on one GPU.

Events are keys of the resident embedding table.  A step looks their rows up, runs one block over
every user's sequence (norm, windowed attention with sinks, gated residual, norm), scores each event,
and goes back: the dense weights take an AdamW step, the looked-up rows a sparse Adagrad step.  The
products with weights are plain torch matmuls.  Afterwards the newest event of each user is answered
from a key/value cache alone and compared with the whole forward.

    python examples/sequence_step.py [--steps 60] [--q8] [--window 16]

The data is synthetic: every item has a hidden value, and an event's label is the sign of the mean over
the events it sees in its window, so the loss falls far only if attention carries what it read.
"""
from __future__ import annotations

import argparse
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import numpy as np  # noqa: E402
import torch  # noqa: E402

from ad_recommendation_amd import dense, emb  # noqa: E402

DEV, HALF = "cuda", torch.float16
DIM, HEADS, HEAD = 64, 4, 16
SINKS, EPS, ALPHA = 2, 1e-6, 1.0


class SequenceModel:
    def __init__(self, n_items: int, window: int, q8: bool, seed: int = 0):
        g = torch.Generator().manual_seed(seed)
        rand = lambda *s, by: by * torch.randn(*s, generator=g)  # noqa: E731
        self.window, self.q8, self.step, self.scale = window, q8, 0, HEAD ** -0.5
        keys = np.arange(1, n_items + 1, dtype=np.int64)  # field 0
        rows = rand(n_items, DIM, by=0.5).to(HALF).numpy()
        self.table = emb.Table([DIM], emb.EMB_F16, True, 1, 0.5, 0.01, keys, rows.reshape(-1), None,
                               rows.astype(np.float32).reshape(-1))
        self.table.flash(DEV)
        w = dict(qkv=rand(DIM, 3 * DIM, by=DIM ** -0.5), out=rand(DIM, DIM, by=DIM ** -0.5),
                 head=rand(DIM, 1, by=DIM ** -0.5), pre=torch.ones(DIM), post=torch.ones(DIM),
                 gate=torch.full((DIM,), 0.5), pre2=torch.ones(DIM))
        self.w = {k: v.to(DEV).contiguous() for k, v in w.items()}  # fp32, what AdamW updates
        self.c = {k: v.to(HALF) for k, v in self.w.items()}         # what the products read
        n = dense.adamw_state_elems(list(self.w.values()))
        if q8:
            self.state = [torch.zeros(x, dtype=torch.uint8, device=DEV) for x in (n, n // dense.ADAMW_BLOCK) * 2]
        else:
            self.state = [torch.zeros(n, device=DEV) for _ in range(2)]

    def lookup(self, keys):
        """The events' rows: bags of one key each."""
        t = keys.numel()
        self.bags = torch.arange(t + 1, dtype=torch.int32, device=DEV)
        x = torch.empty(t, DIM, dtype=HALF, device=DEV)
        self.rowref = torch.empty(t, dtype=torch.int32, device=DEV)
        emb.lookup_pool_fwd(self.table.h, keys, self.bags, t, t, x, emb.EMB_F16, self.rowref)
        return x

    def forward(self, keys, offsets):
        t, new = keys.numel(), lambda *s: torch.empty(*s, dtype=HALF, device=DEV)  # noqa: E731
        x = self.lookup(keys)
        h = new(t, DIM)
        dense.norm_gate_residual_fwd(x, None, None, None, self.w["pre"], 1.0, EPS, None, h)
        qkv = (h @ self.c["qkv"]).view(t, 3 * HEADS, HEAD)
        q, k, v = qkv.split(HEADS, 1)
        o, lse = new(t, HEADS, HEAD), torch.empty(HEADS, t, device=DEV)
        dense.attn_window_fwd(q, k, v, offsets, self.window, SINKS, self.scale, o, lse)
        y = o.view(t, DIM) @ self.c["out"]
        r, h2 = new(t, DIM), new(t, DIM)
        dense.norm_gate_residual_fwd(x, y, self.c["gate"], self.w["post"], self.w["pre2"], ALPHA, EPS, r, h2)
        self.saved = x, h, q, k, v, o, lse, y, r, h2
        return (h2 @ self.c["head"])[:, 0].float()

    def backward(self, dlogit, offsets):
        """Gradients of the dense weights (fp32) and of the looked-up rows."""
        x, h, q, k, v, o, lse, y, r, h2 = self.saved
        t, g = x.shape[0], {k: torch.empty_like(w) for k, w in self.w.items()}
        ws = lambda n: torch.empty(max(n, 16), dtype=torch.uint8, device=DEV)  # noqa: E731
        d = dlogit[:, None].to(HALF)
        g["head"] = (h2.t().float() @ d.float())
        dh2 = d @ self.c["head"].t()
        dx, dy = torch.empty_like(x), torch.empty_like(y)
        norm_ws = ws(dense.norm_gate_residual_bwd_workspace_bytes(t, DIM))
        dense.norm_gate_residual_bwd(r, y, self.c["gate"], self.w["post"], self.w["pre2"], ALPHA, EPS, None, dh2,
                                     dx, dy, g["gate"], g["post"], g["pre2"], norm_ws)
        g["out"] = (o.view(t, DIM).t() @ dy).float()
        do = (dy @ self.c["out"].t()).view(t, HEADS, HEAD)
        dqkv = torch.empty(t, 3 * HEADS, HEAD, dtype=HALF, device=DEV)
        n = dense.attn_window_bwd_workspace_bytes(t, offsets.numel() - 1, HEADS, HEADS, HEAD, SINKS)
        dense.attn_window_bwd(q, k, v, offsets, self.window, SINKS, self.scale, o, lse, do,
                              *dqkv.split(HEADS, 1), ws(n))
        dqkv = dqkv.view(t, 3 * DIM)
        g["qkv"] = (h.t() @ dqkv).float()
        dh = dqkv @ self.c["qkv"].t()
        # the first norm's input is x itself, which the residual reads too: dx flows into it
        dense.norm_gate_residual_bwd(x, None, None, None, self.w["pre"], 1.0, EPS, dx, dh, dx, None, None, None,
                                     g["pre"], norm_ws)
        return g, dx

    def train(self, keys, offsets, labels, lr=3e-3, row_lr=0.05):
        logit = self.forward(keys, offsets)
        loss = torch.nn.functional.binary_cross_entropy_with_logits(logit, labels)
        t = keys.numel()
        # the gradient of the sum, so that half precision holds it; the mean's factor goes to the updates
        g, dx = self.backward(torch.sigmoid(logit) - labels, offsets)
        self.step += 1
        args = (self.step, lr, 0.9, 0.99, 1e-8, [0.01 if w.dim() == 2 else 0.0 for w in self.w.values()])
        more = dict(copies=list(self.c.values()), grad_scale=torch.tensor(1.0 / t, device=DEV))
        if self.q8:
            dense.adamw_step_q8(list(self.w.values()), list(g.values()), *self.state, *args, seed=self.step, **more)
        else:
            dense.adamw_step(list(self.w.values()), list(g.values()), *self.state, *args, **more)
        ws = torch.empty(emb.bwd_workspace_bytes(self.table.h, t, t), dtype=torch.uint8, device=DEV)
        emb.sparse_adagrad_bwd(self.table.h, self.rowref, self.bags, t, t, dx, emb.EMB_F16, row_lr, 1e-8, ws)
        return loss

    def serve(self, k_cache, v_cache, lens, q):
        """The newest event of each user against its cache."""
        out = torch.empty_like(q)
        n, cap = k_cache.shape[:2]
        nb = dense.attn_window_decode_workspace_bytes(n, cap, HEADS, HEADS, HEAD, self.window, SINKS)
        ws = torch.empty(nb, dtype=torch.uint8, device=DEV) if nb else None
        dense.attn_window_decode(q, k_cache, v_cache, lens, self.window, SINKS, self.scale, out, ws)
        return out


def batch(rng, values, window: int, n_seq: int = 64, longest: int = 100):
    lens = rng.integers(2, longest, n_seq)
    off = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    items = rng.integers(0, values.size, off[-1])
    labels = np.empty(off[-1], np.float32)
    for b, e in zip(off[:-1], off[1:]):
        total = np.concatenate([[0.0], np.cumsum(values[items[b:e]])])
        i = np.arange(1, e - b + 1)
        labels[b:e] = total[i] - total[np.maximum(i - window, 0)] > 0
    to = lambda a: torch.from_numpy(a).to(DEV)  # noqa: E731
    return to((items + 1).astype(np.int64)), to(off), to(labels)


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=60)
    ap.add_argument("--items", type=int, default=200)
    ap.add_argument("--window", type=int, default=16)
    ap.add_argument("--q8", action="store_true", help="AdamW states in 8 bits")
    a = ap.parse_args(argv)
    torch.cuda.set_device(0)
    rng = np.random.default_rng(0)
    values = rng.standard_normal(a.items)
    m = SequenceModel(a.items, a.window, a.q8)
    losses = []
    for i in range(a.steps):
        losses.append(m.train(*batch(rng, values, a.window)).item())
        if i % 10 == 0 or i == a.steps - 1:
            print(f"step {i}: loss {losses[-1]:.4f}", flush=True)

    # serving: the caches hold every user's keys and values, the newest event's included
    keys, off, _ = batch(rng, values, a.window, n_seq=8)
    m.forward(keys, off)
    q, k, v, o = m.saved[2:6]
    lens = off[1:] - off[:-1]
    cap = int(lens.max())
    kc, vc = (torch.zeros(lens.numel(), cap, HEADS, HEAD, dtype=HALF, device=DEV) for _ in range(2))
    for s, (b, e) in enumerate(zip(off[:-1].tolist(), off[1:].tolist())):
        kc[s, :e - b], vc[s, :e - b] = k[b:e], v[b:e]
    last = (off[1:] - 1).long()
    served = m.serve(kc, vc, lens, q[last].contiguous())
    worst = (served.float() - o[last].float()).abs().max().item()
    print(f"newest events from the cache differ from the whole forward by at most {worst:.2g}", flush=True)
    m.table.close()
    return losses, worst


if __name__ == "__main__":
    main()

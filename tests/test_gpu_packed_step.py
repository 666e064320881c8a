"""The example's packed training step (examples/packed_step.py) against the
same model in float64 on every sequence alone: losses at each loss position
and the gradient of every weight.

Tolerance: between a weight and its gradient lie at most eight tensors that
are rounded to bf16 once each (half a step 2^-8 relative: embedding path,
projection, rotated q / k, P, attention output, y, logits, their gradients),
so a gradient's 2-norm is off by at most 8 * 2^-8 of itself; log-probabilities
and entropies follow logits of magnitude below 8 (rounded: 8 * 2^-8) whose own
inputs carry three such roundings.
"""
import importlib.util
import os
import sys

import numpy as np
import pytest
import torch

from conftest import ROOT
from sft_trie_build_gb300 import workloads as W

pytestmark = pytest.mark.gpu
spec = importlib.util.spec_from_file_location("packed_step", os.path.join(ROOT, "examples", "packed_step.py"))
EX = importlib.util.module_from_spec(spec)
sys.modules["packed_step"] = EX          # its dataclass looks its module up
spec.loader.exec_module(EX)


def _alone(c, w, seq, train, terms):
    """Sum of the loss terms of one sequence, float64; terms(p) gives the weights at the loss position before p."""
    n, hq, hkv, d = len(seq), c.n_q_heads, c.n_kv_heads, c.head_dim
    x = w["embed"][torch.from_numpy(seq).long()]
    qkv = (x @ w["qkv"]).view(n, hq + 2 * hkv, d)
    ang = torch.arange(n, dtype=torch.float64)[:, None] * 10000.0 ** (-torch.arange(0, d, 2, dtype=torch.float64) / d)
    turn = torch.polar(torch.ones_like(ang), ang)[:, None]

    def rot(a, g):
        a = g * a / (a.square().mean(-1, keepdim=True) + 1e-6).sqrt()
        z = torch.complex(a[..., :d // 2], a[..., d // 2:]) * turn
        return torch.cat((z.real, z.imag), -1)

    q, k = rot(qkv[:, :hq], w["norm_q"]), rot(qkv[:, hq:hq + hkv], w["norm_k"])
    k, v = (a.repeat_interleave(hq // hkv, 1) for a in (k, qkv[:, hq + hkv:]))
    i, j = torch.arange(n)[:, None], torch.arange(n)[None]
    see = (j <= i) & ((i - j < c.window) | (j < c.n_sink))
    p = torch.softmax(torch.einsum("ihd,jhd->hij", q, k).mul(d ** -0.5).masked_fill(~see, float("-inf")), -1)
    y = x + torch.einsum("hij,jhd->ihd", p, v).reshape(n, -1) @ w["out"]
    lp = torch.log_softmax(y @ w["head"], -1)
    total, seen = 0.0, []
    for t in range(1, n):
        if train[t]:
            ids, tl, dist, gl, ge = terms(t)
            lq = torch.log_softmax(tl, -1)
            loss = (lq.exp() * (lq - lp[t - 1, ids])).sum()
            ent = -(lp[t - 1].exp() * lp[t - 1]).sum()
            total = total + dist * loss + gl * lp[t - 1, int(seq[t])] + ge * ent
            seen.append((t - 1, float(loss.detach()), float(lp[t - 1, int(seq[t])].detach()), float(ent.detach())))
    return total, seen


def test_packed_step_equals_sequences_alone():
    c = EX.Config(vocab=96, width=128, n_q_heads=2, n_kv_heads=1, window=20, n_sink=2, teacher_k=8)
    b = W.random_forest(11, n_roots=3, max_depth=2, len_lo=4, len_hi=40, row_len=256, min_shared=4, vocab=c.vocab)
    rows = EX.pack(b)
    w = EX.init_weights(c, seed=3)
    n = rows["token_ids"].size
    g = torch.Generator().manual_seed(5)
    ids = torch.rand(n, c.vocab, generator=g).topk(c.teacher_k, -1).indices.int()
    tl = torch.randn(n, c.teacher_k, generator=g)
    dist, gl, ge = torch.rand(n, generator=g), -torch.rand(n, generator=g), 0.1 * torch.randn(n, generator=g)
    r = EX.step(c, w, rows, ids.cuda(), tl.cuda(), dist.cuda(), gl.cuda(), ge.cuda())

    w64 = {k: v.detach().double().cpu().requires_grad_() for k, v in w.items()}
    flat = rows["gather_index"]
    total, at, checked = 0.0, 0, 0
    for seq, train in zip(b.seqs, b.trainable):
        here = flat[at:at + len(seq)]
        # the loss position of token t is the packed place of its predecessor (the join copy)
        terms = lambda t: (ids[here[t - 1]].long(), tl[here[t - 1]].double(), float(dist[here[t - 1]]),  # noqa: B023,E731
                           float(gl[here[t - 1]]), float(ge[here[t - 1]]))
        s, seen = _alone(c, w64, seq, train, terms)
        total = total + s
        for t, loss, lp, ent in seen:
            x = here[t]
            for name, want in (("loss", loss), ("logprob", lp), ("entropy", ent)):
                assert abs(float(r[name][x]) - want) <= 8 * 4 * 2.0 ** -8, (name, t, float(r[name][x]), want)
            checked += 1
        at += len(seq)
    assert checked == int(rows["loss_mask"].sum()) > 50
    grads = torch.autograd.grad(total, list(w64.values()))
    for (name, _), want in zip(w64.items(), grads):
        got = r["grad"][name].double().cpu()
        assert float((got - want).norm() / want.norm()) <= 8 * 2.0 ** -8, name
    assert np.isfinite(float(sum(x.float().norm() for x in r["grad"].values())))


def test_example_runs():
    EX.main()

"""The example's policy step (examples/packed_step.py: embedding, projection,
norm and rotation, windowed attention, clipped policy loss, and all of it
back) against the same model in float64 on every sequence alone; and its
activations in 8 bits.

Tolerance: between a weight and its gradient lie at most eight tensors that
are rounded to bf16 once each (half a step 2^-8 relative), so a gradient's
2-norm is off by at most 8 * 2^-8 of itself; besides, the derivative of the
loss by a log-probability follows exp(lp - old) and exp(ref - lp), so it is
off by as much as lp (itself 8 * 4 * 2^-8 at most: eight roundings of logits
below 4).
"""
import numpy as np
import pytest
import torch

from oracle import ckpt as OC
from sft_trie_build_gb300 import workloads as W
from test_gpu_packed_step import EX

pytestmark = pytest.mark.gpu


def _setup():
    c = EX.Config(vocab=96, width=128, n_q_heads=2, n_kv_heads=1, window=20, n_sink=2, kl_coef=0.1, entropy_coef=0.05)
    b = W.random_forest(11, n_roots=3, max_depth=2, len_lo=4, len_hi=40, row_len=256, min_shared=4, vocab=c.vocab)
    return c, b, EX.pack(b), EX.init_weights(c, seed=3)


def _layer(c, w, seq):
    """Log-probabilities of every next token of one sequence, float64."""
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
    return torch.log_softmax((x + torch.einsum("hij,jhd->ihd", p, v).reshape(n, -1) @ w["out"]) @ w["head"], -1)


def test_policy_step_equals_sequences_alone():
    c, b, rows, w = _setup()
    n = rows["token_ids"].size
    g = torch.Generator().manual_seed(5)
    adv, weight = torch.randn(n, generator=g), torch.rand(n, generator=g)
    w64 = {k: v.detach().double().cpu().requires_grad_() for k, v in w.items()}
    flat, at, places, lps, ents = rows["gather_index"], 0, [], [], []
    for seq, train in zip(b.seqs, b.trainable):
        here = flat[at:at + len(seq)]
        lp = _layer(c, w64, seq)
        for t in range(1, len(seq)):
            if train[t]:
                places.append(int(here[t - 1]))            # the packed place of the token before: the join copy
                lps.append(lp[t - 1, int(seq[t])])
                ents.append(-(lp[t - 1].exp() * lp[t - 1]).sum())
        at += len(seq)
    places, lp, ent = torch.tensor(places), torch.stack(lps), torch.stack(ents)
    assert len(places) == int(rows["loss_mask"].sum()) > 50
    # some positions well inside the borders, some well outside
    move = torch.tensor([0.05, -0.05, 1.0, -1.0], dtype=torch.float64)[torch.arange(len(places)) % 4]
    old, ref = torch.zeros(n), torch.zeros(n)
    old[places], ref[places] = (lp - move).detach().float(), (lp + 0.2 * move).detach().float()
    r = EX.policy_step(c, w, rows, old.cuda(), ref.cuda(), adv.cuda(), weight.cuda())

    off = float((r["logprob"].double().cpu()[places] - lp.detach()).abs().max())
    assert off <= 8 * 4 * 2.0 ** -8
    a, ratio = adv.double()[places], torch.exp(lp - old.double()[places])
    x = ref.double()[places] - lp
    kl = torch.expm1(x) - x
    loss = -torch.minimum(ratio * a, ratio.clamp(1 - c.clip_low, 1 + c.clip_high) * a) + c.kl_coef * kl - c.entropy_coef * ent
    got = r["loss"].double().cpu()
    # the loss changes by at most |A| r + kl_coef exp(x) per unit of lp, and by entropy_coef per unit of entropy (off by 8 * 4 * 2^-8)
    tol = ((a.abs() * ratio + c.kl_coef * x.exp()) * np.expm1(off) + c.entropy_coef * 8 * 4 * 2.0 ** -8 + 1e-4).detach()
    assert ((got[places] - loss).abs() <= tol).all()
    rest = torch.ones(n, dtype=torch.bool)
    rest[places] = False
    assert not got[rest].any()
    grads = torch.autograd.grad((loss * weight.double()[places]).sum(), list(w64.values()))
    for (name, _), want in zip(w64.items(), grads):
        d = r["grad"][name].double().cpu() - want
        assert float(d.norm() / want.norm()) <= 8 * 2.0 ** -8 + np.expm1(off), name


def test_activations_in_8_bits_change_their_weights_gradients_only(monkeypatch):
    c, b, rows, w = _setup()
    dz, seen, given = None, {}, []
    plain = EX.Kept.weight_grad

    def weight_grad(self, d_y):
        given.append(d_y.double().cpu())
        return plain(self, d_y)

    monkeypatch.setattr(EX.Kept, "weight_grad", weight_grad)
    for kept in (False, True):
        c.ckpt8 = kept
        f = EX.forward(c, w, rows)
        if dz is None:
            dz = torch.randn(f["logits"].shape, generator=torch.Generator().manual_seed(1)).bfloat16().cuda()
            inputs = {"head": f["y"].x.double().cpu(), "qkv": f["x"].x.double().cpu()}
        seen[kept] = {**EX.backward(c, w, f, dz), "logits": f["logits"]}
    for name in ("logits", "out", "norm_q", "norm_k", "embed"):
        assert torch.equal(seen[False][name], seen[True][name]), name
    # the gradients are those of the restored inputs: exact products, sums of n terms
    for name, d in zip(("head", "qkv"), given[2:]):
        x = torch.from_numpy(OC.keep(inputs[name].numpy()))
        assert not torch.equal(x, inputs[name])
        assert ((seen[True][name].double().cpu() - x.T @ d).abs() <= len(d) * 2.0 ** -22 * (x.abs().T @ d.abs())).all(), name


def test_policy_step_in_8_bits_runs_and_repeats():
    c, b, rows, w = _setup()
    c.ckpt8 = True
    n = rows["token_ids"].size
    old, adv, weight = torch.full((n,), -4.0, device="cuda"), torch.ones(n, device="cuda"), torch.full((n,), 1 / n, device="cuda")
    r = [EX.policy_step(c, w, rows, old, old, adv, weight) for _ in range(2)]
    for name in ("qkv", "head", "embed"):
        assert torch.isfinite(r[0]["grad"][name]).all()
    assert torch.equal(r[0]["loss"], r[1]["loss"]) and torch.equal(r[0]["grad"]["head"], r[1]["grad"]["head"])

"""Training steps of a one-layer model on prefix-tree packed rows.

Sequences that share prefixes are packed once; the layer rotates queries and
keys by the packer's position ids and attends within a window along each
token's own path.  `step` gives the loss positions two terms: distillation
from a teacher's top logits, and a policy term (log-probability of the next
token, entropy).  `policy_step` gives them the clipped policy loss with its KL
and entropy terms.  The gradient of every weight follows from the library's
backward calls; the plain matrix products are torch's.  With `ckpt8` the inputs
of the projection and of the head are kept in 8 bits until the backward pass.

    python examples/packed_step.py
"""
from __future__ import annotations

import os
import sys
from dataclasses import dataclass

import numpy as np
import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from sft_trie_build_gb300 import stp  # noqa: E402
from sft_trie_build_gb300 import workloads as W  # noqa: E402


@dataclass
class Config:
    vocab: int = 512   # with ckpt8 a multiple of 8, as every width of a gradient there
    width: int = 256   # a multiple of 8: token vectors are whole 16 bytes
    n_q_heads: int = 4
    n_kv_heads: int = 2
    head_dim: int = 128
    window: int = 48
    n_sink: int = 4
    teacher_k: int = 16
    top_k: int = 3
    ckpt8: bool = False
    clip_low: float = 0.2
    clip_high: float = 0.28
    kl_coef: float = 0.04
    entropy_coef: float = 0.001


def init_weights(c: Config, seed: int = 0, device="cuda") -> dict:
    g = torch.Generator().manual_seed(seed)
    kv = c.n_q_heads + 2 * c.n_kv_heads

    def w(*shape, std):
        return (torch.randn(*shape, generator=g) * std).to(torch.bfloat16).to(device)

    return {"embed": w(c.vocab, c.width, std=1.0),
            "qkv": w(c.width, kv * c.head_dim, std=c.width ** -0.5),
            "out": w(c.n_q_heads * c.head_dim, c.width, std=(c.n_q_heads * c.head_dim) ** -0.5),
            "head": w(c.width, c.vocab, std=c.width ** -0.5),
            "norm_q": 1 + 0.1 * torch.randn(c.head_dim, generator=g).to(device),
            "norm_k": 1 + 0.1 * torch.randn(c.head_dim, generator=g).to(device)}


def pack(batch: W.SeqBatch) -> dict:
    """Host arrays of the packed rows, and next-token targets (-1 off the loss mask)."""
    tokens, offsets, train = batch.flat()
    plan = stp.stp_pack(tokens, offsets, train, batch.family, row_len=batch.row_len, min_shared=batch.min_shared)
    rows = stp.stp_plan_write(plan)
    nxt = np.roll(rows["token_ids"], -1, axis=1)
    rows["targets"] = np.where(rows["loss_mask"] != 0, nxt, -1).astype(np.int32)
    return rows


def check(**spaces):
    for name, space in spaces.items():
        if stp.stp_device_status(space) != stp.STP_OK:
            raise RuntimeError(f"device check of {name} failed")


class Kept:
    """A layer's input until its weight's gradient is due: in 8 bits, or as it is."""

    def __init__(self, x, ckpt8: bool):
        self.x, self.desc = x, None
        if ckpt8:
            self.desc = stp.ckpt_desc(*x.shape)
            self.x = torch.empty(stp.stp_ckpt_size(self.desc), dtype=torch.uint8, device=x.device)
            stp.stp_ckpt_save(self.desc, x, self.x)

    def weight_grad(self, d_y):
        """x^T d_y, x as it was kept."""
        if self.desc is None:
            return self.x.T @ d_y
        cols = d_y.shape[1]
        dw = torch.empty(self.desc.dim, cols, dtype=torch.float32, device=d_y.device)
        ws = torch.empty(stp.stp_ckpt_wgrad_workspace_size(self.desc, cols), dtype=torch.uint8, device=d_y.device)
        stp.stp_ckpt_wgrad(self.desc, cols, self.x, d_y, d_y.stride(0), False, dw, ws)
        check(weight_gradient=ws)
        return dw


def forward(c: Config, w: dict, rows: dict) -> dict:
    """Logits of every position, and what the backward pass needs."""
    dev = w["embed"].device
    R, T = rows["token_ids"].shape
    n, hq, hkv, d = R * T, c.n_q_heads, c.n_kv_heads, c.head_dim
    width = (hq + 2 * hkv) * d
    tok, pos, se = (torch.from_numpy(rows[k]).to(dev) for k in ("token_ids", "position_ids", "subtree_end"))

    def empty(*shape, dtype=torch.bfloat16):
        return torch.empty(*shape, dtype=dtype, device=dev)

    # token vectors, projection, norm and rotation of q and k, windowed attention
    ed = stp.embed_desc(n, c.vocab, c.width)
    x, embed_ws = empty(n, c.width), empty(stp.stp_embed_workspace_size(ed), dtype=torch.uint8)
    stp.stp_embed_fwd(ed, w["embed"], tok, x, embed_ws)
    qkv = x @ w["qkv"]
    inv_freq = 10000.0 ** (-np.arange(0, d, 2, dtype=np.float64) / d)
    qk = stp.qk_desc(n, hq, hkv, d, q_stride=width, k_stride=width)
    q, k = empty(R, T, hq, d), empty(R, T, hkv, d)
    q_in, k_in = qkv[:, :hq * d], qkv[:, hq * d:(hq + hkv) * d]
    stp.stp_qk_norm_rope_fwd(qk, q_in, k_in, w["norm_q"], w["norm_k"], inv_freq, pos, q, k)
    v = qkv[:, (hq + hkv) * d:].reshape(R, T, hkv, d).contiguous()
    pairs = stp.stp_count_window_tile_pairs(rows["subtree_end"], rows["position_ids"], c.window, c.n_sink)
    attn = stp.Desc(R, T, hq, hkv, d, stp.STP_BF16, d ** -0.5, pairs)
    buf = stp.Buffers(attn, dev)
    o, lse = torch.empty_like(q), empty(R, hq, T, dtype=torch.float32)
    stp.stp_classify_window(attn, c.window, c.n_sink, se, pos, buf.tile_meta)
    stp.stp_attn_window_fwd(attn, c.window, c.n_sink, q, k, v, se, pos, buf.tile_meta, o, lse, buf.fwd_ws)
    y = x + o.view(n, hq * d) @ w["out"]
    logits = y @ w["head"]
    check(tokens=embed_ws, classes=buf.tile_meta, attention=buf.fwd_ws)
    return {"logits": logits, "x": Kept(x, c.ckpt8), "y": Kept(y, c.ckpt8), "tok": tok, "pos": pos, "se": se, "embed": ed,
            "embed_ws": embed_ws, "qk": qk, "inv_freq": inv_freq, "qkv": qkv, "q": q, "k": k, "v": v, "attn": attn, "buf": buf,
            "o": o, "lse": lse}


def backward(c: Config, w: dict, f: dict, dz) -> dict:
    """Gradient of every weight from the gradient dz by the logits."""
    dev = dz.device
    (R, T, hq, d), hkv = f["q"].shape, c.n_kv_heads
    n = R * T

    def empty(*shape, dtype=torch.bfloat16):
        return torch.empty(*shape, dtype=dtype, device=dev)

    grad = {"head": f["y"].weight_grad(dz)}
    dy = dz @ w["head"].T
    grad["out"] = f["o"].view(n, hq * d).T @ dy
    do = (dy @ w["out"].T).view(R, T, hq, d)
    dq, dk, dv = torch.empty_like(f["q"]), torch.empty_like(f["k"]), torch.empty_like(f["v"])
    stp.stp_attn_window_bwd(f["attn"], c.window, c.n_sink, f["q"], f["k"], f["v"], f["o"], f["lse"], do, f["se"], f["pos"],
                            f["buf"].tile_meta, dq, dk, dv, f["buf"].bwd_ws)
    qkv = f["qkv"]
    dqkv = torch.empty_like(qkv)
    grad["norm_q"], grad["norm_k"] = empty(d, dtype=torch.float32), empty(d, dtype=torch.float32)
    ws = empty(stp.stp_qk_norm_rope_workspace_size(f["qk"]), dtype=torch.uint8)
    stp.stp_qk_norm_rope_bwd(f["qk"], qkv[:, :hq * d], qkv[:, hq * d:(hq + hkv) * d], w["norm_q"], w["norm_k"], f["inv_freq"],
                             f["pos"], dq, dk, dqkv[:, :hq * d], dqkv[:, hq * d:(hq + hkv) * d], grad["norm_q"],
                             grad["norm_k"], ws)
    dqkv[:, (hq + hkv) * d:] = dv.view(n, hkv * d)
    grad["qkv"] = f["x"].weight_grad(dqkv)
    dx = dy + dqkv @ w["qkv"].T
    grad["embed"] = empty(c.vocab, c.width, dtype=torch.float32)
    stp.stp_embed_bwd(f["embed"], dx, f["tok"], False, grad["embed"], f["embed_ws"])
    check(backward=f["buf"].bwd_ws, tokens=f["embed_ws"])
    return grad


def step(c: Config, w: dict, rows: dict, teacher_ids, teacher_logits, distill_weight, g_logprob, g_entropy) -> dict:
    """Losses, statistics and the gradient of
        sum over loss positions of distill_weight * distillation + g_logprob * logprob + g_entropy * entropy
    for per-position float32 [N] weights on the device."""
    f = forward(c, w, rows)
    logits, dev = f["logits"], f["logits"].device
    n = logits.shape[0]
    mask, targets = (torch.from_numpy(rows[k]).to(dev) for k in ("loss_mask", "targets"))

    def empty(*shape, dtype=torch.float32):
        return torch.empty(*shape, dtype=dtype, device=dev)

    # the two losses and their gradients on the logits
    dd = stp.distill_desc(n, c.vocab, c.teacher_k)
    loss, loss_lse, dz = empty(n), empty(n), torch.empty_like(logits)
    ws = empty(max(256, stp.stp_distill_workspace_size(dd)), dtype=torch.uint8)
    stp.stp_distill_step(dd, logits, teacher_ids, teacher_logits, mask, distill_weight, loss, loss_lse, dz, ws)
    sd = stp.stats_desc(n, c.vocab, c.top_k)
    logprob, entropy, stat_lse = empty(n), empty(n), empty(n)
    top_id, top_lp = empty(n, c.top_k, dtype=torch.int32), empty(n, c.top_k)
    ws2, dz2 = empty(max(256, stp.stp_token_stats_workspace_size(sd)), dtype=torch.uint8), torch.empty_like(logits)
    stp.stp_token_stats_fwd(sd, logits, targets, logprob, entropy, stat_lse, top_id, top_lp, ws2)
    stp.stp_token_stats_bwd(sd, logits, targets, stat_lse, entropy, g_logprob, g_entropy, dz2)
    grad = backward(c, w, f, dz + dz2)
    check(distillation=ws, statistics=ws2)
    return {"loss": loss, "logprob": logprob, "entropy": entropy, "top_id": top_id, "top_logprob": top_lp, "grad": grad}


def policy_step(c: Config, w: dict, rows: dict, old_logprob, ref_logprob, advantage, weight) -> dict:
    """The clipped policy loss of every loss position, its terms, and the gradient of their sum with the given weights;
    per-position float32 [N] arrays on the device."""
    f = forward(c, w, rows)
    logits, dev = f["logits"], f["logits"].device
    n = logits.shape[0]
    targets = torch.from_numpy(rows["targets"]).to(dev)
    desc = stp.policy_desc(n, c.vocab, stp.STP_BF16, 1.0, c.clip_low, c.clip_high, c.kl_coef, c.entropy_coef)
    out = {k: torch.empty(n, device=dev) for k in ("loss", "logprob", "entropy", "lse", "kl")}
    ws = torch.empty(stp.stp_policy_workspace_size(desc), dtype=torch.uint8, device=dev)
    # the gradient takes the logits' place
    stp.stp_policy_step(desc, logits, targets, old_logprob, ref_logprob, advantage, weight, *out.values(), logits, ws)
    grad = backward(c, w, f, logits)
    check(policy=ws)
    return {**out, "grad": grad}


def main():
    c = Config()
    batch = W.random_forest(4, n_roots=3, max_depth=3, len_lo=8, len_hi=120, row_len=512, min_shared=16, vocab=c.vocab)
    rows = pack(batch)
    w = init_weights(c)
    n = rows["token_ids"].size
    g = torch.Generator(device="cuda").manual_seed(1)
    ids = torch.rand(n, c.vocab, generator=g, device="cuda").topk(c.teacher_k, -1).indices.int()
    tl = torch.randn(n, c.teacher_k, generator=g, device="cuda") * 2
    n_loss = max(1, int(rows["loss_mask"].sum()))
    weight = torch.full((n,), 1.0 / n_loss, device="cuda")
    r = step(c, w, rows, ids, tl, weight, -0.1 * weight, -0.01 * weight)
    print(f"{rows['token_ids'].shape[0]} packed rows, {n_loss} loss positions: distillation {float(r['loss'].sum()) / n_loss:.4f}, "
          f"logprob {float(r['logprob'].sum()) / n_loss:.4f}, entropy {float(r['entropy'].sum()) / n_loss:.4f}")
    for name, x in r["grad"].items():
        print(f"  |d {name}| = {float(x.float().norm()):.5f}")
    # a policy step on the same rows: sampled under these weights, the inputs kept in 8 bits
    c.ckpt8 = True
    adv = torch.randn(n, generator=g, device="cuda")
    r = policy_step(c, w, rows, r["logprob"], r["logprob"] + 0.1 * torch.randn(n, generator=g, device="cuda"), adv, weight)
    print(f"policy loss {float(r['loss'].sum()) / n_loss:.4f}, KL {float(r['kl'].sum()) / n_loss:.4f}")
    for name, x in r["grad"].items():
        print(f"  |d {name}| = {float(x.float().norm()):.5f}")


if __name__ == "__main__":
    main()

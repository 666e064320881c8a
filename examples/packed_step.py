"""One training step of a one-layer model on prefix-tree packed rows.

Sequences that share prefixes are packed once; the layer rotates queries and
keys by the packer's position ids, attends within a window along each token's
own path, and the loss positions get two terms: distillation from a teacher's
top logits, and a policy term (log-probability of the next token, entropy).
The gradient of every weight follows from the library's backward calls; the
plain matrix products are torch's.

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
    vocab: int = 512
    width: int = 256
    n_q_heads: int = 4
    n_kv_heads: int = 2
    head_dim: int = 128
    window: int = 48
    n_sink: int = 4
    teacher_k: int = 16
    top_k: int = 3


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


def step(c: Config, w: dict, rows: dict, teacher_ids, teacher_logits, distill_weight, g_logprob, g_entropy) -> dict:
    """Losses, statistics and the gradient of
        sum over loss positions of distill_weight * distillation + g_logprob * logprob + g_entropy * entropy
    for per-position float32 [N] weights on the device."""
    dev = w["embed"].device
    R, T = rows["token_ids"].shape
    n, hq, hkv, d = R * T, c.n_q_heads, c.n_kv_heads, c.head_dim
    width = (hq + 2 * hkv) * d
    tok, pos, se, mask, targets = (torch.from_numpy(rows[k]).to(dev) for k in
                                   ("token_ids", "position_ids", "subtree_end", "loss_mask", "targets"))
    tok = tok.reshape(-1).long()

    def empty(*shape, dtype=torch.bfloat16):
        return torch.empty(*shape, dtype=dtype, device=dev)

    # forward: projection, norm and rotation of q and k, windowed attention
    x = w["embed"][tok]
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

    # the two losses and their gradients on the logits
    row = lambda: empty(n, dtype=torch.float32)  # noqa: E731
    dd = stp.distill_desc(n, c.vocab, c.teacher_k)
    loss, loss_lse, dz = row(), row(), torch.empty_like(logits)
    ws = empty(max(256, stp.stp_distill_workspace_size(dd)), dtype=torch.uint8)
    stp.stp_distill_step(dd, logits, teacher_ids, teacher_logits, mask, distill_weight, loss, loss_lse, dz, ws)
    sd = stp.stats_desc(n, c.vocab, c.top_k)
    logprob, entropy, stat_lse = row(), row(), row()
    top_id, top_lp = empty(n, c.top_k, dtype=torch.int32), empty(n, c.top_k, dtype=torch.float32)
    ws2, dz2 = empty(max(256, stp.stp_token_stats_workspace_size(sd)), dtype=torch.uint8), torch.empty_like(logits)
    stp.stp_token_stats_fwd(sd, logits, targets, logprob, entropy, stat_lse, top_id, top_lp, ws2)
    stp.stp_token_stats_bwd(sd, logits, targets, stat_lse, entropy, g_logprob, g_entropy, dz2)
    dz = dz + dz2

    # and back through the layer
    grad = {"head": y.T @ dz}
    dy = dz @ w["head"].T
    grad["out"] = o.view(n, hq * d).T @ dy
    do = (dy @ w["out"].T).view(R, T, hq, d)
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    stp.stp_attn_window_bwd(attn, c.window, c.n_sink, q, k, v, o, lse, do, se, pos, buf.tile_meta, dq, dk, dv, buf.bwd_ws)
    dqkv = torch.empty_like(qkv)
    grad["norm_q"], grad["norm_k"] = empty(d, dtype=torch.float32), empty(d, dtype=torch.float32)
    ws3 = empty(stp.stp_qk_norm_rope_workspace_size(qk), dtype=torch.uint8)
    stp.stp_qk_norm_rope_bwd(qk, q_in, k_in, w["norm_q"], w["norm_k"], inv_freq, pos, dq, dk, dqkv[:, :hq * d],
                             dqkv[:, hq * d:(hq + hkv) * d], grad["norm_q"], grad["norm_k"], ws3)
    dqkv[:, (hq + hkv) * d:] = dv.view(n, hkv * d)
    grad["qkv"] = x.T @ dqkv
    dx = (dy + dqkv @ w["qkv"].T).float()
    grad["embed"] = torch.zeros_like(w["embed"], dtype=torch.float32).index_add_(0, tok, dx)
    for name, space in (("classes", buf.tile_meta), ("attention", buf.fwd_ws), ("its backward", buf.bwd_ws),
                        ("distillation", ws), ("statistics", ws2)):
        if stp.stp_device_status(space) != stp.STP_OK:
            raise RuntimeError(f"device check of {name} failed")
    return {"loss": loss, "logprob": logprob, "entropy": entropy, "top_id": top_id, "top_logprob": top_lp, "grad": grad}


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


if __name__ == "__main__":
    main()

"""Four operators around tree attention on packed rows, as cases that can be timed and compared:

  rope     norm of queries and keys for each head and the rotation by position, in one pass (fwd, bwd)
  window   tree attention with a sliding window along each token's own path and a few first tokens that stay
           visible (fwd; step = forward then backward)
  stats    log-probability of a given token, entropy and top alternatives of rows of logits (fwd; step = forward
           then the gradient of both)
  distill  loss against a teacher's top logits (fwd; step = loss and its gradient)

`own` false computes them in elementary torch operations in 32 bits; `own` true calls the library."""
import math

import numpy as np
import torch

own = False

NEG = float("-inf")


def listed():
    return [
        # one decoding step of eight sequences: one token each, far into their contexts
        dict(name="rope-decode", op="rope", dir="fwd", n=8, hq=32, hkv=8, d=128, rot=128, inter=False, dtype="bf16", far=131072),
        # a packed 16384-token row of a training step, from the fused projection
        dict(name="rope-row", op="rope", dir="fwd", n=16384, hq=32, hkv=8, d=128, rot=128, inter=False, dtype="bf16", far=6000),
        # the same row's way back
        dict(name="rope-row-bwd", op="rope", dir="bwd", n=16384, hq=32, hkv=8, d=128, rot=128, inter=False, dtype="bf16", far=6000),
        # a short row while a model is tried out
        dict(name="window-short-step", op="window", dir="step", rows=1, t=512, hq=4, hkv=2, d=128, dtype="bf16", prefix=130, window=100, sinks=4),
        # one group of rollouts over a 5000-token prefix, scored under the current weights
        dict(name="window-group", op="window", dir="fwd", rows=1, t=16384, hq=32, hkv=8, d=128, dtype="bf16", prefix=5000, window=1024, sinks=4),
        # sixteen 4096-token rows of many small groups, trained on
        dict(name="window-rows-step", op="window", dir="step", rows=16, t=4096, hq=16, hkv=8, d=128, dtype="bf16", prefix=650, window=512, sinks=16),
        # eight sequences of a server that reports log-probabilities and alternatives
        dict(name="stats-decode", op="stats", dir="fwd", n=8, v=151936, k=20, dtype="bf16", scale=1.0, skip=0.0, pad=0),
        # every loss position of a group of rollouts, with a few alternatives
        dict(name="stats-group", op="stats", dir="fwd", n=8192, v=151936, k=5, dtype="bf16", scale=1.0, skip=0.0, pad=271),
        # a policy step with an entropy term at a temperature, on rows that hold prompt positions too; an odd vocabulary
        dict(name="stats-step-odd", op="stats", dir="step", n=4096, v=32003, k=1, dtype="fp32", scale=1.25, skip=0.3, pad=0),
        # distillation of a few short answers
        dict(name="distill-short-step", op="distill", dir="step", n=61, v=32000, k=16, dtype="bf16", scale=1.0, skip=0.1),
        # the loss alone, for an evaluation
        dict(name="distill-eval", op="distill", dir="fwd", n=2048, v=151936, k=64, dtype="bf16", scale=0.5, skip=0.0),
        # a training step against a teacher's 64 top logits
        dict(name="distill-step", op="distill", dir="step", n=4096, v=151936, k=64, dtype="bf16", scale=1.0, skip=0.1),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    op = rng.choice(["rope", "window", "stats", "distill"])
    dtype = rng.choice(["bf16", "bf16", "fp32"])
    if op == "rope":
        d = rng.choice([32, 64, 80, 96, 128, 128, 192, 256])
        rot = rng.choice([d, d, 16 * rng.randint(1, d // 16)])
        hkv = rng.randint(1, 8)
        hq = hkv * rng.randint(1, 8)
        most = 16384 * 40 * 128 // ((hq + hkv) * d * (2 if dtype == "fp32" else 1))
        return dict(op=op, dir=rng.choice(["fwd", "bwd"]), n=_log(rng, 1, min(most, 40000)), hq=hq, hkv=hkv, d=d, rot=rot,
                    inter=rng.random() < 0.3, dtype=dtype, far=_log(rng, 1000, 1000000))
    if op == "window":
        fp32 = dtype == "fp32"
        t = 128 * _log(rng, 1, 8 if fp32 else 64)
        rows = _log(rng, 1, max(1, (2048 if fp32 else 32768) // t))
        hkv = rng.choice([1, 2, 4] if fp32 else [1, 2, 4, 8])
        hq = hkv * rng.choice([1, 2] if fp32 else [1, 2, 3, 4, 8])
        return dict(op=op, dir=rng.choice(["fwd", "step"]), rows=rows, t=t, hq=min(hq, 32), hkv=hkv,
                    d=rng.choice([64, 128]) if fp32 else 128, dtype=dtype, prefix=rng.randint(8, t // 2),
                    window=_log(rng, 1, t), sinks=rng.choice([0, 1, 4, 64, rng.randint(0, 200)]))
    v = _log(rng, 100, 200000)
    most = (4096 if op == "distill" else 8192) * 151936 // (v * (2 if dtype == "fp32" else 1))
    n = _log(rng, 1, max(1, min(most // 2, 20000)))
    case = dict(op=op, dir=rng.choice(["fwd", "step"]), n=n, v=v, dtype=dtype, scale=rng.choice([1.0, 1.0, 0.7, 1.25]),
                skip=rng.choice([0.0, 0.2, 0.9]))
    if op == "stats":
        case |= dict(k=rng.randint(1, 32), pad=rng.choice([0, 0, rng.randint(1, max(1, v // 3))]))
    else:
        case |= dict(k=min(v // 2, _log(rng, 1, 256)))
    return case


def _dtype(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def _bytes(case):
    return 2 if case["dtype"] == "bf16" else 4


# ---------------------------------------------------------------------------------------------- inputs

def _tree(case, seed):
    """subtree_end and position_ids, int32 [rows, t]: in each row one root of about `prefix` tokens with branches of
    random lengths, some of which branch again, further small trees while the row has room, then pads."""
    rng = np.random.default_rng(seed)
    rows, t = case["rows"], case["t"]
    se, pos = np.tile(np.arange(t, dtype=np.int32), (rows, 1)), np.zeros((rows, t), np.int32)

    def lay(r, x, depth, length, level, limit):
        """One segment at x and what is below it; returns where it ends."""
        length = min(length, limit - x)
        pos[r, x:x + length] = np.arange(depth, depth + length)
        at = x + length
        if level > 0:
            for _ in range(int(rng.integers(2, 9 if level > 1 else 4))):
                if at < limit:
                    below = int(rng.integers(1, 1 + max(1, case["prefix"] // 4)))
                    at = lay(r, at, depth + length, below, level - 1 if rng.random() < 0.4 else 0, limit)
        se[r, x:x + length] = at - 1
        return at

    for r in range(rows):
        used = t - int(rng.integers(0, 1 + t // 16))
        x = lay(r, 0, 0, case["prefix"], 2, used)
        while x < used:
            x = lay(r, x, 0, int(rng.integers(1, 1 + case["prefix"])), 2, used)
    return se, pos


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = _dtype(case)

    def normal(*shape, std=1.0, dtype=dt):
        return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32).mul_(std).to(dtype)

    s = {"case": case}
    if case["op"] == "rope":
        n, hq, hkv, d = case["n"], case["hq"], case["hkv"], case["d"]
        # the fused projection's output: a token's queries, keys and values in one row
        s["qkv"] = normal(n, (hq + 2 * hkv) * d, std=1.5)
        s["w_q"], s["w_k"] = (1 + normal(d, std=0.2, dtype=torch.float32) for _ in range(2))
        s["pos"] = torch.randint(0, case["far"], (n,), generator=g, device="cuda", dtype=torch.int32)
        s["inv_freq"] = 10000.0 ** (-np.arange(0, case["rot"], 2, dtype=np.float64) / case["rot"])
        if case["dir"] == "bwd":
            s["dq"], s["dk"] = normal(n, hq, d), normal(n, hkv, d)
    elif case["op"] == "window":
        rows, t, hq, hkv, d = case["rows"], case["t"], case["hq"], case["hkv"], case["d"]
        s["se_host"], s["pos_host"] = _tree(case, seed)
        s["se"], s["pos"] = torch.from_numpy(s["se_host"]).cuda(), torch.from_numpy(s["pos_host"]).cuda()
        s["q"] = normal(rows, t, hq, d, std=0.5)
        s["k"], s["v"] = (normal(rows, t, hkv, d, std=0.5) for _ in range(2))
        if case["dir"] == "step":
            s["do"] = normal(rows, t, hq, d)
    else:
        n, v, k = case["n"], case["v"], case["k"]
        z = torch.randn(n, v, generator=g, device="cuda", dtype=torch.float32).mul_(2.0)
        likely = torch.randint(0, v, (n, 1), generator=g, device="cuda")
        if case["op"] == "stats":
            # a model's rows: one likely token each; columns that pad the vocabulary are -inf
            z.scatter_add_(1, likely, 5 + normal(n, 1, std=3.0, dtype=torch.float32))
            if case["pad"]:
                z[:, v - case["pad"]:] = NEG
            s["targets"] = torch.where(torch.rand(n, generator=g, device="cuda") < 0.6, likely[:, 0],
                                       torch.randint(0, v - case["pad"], (n,), generator=g, device="cuda")).to(torch.int32)
            s["targets"][torch.rand(n, generator=g, device="cuda") < case["skip"]] = -1
            if case["dir"] == "step":
                s["d_logprob"], s["d_entropy"] = normal(n, dtype=torch.float32), normal(n, std=0.01, dtype=torch.float32)
        else:
            # the teacher's k ids of a row, which the student finds likely too, and the teacher's logits there
            ids = (likely + torch.arange(k, device="cuda") * (v // k)) % v
            bump = torch.linspace(9, 0, k, device="cuda") + normal(n, k, std=1.0, dtype=torch.float32)
            z.scatter_add_(1, ids, bump)
            s["teacher_logits"] = bump * 1.1 + normal(n, k, std=0.5, dtype=torch.float32)
            ids[torch.rand(n, k, generator=g, device="cuda") < 0.03] = -1
            s["teacher_ids"] = ids.to(torch.int32)
            s["mask"] = (torch.rand(n, generator=g, device="cuda") >= case["skip"]).to(torch.uint8)
            if case["dir"] == "step":
                s["d_loss"] = (0.5 + torch.rand(n, generator=g, device="cuda")) / n
        s["logits"] = z.to(dt)
    if own:
        _keep(s)
    return s


def _keep(s):
    """What a program that uses the library keeps beside its inputs: descriptors, output buffers and workspaces."""
    from sft_trie_build_gb300 import stp

    case, dt = s["case"], _dtype(s["case"])
    code = stp.STP_BF16 if case["dtype"] == "bf16" else stp.STP_FP32

    def empty(*shape, dtype=dt):
        return torch.empty(*shape, dtype=dtype, device="cuda")

    def space(size):
        return empty(max(256, size), dtype=torch.uint8)

    if case["op"] == "rope":
        n, hq, hkv, d = case["n"], case["hq"], case["hkv"], case["d"]
        width = (hq + 2 * hkv) * d
        s["desc"] = stp.qk_desc(n, hq, hkv, d, case["rot"], case["inter"], code, q_stride=width, k_stride=width)
        if case["dir"] == "fwd":
            s["out"] = empty(n, hq, d), empty(n, hkv, d)
        else:
            s["dqkv"] = torch.zeros_like(s["qkv"])
            s["dw"] = empty(d, dtype=torch.float32), empty(d, dtype=torch.float32)
            s["ws"] = space(stp.stp_qk_norm_rope_workspace_size(s["desc"]))
    elif case["op"] == "window":
        rows, t, hq, hkv, d = case["rows"], case["t"], case["hq"], case["hkv"], case["d"]
        pairs = stp.stp_count_window_tile_pairs(s["se_host"], s["pos_host"], case["window"], case["sinks"])
        s["desc"] = stp.Desc(rows, t, hq, hkv, d, code, d ** -0.5, pairs)
        meta, fwd, bwd = stp.stp_workspace_size(s["desc"])
        s["meta"], s["ws"] = space(meta), space(fwd)
        s["o"], s["lse"] = torch.empty_like(s["q"]), empty(rows, hq, t, dtype=torch.float32)
        if case["dir"] == "step":
            s["ws_bwd"] = space(bwd)
            s["dqkv"] = tuple(torch.empty_like(s[x]) for x in "qkv")
    else:
        n, v, k = case["n"], case["v"], case["k"]

        def row():
            return empty(n, dtype=torch.float32)

        if case["op"] == "stats":
            s["desc"] = stp.stats_desc(n, v, k, code, case["scale"])
            s["out"] = row(), row(), row(), empty(n, k, dtype=torch.int32), empty(n, k, dtype=torch.float32)
            s["ws"] = space(stp.stp_token_stats_workspace_size(s["desc"]))
        else:
            s["desc"] = stp.distill_desc(n, v, k, code, case["scale"])
            s["out"] = row(), row()
            s["ws"] = space(stp.stp_distill_workspace_size(s["desc"]))
        if case["dir"] == "step":
            s["dz"] = torch.empty_like(s["logits"])


# ---------------------------------------------------------------------------------------------- one pass

def run(s):
    return (_run_own if own else _run_plain)(s)


def _run_own(s):
    from sft_trie_build_gb300 import stp

    case = s["case"]
    if case["op"] == "rope":
        hq, hkv, d = case["hq"], case["hkv"], case["d"]
        q, k = s["qkv"][:, :hq * d], s["qkv"][:, hq * d:]
        if case["dir"] == "fwd":
            stp.stp_qk_norm_rope_fwd(s["desc"], q, k, s["w_q"], s["w_k"], s["inv_freq"], s["pos"], *s["out"])
            return {"q": s["out"][0], "k": s["out"][1]}
        dxq, dxk = s["dqkv"][:, :hq * d], s["dqkv"][:, hq * d:(hq + hkv) * d]
        stp.stp_qk_norm_rope_bwd(s["desc"], q, k, s["w_q"], s["w_k"], s["inv_freq"], s["pos"], s["dq"], s["dk"], dxq, dxk,
                                 *s["dw"], s["ws"])
        return {"dxq": dxq, "dxk": dxk, "dw_q": s["dw"][0], "dw_k": s["dw"][1]}
    if case["op"] == "window":
        w, m = case["window"], case["sinks"]
        stp.stp_classify_window(s["desc"], w, m, s["se"], s["pos"], s["meta"])
        stp.stp_attn_window_fwd(s["desc"], w, m, s["q"], s["k"], s["v"], s["se"], s["pos"], s["meta"], s["o"], s["lse"], s["ws"])
        if case["dir"] == "fwd":
            return {"o": s["o"], "lse": s["lse"]}
        stp.stp_attn_window_bwd(s["desc"], w, m, s["q"], s["k"], s["v"], s["o"], s["lse"], s["do"], s["se"], s["pos"], s["meta"],
                                *s["dqkv"], s["ws_bwd"])
        return {"o": s["o"], "lse": s["lse"], "dq": s["dqkv"][0], "dk": s["dqkv"][1], "dv": s["dqkv"][2]}
    if case["op"] == "stats":
        stp.stp_token_stats_fwd(s["desc"], s["logits"], s["targets"], *s["out"], s["ws"])
        out = dict(zip(("logprob", "entropy", "lse", "top_id", "top_logprob"), s["out"]))
        if case["dir"] == "step":
            stp.stp_token_stats_bwd(s["desc"], s["logits"], s["targets"], out["lse"], out["entropy"], s["d_logprob"],
                                    s["d_entropy"], s["dz"])
            out["dz"] = s["dz"]
        return out
    if case["dir"] == "fwd":
        stp.stp_distill_fwd(s["desc"], s["logits"], s["teacher_ids"], s["teacher_logits"], s["mask"], *s["out"], s["ws"])
        return {"loss": s["out"][0], "lse": s["out"][1]}
    stp.stp_distill_step(s["desc"], s["logits"], s["teacher_ids"], s["teacher_logits"], s["mask"], s["d_loss"], *s["out"],
                         s["dz"], s["ws"])
    return {"loss": s["out"][0], "lse": s["out"][1], "dz": s["dz"]}


def _run_plain(s):
    return {"rope": _rope, "window": _window, "stats": _stats, "distill": _distill}[s["case"]["op"]](s)


def _turn(x, cos, sin, inter):
    """Rotates the first 2 * cos.shape[-1] channels of x [n, h, d]: pairs (c, c + half), or (2c, 2c + 1) if `inter`."""
    half = cos.shape[-1]
    if inter:
        a, b = x[..., 0:2 * half:2], x[..., 1:2 * half:2]
        y = torch.stack((a * cos - b * sin, a * sin + b * cos), -1).flatten(-2)
    else:
        a, b = x[..., :half], x[..., half:2 * half]
        y = torch.cat((a * cos - b * sin, a * sin + b * cos), -1)
    return torch.cat((y, x[..., 2 * half:]), -1)


def _rope(s):
    case = s["case"]
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    angle = s["pos"].double()[:, None, None] * torch.from_numpy(s["inv_freq"]).cuda()  # far positions need 64 bits
    cos, sin = angle.cos().float(), angle.sin().float()
    x = s["qkv"].view(case["n"], hq + 2 * hkv, d)[:, :hq + hkv].float()
    w = torch.cat((s["w_q"].expand(hq, d), s["w_k"].expand(hkv, d)))
    r = torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6)
    if case["dir"] == "fwd":
        y = _turn(x * r * w, cos, sin, case["inter"]).to(s["qkv"].dtype)
        return {"q": y[:, :hq].contiguous(), "k": y[:, hq:].contiguous()}
    dy = _turn(torch.cat((s["dq"], s["dk"]), 1).float(), cos, -sin, case["inter"])
    xn = x * r
    dw = (dy * xn).sum(0)
    dn = dy * w
    dx = (r * (dn - xn * (dn * xn).mean(-1, keepdim=True))).to(s["qkv"].dtype)
    return {"dxq": dx[:, :hq].flatten(1), "dxk": dx[:, hq:].flatten(1), "dw_q": dw[:hq].sum(0), "dw_k": dw[hq:].sum(0)}


def _window(s):
    case = s["case"]
    rows, t, hq, hkv, d = case["rows"], case["t"], case["hq"], case["hkv"], case["d"]
    i, j = torch.arange(t, device="cuda")[:, None], torch.arange(t, device="cuda")[None]
    see = (j <= i) & (s["se"][:, None] >= i)
    see &= (s["pos"][:, :, None] - s["pos"][:, None] < case["window"]) | (s["pos"][:, None] < case["sinks"])
    see = see[:, None]                                                     # [rows, 1, t, t]
    o, lse = torch.empty_like(s["q"]), torch.empty(rows, hq, t, device="cuda")
    dq, dk, dv = (torch.empty_like(s[x]) for x in "qkv")
    each = hq // hkv
    some = max(1, min(hkv, (1 << 31) // (rows * t * t * each)))            # kv heads at a time, as memory allows
    for g in range(0, hkv, some):
        h, n = slice(g * each, (g + some) * each), min(some, hkv - g)
        q = s["q"][:, :, h].float().transpose(1, 2)                        # [rows, heads, t, d]
        k, v = (s[x][:, :, g:g + some].float().transpose(1, 2).repeat_interleave(each, 1) for x in "kv")
        a = (q @ k.transpose(2, 3)).mul_(d ** -0.5).masked_fill_(~see, NEG)
        top = a.amax(-1, keepdim=True)
        p = a.sub_(top).exp_()
        z = p.sum(-1, keepdim=True)
        p = p.div_(z)
        y = p @ v
        o[:, :, h], lse[:, h] = y.transpose(1, 2).to(o.dtype), (top + z.log())[..., 0]
        if case["dir"] == "step":
            do = s["do"][:, :, h].float().transpose(1, 2)
            ds = (do @ v.transpose(2, 3)).sub_((do * y).sum(-1, keepdim=True)).mul_(p)
            dq[:, :, h] = (ds @ k * d ** -0.5).transpose(1, 2).to(dq.dtype)
            for out, grad in ((dk, ds.transpose(2, 3) @ q * d ** -0.5), (dv, p.transpose(2, 3) @ do)):
                out[:, :, g:g + some] = grad.view(rows, n, each, t, d).sum(2).transpose(1, 2).to(out.dtype)
    return {"o": o, "lse": lse, "dq": dq, "dk": dk, "dv": dv} if case["dir"] == "step" else {"o": o, "lse": lse}


def _lse(z):
    top = z.amax(-1, keepdim=True)
    return top + (z - top).exp().sum(-1, keepdim=True).log()


def _stats(s):
    case, raw = s["case"], s["logits"].float()
    z = raw * case["scale"]
    on = (s["targets"] >= 0)[:, None]
    at = s["targets"].clamp(min=0).long()[:, None]
    lse = _lse(z)
    lp = z - lse
    p = lp.exp()
    lp0 = lp.masked_fill(lp == NEG, 0)                                       # 0 ln 0 = 0
    ent = -(p * lp0).sum(-1, keepdim=True)
    # the k largest, ties to the lowest id: one whole number orders by value, then by id
    bits = raw.add(0.0).view(torch.int32)
    key = torch.where(bits < 0, bits ^ 0x7fffffff, bits).long() * (1 << 24) - torch.arange(case["v"], device="cuda")
    ids = key.topk(min(case["k"], case["v"]), -1).indices
    top = lp.gather(1, ids)
    ids = ids.masked_fill((top == NEG) | ~on, -1).int()
    top = top.masked_fill(ids < 0, NEG)
    out = {"logprob": lp.gather(1, at).masked_fill(~on, 0)[:, 0], "entropy": ent.masked_fill(~on, 0)[:, 0],
           "lse": lse.masked_fill(~on, 0)[:, 0], "top_id": ids, "top_logprob": top}
    if case["dir"] == "step":
        hot = torch.zeros_like(p).scatter_(1, at, 1.0)
        dz = s["d_logprob"][:, None] * (hot - p) - s["d_entropy"][:, None] * p * (lp0 + ent)
        out["dz"] = (dz * case["scale"]).masked_fill(~on, 0).to(s["logits"].dtype)
    return out


def _distill(s):
    case = s["case"]
    z = s["logits"].float() * case["scale"]
    there = s["teacher_ids"] >= 0
    on = (s["mask"] != 0) & there.any(-1)
    at = s["teacher_ids"].clamp(min=0).long()
    a = (s["teacher_logits"] * case["scale"]).masked_fill(~there, NEG)
    lq = a - _lse(a)
    q = lq.exp().masked_fill(~there, 0)
    lse = _lse(z)
    loss = (q * (lq - (z.gather(1, at) - lse)).masked_fill(~there, 0)).sum(-1)
    out = {"loss": loss.masked_fill(~on, 0), "lse": lse[:, 0].masked_fill(~on, 0)}
    if case["dir"] == "step":
        dz = (z - lse).exp().scatter_add_(1, at, -q)
        out["dz"] = (dz * (s["d_loss"] * case["scale"])[:, None]).masked_fill(~on[:, None], 0).to(s["logits"].dtype)
    return out


# ---------------------------------------------------------------------------------------------- what a pass needs

def work(case):
    b = _bytes(case)
    if case["op"] == "rope":
        x = case["n"] * (case["hq"] + case["hkv"]) * case["d"]
        return {"bytes": x * b * (2 if case["dir"] == "fwd" else 3) + 4 * case["n"] + 8 * case["d"] * (1 if case["dir"] == "fwd" else 2),
                "flops": x * (8 if case["dir"] == "fwd" else 18)}
    if case["op"] == "window":
        se, pos = _tree(case, 0)
        # a query at depth p sees the `window` tokens up to itself and the sinks before them
        p = np.concatenate([pos[r] for r in range(case["rows"])]).astype(np.int64) + 1
        seen = np.minimum(p, case["window"])
        pairs = int((seen + np.minimum(p - seen, case["sinks"])).sum()) * case["hq"]
        tokens = case["rows"] * case["t"]
        x, y = tokens * case["hq"] * case["d"] * b, tokens * case["hkv"] * case["d"] * b
        step = case["dir"] == "step"
        return {"bytes": 2 * x + 2 * y + 4 * tokens * case["hq"] + 8 * tokens + (2 * x + 2 * y if step else 0),
                "flops": pairs * case["d"] * (14 if step else 4)}
    rows = case["n"] * (1 - case["skip"])
    step = case["dir"] == "step"
    z = rows * case["v"] * b + (case["n"] * case["v"] * b if step else 0)
    return {"bytes": int(z + case["n"] * (16 + 8 * case["k"])), "flops": int(rows * case["v"] * (12 if step else 6))}


# ---------------------------------------------------------------------------------------------- 64 bits

def exact(case, seed):
    keep = globals()["own"]
    globals()["own"] = False
    try:
        s = prepare(case, seed)
    finally:
        globals()["own"] = keep
    return {"rope": _rope64, "window": _window64, "stats": _stats64, "distill": _distill64}[case["op"]](s)


def _rope64(s):
    case = s["case"]
    n, hq, hkv, d, rot = (case[x] for x in ("n", "hq", "hkv", "d", "rot"))
    x = s["qkv"].view(n, -1, d).double()
    unit = torch.polar(torch.ones((), dtype=torch.float64, device="cuda"),
                       torch.outer(s["pos"].double(), torch.from_numpy(s["inv_freq"]).cuda()))[:, None]

    def forward(x, w):
        y = w * x / (x.square().mean(-1, keepdim=True) + 1e-6).sqrt()
        c, rest = y[..., :rot], y[..., rot:]
        pair = c.unflatten(-1, (rot // 2, 2)) if case["inter"] else c.unflatten(-1, (2, rot // 2)).transpose(-1, -2)
        turned = torch.view_as_real(torch.view_as_complex(pair.contiguous()) * unit)
        c = turned.flatten(-2) if case["inter"] else turned.transpose(-1, -2).flatten(-2)
        return torch.cat((c, rest), -1)

    out = {}
    for name, heads, w, dy in (("q", slice(0, hq), s["w_q"], s.get("dq")), ("k", slice(hq, hq + hkv), s["w_k"], s.get("dk"))):
        x0, w0 = x[:, heads].clone().requires_grad_(), w.double().requires_grad_()
        y = forward(x0, w0)
        if dy is None:
            out[name] = y.detach()
        else:
            dx, dw = torch.autograd.grad(y, (x0, w0), dy.double())
            out["dx" + name], out["dw_" + name] = dx.flatten(1), dw
    return out


def _window64(s):
    case = s["case"]
    rows, t, hq, hkv, d = case["rows"], case["t"], case["hq"], case["hkv"], case["d"]
    each, c = hq // hkv, d ** -0.5
    o, lse = torch.zeros(rows, t, hq, d, dtype=torch.float64, device="cuda"), torch.zeros(rows, hq, t, dtype=torch.float64, device="cuda")
    dq, dk, dv = (torch.zeros(s[x].shape, dtype=torch.float64, device="cuda") for x in "qkv")
    for r in range(rows):
        se, pos = s["se"][r].long(), s["pos"][r].long()
        for a in range(0, t, 256):
            i = torch.arange(a, min(t, a + 256), device="cuda")
            j = torch.arange(int(i[-1]) + 1, device="cuda")
            hid = (j[None] > i[:, None]) | (se[j][None] < i[:, None])
            hid |= (pos[i][:, None] - pos[j][None] >= case["window"]) & (pos[j][None] >= case["sinks"])
            j = torch.nonzero(~hid.all(0))[:, 0]
            hid = hid[:, j]
            q = s["q"][r, i].double().view(len(i), hkv, each, d)
            k, v = s["k"][r, j].double(), s["v"][r, j].double()
            x = torch.einsum("ighd,jgd->ghij", q, k) * c
            x = x.masked_fill(hid, NEG)
            z = torch.logsumexp(x, -1, keepdim=True)
            p = torch.exp(x - z)
            y = torch.einsum("ghij,jgd->ighd", p, v)
            o[r, i], lse[r, :, i] = y.reshape(len(i), hq, d), z.reshape(hq, len(i))
            if case["dir"] == "step":
                do = s["do"][r, i].double().view(len(i), hkv, each, d)
                dx = p * (torch.einsum("ighd,jgd->ghij", do, v) - torch.einsum("ighd,ighd->ghi", do, y)[..., None]) * c
                dq[r, i] = torch.einsum("ghij,jgd->ighd", dx, k).reshape(len(i), hq, d)
                dk[r].index_add_(0, j, torch.einsum("ghij,ighd->jgd", dx, q))
                dv[r].index_add_(0, j, torch.einsum("ghij,ighd->jgd", p, do))
    return {"o": o, "lse": lse, "dq": dq, "dk": dk, "dv": dv} if case["dir"] == "step" else {"o": o, "lse": lse}


def _blocks(n, v):
    size = max(1, (1 << 28) // v)
    return [slice(a, min(n, a + size)) for a in range(0, n, size)]


def _stats64(s):
    case = s["case"]
    out = []
    for b in _blocks(case["n"], case["v"]):
        z = s["logits"][b].double().requires_grad_()
        y = torch.log_softmax(z * case["scale"], -1)
        skip = s["targets"][b] < 0
        lp = y.gather(1, s["targets"][b].clamp(min=0).long()[:, None])[:, 0]
        safe = torch.where(torch.isinf(y), torch.zeros_like(y), y)
        ent = -(torch.exp(y) * safe).sum(-1)
        lse = torch.logsumexp(z.detach() * case["scale"], -1)
        k = min(case["k"], case["v"])
        top = y.detach().topk(k, -1).values.masked_fill(skip[:, None], NEG)
        got = {"logprob": lp.detach().masked_fill(skip, 0), "entropy": ent.detach().masked_fill(skip, 0),
               "lse": lse.masked_fill(skip, 0), "top_logprob": top}
        if case["dir"] == "step":
            total = (s["d_logprob"][b].double() * lp + s["d_entropy"][b].double() * ent).masked_fill(skip, 0).sum()
            dz, = torch.autograd.grad(total, z)
            got["dz"] = dz.nan_to_num(0.0)
        out.append(got)
    out = {x: torch.cat([g[x] for g in out]) for x in out[0]}
    return {**out, "top_id": None}


def _distill64(s):
    case = s["case"]
    out = []
    for b in _blocks(case["n"], case["v"]):
        z = s["logits"][b].double().requires_grad_()
        y = torch.log_softmax(z * case["scale"], -1)
        ids = s["teacher_ids"][b].long()
        a = torch.where(ids < 0, torch.full_like(ids, NEG, dtype=torch.float64), s["teacher_logits"][b].double() * case["scale"])
        live = (s["mask"][b] != 0) & (ids >= 0).any(-1)
        lq = torch.log_softmax(torch.where(live[:, None], a, torch.zeros_like(a)), -1)
        lq = torch.where(ids < 0, torch.zeros_like(lq), lq)
        q = torch.where(ids < 0, torch.zeros_like(lq), lq.exp())
        loss = (q * (lq - y.gather(1, ids.clamp(min=0)))).sum(-1)
        loss = torch.where(live, loss, torch.zeros_like(loss))
        got = {"loss": loss.detach(), "lse": torch.logsumexp(z.detach() * case["scale"], -1).masked_fill(~live, 0)}
        if case["dir"] == "step":
            got["dz"], = torch.autograd.grad((loss * s["d_loss"][b].double()).sum(), z)
        out.append(got)
    return {x: torch.cat([g[x] for g in out]) for x in out[0]}

"""Both ends of a training step on packed rows and what is kept in between, as cases that can be timed and compared:

  embed   token vectors from a table, scaled, and the table's gradient, summed by token (fwd, bwd)
  policy  clipped policy loss with a KL term and an entropy term on rows of logits (fwd; step = loss and its gradient)
  ckpt    activations kept in 8 bits, with a scale for 32 channels of a token (keep = store, then restore)
  grad    weight gradient of a projection, from its kept input and its output's gradient

`own` false computes them in elementary torch operations in 32 bits; `own` true calls the library."""
import math

import numpy as np
import torch

own = False

NEG = float("-inf")


def listed():
    return [
        # a short row while a model is tried out
        dict(name="embed-short", op="embed", dir="fwd", n=512, v=512, c=256, dtype="bf16", scale=1.0, skip=0.0),
        # a packed 16384-token row enters the model, scaled by the root of the width
        dict(name="embed-row", op="embed", dir="fwd", n=16384, v=151936, c=4096, dtype="bf16", scale=64.0, skip=0.0),
        # the same row's way back, over a smaller table
        dict(name="embed-row-bwd", op="embed", dir="bwd", n=16384, v=32000, c=4096, dtype="bf16", scale=64.0, skip=0.0),
        # about sixteen 4096-token rows at once; an odd vocabulary, pads that have no token
        dict(name="embed-rows-odd-bwd", op="embed", dir="bwd", n=65531, v=32003, c=1000, dtype="fp32", scale=1.0, skip=0.05),
        # the loss positions of a few short answers
        dict(name="policy-short-step", op="policy", dir="step", n=61, v=32000, dtype="bf16", scale=1.0, skip=0.1, kl=0.04, ent=0.0),
        # the loss alone of a batch at a temperature, on rows that hold prompt positions too; an odd vocabulary
        dict(name="policy-eval-odd", op="policy", dir="fwd", n=8192, v=32003, dtype="fp32", scale=1.25, skip=0.3, kl=0.0, ent=0.01),
        # a training step over a group of rollouts, with all terms
        dict(name="policy-step", op="policy", dir="step", n=4096, v=151936, dtype="bf16", scale=1.0, skip=0.1, kl=0.04, ent=0.001),
        # a small batch of an odd width, in 32 bits
        dict(name="ckpt-odd", op="ckpt", n=1021, c=1000, dtype="fp32"),
        # a layer's input over a packed 16384-token row
        dict(name="ckpt-row", op="ckpt", n=16384, c=4096, dtype="bf16"),
        # a short row while a model is tried out
        dict(name="grad-short", op="grad", n=512, c=256, m=1024),
        # a narrow projection over many tokens, of odd sizes
        dict(name="grad-rows-odd", op="grad", n=65531, c=1000, m=523),
        # the fused query, key and value projection over a packed 16384-token row
        dict(name="grad-row", op="grad", n=16384, c=4096, m=6144),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    op = rng.choice(["embed", "policy", "ckpt", "grad"])
    dtype = rng.choice(["bf16", "bf16", "fp32"])
    wide = 2 if dtype == "fp32" else 1
    if op == "embed":
        c = 8 * _log(rng, 1, 1024)
        return dict(op=op, dir=rng.choice(["fwd", "bwd"]), n=_log(rng, 1, min(70000, 16384 * 4096 // (c * wide))),
                    v=_log(rng, 1, min(160000, 32000 * 4096 // c)), c=c, dtype=dtype, scale=rng.choice([1.0, 0.5, c ** 0.5]),
                    skip=rng.choice([0.0, 0.1, 0.9]))
    if op == "policy":
        v = _log(rng, 100, 200000)
        return dict(op=op, dir=rng.choice(["fwd", "step"]), n=_log(rng, 1, min(20000, max(1, 2048 * 151936 // (v * wide)))), v=v,
                    dtype=dtype, scale=rng.choice([1.0, 1.0, 0.7, 1.25]), skip=rng.choice([0.0, 0.2, 0.9]),
                    kl=rng.choice([0.0, 0.04, 0.5]), ent=rng.choice([0.0, 0.001, 0.01]))
    if op == "ckpt":
        c = _log(rng, 1, 8192)
        return dict(op=op, n=_log(rng, 1, min(70000, 16384 * 4096 // (c * wide))), c=c, dtype=dtype)
    c, m = _log(rng, 1, 8192), _log(rng, 1, 8192)
    return dict(op=op, n=_log(rng, 1, min(70000, max(1, 16384 * 4096 * 4096 // (c * m)))), c=c, m=m)


def _dtype(case):
    return torch.float32 if case.get("dtype") == "fp32" else torch.bfloat16


def _bytes(case):
    return 4 if case.get("dtype") == "fp32" else 2


# ---------------------------------------------------------------------------------------------- inputs

def _tokens(case, seed):
    """Token ids int32 [n]: few tokens make up much of a text (a token's share falls with its rank); -1 where a
    position has none."""
    rng = np.random.default_rng(seed)
    v, n = case["v"], case["n"]
    rank = np.minimum(np.floor(np.exp(rng.random(n) * math.log(v + 1))).astype(np.int64), v) - 1
    tok = (rank * 7919 + 11) % v if v % 7919 else rank
    tok[rng.random(n) < case["skip"]] = -1
    return tok.astype(np.int32)


LOW, HIGH = 0.2, 0.28   # how far a policy step may move a ratio


def _inputs(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = _dtype(case)

    def normal(*shape, std=1.0, dtype=dt):
        return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32).mul_(std).to(dtype)

    s = {"case": case}
    n = case["n"]
    if case["op"] == "embed":
        s["tok"] = torch.from_numpy(_tokens(case, seed)).cuda()
        if case["dir"] == "fwd":
            s["table"] = normal(case["v"], case["c"], std=0.02)
        else:
            s["d_out"] = normal(n, case["c"])
    elif case["op"] == "policy":
        v = case["v"]
        z = normal(n, v, std=2.0, dtype=torch.float32)
        likely = torch.randint(0, v, (n, 1), generator=g, device="cuda")
        z.scatter_add_(1, likely, 5 + normal(n, 1, std=3.0, dtype=torch.float32))
        s["logits"] = z.to(dt)
        # most tokens were sampled from a policy near this one
        t = torch.where(torch.rand(n, 1, generator=g, device="cuda") < 0.7, likely, torch.randint(0, v, (n, 1), generator=g, device="cuda"))
        z = s["logits"].float() * case["scale"]
        lp = (z.gather(1, t) - _lse(z))[:, 0]
        del z
        move = normal(n, std=0.15, dtype=torch.float32)
        for edge in (math.log(1 - LOW), math.log(1 + HIGH)):   # the gradient jumps there: no value next to it
            move = torch.where((move - edge).abs() < 2e-3, move + 4e-3, move)
        s["old"] = lp - move
        s["ref"] = lp + normal(n, std=0.3, dtype=torch.float32) if case["kl"] else None
        s["adv"] = normal(n, dtype=torch.float32)
        s["targets"] = t[:, 0].to(torch.int32)
        s["targets"][torch.rand(n, generator=g, device="cuda") < case["skip"]] = -1
        if case["dir"] == "step":
            s["d_loss"] = (0.5 + torch.rand(n, generator=g, device="cuda")) / n
    else:
        # a layer's input: a few channels are far larger than the others
        c = case["c"]
        width = normal(c, std=0.5, dtype=torch.float32).exp_()
        width[torch.rand(c, generator=g, device="cuda") < 0.01] *= 20.0
        s["x"] = (normal(n, c, dtype=torch.float32) * width).to(dt)
        if case["op"] == "grad":
            m = case["m"]
            s["dy"] = normal(n, -(-m // 8) * 8, std=0.1)[:, :m]   # rows start at whole 16 bytes
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    if own:
        _keep(s)
    elif case["op"] == "grad":
        s["codes"], s["scales"] = _quantise(s["x"])
    if case["op"] == "grad":
        del s["x"]   # the forward pass has stored it
    return s


def _keep(s):
    """What a program that uses the library keeps beside its inputs: descriptors, output buffers, workspaces and, for a
    weight gradient, the input that its forward pass has stored."""
    from sft_trie_build_gb300 import stp

    case, dt = s["case"], _dtype(s["case"])
    code, n = stp.STP_FP32 if dt is torch.float32 else stp.STP_BF16, case["n"]

    def empty(*shape, dtype=dt):
        return torch.empty(*shape, dtype=dtype, device="cuda")

    def space(size):
        return empty(max(256, size), dtype=torch.uint8)

    if case["op"] == "embed":
        s["desc"] = stp.embed_desc(n, case["v"], case["c"], code, case["scale"])
        s["ws"] = space(stp.stp_embed_workspace_size(s["desc"]))
        s["out"] = empty(n, case["c"]) if case["dir"] == "fwd" else empty(case["v"], case["c"], dtype=torch.float32)
    elif case["op"] == "policy":
        s["desc"] = stp.policy_desc(n, case["v"], code, case["scale"], LOW, HIGH, case["kl"], case["ent"])
        s["ws"] = space(stp.stp_policy_workspace_size(s["desc"]))
        s["out"] = tuple(empty(n, dtype=torch.float32) for _ in range(5))
        if case["dir"] == "step":
            s["dz"] = torch.empty_like(s["logits"])
    else:
        s["desc"] = stp.ckpt_desc(n, case["c"], code)
        s["ckpt"] = space(stp.stp_ckpt_size(s["desc"]))
        if case["op"] == "ckpt":
            s["out"] = torch.empty_like(s["x"])
        else:
            stp.stp_ckpt_save(s["desc"], s["x"], s["ckpt"])
            s["ws"] = space(stp.stp_ckpt_wgrad_workspace_size(s["desc"], case["m"]))
            s["dw"] = empty(case["c"], case["m"], dtype=torch.float32)


# ---------------------------------------------------------------------------------------------- one pass

def run(s):
    return (_run_own if own else _run_plain)(s)


def _run_own(s):
    from sft_trie_build_gb300 import stp

    case = s["case"]
    if case["op"] == "embed":
        if case["dir"] == "fwd":
            stp.stp_embed_fwd(s["desc"], s["table"], s["tok"], s["out"], s["ws"])
            return {"out": s["out"]}
        stp.stp_embed_bwd(s["desc"], s["d_out"], s["tok"], False, s["out"], s["ws"])
        return {"d_table": s["out"]}
    if case["op"] == "policy":
        given = s["logits"], s["targets"], s["old"], s["ref"], s["adv"]
        out = dict(zip(("loss", "logprob", "entropy", "lse", "kl"), s["out"]))
        if case["dir"] == "fwd":
            stp.stp_policy_fwd(s["desc"], *given, *s["out"], s["ws"])
        else:
            stp.stp_policy_step(s["desc"], *given, s["d_loss"], *s["out"], s["dz"], s["ws"])
            out["dz"] = s["dz"]
        return out
    if case["op"] == "ckpt":
        stp.stp_ckpt_save(s["desc"], s["x"], s["ckpt"])
        stp.stp_ckpt_load(s["desc"], s["ckpt"], s["out"])
        return {"x": s["out"]}
    stp.stp_ckpt_wgrad(s["desc"], case["m"], s["ckpt"], s["dy"], s["dy"].stride(0), False, s["dw"], s["ws"])
    return {"dw": s["dw"]}


def _run_plain(s):
    return {"embed": _embed, "policy": _policy, "ckpt": _ckpt, "grad": _grad}[s["case"]["op"]](s)


def _embed(s):
    case, there = s["case"], s["tok"] >= 0
    if case["dir"] == "fwd":
        x = s["table"][s["tok"].clamp(min=0).long()].float() * case["scale"]
        return {"out": x.masked_fill_(~there[:, None], 0).to(s["table"].dtype)}
    d = torch.zeros(case["v"], case["c"], device="cuda")
    return {"d_table": d.index_add_(0, s["tok"][there].long(), s["d_out"][there].float()).mul_(case["scale"])}


def _lse(z):
    top = z.amax(-1, keepdim=True)
    return top + (z - top).exp().sum(-1, keepdim=True).log()


def _policy(s):
    case = s["case"]
    z = s["logits"].float() * case["scale"]
    on = s["targets"] >= 0
    at = s["targets"].clamp(min=0).long()[:, None]
    lse = _lse(z)
    y = z - lse
    p = y.exp()
    ent = -(p * y).sum(-1)
    lp = y.gather(1, at)[:, 0]
    r, a = (lp - s["old"]).exp(), s["adv"]
    loss = -torch.minimum(r * a, r.clamp(1 - LOW, 1 + HIGH) * a) - case["ent"] * ent
    kl = torch.zeros_like(lp)
    if s["ref"] is not None:
        x = s["ref"] - lp
        kl = x.expm1() - x
        loss = loss + case["kl"] * kl
    out = {"loss": loss, "logprob": lp, "entropy": ent, "lse": lse[:, 0], "kl": kl}
    out = {k: v.masked_fill(~on, 0) for k, v in out.items()}
    if case["dir"] == "step":
        live = torch.where(a >= 0, r <= 1 + HIGH, r >= 1 - LOW)
        g = -(a * r) * live
        if s["ref"] is not None:
            g = g - case["kl"] * (s["ref"] - lp).expm1()
        hot = torch.zeros_like(p).scatter_(1, at, 1.0)
        dz = g[:, None] * (hot - p) + case["ent"] * p * (y + ent[:, None])
        dz = dz * (s["d_loss"] * case["scale"])[:, None]
        out["dz"] = dz.masked_fill_(~on[:, None], 0).to(s["logits"].dtype)
    return out


def _quantise(x):
    """Codes float8_e4m3 [n, blocks, 32] and scales float32 [n, blocks, 1]: the smallest power of two (from 2^-117 on)
    at which the block's largest value is at most 448; NaN where the block holds an infinity or a NaN."""
    n, c = x.shape
    x = torch.nn.functional.pad(x.float(), (0, -c % 32)).view(n, -1, 32)
    top = x.abs().amax(-1, keepdim=True)
    m, e = torch.frexp(top)
    k = torch.where(m > 0.875, e - 8, e - 9).clamp(min=-117)
    bad = ~torch.isfinite(top)
    k = k.masked_fill(bad | (top == 0), 0).int()
    codes = (x * ((127 - k) << 23).view(torch.float32)).masked_fill(bad, 0).to(torch.float8_e4m3fn)
    return codes, ((127 + k) << 23).view(torch.float32).masked_fill(bad, float("nan"))


def _ckpt(s):
    codes, scales = _quantise(s["x"])
    return {"x": (codes.float() * scales).flatten(1)[:, :s["case"]["c"]].to(s["x"].dtype)}


def _grad(s):
    x = (s["codes"].float() * s["scales"]).flatten(1)[:, :s["case"]["c"]]
    return {"dw": x.T @ s["dy"].float()}


# ---------------------------------------------------------------------------------------------- what a pass needs

def work(case):
    b, n = _bytes(case), case["n"]
    if case["op"] == "embed":
        x = n * case["c"]
        tok = _tokens(case, 0)
        rows = len(np.unique(tok[tok >= 0])) * case["c"] * b if case["dir"] == "fwd" else case["v"] * case["c"] * 4
        return {"bytes": int(4 * n + rows + x * b * (1 if case["dir"] == "fwd" else 1 - case["skip"])), "flops": x}
    if case["op"] == "policy":
        rows = n * (1 - case["skip"])
        step = case["dir"] == "step"
        return {"bytes": int(rows * case["v"] * b + (n * case["v"] * b if step else 0) + n * 40),
                "flops": int(rows * case["v"] * (12 if step else 6))}
    x = n * case["c"]
    if case["op"] == "ckpt":
        return {"bytes": 2 * x * b + 2 * x * 33 // 32, "flops": 4 * x}
    return {"bytes": x * 33 // 32 + 2 * n * case["m"] + 4 * case["c"] * case["m"], "flops": 2 * x * case["m"]}


# ---------------------------------------------------------------------------------------------- 64 bits

def exact(case, seed):
    return {"embed": _embed64, "policy": _policy64, "ckpt": _ckpt64, "grad": _grad64}[case["op"]](_inputs(case, seed))


def _embed64(s):
    case = s["case"]
    tok = s["tok"].long()
    if case["dir"] == "fwd":
        rows = torch.cat((s["table"].double() * case["scale"], torch.zeros(1, case["c"], dtype=torch.float64, device="cuda")))
        return {"out": rows[torch.where(tok < 0, torch.full_like(tok, case["v"]), tok)]}
    d = torch.zeros(case["v"] + 1, case["c"], dtype=torch.float64, device="cuda")
    d.index_add_(0, torch.where(tok < 0, torch.full_like(tok, case["v"]), tok), s["d_out"].double() * case["scale"])
    return {"d_table": d[:-1]}


def _policy64(s):
    case = s["case"]
    out = []
    size = max(1, (1 << 28) // case["v"])
    for a in range(0, case["n"], size):
        b = slice(a, min(case["n"], a + size))
        z = s["logits"][b].double().requires_grad_()
        y = torch.log_softmax(z * case["scale"], -1)
        skip = s["targets"][b] < 0
        lp = y.gather(1, s["targets"][b].clamp(min=0).long()[:, None])[:, 0]
        ent = -(torch.exp(y) * y).sum(-1)
        ratio, adv = torch.exp(lp - s["old"][b].double()), s["adv"][b].double()
        # the surrogate by cases: what a large step would gain (or lose) beyond the border does not count
        bound = torch.where(adv >= 0, torch.full_like(adv, 1 + HIGH), torch.full_like(adv, 1 - LOW))
        out_of = torch.where(adv >= 0, ratio > bound, ratio < bound)
        loss = -adv * torch.where(out_of, bound, ratio) - case["ent"] * ent
        kl = torch.zeros_like(lp)
        if s["ref"] is not None:
            rel = torch.exp(s["ref"][b].double() - lp)
            kl = rel - 1 - torch.log(rel)
            loss = loss + case["kl"] * kl
        loss = loss.masked_fill(skip, 0)
        got = {"loss": loss, "logprob": lp, "entropy": ent, "lse": torch.logsumexp(z * case["scale"], -1), "kl": kl}
        got = {k: v.detach().masked_fill(skip, 0) for k, v in got.items()}
        if case["dir"] == "step":
            got["dz"], = torch.autograd.grad((loss * s["d_loss"][b].double()).sum(), z)
        out.append(got)
    return {x: torch.cat([g[x] for g in out]) for x in out[0]}


def _kept64(x):
    """What 8 bits keep of x: eight steps between powers of two down to 2^-6 of the scale, even steps below."""
    n, c = x.shape
    x = torch.nn.functional.pad(x.double(), (0, -c % 32)).reshape(n, -1, 32)
    top = x.abs().amax(-1, keepdim=True)
    tiny = 1e-9   # beyond the error of log2 at powers of two, below the distance of any other value
    scale = torch.exp2(torch.ceil(torch.log2(top / 448) - tiny).clamp(min=-117.0))
    v = x / scale
    step = torch.exp2(torch.floor(torch.log2(v.abs()) + tiny).clamp(min=-6.0) - 3)
    return (torch.round(v / step) * step * scale).reshape(n, -1)[:, :c]


def _ckpt64(s):
    return {"x": _kept64(s["x"])}


def _grad64(s):
    return {"dw": _kept64(s["x"]).T @ s["dy"].double()}

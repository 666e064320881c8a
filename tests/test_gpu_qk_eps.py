"""q/k norm with rotation at eps = 0 and with heads that do not fill a warp's
pass, and with tolerances taken from each head vector by itself.

Tolerance: as in test_gpu_qk.py, an output is rounded once (u = eps / 2 of its
type) after float32 work within W = 64 * 2^-24 of the largest terms of its own
vector; dw sums N H products, 96 * 2^-24 of the sum of their absolute values.
"""
import numpy as np
import pytest
import torch

from oracle import qk as OQ
from sft_trie_build_gb300 import stp

pytestmark = pytest.mark.gpu
WORK = 64 * 2.0 ** -24
DT = {stp.STP_BF16: torch.bfloat16, stp.STP_FP32: torch.float32}


@pytest.mark.parametrize("dtype", [stp.STP_BF16, stp.STP_FP32])
@pytest.mark.parametrize("n,hq,hkv,d,rot,eps", [
    (1, 1, 1, 16, 16, 0.0),        # one head where a pass takes 32
    (5, 3, 2, 128, 128, 0.0),      # a pass takes four
    (70, 8, 2, 128, 64, 0.0),      # queries fill their passes, keys do not
    (33, 5, 3, 64, 64, 0.0),
    (9, 2, 1, 48, 48, 0.0),        # and idle lanes within a head
    (7, 1, 3, 256, 256, 0.0),
    (3, 2, 1, 512, 512, 0.0),
    (40, 3, 2, 128, 128, 1e-6), (40, 3, 2, 128, 128, 1.0),
])
def test_eps_and_unfilled_passes(n, hq, hkv, d, rot, eps, dtype):
    g = torch.Generator().manual_seed(n + d)
    dt, u = DT[dtype], torch.finfo(DT[dtype]).eps / 2
    x = {"q": torch.randn(n, hq, d, generator=g).to(dt), "k": torch.randn(n, hkv, d, generator=g).to(dt)}
    dy = {"q": torch.randn(n, hq, d, generator=g).to(dt), "k": torch.randn(n, hkv, d, generator=g).to(dt)}
    for y in "qk":                 # vectors of very different length, each with its own bound
        x[y] = (x[y] * torch.logspace(-2, 2, n)[:, None, None]).to(dt)
        if eps > 0:
            x[y][n // 2, 0] = 0.0  # the norm of nothing: eps alone
    w = {y: 1 + 0.3 * torch.randn(d, generator=g) for y in "qk"}
    pos = torch.randint(0, 5000, (n,), generator=g).to(torch.int32)
    freq = 10000.0 ** (-np.arange(rot // 2) / (rot // 2))
    desc = stp.qk_desc(n, hq, hkv, d, rot, False, dtype, eps)
    c = {k: v.cuda() for k, v in (("q", x["q"]), ("k", x["k"]), ("dq", dy["q"]), ("dk", dy["k"]), ("wq", w["q"]),
                                  ("wk", w["k"]), ("pos", pos))}
    out = {k: torch.full_like(c[k[-1]], float("nan")) for k in ("yq", "yk", "xq", "xk")}
    dw = {y: torch.full((d,), float("nan"), device="cuda") for y in "qk"}
    ws = torch.empty(stp.stp_qk_norm_rope_workspace_size(desc), dtype=torch.uint8, device="cuda")
    stp.stp_qk_norm_rope_fwd(desc, c["q"], c["k"], c["wq"], c["wk"], freq, c["pos"], out["yq"], out["yk"])
    stp.stp_qk_norm_rope_bwd(desc, c["q"], c["k"], c["wq"], c["wk"], freq, c["pos"], c["dq"], c["dk"], out["xq"],
                             out["xk"], dw["q"], dw["k"], ws)
    torch.cuda.synchronize()
    for y in "qk":
        xs, ws_, gs = x[y].double().numpy(), w[y].double().numpy(), dy[y].double().numpy()
        r = 1 / np.sqrt((xs ** 2).mean(-1, keepdims=True) + eps)
        want = OQ.forward(xs, ws_, pos.numpy(), freq, rot, eps=eps)
        big = np.abs(xs * ws_).max(-1, keepdims=True) * r
        got = out["y" + y].double().cpu().numpy()
        assert (np.abs(got - want) <= u * np.abs(want) + WORK * big).all(), y
        dx, dwant = OQ.backward(xs, ws_, pos.numpy(), freq, rot, gs, eps=eps)
        big = (np.abs(gs).max(-1, keepdims=True) * 1.5 * np.abs(ws_).max() * r) * (1 + np.abs(xs * r))
        got = out["x" + y].double().cpu().numpy()
        assert (np.abs(got - dx) <= u * np.abs(dx) + 4 * WORK * big).all(), "dx " + y
        terms = 1.5 * np.abs(gs).max() * np.abs(xs * r).sum((0, 1))
        assert (np.abs(dw[y].double().cpu().numpy() - dwant) <= 96 * 2.0 ** -24 * terms).all(), "dw " + y

"""The embedding, the policy loss and the activations in 8 bits where element
offsets pass 2^31, and calls that run at the same time on two streams.

Whole numbers are used wherever sums are compared, small enough that every
order gives the same float32 result; other bounds are those of the operators'
own tests."""
import numpy as np
import pytest
import torch

from oracle import policy as OP
from sft_trie_build_gb300 import stp

pytestmark = pytest.mark.gpu


def _space(size):
    return torch.full((max(256, size),), 255, dtype=torch.uint8, device="cuda")


def test_embedding_of_a_table_beyond_2_31_elements():
    v, c, n = 300000, 8192, 333                            # 2.46e9 elements
    tok = np.random.default_rng(0).integers(0, v, n).astype(np.int32)
    tok[:5] = [v - 1, v - 1, 0, v - 2, v // 2]
    t = torch.from_numpy(tok).cuda()
    desc = stp.embed_desc(n, v, c)
    ws = _space(stp.stp_embed_workspace_size(desc))
    table = torch.zeros(v, c, dtype=torch.bfloat16, device="cuda")
    rows = torch.randint(-100, 101, (n, c), generator=torch.Generator().manual_seed(1)).float()
    rows[1] = rows[0]
    for i in range(n):                                     # the last of equal tokens counts in the table
        table[int(tok[i])] = rows[i].bfloat16().cuda()
    out = torch.empty(n, c, dtype=torch.bfloat16, device="cuda")
    stp.stp_embed_fwd(desc, table, t, out, ws)
    assert torch.equal(out, table[t.long()]) and stp.stp_device_status(ws) == stp.STP_OK
    del table
    d = rows.bfloat16().cuda()
    grad = torch.full((v, c), float("nan"), device="cuda")
    stp.stp_embed_bwd(desc, d, t, False, grad, ws)
    assert stp.stp_device_status(ws) == stp.STP_OK
    uniq, inv = torch.unique(t.long(), return_inverse=True)
    want = torch.zeros(len(uniq), c, device="cuda").index_add_(0, inv, d.float())
    assert torch.equal(grad[uniq], want)
    grad[uniq] = 0
    assert not bool(grad.any())


@pytest.mark.parametrize("n,v,c", [(300001, 5000, 8), (200000, 3, 40)])
def test_embedding_gradient_of_many_tokens(n, v, c):
    # several rounds of the walk over the positions; tokens by the ten thousand
    rng = np.random.default_rng(n)
    tok = np.minimum(np.exp(rng.random(n) * np.log(v + 1)).astype(np.int64), v).astype(np.int32) - 1
    tok[rng.random(n) < 0.1] = -1
    d = torch.from_numpy(rng.integers(-8, 9, (n, c)).astype(np.float32)).bfloat16().cuda()
    t = torch.from_numpy(tok).cuda()
    desc = stp.embed_desc(n, v, c)
    ws, grad = _space(stp.stp_embed_workspace_size(desc)), torch.full((v, c), float("nan"), device="cuda")
    stp.stp_embed_bwd(desc, d, t, False, grad, ws)
    assert stp.stp_device_status(ws) == stp.STP_OK
    want = torch.zeros(v, c, dtype=torch.float64, device="cuda").index_add_(0, t[t >= 0].long(), d[t >= 0].double())
    assert float(want.abs().max()) < 2 ** 24 and torch.equal(grad.double(), want)


def test_policy_rows_beyond_2_31_elements():
    n, v = 20000, 120000                                   # 2.4e9 elements
    z = torch.empty(n, v, dtype=torch.bfloat16, device="cuda")
    z.normal_(generator=torch.Generator(device="cuda").manual_seed(0))
    rng = np.random.default_rng(1)
    t = np.full(n, -1, np.int32)
    at = [0, 17, n // 2, n - 2, n - 1]
    t[at] = [5, v - 1, 77, 0, v - 1]
    old, adv, w = (rng.standard_normal(n).astype(np.float32) * 0.1 for _ in range(3))
    old -= 12.0
    given = [torch.from_numpy(x).cuda() for x in (t, old, adv, w)]
    out = [torch.full((n,), float("nan"), device="cuda") for _ in range(5)]
    desc, ws = stp.policy_desc(n, v), _space(256)
    rows = z[at].double().cpu().numpy()
    stp.stp_policy_step(desc, z, given[0], given[1], None, given[2], given[3], *out, z, ws)
    assert stp.stp_device_status(ws) == stp.STP_OK
    for k, i in enumerate(at):
        loss, lp, _, _, _, dz = OP.row(rows[k], t[i], float(old[i]), None, float(adv[i]), 0.2, 0.2, 0.0, 0.0)
        assert abs(float(out[1][i]) - lp) <= 1e-4 and abs(float(out[0][i]) - loss) <= 1e-3 * (1 + abs(loss))
        got = z[i].double().cpu().numpy()
        # p and the ratio are off by 1e-4 relative at most, and the result is rounded once
        assert (np.abs(got - w[i] * dz) <= (2.0 ** -8 + 1e-3) * np.abs(w[i] * dz) + 1e-12).all()
        z[i] = 0
    assert not bool(z.any())


def test_activations_beyond_2_31_elements():
    n, c, m = 600000, 4096, 24                             # 2.46e9 elements
    g = torch.Generator(device="cuda").manual_seed(0)
    x = torch.randint(-8, 9, (n, c), generator=g, device="cuda", dtype=torch.int8).to(torch.bfloat16)
    dy = torch.randint(-4, 5, (n, m), generator=g, device="cuda", dtype=torch.int8).to(torch.bfloat16)
    desc = stp.ckpt_desc(n, c)
    ckpt = _space(stp.stp_ckpt_size(desc))
    stp.stp_ckpt_save(desc, x, ckpt)
    out = torch.empty_like(x)
    stp.stp_ckpt_load(desc, ckpt, out)
    assert torch.equal(out, x)                             # whole numbers up to 8 are kept as they are
    ws, dw = _space(stp.stp_ckpt_wgrad_workspace_size(desc, m)), torch.full((c, m), float("nan"), device="cuda")
    stp.stp_ckpt_wgrad(desc, m, ckpt, dy, m, False, dw, ws)
    assert stp.stp_device_status(ws) == stp.STP_OK
    want = torch.zeros(c, m, dtype=torch.float64, device="cuda")
    for a in range(0, n, 50000):
        want += x[a:a + 50000].double().T @ dy[a:a + 50000].double()
    assert float(want.abs().max()) < 2 ** 24 and torch.equal(dw.double(), want)


def test_calls_at_the_same_time_on_two_streams():
    g = torch.Generator().manual_seed(3)
    jobs = []
    for n, c, m, v in ((20001, 300, 500, 700), (9000, 1000, 1100, 60000)):
        x = torch.randint(-8, 9, (n, c), generator=g).bfloat16()
        dy = torch.randint(-4, 5, (n, m // 8 * 8), generator=g).bfloat16()
        tok = torch.randint(-1, v, (n,), generator=g, dtype=torch.int32)
        cd, ed = stp.ckpt_desc(n, c // 8 * 8, stride=c), stp.embed_desc(n, v, c // 8 * 8, stride=(c + 7) // 8 * 8)
        wide = torch.zeros(n, (c + 7) // 8 * 8, dtype=torch.bfloat16)
        wide[:, :c] = x
        jobs.append(dict(stream=torch.cuda.Stream(), x=x.cuda(), dy=dy.cuda(), tok=tok.cuda(), cd=cd, ed=ed, m=m // 8 * 8, wide=wide.cuda(),
                         ck=_space(stp.stp_ckpt_size(cd)), ws=_space(stp.stp_ckpt_wgrad_workspace_size(cd, m // 8 * 8)),
                         ews=_space(stp.stp_embed_workspace_size(ed)), dw=torch.zeros(c // 8 * 8, m // 8 * 8, device="cuda"),
                         grad=torch.zeros(v, c // 8 * 8, device="cuda")))
    torch.cuda.synchronize()
    for _ in range(4):
        for j in jobs:
            stp.stp_ckpt_save(j["cd"], j["x"], j["ck"], stream=j["stream"])
            stp.stp_ckpt_wgrad(j["cd"], j["m"], j["ck"], j["dy"], j["m"], True, j["dw"], j["ws"], stream=j["stream"])
            stp.stp_embed_bwd(j["ed"], j["wide"], j["tok"], True, j["grad"], j["ews"], stream=j["stream"])
    torch.cuda.synchronize()
    for j in jobs:
        assert stp.stp_device_status(j["ws"]) == stp.stp_device_status(j["ews"]) == stp.STP_OK
        c = j["cd"].dim
        x = j["x"][:, :c].double()
        assert torch.equal(j["dw"].double(), 4 * (x.T @ j["dy"].double()))
        on = j["tok"] >= 0
        want = torch.zeros(j["grad"].shape, dtype=torch.float64, device="cuda").index_add_(0, j["tok"][on].long(), x[on])
        assert torch.equal(j["grad"].double(), 4 * want)

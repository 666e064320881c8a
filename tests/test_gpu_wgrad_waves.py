"""Weight gradients from 8-bit checkpoints whose launch has whole tiles and a
last wave that is cut along the tokens, and how exact their sums are over many
tokens.

Whole numbers, whose sums stay below 2^24, must come out exactly.  For other
values: a product is exact, the tensor core takes 16 tokens a step and drops
less than one unit of the last place of the sum so far (2^-23 of it), the sums
are taken out every 2048 tokens (128 steps) and added in float32 (2^-24 of the sum
each).  With all terms positive no sum so far is above the result, a chunk's
not above its share: (128 * 2^-23 + n / 2048 * 2^-24) of the result, and as
much again from the parts' joining, 2^-24 for each of at most 76.
"""
import pytest
import torch

from sft_trie_build_gb300 import stp

pytestmark = pytest.mark.gpu
PART = 2 * 128 * 256 * 4                                              # bytes of a tile's part in the workspace


def _space(size):
    return torch.full((max(256, size),), 255, dtype=torch.uint8, device="cuda")


def _form(n, c, m):
    """(whole waves, tiles of the last one, pairs of blocks that work on them) of a call on this device; the tiles are
    256 channels x at most 256 columns, as long as there are more of them than pairs, or parts."""
    pairs = torch.cuda.get_device_properties(0).multi_processor_count // 2
    tiles = -(-c // 256) * -(-m // 256)
    cut = (stp.stp_ckpt_wgrad_workspace_size(stp.ckpt_desc(n, c), m) - 256) // PART
    return tiles // pairs, tiles % pairs, cut


def _run(x, dy, add=None):
    n, c = x.shape
    m = dy.shape[1]
    desc = stp.ckpt_desc(n, c)
    ckpt, ws = _space(stp.stp_ckpt_size(desc)), _space(stp.stp_ckpt_wgrad_workspace_size(desc, m))
    y = torch.full((n, (m + 7) // 8 * 8), float("nan"), dtype=torch.bfloat16, device="cuda")
    y[:, :m] = dy
    dw = torch.full((c, m), float("nan"), device="cuda") if add is None else add.clone()
    stp.stp_ckpt_save(desc, x, ckpt)
    stp.stp_ckpt_wgrad(desc, m, ckpt, y, y.stride(0), add is not None, dw, ws)
    torch.cuda.synchronize()
    assert stp.stp_device_status(ws) == stp.STP_OK
    return dw


@pytest.mark.parametrize("add", [False, True])
@pytest.mark.parametrize("n,c,m", [(4096, 4096, 1300), (4001, 4111, 1291), (3000, 5120, 2000), (6100, 2560, 4000), (9001, 9990, 1023)])
def test_whole_waves_and_a_cut_one(n, c, m, add):
    whole, rest, cut = _form(n, c, m)
    assert whole >= 1 and cut >= 2 * rest > 0
    g = torch.Generator(device="cuda").manual_seed(n + c + m)
    x = torch.randint(-8, 9, (n, c), generator=g, device="cuda", dtype=torch.int8).bfloat16()
    dy = torch.randint(-4, 5, (n, m), generator=g, device="cuda", dtype=torch.int8).bfloat16()
    assert 32 * n < 2 ** 24
    start = torch.arange(c * m, device="cuda", dtype=torch.float32).remainder_(1000).view(c, m) if add else None
    want = x.double().T @ dy.double()
    if add:
        want += start.double()
    assert torch.equal(_run(x, dy, start).double(), want)


def test_forms_that_the_sizes_above_stand_for():
    forms = [_form(*s) for s in ((4096, 4096, 1300), (4001, 4111, 1291), (3000, 5120, 2000), (6100, 2560, 4000), (9001, 9990, 1023))]
    pairs = torch.cuda.get_device_properties(0).multi_processor_count // 2
    assert any(w >= 2 for w, _, _ in forms)                           # several whole waves
    assert any(cut < pairs for _, _, cut in forms)                    # pairs without a part


# all tokens in one block's hands (as many tiles as pairs of blocks: 34 takings of the sums), and in parts
@pytest.mark.parametrize("n,c,m", [(70001, 4860, 1020), (70001, 64, 64), (20001, 130, 300), (16384, 300, 1100)])
def test_sums_over_many_tokens(n, c, m):
    if c == 4860:
        assert _form(n, c, m)[0] >= 1
    g = torch.Generator(device="cuda").manual_seed(n)
    x = torch.rand(n, c, generator=g, device="cuda").add_(0.5)
    dy = torch.rand(n, m, generator=g, device="cuda").add_(0.5).bfloat16()
    desc = stp.ckpt_desc(n, c, stp.STP_FP32)
    ckpt, kept = _space(stp.stp_ckpt_size(desc)), torch.empty_like(x)
    stp.stp_ckpt_save(desc, x, ckpt)
    stp.stp_ckpt_load(desc, ckpt, kept)
    want = kept.double().T @ dy.double()
    got = _run(kept.bfloat16(), dy).double()                          # what is restored is kept as it is
    bound = 128 * 2.0 ** -23 + -(-n // 2048) * 2.0 ** -24 + 76 * 2.0 ** -24
    assert float(((got - want).abs() / want).max()) <= bound

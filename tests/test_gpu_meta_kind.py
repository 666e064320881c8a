"""A tile_meta that was classified for one kind of attention, given to calls of
another (no window, a window, another window or number of first tokens): the
device error word says so and no output is written."""
import pytest
import torch

from oracle import pack as OP
from sft_trie_build_gb300 import stp
from sft_trie_build_gb300 import workloads as W

pytestmark = pytest.mark.gpu
PLAIN = None


class Calls:
    def __init__(self, dtype):
        b = W.random_forest(3, n_roots=3, max_depth=3, len_lo=5, len_hi=80, row_len=384, min_shared=8)
        plan = OP.pack(b.seqs, b.trainable, b.row_len, b.min_shared)
        R, T = plan.subtree_end.shape
        dt = torch.bfloat16 if dtype == stp.STP_BF16 else torch.float32
        g = torch.Generator().manual_seed(0)
        r = lambda h: torch.randn(R, T, h, 128, generator=g).to(dt).cuda()  # noqa: E731
        self.q, self.k, self.v, self.do = r(2), r(1), r(1), r(2)
        self.desc = stp.Desc(R, T, 2, 1, 128, dtype, 0.0, 0)
        self.buf = stp.Buffers(self.desc)
        self.se, self.pos = torch.from_numpy(plan.subtree_end).cuda(), torch.from_numpy(plan.position_ids).cuda()
        self.lse = torch.empty(R, 2, T, device="cuda")
        self.o, self.dq, self.dk, self.dv = (torch.empty_like(x) for x in (self.q, self.q, self.k, self.v))
        # finite forward results for the backward's own reading
        self.classify(PLAIN)
        self.forward(PLAIN)

    def classify(self, kind, noalloc=False):
        if kind is not PLAIN:
            stp.stp_classify_window(self.desc, *kind, self.se, self.pos, self.buf.tile_meta)
        else:
            (stp.stp_classify_noalloc if noalloc else stp.stp_classify)(self.desc, self.se, self.buf.tile_meta)

    def forward(self, kind):
        if kind is PLAIN:
            stp.stp_attn_fwd(self.desc, self.q, self.k, self.v, self.se, self.buf.tile_meta, self.o, self.lse, self.buf.fwd_ws)
        else:
            stp.stp_attn_window_fwd(self.desc, *kind, self.q, self.k, self.v, self.se, self.pos, self.buf.tile_meta, self.o,
                                    self.lse, self.buf.fwd_ws)

    def backward(self, kind):
        out = (self.dq, self.dk, self.dv, self.buf.bwd_ws)
        if kind is PLAIN:
            stp.stp_attn_bwd(self.desc, self.q, self.k, self.v, self.o, self.lse, self.do, self.se, self.buf.tile_meta, *out)
        else:
            stp.stp_attn_window_bwd(self.desc, *kind, self.q, self.k, self.v, self.o, self.lse, self.do, self.se, self.pos,
                                    self.buf.tile_meta, *out)


@pytest.mark.parametrize("dtype", [stp.STP_BF16, stp.STP_FP32])
@pytest.mark.parametrize("made,used", [((40, 4), PLAIN), (PLAIN, (40, 4)), ((40, 4), (41, 4)), ((40, 4), (40, 3)),
                                       ((2 ** 31 - 1, 0), PLAIN), (PLAIN, (2 ** 31 - 1, 0))])
def test_other_kinds_are_refused(made, used, dtype):
    c = Calls(dtype)
    c.classify(made)
    o, lse = c.o.clone(), c.lse.clone()
    for x in (c.dq, c.dk, c.dv):
        x.fill_(7.0)
    c.backward(used)
    assert stp.stp_device_status(c.buf.bwd_ws) == stp.STP_EDEVICE
    c.o.fill_(7.0)
    c.lse.fill_(7.0)
    c.forward(used)
    assert stp.stp_device_status(c.buf.fwd_ws) == stp.STP_EDEVICE
    for x in (c.o, c.lse, c.dq, c.dk, c.dv):
        assert (x == 7.0).all()
    # and the kind that it is for goes on working
    c.o.copy_(o)
    c.lse.copy_(lse)
    c.forward(made)
    c.backward(made)
    for ws in (c.buf.tile_meta, c.buf.fwd_ws, c.buf.bwd_ws):
        assert stp.stp_device_status(ws) == stp.STP_OK
    for x in (c.o, c.lse, c.dq, c.dk, c.dv):
        assert torch.isfinite(x).all() and not (x == 7.0).all()


@pytest.mark.parametrize("noalloc", [False, True])
def test_classifying_again_changes_the_kind(noalloc):
    c = Calls(stp.STP_BF16)
    want = c.o.clone()
    c.classify((9, 0))
    c.classify(PLAIN, noalloc)
    c.forward(PLAIN)
    assert stp.stp_device_status(c.buf.fwd_ws) == stp.STP_OK and torch.equal(c.o, want)
    # windows that hide nothing are one kind
    c.classify((1 << 30, 0))
    c.forward((2 ** 31 - 1, 0))
    assert stp.stp_device_status(c.buf.fwd_ws) == stp.STP_OK and torch.equal(c.o, want)


def test_index_refuses_windowed_classes():
    c = Calls(stp.STP_BF16)
    R, T = c.se.shape
    desc = stp.index_desc(R, T, 2, 128, 16, 0)
    ws = torch.empty(stp.stp_index_workspace_size(desc), dtype=torch.uint8, device="cuda")
    idx, score = torch.empty(R, T, 16, dtype=torch.int32, device="cuda"), torch.empty(R, T, 16, device="cuda")
    k, w = c.k.view(R, T, 128), torch.ones(R, T, 2, device="cuda")
    for kind, status in ((PLAIN, stp.STP_OK), ((9, 0), stp.STP_EDEVICE), (PLAIN, stp.STP_OK)):
        c.classify(kind)
        stp.stp_index_topk(desc, c.q, k, w, c.se, c.buf.tile_meta, idx, score, ws)
        assert stp.stp_device_status(ws) == status
        assert ((idx[:, :, 0] >= 0) == (status == stp.STP_OK)).all()


def test_host_step_refuses_windowed_classes():
    c = Calls(stp.STP_BF16)
    c.classify((9, 0))
    scratch = torch.zeros(stp.stp_step_scratch_size(c.desc, 1), dtype=torch.uint8, device="cuda")
    host = [x.cpu().pin_memory() for x in (c.q, c.k, c.v, c.do)]
    out = [torch.empty(x.shape, dtype=x.dtype).pin_memory() for x in (c.o, c.lse, c.dq, c.dk, c.dv)]
    stp.stp_attn_step_host(c.desc, 1, *host, c.se, c.buf.tile_meta, *out, scratch)
    torch.cuda.synchronize()
    assert stp.stp_device_status(scratch) == stp.STP_EDEVICE

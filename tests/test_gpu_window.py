"""Windowed tree attention on the GPU (stp_classify_window,
stp_attn_window_fwd / _bwd) against the float64 oracle (oracle/window.py).

Tolerance: the oracle gives, per element, what rounding P, dS and the stored O
once by a relative half step u does at most (o_tol, dq_tol, ...; u = 2^-8 for
bf16, 2^-24 for float32).  To this comes float32 work: sums of at most 1024
terms and exponents of |s log2 e| < 64, within 512 * 2^-24 of the same sums of
absolute values.  LSE: the same work on a value below 32 in magnitude.
"""
import numpy as np
import pytest
import torch

from oracle import pack as OP
from oracle import window as OW
from sft_trie_build_gb300 import stp
from sft_trie_build_gb300 import workloads as W

pytestmark = pytest.mark.gpu
WORK = 512 * 2.0 ** -24


class Run:
    def __init__(self, se, pos, hq, hkv, d, dtype, window, sinks, seed=0, stream=None, ds_groups=0):
        R, T = se.shape
        dt = torch.bfloat16 if dtype == stp.STP_BF16 else torch.float32
        g = torch.Generator().manual_seed(seed)
        self.window, self.sinks, self.stream = window, sinks, stream
        self.q = torch.randn(R, T, hq, d, generator=g).to(dt).cuda()
        self.k, self.v = (torch.randn(R, T, hkv, d, generator=g).to(dt).cuda() for _ in range(2))
        self.do = torch.randn(R, T, hq, d, generator=g).to(dt).cuda()
        self.pairs = stp.stp_count_window_tile_pairs(se, pos, window, sinks)
        self.desc = stp.Desc(R, T, hq, hkv, d, dtype, 0.0, self.pairs, ds_groups)
        self.buf = stp.Buffers(self.desc)
        self.se, self.pos = torch.from_numpy(se).cuda(), torch.from_numpy(pos).cuda()
        self.o, self.dq = torch.full_like(self.q, float("nan")), torch.full_like(self.q, float("nan"))
        self.dk, self.dv = torch.full_like(self.k, float("nan")), torch.full_like(self.k, float("nan"))
        self.lse = torch.full((R, hq, T), float("nan"), device="cuda")
        torch.cuda.synchronize()

    def classify(self):
        stp.stp_classify_window(self.desc, self.window, self.sinks, self.se, self.pos, self.buf.tile_meta, stream=self.stream)

    def step(self):
        self.classify()
        stp.stp_attn_window_fwd(self.desc, self.window, self.sinks, self.q, self.k, self.v, self.se, self.pos,
                                self.buf.tile_meta, self.o, self.lse, self.buf.fwd_ws, stream=self.stream)
        stp.stp_attn_window_bwd(self.desc, self.window, self.sinks, self.q, self.k, self.v, self.o, self.lse, self.do,
                                self.se, self.pos, self.buf.tile_meta, self.dq, self.dk, self.dv, self.buf.bwd_ws,
                                stream=self.stream)

    def classes(self):
        n = self.desc.row_len // 128
        c = torch.empty(self.desc.n_rows, n, n, dtype=torch.int8, device="cuda")
        stp.stp_read_tile_classes(self.desc, self.buf.tile_meta, c, stream=self.stream)
        torch.cuda.synchronize()
        return c.cpu().numpy()

    def outputs(self):
        torch.cuda.synchronize()
        for ws in (self.buf.tile_meta, self.buf.fwd_ws, self.buf.bwd_ws):
            assert stp.stp_device_status(ws) == stp.STP_OK
        return {x: getattr(self, x).double().cpu().numpy() for x in ("o", "lse", "dq", "dk", "dv")}


def _forest(seed, T, **kw):
    kw = dict(n_roots=4, max_depth=3, len_lo=3, len_hi=90, min_shared=8) | kw
    b = W.random_forest(seed, row_len=T, **kw)
    return OP.pack(b.seqs, b.trainable, T, b.min_shared)


def _check(run, m):
    run.step()
    got = run.outputs()
    want = OW.attention(m, *(x.double().cpu().numpy() for x in (run.q, run.k, run.v)), run.desc.c().scale,
                        run.do.double().cpu().numpy())
    u = torch.finfo(run.q.dtype).eps / 2 + WORK
    assert np.abs(got["lse"] - want["lse"]).max() <= 32 * WORK
    for x in ("o", "dq", "dk", "dv"):
        off = np.abs(got[x] - want[x]) - u * want[x + "_tol"]
        assert off.max() <= 1e-6, (x, off.max())
    # the classes: what is visible lies in listed tiles, what is FULL is visible
    c, R, n = run.classes(), len(m), m.shape[1] // 128
    tiles = m.reshape(R, n, 128, n, 128)
    assert not (tiles.any((2, 4)) & (c == 0)).any()
    assert not (~tiles.all((2, 4)) & (c == 2)).any()
    assert (c != 0).sum() == run.pairs
    return c


@pytest.mark.parametrize("hq,hkv,window,sinks", [(2, 1, 1, 0), (1, 1, 1, 1), (4, 2, 37, 4), (3, 1, 128, 0), (8, 1, 129, 300),
                                                 (2, 2, 500, 2), (2, 1, 2 ** 31 - 1, 0)])
def test_bf16_forests(hq, hkv, window, sinks):
    plan = _forest(hq * 10 + window % 97, 512)
    _check(Run(plan.subtree_end, plan.position_ids, hq, hkv, 128, stp.STP_BF16, window, sinks, seed=window % 89),
           OW.mask(plan, window, sinks))


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("window,sinks", [(1, 0), (50, 3), (1000, 0)])
def test_fp32_forests(d, window, sinks):
    plan = _forest(d + window, 256, len_hi=60)
    _check(Run(plan.subtree_end, plan.position_ids, 2, 1, d, stp.STP_FP32, window, sinks, seed=window),
           OW.mask(plan, window, sinks))


@pytest.mark.parametrize("window,sinks", [(1, 0), (127, 0), (129, 4), (300, 130)])
def test_one_long_sequence_drops_far_tiles(window, sinks):
    T = 1024
    se, pos = np.full((1, T), T - 1, np.int32), np.arange(T, dtype=np.int32)[None]
    i, j = np.arange(T)[:, None], np.arange(T)[None]
    m = ((j <= i) & ((i - j < window) | (j < sinks)))[None]
    c = _check(Run(se, pos, 2, 1, 128, stp.STP_BF16, window, sinks, seed=3), m)
    assert ((c != 0) == m.reshape(1, 8, 128, 8, 128).any((2, 4))).all()       # no tile more than needed


def test_row_of_pads_and_one_tile():
    T = 128
    se, pos = np.tile(np.arange(T, dtype=np.int32), (2, 1)), np.zeros((2, T), np.int32)
    se[1, :50], pos[1, :50] = 49, np.arange(50)        # the second row holds one sequence
    m = np.zeros((2, T, T), bool)
    m[:, np.arange(T), np.arange(T)] = True
    for i in range(50):
        m[1, i, max(0, i - 6):i + 1] = True
        m[1, i, :min(i + 1, 2)] = True
    _check(Run(se, pos, 2, 2, 128, stp.STP_BF16, 7, 2), m)


def test_a_window_of_everything_is_tree_attention():
    """A window that hides nothing gives the bits of the unwindowed calls."""
    plan = _forest(5, 1024)
    r = Run(plan.subtree_end, plan.position_ids, 4, 2, 128, stp.STP_BF16, 1 << 30, 0, seed=2)
    r.step()
    a = r.outputs()
    stp.stp_classify(r.desc, r.se, r.buf.tile_meta)
    stp.stp_attn_fwd(r.desc, r.q, r.k, r.v, r.se, r.buf.tile_meta, r.o, r.lse, r.buf.fwd_ws)
    stp.stp_attn_bwd(r.desc, r.q, r.k, r.v, r.o, r.lse, r.do, r.se, r.buf.tile_meta, r.dq, r.dk, r.dv, r.buf.bwd_ws)
    b = r.outputs()
    for x in a:
        assert np.array_equal(a[x], b[x]), x


def test_same_bits_with_bounded_workspace_and_on_another_stream():
    plan = _forest(6, 512)
    args = (plan.subtree_end, plan.position_ids, 8, 4, 128, stp.STP_BF16, 40, 4)
    outs = []
    for r in (Run(*args), Run(*args), Run(*args, ds_groups=1), Run(*args, stream=torch.cuda.Stream())):
        r.step()
        outs.append(r.outputs())
    for o in outs[1:]:
        for x in o:
            assert np.array_equal(o[x], outs[0][x]), x


def test_captured_step():
    plan = _forest(7, 512)
    r = Run(plan.subtree_end, plan.position_ids, 4, 2, 128, stp.STP_BF16, 64, 4)
    r.step()                                    # the first call of a process creates the library's streams
    want = r.outputs()
    for x in ("o", "dq", "dk", "dv", "lse"):
        getattr(r, x).fill_(float("nan"))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        r.stream = torch.cuda.current_stream()
        r.step()
    g.replay()
    got = r.outputs()
    for x in want:
        assert np.array_equal(got[x], want[x]), x


def test_bad_positions_set_the_device_error_word():
    plan = _forest(8, 256)
    r = Run(plan.subtree_end, plan.position_ids, 1, 1, 128, stp.STP_BF16, 9, 0)
    for bad in (-1, 1 << 30):
        r.pos[0, 100] = bad
        r.classify()
        assert stp.stp_device_status(r.buf.tile_meta) == stp.STP_EDEVICE
    r.pos[0, 100] = int(plan.position_ids[0, 100])
    r.classify()
    assert stp.stp_device_status(r.buf.tile_meta) == stp.STP_OK

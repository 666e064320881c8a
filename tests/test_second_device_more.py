"""The policy loss, the embedding's gradient and the weight gradient from 8-bit
checkpoints in a process that uses two devices: their kernels' shared-memory
limits are raised on each device before the first launch there.  As
tests/test_second_device.py, against its stand-in for the CUDA runtime; no GPU
is touched."""
import subprocess
import sys
import textwrap

from conftest import ROOT
from test_second_device import fake_lib  # noqa: F401

CALLS = """
import ctypes, sys
sys.path.insert(0, sys.argv[2])
from sft_trie_build_gb300 import stp
stp.LIB_PATH = sys.argv[1]
fake = ctypes.CDLL(sys.argv[1])
A = 1 << 20
B, F = stp.STP_BF16, stp.STP_FP32

def policy(dt, n):
    d = stp.policy_desc(n, 40000, dt, kl_coef=0.1)
    stp.stp_policy_fwd(d, *[A] * 11, stream=0)
    stp.stp_policy_bwd(d, *[A] * 10, stream=0)
    stp.stp_policy_step(d, *[A] * 13, stream=0)

def embed(dt, n):
    d = stp.embed_desc(n, 1000, 64, dt)
    stp.stp_embed_fwd(d, A, A, A, A, stream=0)
    stp.stp_embed_bwd(d, A, A, 0, A, A, stream=0)

def wgrad(dt, n):
    d = stp.ckpt_desc(n, 300, dt)
    stp.stp_ckpt_save(d, A, A, stream=0)
    stp.stp_ckpt_wgrad(d, 500, A, A, 504, 0, A, A, stream=0)

calls = [lambda dt=dt, n=n, f=f: f(dt, n) for f in (policy, embed, wgrad) for dt in (B, F) for n in (2, 7000)]
for device in (0, 1, 5, 0):
    fake.fake_device(device)
    for call in calls:
        call()
assert fake.fake_launches() > 4 * len(calls)
assert fake.fake_bad() == 0, f"{fake.fake_bad()} of {fake.fake_launches()} launches refused"
# a setting that fails once is an error of that call alone
fake.fake_device(7)
for call in calls:
    fake.fake_fail(1)
    try:
        call()
    except stp.StpError as e:
        assert e.status == stp.STP_ECUDA
    fake.fake_fail(0)
    call()
assert fake.fake_bad() == 0
print("done")
"""


def test_limits_are_raised_on_every_device(fake_lib):  # noqa: F811
    p = subprocess.run([sys.executable, "-c", textwrap.dedent(CALLS), fake_lib, ROOT], capture_output=True, text=True,
                       timeout=300)
    assert p.returncode == 0 and "done" in p.stdout, p.stdout + p.stderr

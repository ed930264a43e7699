"""The feed-forward handle with two devices, on a CUDA runtime made for it
(tests/host_fakes): no GPU is used, and a child process keeps the preloaded
runtime to itself."""
import os
import shutil
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SRC = os.path.join(ROOT, "tests", "host_fakes", "two_devices.c")

pytestmark = pytest.mark.skipif(not shutil.which("gcc"), reason="no C compiler")


@pytest.fixture(scope="module")
def runtime(tmp_path_factory):
    out = tmp_path_factory.mktemp("fake") / "two_devices.so"
    subprocess.run(["gcc", "-O1", "-std=gnu11", "-Wall", "-shared", "-fPIC", "-I", "/usr/local/cuda/include", SRC, "-o",
                    str(out)], check=True)
    return str(out)


PROLOGUE = """
import ctypes, sys
sys.path.insert(0, {root!r})
import layout_aware_collectives_gb300 as tide
fake = ctypes.CDLL({fake!r})
A = 4096  # an address that nothing reads

def on(device):
    fake.cudaSetDevice(device)

def bound(device):
    c = tide.Compute()
    on(device)
    c.fp8_store(1, 128, A, A, A)
    return c

def refused(status, call, *a):
    try:
        call(*a)
    except tide.TideError as e:
        assert e.status == status, e
        return
    raise AssertionError("not refused")
"""


def child(runtime, body):
    code = PROLOGUE.format(root=ROOT, fake=runtime) + body
    env = dict(os.environ, LD_PRELOAD=runtime)
    res = subprocess.run([sys.executable, "-c", code], env=env, capture_output=True, text=True, timeout=120)
    assert res.returncode == 0, res.stdout + res.stderr


def test_check_device_is_of_the_handle_s_device(runtime):
    """With another device current the handle's kernels may still be running:
    the check waits for no other device, and misses no error."""
    child(runtime, """
c = bound(0)
assert fake.fake_launches() == 1
fake.fake_error_at_sync(0, 1)
on(1)
before = fake.fake_syncs(1)
refused(tide.TIDE_ERR_INVALID_ARG, c.check_device)
assert fake.fake_syncs(1) == before and fake.fake_syncs(0) == 0
on(0)
refused(tide.TIDE_ERR_TIMEOUT, c.check_device)
assert fake.fake_syncs(0) == 1
fake.fake_error_at_sync(0, 0)
c.check_device()
""")


def test_handle_keeps_its_own_device_s_properties(runtime):
    """How a contraction is split, and with it the order of its sums, goes by
    the handle's own device, whatever handle was bound since."""
    child(runtime, """
def shapes(c):
    out = []
    def note(call, *a, **kw):
        call(*a, **kw)
        out.append((fake.fake_grid(0), fake.fake_grid(1), fake.fake_grid(2), fake.fake_cluster()))
    for m, n, k in ((1, 2048, 8192), (1014, 752, 9200), (200, 2368, 7904)):
        note(c.fp8_matmul, m, n, k, A, A, A, A, A)
    for t, k, f in ((1, 2048, 8192), (40, 2048, 768), (1014, 9200, 752), (200, 7904, 2368)):
        note(c.gated_forward, t, k, f, A, A, A, A)
    return out

first = bound(0)
want = shapes(first)
assert any(s[3] > 2 for s in want)
second = bound(1)
other = shapes(second)
assert other != want
on(0)
assert shapes(first) == want, (shapes(first), want)
third = bound(0)
assert shapes(third) == want
on(1)
assert shapes(second) == other
""")

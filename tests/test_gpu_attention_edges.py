"""GPU tests of the attention entry points at their edges."""
import os
import subprocess
import sys

import pytest

from test_gpu_attention import _Case, env  # noqa: F401

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


# ------------------------------------------------------------------ kv_plan ----

def test_plan_around_the_default_shared_memory_limit(env):
    """Four ints a sequence and a few static bytes pass 48 KB between 3056 and 3057 sequences.
    In a process of its own: a larger call would raise the limit for the ones after it."""
    code = """
import sys, torch
sys.path[:0] = [{root!r}, {tests!r}]
import split_switched_decode_gb300 as ssd
from test_gpu_attention import _check_plan, _plan_case
env = (torch, ssd, torch.device("cuda:0"))
for S in (3056, 3057, 3072, 3073):
    for max_tokens in (4096, 5000):          # one CTA, a cluster
        kv, new, table, free = _plan_case(S, S, 16, 40, 2)
        _check_plan(env, kv, new, table, free, 0, 16, max_tokens)
print("plans agree")
""".format(root=ROOT, tests=os.path.join(ROOT, "tests"))
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "plans agree" in r.stdout, r.stdout + r.stderr


# ----------------------------------------------------------- waits that run out ----

def _held(env, c):
    """Runs the case with the multiplying warps waiting for what never comes; then, on a
    zero-filled workspace, as ever. Outputs have to be what they were, and the time-out known."""
    torch, ssd, dev = env
    want, want_lse = c.check() if sum(c.lengths) < 5000 else c.run()
    assert ssd.dec_sync_status() == ssd.DEC_OK
    ssd.dec_set_wait_limit_ns(1_000_000)
    ssd.dec_debug_attn_timeout(True)
    try:
        c.run()
        assert ssd.dec_sync_status() == ssd.DEC_ERR_TIMEOUT
    finally:
        ssd.dec_debug_attn_timeout(False)
        ssd.dec_set_wait_limit_ns(2_000_000_000)
    c.ws.zero_()
    got, lse = c.run()
    assert ssd.dec_sync_status() == ssd.DEC_OK
    assert torch.equal(got, want) and torch.equal(lse, want_lse)


@pytest.mark.parametrize("lengths", [[40], [300, 70, 0, 1000], [6000] * 20])
@pytest.mark.parametrize("page", [16, 13])
@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_attn_wait_that_runs_out(env, D, e4m3, page, lengths):
    """Boxes (pages of 16) and 16-byte copies (of 13); ranges that end before the time-out does
    (the copying warps are done with their stages by then) and longer ones."""
    _held(env, _Case(env, lengths, [1] * len(lengths), 8, 1, D, page, e4m3, seed=D))


@pytest.mark.parametrize("lengths", [[40], [300, 70, 0, 1000], [6000] * 20])
@pytest.mark.parametrize("rows", [4, 8, 16])
@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_attn_many_rows_wait_that_runs_out(env, D, e4m3, rows, lengths):
    """The same with products in flight as well, in items of 32, 64 and 128 rows."""
    _held(env, _Case(env, lengths, [rows] * len(lengths), 8, 1, D, 16, e4m3, seed=rows))

"""GPU tests of the attention entry points at their edges."""
import os
import subprocess
import sys

import pytest

from test_gpu_attention import env  # noqa: F401

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

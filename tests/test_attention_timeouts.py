"""What the attention kernels do when a wait runs out, as far as that can be seen without a
GPU: whether copies or products are still in flight may be decided only once no role of the
CTA can run into a time-out any more. Read from the kernels' sources."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "split_switched_decode_gb300", "csrc")
FLAG = "*static_cast<volatile int *>(&abort_flag)"


def _kernel(name, file):
    """The body of __global__ function `name`, comments taken out."""
    with open(os.path.join(CSRC, file)) as f:
        text = re.sub(r"//[^\n]*", "", f.read())
    at = text.index("{", text.index(f" {name}("))
    depth = 0
    for i in range(at, len(text)):
        depth += {"{": 1, "}": -1}.get(text[i], 0)
        if depth == 0:
            return text[at:i + 1]
    raise AssertionError(f"{name}: no end")


def _only(text, part):
    assert text.count(part) == 1, (part, text.count(part))
    return text.index(part)


def test_copies_are_drained_after_the_last_wait_of_the_multiplying_warps():
    body = _kernel("attn_decode_kernel", "attn_kernel.cuh")
    roles = body.index("if (warp >= AT_CWARPS) {")
    end = body.index("return;", roles)
    copying, multiplying = body[roles:end], body[end + len("return;"):]
    met = _only(copying, "named_bar_sync(3, AT_THREADS)")
    assert copying.rindex("mbar_wait_bounded(") < met
    assert met < _only(copying, FLAG) < _only(copying, "mbar_wait_drain(")
    assert multiplying.rindex("mbar_wait_bounded(") < _only(multiplying,
                                                            "named_bar_arrive(3, AT_THREADS)")
    assert "return;" not in multiplying


def test_products_and_copies_are_drained_before_tensor_memory_is_released():
    body = _kernel("attn_tc_kernel", "attn_tc.cuh")
    joins = _only(body, "run_joins<")          # by every thread, after the roles
    met = body.index("__syncthreads();", joins)
    flag = _only(body, FLAG)
    assert "wait(" not in body[joins:] and "wait_pv(" not in body[joins:]
    assert joins < met < flag < body.index("tc_commit(bar)", flag)
    assert body.index("mbar_wait_drain(") > flag and body.count("mbar_wait_drain(") == 2
    assert body.rindex("mbar_wait_drain(") < body.rindex("__syncthreads();")
    assert body.rindex("__syncthreads();") < _only(body, "tmem_dealloc(")
    # no role leaves before the joins (only a CTA without work, as a whole)
    assert body.count("return;") == 1 and body.index("return;") < body.index("tmem_alloc(")


@pytest.mark.parametrize("on,status", [(2, 1), (-1, 1), (1, 0), (0, 0)])
def test_the_self_test_is_switched_on_and_off(on, status):
    import split_switched_decode_gb300 as ssd
    ssd.build()
    try:
        assert ssd.lib().dec_debug_attn_timeout(on) == status
    finally:
        ssd.dec_debug_attn_timeout(False)

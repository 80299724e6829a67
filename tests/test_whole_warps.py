"""Reads and writes of tensor memory (tcgen05 .sync.aligned) are executed by whole warps: read from
the kernels' sources, as a warp that is split there may stop the GPU. A loop that meets such an
instruction again must not go back to its head from a branch that rows take differently, and where
such a branch ended, the warp meets before the next one."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "split_switched_decode_gb300", "csrc")
ALIGNED = re.compile(r"\btmem_(ld|st|wait_ld|wait_st)\w*(<\w+>)?\(")
# conditions that all threads of a warp share
UNIFORM = {"k % GROUPS != grp"}


def _text(file):
    with open(os.path.join(CSRC, file)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


def _close(text, at, pair):
    depth = 0
    for i in range(at, len(text)):
        depth += (text[i] == pair[0]) - (text[i] == pair[1])
        if depth == 0:
            return i
    raise AssertionError("no end")


def _loops(text):
    """The bodies in braces of all for and while loops, outer ones before those inside."""
    for m in re.finditer(r"\b(for|while) \(", text):
        head = _close(text, m.end() - 1, "()")
        if text[head + 1:].lstrip().startswith("{"):
            at = text.index("{", head)
            yield text[at:_close(text, at, "{}") + 1]


def _condition(body, at):
    """Of the `if` whose statement is the `continue` at `at`."""
    head = max(body.rfind("if (", 0, at), 0)
    end = _close(body, head + 3, "()")
    return body[head + 4:end] if body[end + 1:at].strip() in ("", "{") else None


@pytest.mark.parametrize("file", ["attn_tc.cuh", "latent_decode.cuh", "latent_prompt.cu", "latent_project.cu"])
def test_loops_over_tensor_memory_do_not_start_again_from_a_branch(file):
    looked = 0
    for body in _loops(_text(file)):
        if not ALIGNED.search(body):
            continue
        looked += 1
        for inner in _loops(body[1:]):  # their `continue` is their own
            body = body.replace(inner, "{}") if not ALIGNED.search(inner) else body
        for m in re.finditer(r"\bcontinue;", body):
            assert _condition(body, m.start()) in UNIFORM, _condition(body, m.start())
    assert looked > 0


@pytest.mark.parametrize("file,after", [
    ("latent_prompt.cu", "o[e] += w * bf16_to_f32(v[e]);"),  # rows that see a value, and others
    ("latent_prompt.cu", "pack2<false>(y[4], y[5])"),        # rows that exist, and others
    ("latent_decode.cuh", "slot[(r0 + e) * DP + dim] = o[e];"),
    ("attn_tc.cuh", "o[e] += pr * to_f32<E4M3>(y);"),
    ("attn_tc.cuh", "make_float4(o[e], o[e + 1], o[e + 2], o[e + 3]);"),
])
def test_warps_meet_behind_branches_of_rows(file, after):
    text = _text(file)
    assert text.count(after) == 1
    behind = text[text.index(after):]
    met = behind.index("__syncwarp();")
    again = ALIGNED.search(behind)
    assert again is None or met < again.start()
    assert not re.search(r"\b(for|while) \(", behind[:met])
    # the last thing of its loop
    assert behind[met + len("__syncwarp();"):].lstrip().startswith("}")

"""Attention entry points without a GPU: host argument checks answer before any CUDA call,
the frequency tables follow their formulas, and the plain 64-bit forms that the GPU tests
compare with give what can be worked out by hand."""
import ctypes
import math

import numpy as np
import pytest

import attn_ref


@pytest.fixture(scope="module")
def ssd():
    import split_switched_decode_gb300 as m
    m.build()
    return m


A, U, N0 = ctypes.c_void_p(0x1000), ctypes.c_void_p(0x1002), None  # never dereferenced
B = ctypes.c_void_p(0x900000)


def _changed(args, changes):
    args = list(args)
    for i, v in changes.items():
        args[i] = v
    return args


#            kv new S  ps tab mp free nf used len qst pos slo max sum s
PLAN_ARGS = [A, A, 4, 16, A, 8, A, 32, A, A, A, A, A, 64, A, None]


@pytest.mark.parametrize("changes,status", [
    ({0: N0}, "INVALID_ARG"), ({2: 0}, "INVALID_ARG"), ({3: 0}, "INVALID_ARG"),
    ({4: N0}, "INVALID_ARG"), ({5: 0}, "INVALID_ARG"), ({6: N0}, "INVALID_ARG"),
    ({7: -1}, "INVALID_ARG"), ({9: N0}, "INVALID_ARG"), ({10: N0}, "INVALID_ARG"),
    ({11: N0}, "INVALID_ARG"), ({12: N0}, "INVALID_ARG"), ({13: 0}, "INVALID_ARG"),
    ({14: N0}, "INVALID_ARG"), ({2: 8193}, "UNSUPPORTED_SHAPE"), ({0: U}, "MISALIGNED"),
    ({13: (1 << 28) + 1}, "UNSUPPORTED_SHAPE"), ({8: U}, "MISALIGNED"), ({14: U}, "MISALIGNED"),
])
def test_kv_plan_refusals(ssd, changes, status):
    assert ssd.lib().kv_plan(*_changed(PLAN_ARGS, changes)) == getattr(ssd, "DEC_ERR_" + status)


#            q qs   k  ks   v  vs   pos sl inv mag T Hq Hkv D  rot il out os  kc vc ty
ROPE_ARGS = [A, 512, A, 128, A, 128, A, A, A, 1.0, 2, 4, 1, 128, 128, 0, B, 512, A, A, 0,
             # ksc vsc pages ps  page   head token stream
             N0, N0, 10, 16, 2048, 2048, 128, None]


@pytest.mark.parametrize("changes,status", [
    ({0: N0}, "INVALID_ARG"), ({2: N0}, "INVALID_ARG"), ({4: N0}, "INVALID_ARG"),
    ({6: N0}, "INVALID_ARG"), ({7: N0}, "INVALID_ARG"), ({8: N0}, "INVALID_ARG"),
    ({16: N0}, "INVALID_ARG"), ({18: N0}, "INVALID_ARG"), ({19: N0}, "INVALID_ARG"),
    ({10: 0}, "INVALID_ARG"), ({11: 0}, "INVALID_ARG"), ({12: 0}, "INVALID_ARG"),
    ({14: 127}, "INVALID_ARG"), ({14: 130}, "INVALID_ARG"), ({14: -2}, "INVALID_ARG"),
    ({15: 2}, "INVALID_ARG"), ({20: 2}, "INVALID_ARG"), ({23: 0}, "INVALID_ARG"),
    ({24: 0}, "INVALID_ARG"), ({1: 504}, "INVALID_ARG"), ({3: 120}, "INVALID_ARG"),
    ({16: A, 17: 520}, "INVALID_ARG"),                 # in place with another stride
    ({13: 120}, "UNSUPPORTED_SHAPE"), ({13: 272}, "UNSUPPORTED_SHAPE"),
    ({10: (1 << 20) + 1}, "UNSUPPORTED_SHAPE"), ({11: 1025, 1: 1 << 20, 17: 1 << 20},
                                                 "UNSUPPORTED_SHAPE"),
    ({23: 1 << 20, 24: 1 << 12}, "UNSUPPORTED_SHAPE"),  # a slot passes int32
    ({0: U}, "MISALIGNED"), ({18: U}, "MISALIGNED"), ({1: 516}, "MISALIGNED"),
    ({25: 2044}, "MISALIGNED"), ({20: 1, 27: 136}, "MISALIGNED"),  # e4m3 rows of 16 bytes
])
def test_rope_append_refusals(ssd, changes, status):
    got = ssd.lib().rope_append(*_changed(ROPE_ARGS, changes))
    assert got == getattr(ssd, "DEC_ERR_" + status)


#            q qs   kc vc ty ksc vsc pg ps page   head  tok  tab mp len qst S T Hq Hkv D
ATTN_ARGS = [A, 512, A, A, 0, N0, N0, 10, 16, 2048, 2048, 128, A, 8, A, A, 2, 3, 4, 1, 128,
             # scale win out os  lse ws bytes    stream
             0.1, 0, B, 512, A, A, 1 << 30, None]


@pytest.mark.parametrize("changes,status", [
    ({0: N0}, "INVALID_ARG"), ({2: N0}, "INVALID_ARG"), ({3: N0}, "INVALID_ARG"),
    ({12: N0}, "INVALID_ARG"), ({14: N0}, "INVALID_ARG"), ({23: N0}, "INVALID_ARG"),
    ({26: N0}, "INVALID_ARG"), ({16: 0}, "INVALID_ARG"), ({17: 0}, "INVALID_ARG"),
    ({18: 0}, "INVALID_ARG"), ({19: 0}, "INVALID_ARG"), ({20: 0}, "INVALID_ARG"),
    ({13: 0}, "INVALID_ARG"), ({22: -1}, "INVALID_ARG"), ({4: 7}, "INVALID_ARG"),
    ({15: N0}, "INVALID_ARG"),                          # no q_start, but T != S
    ({19: 3}, "INVALID_ARG"), ({23: A}, "INVALID_ARG"), ({24: 504}, "INVALID_ARG"),
    ({16: 8193}, "UNSUPPORTED_SHAPE"), ({17: 65537}, "UNSUPPORTED_SHAPE"),
    ({20: 264}, "UNSUPPORTED_SHAPE"), ({20: 24}, "UNSUPPORTED_SHAPE"),
    ({18: 1028, 24: 1 << 20}, "UNSUPPORTED_SHAPE"),
    ({0: U}, "MISALIGNED"), ({2: U}, "MISALIGNED"), ({26: U}, "MISALIGNED"),
    ({1: 516}, "MISALIGNED"), ({11: 129}, "MISALIGNED"),
])
def test_attn_decode_refusals(ssd, changes, status):
    got = ssd.lib().attn_decode(*_changed(ATTN_ARGS, changes))
    assert got == getattr(ssd, "DEC_ERR_" + status)


def test_workspace_of_unsupported_shapes_is_zero(ssd):
    for shape in ((0, 1, 1, 1, 64), (1, 1, 3, 2, 64), (1, 1, 4, 2, 24), (1, 1, 4, 2, 512)):
        assert ssd.attn_decode_workspace_bytes(*shape) == 0


def _relative(got, want):
    return np.max(np.abs(got.numpy().astype(np.float64) - want) / want)


@pytest.mark.parametrize("rot,base", [(2, 10000.0), (64, 10000.0), (128, 500000.0), (256, 1e6)])
def test_frequencies_plain_linear_base(ssd, rot, base):
    i = np.arange(rot // 2)
    plain = base ** (-2.0 * i / rot)
    inv, mag = ssd.rope_frequencies(rot, base)
    assert mag == 1.0 and _relative(inv, plain) <= 2.0 ** -24  # rounded once
    inv, mag = ssd.rope_frequencies(rot, base, ssd.ROPE_LINEAR, 8.0)
    assert mag == 1.0 and _relative(inv, plain / 8.0) <= 2.0 ** -24
    if rot >= 4:
        inv, mag = ssd.rope_frequencies(rot, base, ssd.ROPE_BASE, 8.0)
        assert mag == 1.0 and inv[0] == 1.0
        # the slowest pair is interpolated by exactly the factor
        assert abs(float(inv[-1]) / (plain[-1] / 8.0) - 1.0) <= 2.0 ** -23


def test_frequencies_by_parts(ssd):
    rot, base, factor, orig = 128, 10000.0, 4.0, 4096
    inv, mag = ssd.rope_frequencies(rot, base, ssd.ROPE_PARTS, factor, orig)
    assert mag == np.float32(0.1 * math.log(factor) + 1.0)
    plain = base ** (-2.0 * np.arange(rot // 2) / rot)
    turns = orig * plain / (2 * math.pi)
    ratio = inv.numpy() / plain
    # more than 32 turns: kept; less than one: interpolated (one pair of slack for the
    # ramp's whole-numbered ends); monotone between
    assert np.allclose(ratio[turns > 33 * base ** (2.0 / rot)], 1.0, atol=1e-6)
    assert np.allclose(ratio[turns < 1 / base ** (2.0 / rot)], 1.0 / factor, atol=1e-6)
    assert np.all(np.diff(ratio) <= 1e-6) and ratio[0] > ratio[-1]


@pytest.mark.parametrize("args", [
    (0, 10000.0), (3, 10000.0), (258, 10000.0), (64, 1.0), (64, float("nan")),
    (64, float("inf")), (64, 10000.0, 4), (64, 10000.0, 1, 0.5), (64, 10000.0, 1, float("nan")),
    (2, 10000.0, 2, 2.0), (64, 10000.0, 3, 2.0, 0), (64, 10000.0, 3, 2.0, 4096, 1.0, 1.0),
    (64, 10000.0, 3, 2.0, 4096, 32.0, 0.0),
])
def test_frequencies_refusals(ssd, args):
    with pytest.raises(ssd.DecError) as e:
        ssd.rope_frequencies(*args)
    assert e.value.status == ssd.DEC_ERR_INVALID_ARG


# ------------------------------------------------- the plain forms themselves ----

def test_plain_plan_by_hand():
    table = np.full((3, 3), -1)
    table[0, 0], table[2, 0], table[2, 1] = 7, 5, 6
    got = attn_ref.kv_plan([3, 0, 8], [2, 0, 1], table, [11, 12, 13], 1, 4, 4)
    assert got[0].tolist() == [[7, 12, -1], [-1, -1, -1], [5, 6, 13]]
    assert got[1].tolist() == [5, 0, 9] and got[2].tolist() == [0, 2, 2, 3]
    assert got[3].tolist() == [3, 4, 8, 0] and got[4].tolist() == [31, 48, 52, -1]
    assert got[5].tolist() == [3, 3, 0, 0]


def test_plain_rotation_keeps_length_and_composes():
    rng = np.random.default_rng(0)
    x = rng.standard_normal((2, 8))
    inv = np.array([1.0, 0.1, 0.01])
    for il in (False, True):
        y, _ = attn_ref.rotate(x, 5, inv, 1.0, il)
        z, _ = attn_ref.rotate(y, 7, inv, 1.0, il)
        w, _ = attn_ref.rotate(x, 12, inv, 1.0, il)
        assert np.allclose(z, w) and np.allclose(y[:, 6:], x[:, 6:])
        assert np.allclose(np.linalg.norm(y, axis=1), np.linalg.norm(x, axis=1))
    # a quarter turn of the first pair, by hand
    y, _ = attn_ref.rotate(np.array([[1.0, 2.0, 3.0, 4.0]]), 1, [math.pi / 2], 2.0, False)
    assert np.allclose(y, [[-4.0, 2.0, 3.0, 4.0]])


def test_plain_attention_by_hand():
    # equal scores: the mean of what is seen; the causal row sees one key less
    q, k = np.zeros((2, 2, 4)), np.ones((3, 1, 4))
    v = np.arange(12, dtype=float).reshape(3, 1, 4)
    out, lse, _, _ = attn_ref.attention(q, k, v, np.ones(3, bool), 1.0, 0)
    assert np.allclose(out[0, 0], v[:2, 0].mean(0)) and np.allclose(out[1, 1], v[:, 0].mean(0))
    assert np.allclose(lse[:, 0], [math.log(2), math.log(3)])
    out, lse, _, _ = attn_ref.attention(q, k, v, np.ones(3, bool), 1.0, 1)
    assert np.allclose(out[:, 0], v[1:, 0]) and np.allclose(lse, 0.0)
    out, lse, _, _ = attn_ref.attention(q, k, v, np.zeros(3, bool), 1.0, 0)
    assert not out.any() and np.all(lse == -np.inf)

"""GPU tests of the attention entry points at their edges."""
import math
import os
import subprocess
import sys

import numpy as np
import pytest

import attn_ref
from test_gpu_attention import U, _Case, _f64, _i32, env  # noqa: F401

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


@pytest.mark.parametrize("rows", [1, 8])
@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("D", [64, 128])
def test_attn_segments_longer_than_the_wait_limit(env, D, e4m3, rows):
    """Every stage comes in time, so nothing runs out, however long a CTA is at one item: some
    117 million tokens (the same four pages again and again) take several milliseconds under
    a limit of one. Repeated tokens change the sum of the weights, not the mean.

    Tolerance: that of the other cases, and 2^-23 for each of the up to 12000 * 4 sums of
    products that an output adds up (2^-24 for the 12000 of a row's sum)."""
    torch, ssd, dev = env
    page, pages, times, Hq = 4096, 4, 7168, 8
    n = page * pages
    g = torch.Generator(device=dev).manual_seed(D)
    dt = torch.float8_e4m3fn if e4m3 else torch.bfloat16
    kc, vc = (torch.randn((pages, 1, page, D), generator=g, device=dev).to(dt) for _ in range(2))
    q = torch.randn((rows, Hq, D), generator=g, device=dev).to(torch.bfloat16)
    table = torch.arange(pages * times, dtype=torch.int32, device=dev).view(1, -1) % pages
    out = torch.zeros_like(q)
    lse = torch.zeros((rows, Hq), dtype=torch.float32, device=dev)
    ws = ssd.workspace(ssd.attn_decode_workspace_bytes(1, rows, Hq, 1, D))
    ssd.dec_set_wait_limit_ns(1_000_000)
    try:
        ssd.attn_decode(q, kc, vc, table, _i32(torch, [n * times], dev), out, ws,
                        q_start=_i32(torch, [0, rows], dev), lse=lse)
        assert ssd.dec_sync_status() == ssd.DEC_OK
    finally:
        ssd.dec_set_wait_limit_ns(2_000_000_000)
    k, v = (_f64(c).reshape(n, 1, D) for c in (kc, vc))
    for i in range(rows):  # each alone over all tokens: what the others do not see is 2^-24
        want, wl, size, reach = attn_ref.attention(_f64(q[i:i + 1]), k, v, np.ones(n, bool),
                                                   D ** -0.5, 0)
        score = (D + 16) * 2.0 ** -24 * reach
        extra = 12000 * (4 * 2.0 ** -23 + 2.0 ** -24)
        bound = U * np.abs(want) + (U + 2 * score[..., None] + 2.0 ** -18 + extra) * size
        assert np.all(np.abs(_f64(out[i:i + 1]) - want) <= bound)
        got = lse[i:i + 1].cpu().numpy().astype(np.float64)
        assert np.all(np.abs(got - wl - math.log(times))
                      <= score + 12000 * 2.0 ** -24 + 2.0 ** -18)


# ------------------------------------------------------------------ flat tails ----

@pytest.mark.parametrize("peak", [10.0, 14.0, 16.0, 18.0, 20.0])
@pytest.mark.parametrize("rows,n", [(1, 100), (1, 1000), (2, 300), (4, 500), (8, 500), (16, 900)])
@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("D", [64, 256])
def test_attn_flat_tail_under_a_peak(env, D, e4m3, rows, n, peak):
    """One key 14 to 29 powers of two above all others, whose values alone count (the peak's is
    zero): what is lost of the others' weights is lost of the outputs.

    Weights round by 2^-8 (bf16) or 2^-11 of themselves or 2^-32 of the largest (f16), outputs
    by 2^-8."""
    torch, ssd, dev = env
    c = _Case(env, [n], [rows], 8, 1, D, 16, e4m3, seed=n)
    one = torch.ones(1, device=dev)
    c.ks = c.vs = one if e4m3 else None
    kind = torch.uint8 if e4m3 else torch.int16
    keys = torch.zeros((n, D), device=dev)
    keys[:, 0] = 0.125
    keys[3, 0] = peak
    values = torch.randint(8, 16, (n, D), device=dev, generator=torch.Generator(dev).manual_seed(1))
    values = values.float() / 8                 # 1 to 2, in steps that both types have
    values[3] = 0.0
    for cache, x in ((c.kc, keys), (c.vc, values)):
        x = x.to(cache.dtype).view(kind)
        for i in range(0, n, 16):
            cache[int(c.table[0, i // 16]), 0, :len(x[i:i + 16])].view(kind).copy_(x[i:i + 16])
    c.q.zero_()
    c.q[:, :, 0] = 1.0
    c.scale = 1.0
    got, lse = (_f64(t) for t in c.run())
    w = np.exp(_f64(keys)[:, 0] - peak)
    v = _f64(values)
    u = 2.0 ** -11 if e4m3 else U
    floor = 2.0 ** -32 if e4m3 else 0.0
    for i in range(rows):
        seen = n - rows + i + 1
        total = w[:seen].sum()
        want, size = w[:seen] @ v[:seen] / total, w[:seen] @ np.abs(v[:seen]) / total
        # scores of one product each: 2^-22 |z| for the scaling and the difference
        bound = U * want + (u + 2.0 ** -21 * peak + 2.0 ** -18) * size \
            + floor * np.abs(v[:seen]).sum(0) / total
        assert np.all(np.abs(got[i] - want) <= bound), i
        assert np.all(np.abs(lse[i] - (peak + math.log(total))) <= 2.0 ** -21 * peak + 2.0 ** -18)


# -------------------------------------------- values that are not finite, little weight ----

def _peak_and_bad_value(env, n, rows, D, e4m3, peak, bad):
    """Token `peak` 200 above all others, and a value that is not finite, in element 5 of token
    `bad`: every row that sees it has an infinity or NaN there, little as the token weighs
    (2^-288), and is left alone elsewhere; rows that do not see it are as without it."""
    torch, ssd, dev = env
    c = _Case(env, [n], [rows], 8, 1, D, 16, e4m3, seed=n + rows)
    c.ks = None
    kind = torch.uint8 if e4m3 else torch.int16
    keys = torch.zeros((n, D), device=dev)
    keys[peak, 0] = 20.0
    keys = keys.to(c.kc.dtype).view(kind)
    for i in range(0, n, 16):
        page = c.kc[int(c.table[0, i // 16]), 0].view(kind)
        page[:min(16, n - i)].copy_(keys[i:i + 16])
    c.q.zero_()
    c.q[:, :, 0] = 10.0
    c.scale = 1.0
    want, want_lse = c.run()
    value = torch.full((1,), float("nan") if e4m3 else float("inf"), device=dev)
    cell = c.vc[int(c.table[0, bad // 16]), 0, bad % 16].view(kind)
    cell[5:6].copy_(value.to(c.vc.dtype).view(kind))
    got, lse = c.run()
    assert bool(torch.isfinite(want.float()).all())
    assert torch.equal(lse, want_lse)
    rest = [d for d in range(D) if d != 5]
    for i in range(rows):
        if n - rows + i >= bad:
            assert not bool(torch.isfinite(got[i, :, 5].float()).any()), i
            assert torch.equal(got[i][:, rest], want[i][:, rest]), i
        else:
            assert torch.equal(got[i], want[i]), i


@pytest.mark.parametrize("n,rows,peak,bad", [
    (100, 1, 97, 99), (100, 2, 97, 99), (100, 4, 96, 98), (100, 8, 96, 98), (104, 16, 96, 102),
])
@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_attn_bad_value_of_little_weight_that_some_rows_see(env, D, e4m3, n, rows, peak, bad):
    """Among the new tokens, beside the peak."""
    _peak_and_bad_value(env, n, rows, D, e4m3, peak, bad)


@pytest.mark.parametrize("n,rows,peak,bad", [
    (100, 1, 3, 40), (100, 4, 3, 40), (100, 8, 3, 40), (200, 8, 3, 70), (100, 16, 3, 40),
    (700, 16, 3, 150), (100, 8, 90, 5),
])
@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_attn_bad_value_of_little_weight_in_another_part(env, D, e4m3, n, rows, peak, bad):
    """Where the peak is another copy's, another softmax group's or another worker's, whose part
    makes that of the value's own vanish when they are joined."""
    _peak_and_bad_value(env, n, rows, D, e4m3, peak, bad)


# ------------------------------------------------------------------- workspaces ----

def test_attn_one_workspace_for_calls_of_any_sizes(env):
    """Counters stand at one place whatever the heads, rows, pages and cache type are."""
    torch, ssd, dev = env
    cases = [_Case(env, [2500, n], [rows, 1], Hq, Hkv, D, page, e4m3, seed=D + rows)
             for n, rows, Hq, Hkv, D, page, e4m3 in (
                 (3, 1, 8, 1, 64, 16, False), (90, 8, 8, 1, 256, 16, False),
                 (700, 2, 6, 3, 128, 13, True), (40, 16, 8, 2, 128, 32, False),
                 (1, 6, 16, 1, 256, 64, True), (500, 9, 8, 1, 64, 8, True))]
    ws = max((c.ws for c in cases), key=lambda t: t.numel())
    for c in cases:
        c.ws = ws
    wants = [c.check() for c in cases]
    for _ in range(2):
        for c, (out, lse) in zip(cases, wants):
            got, l = c.run()
            assert torch.equal(got, out) and torch.equal(l, lse)
    assert ssd.dec_sync_status() == ssd.DEC_OK


# ---------------------------------------------------------------- infinite queries ----

@pytest.mark.parametrize("rows", [1, 2, 8])
@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("D", [64, 128])
def test_attn_infinite_query_beside_large_ones(env, D, e4m3, rows):
    """A query of -infinity in one element makes every score -infinity where the keys are
    positive there, however large its other elements are: nothing is seen."""
    torch, ssd, dev = env
    c = _Case(env, [70, 300], [rows, rows], 8, 1, D, 16, e4m3, seed=D)
    kind = torch.uint8 if e4m3 else torch.int16
    for s, n in enumerate(c.lengths):
        for i in range(0, n, 16):
            cell = c.kc[int(c.table[s, i // 16]), 0, :min(16, n - i)]
            ones = torch.ones(cell.shape, device=dev).to(c.kc.dtype)
            cell.view(kind).copy_(ones.view(kind))
    want, want_lse = c.run()
    c.q[0] = 1e30
    c.q[0, :, 1] = -math.inf
    got, lse = c.run()
    assert not got[0].any() and bool((lse[0] == -math.inf).all())
    assert torch.equal(got[1:], want[1:]) and torch.equal(lse[1:], want_lse[1:])


@pytest.mark.parametrize("power", [10, 18, 24])
@pytest.mark.parametrize("rows", [1, 2, 8])
@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("D", [64, 256])
def test_attn_query_with_one_large_element(env, D, e4m3, rows, power):
    """An element of q far above the others that meets keys of zero: what the others give is as
    exact as without it."""
    torch, ssd, dev = env
    c = _Case(env, [70, 300], [rows, rows], 8, 1, D, 16, e4m3, seed=D + power)
    kind = torch.uint8 if e4m3 else torch.int16
    for s, n in enumerate(c.lengths):
        c.k[s][:, :, 3] = 0.0
        for i in range(0, n, 16):
            c.kc[int(c.table[s, i // 16]), :, :min(16, n - i), 3].view(kind).zero_()
    c.q[:, :, 3] = 2.0 ** power
    c.check()

"""GPU tests of latent attention where rows of a warp differ. Tolerances as in test_gpu_latent.py."""
import math
import time

import pytest

from test_gpu_latent import U, _Decode, _Prompt, _within, env  # noqa: F401 (a fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("V", [64, 128])
@pytest.mark.parametrize("H", [2, 160])  # (128 and 256 rows a CTA)
def test_prompt_values_not_finite_in_many_tokens(env, H, V):  # noqa: F811
    """Several values that are not finite in a tile, some rows of a warp that see them and some
    that do not, warps of which only some rows exist: rows that see one have it, the others keep
    their bits."""
    torch, ssd, dev = env
    p = _Prompt(env, [300, 77, 1], [300, 90, 40], H, V=V)
    p.run()
    assert ssd.dec_sync_status() == ssd.DEC_OK
    p.check()
    clean = p.out.clone()
    at = [(5, 3, math.inf), (40, 9, -math.inf), (41, 10, math.nan), (131, 17, math.inf), (290, 60, math.inf),
          (299, 61, math.nan), (300 + 20, 30, math.inf), (300 + 89, 31, -math.inf), (390 + 39, 5, math.inf)]
    for j, e, value in at:
        p.v[j, 1, e] = value
    p.out.fill_(5.0)
    p.run()
    assert ssd.dec_sync_status() == ssd.DEC_OK
    want = clean.clone()
    # token j of the keys belongs to row j - 300 - 13 + 300 of the second sequence, the last to the third's
    for j, e, value in at:
        rows = slice(j, 300) if j < 300 else (slice(max(300, j - 13), 377) if j < 390 else slice(377, 378))
        got = p.out[rows, 1, e]
        assert bool(got.isnan().all() if math.isnan(value) else (got == value).all()), (j, e)
        want[rows, 1, e] = got
    first = min(j for j, _, _ in at)
    assert torch.equal(p.out[:first], want[:first]) and torch.equal(p.out[:, 0], clean[:, 0])
    fine = want.isfinite()
    assert torch.equal(fine, p.out.isfinite())
    assert bool((p.out.float() - want.float())[fine].abs().max() <= 2.0 ** -7 * want.float()[fine].abs().max())


def test_decode_workspace_of_the_largest_call_serves_smaller_ones(env):  # noqa: F811
    """Sized once for a batch of single tokens, then used by fewer sequences with more rows each."""
    torch, ssd, dev = env
    size = lambda S, T, H: ssd.latent_decode_workspace_bytes(S, T, H, 512, 64)
    for most in ((64, 64, 16), (300, 300, 3), (5, 40, 128), (8192, 8192, 4)):
        for part in ((1, 1), (1, 2), (2, 1), (8, 3), (64, 64), (1, 4)):
            S, T = max(1, most[0] // part[0]), max(1, most[1] // part[1])
            for H in {most[2], max(1, most[2] // 2), 1}:
                assert size(S, T, H) <= size(*most), (most, S, T, H)
    ws = ssd.workspace(size(64, 64, 16), dev)
    for lens, rows, H in (([500] * 64, [1] * 64, 16), ([9000], [8], 16), ([3000, 20], [3, 20], 16),
                          ([9000], [64], 5), ([70] * 3, [21] * 3, 16)):
        for e4m3 in (False, True):
            d = _Decode(env, lens, rows, H, e4m3=e4m3)
            d.q, d.out, d.lse = d.q[:d.T], d.out[:d.T], d.lse[:d.T]
            d.ws = ws
            d.run()
            assert ssd.dec_sync_status() == ssd.DEC_OK
            d.check()


# ----------------------------------------------------------- waits that run out ----

def _held(env, run, outputs):  # noqa: F811
    """Runs with the warps that read the products waiting for what never comes, under a limit of a
    millisecond: that is told, soon, and the next call gives what the first one gave."""
    torch, ssd, dev = env
    run()
    assert ssd.dec_sync_status() == ssd.DEC_OK
    want = [x.clone() for x in outputs]
    ssd.dec_set_wait_limit_ns(1_000_000)
    ssd.dec_debug_attn_timeout(True)
    try:
        began = time.monotonic()
        run()
        assert ssd.dec_sync_status() == ssd.DEC_ERR_TIMEOUT
        took = time.monotonic() - began
    finally:
        ssd.dec_debug_attn_timeout(False)
        ssd.dec_set_wait_limit_ns(2_000_000_000)
    for x in outputs:
        x.fill_(5.0)
    run()
    assert ssd.dec_sync_status() == ssd.DEC_OK
    for x, y in zip(outputs, want):
        assert torch.equal(x, y)
    return took


# Each CTA meets the limit and then waits for its copies and products: 1 ms, and at most 10 ms for
# products, 20 for queries, 40 for tiles that were requested in part, whatever the lengths.
@pytest.mark.parametrize("rows,keys,H", [
    ([1], [1], 1), ([777], [777], 16), ([300, 0, 5], [300, 40, 700], 3), ([128], [60000], 2),
    ([300, 77], [300, 90], 160), ([256], [60000], 160),
])
def test_prompt_wait_that_runs_out(env, rows, keys, H):  # noqa: F811
    p = _Prompt(env, rows, keys, H, extra=0)
    took = _held(env, p.run, (p.out, p.lse))
    blocks = sum(-(-n // 128) for n in rows) * H
    assert took < 0.5 + 0.071 * -(-blocks // 152)


@pytest.mark.parametrize("T,H,K,N", [(1, 1, 8, 8), (1, 64, 128, 512), (65, 4, 128, 512), (128, 2, 64, 64),
                                     (4096, 64, 128, 512), (20000, 16, 512, 128)])
def test_project_wait_that_runs_out(env, T, H, K, N):  # noqa: F811
    """Few tiles, several a CTA, and thousands."""
    torch, ssd, dev = env
    g = torch.Generator(device=dev).manual_seed(T)
    x, w = (torch.randn(s, generator=g, device=dev).to(torch.bfloat16) for s in ((T, H, K), (H, N, K)))
    y = torch.empty((T, H, N), dtype=torch.bfloat16, device=dev)
    took = _held(env, lambda: ssd.latent_project(x, w, y), (y,))
    assert took < 0.5


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("H", [16, 64])
def test_decode_wait_that_runs_out_over_a_long_sequence(env, H, e4m3):  # noqa: F811
    """33 million tokens (four pages again and again) are more than 3000 stages a CTA; what is left of
    them after the time-out takes some ten microseconds each, not a hundred."""
    torch, ssd, dev = env
    page, times = 4096, 2048
    g = torch.Generator(device=dev).manual_seed(H)
    kind = torch.float8_e4m3fn if e4m3 else torch.bfloat16
    cache = torch.randn((4, page, 576), generator=g, device=dev).to(kind)
    table = (torch.arange(4 * times, dtype=torch.int32, device=dev).view(1, -1) % 4).contiguous()
    lens = torch.tensor([4 * page * times], dtype=torch.int32, device=dev)
    q = torch.randn((1, H, 576), generator=g, device=dev).to(torch.bfloat16)
    out = torch.empty((1, H, 512), dtype=torch.bfloat16, device=dev)
    lse = torch.empty((1, H), device=dev)
    ws = ssd.workspace(ssd.latent_decode_workspace_bytes(1, 1, H, 512, 64), dev)
    took = _held(env, lambda: ssd.latent_decode(q, cache, table, lens, out, ws, 0.05, lse=lse), (out, lse))
    assert took < 0.15


@pytest.mark.parametrize("strided", [False, True])  # rows of q in boxes, or copied
@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("H", [16, 64])
def test_decode_segments_longer_than_the_wait_limit(env, H, e4m3, strided):  # noqa: F811
    """Every stage comes in time, so nothing runs out, however long a CTA is at one sequence before it
    turns to the next: 11 million tokens, 100 and 22 million (four pages again and again) take
    milliseconds under a limit of one. Repeated tokens change the sum of the weights, not the mean.

    Tolerance: that of the other cases, and for each of a CTA's 3500 stages 2^-23 for each of the
    four sums of products that an output adds up, 2^-24 for that of its weights."""
    torch, ssd, dev = env
    import latent_ref
    page, R, W, scale = 4096, 512, 576, 0.05
    n, times = 4 * page, (683, 0, 1365)
    g = torch.Generator(device=dev).manual_seed(H)
    kind = torch.float8_e4m3fn if e4m3 else torch.bfloat16
    cache = torch.randn((4, page, W), generator=g, device=dev).to(kind)
    table = torch.arange(4 * max(times), dtype=torch.int32, device=dev).expand(3, -1) % 4
    lens = torch.tensor([n * times[0], 100, n * times[2]], dtype=torch.int32, device=dev)
    q = torch.randn((3, H * W + (64 if strided else 0)), generator=g, device=dev).to(torch.bfloat16)
    q = q[:, :H * W].unflatten(1, (H, W))
    out = torch.empty((3, H, R), dtype=torch.bfloat16, device=dev)
    lse = torch.empty((3, H), device=dev)
    ws = ssd.workspace(ssd.latent_decode_workspace_bytes(3, 3, H, R, W - R), dev)
    ssd.dec_set_wait_limit_ns(1_000_000)
    try:
        ssd.latent_decode(q, cache, table.contiguous(), lens, out, ws, scale, lse=lse)
        assert ssd.dec_sync_status() == ssd.DEC_OK
    finally:
        ssd.dec_set_wait_limit_ns(2_000_000_000)
    keys = cache.float().double().view(1, n, W)
    extra = 3500 * (4 * 2.0 ** -23 + 2.0 ** -24)
    for s in range(3):
        k = keys if times[s] else keys[:, :100]
        at = torch.full((1,), k.shape[1] - 1, device=dev)
        want, wl, size, reach = latent_ref.attend(q[s:s + 1].double(), k, k[..., :R], at, scale)
        score = (W + 16) * 2.0 ** -24 * reach + 2.0 ** -18  # as in _Decode.check
        _within(out[s:s + 1], want, U * want.abs() + (U + 2 * score[..., None] + extra) * size, "out")
        wl = wl + math.log(max(times[s], 1))
        _within(lse[s:s + 1], wl, score + 2.0 ** -22 * wl.abs() + 3500 * 2.0 ** -24, "lse")

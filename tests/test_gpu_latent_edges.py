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


# ------------------------------------------------------------- values at the edges ----

def _one_sequence(env, tokens, q, scale, e4m3, R, page=16):  # noqa: F811
    """latent_decode of one sequence whose cached rows are `tokens` (exact in the cache's type), the rows
    q [n, H, W] at its end."""
    torch, ssd, dev = env
    L, W = tokens.shape
    n, H = q.shape[:2]
    used = -(-L // page)
    kind = torch.float8_e4m3fn if e4m3 else torch.bfloat16
    cache = torch.zeros((used, page, W), device=dev)
    cache.view(-1, W)[:L] = tokens
    out = torch.empty((n, H, R), dtype=torch.bfloat16, device=dev)
    lse = torch.empty((n, H), device=dev)
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device=dev)
    ws = ssd.workspace(ssd.latent_decode_workspace_bytes(1, n, H, R, W - R), dev)
    ssd.latent_decode(q, cache.to(kind), torch.arange(used, dtype=torch.int32, device=dev).view(1, -1), i32(L),
                      out, ws, scale, q_start=i32(0, n), lse=lse)
    assert ssd.dec_sync_status() == ssd.DEC_OK
    return out, lse


@pytest.mark.parametrize("peak", [10.0, 14.0, 16.0, 18.0, 20.0])
@pytest.mark.parametrize("rows,n,H", [(1, 100, 16), (1, 9000, 16), (2, 300, 16), (3, 500, 32), (1, 3000, 64)])
@pytest.mark.parametrize("e4m3", [False, True])
def test_decode_flat_tail_under_a_peak(env, e4m3, rows, n, H, peak):  # noqa: F811
    """One token 14 to 29 powers of two above all others, whose other elements are zero: what is lost
    of the others' weights is lost of the outputs.

    Weights round by 2^-8 (bf16) or 2^-11 of themselves or 2^-32 of the largest (f16), outputs by
    2^-8; scores of one product each: 2^-22 |z| for the scaling and the difference."""
    torch, ssd, dev = env
    R, W = 128, 192
    tokens = torch.randint(8, 16, (n, W), device=dev, generator=torch.Generator(dev).manual_seed(1)).float() / 8
    tokens[:, 0] = 0.125
    tokens[3] = 0.0
    tokens[3, 0] = peak
    q = torch.zeros((rows, H, W), dtype=torch.bfloat16, device=dev)
    q[:, :, 0] = 1.0
    got, lse = _one_sequence(env, tokens, q, 1.0, e4m3, R)
    w, v = (tokens[:, 0].double() - peak).exp(), tokens[:, 1:R].double()
    u, floor = (2.0 ** -11, 2.0 ** -32) if e4m3 else (U, 0.0)
    for i in range(rows):
        seen = n - rows + i + 1
        total = w[:seen].sum()
        want = (w[:seen] @ v[:seen] / total).expand(H, -1)
        bound = U * want + (u + 2.0 ** -21 * peak + 2.0 ** -18) * want + floor * v[:seen].sum(0) / total
        _within(got[i, :, 1:], want, bound, "out")
        _within(lse[i], (peak + total.log()).expand(H), torch.full((H,), 2.0 ** -21 * peak + 2.0 ** -18,
                                                                  device=dev), "lse")


@pytest.mark.parametrize("H", [16, 64])
@pytest.mark.parametrize("e4m3", [False, True])
def test_decode_infinite_query_beside_large_ones(env, e4m3, H):  # noqa: F811
    """A query of -infinity in one element makes every score -infinity where the tokens are positive
    there, however large its other elements are: nothing is seen."""
    torch, ssd, dev = env
    for n in (70, 9000):
        tokens = torch.ones((n, 576), device=dev)
        q = torch.randn((3, H, 576), device=dev, generator=torch.Generator(dev).manual_seed(2)).to(torch.bfloat16)
        want, want_lse = _one_sequence(env, tokens, q, 0.05, e4m3, 512)
        q[0] = 1e30
        q[0, :, 1] = -math.inf
        got, lse = _one_sequence(env, tokens, q, 0.05, e4m3, 512)
        assert not got[0].any() and bool((lse[0] == -math.inf).all())
        assert torch.equal(got[1:], want[1:]) and torch.equal(lse[1:], want_lse[1:])


class _Scaled(_Decode):
    """On an e4m3 cache q goes to f16 with its row's largest, 2^power here, at 2^14: in steps of 2^-24
    there, so that an element is off by 2^-25 * 2^(power - 14) at most, and a score by that times
    sum_d |k_d|. check() counts (W + 16) 2^-24 of what stands in the last of the results."""
    power = 0

    def reference(self):
        out, lse, size, reach = super().reference()
        if self.c_scale is not None:
            k = self.cache.float().double().abs().sum(-1).max() * self.c_scale.double()
            off = abs(self.scale) * 2.0 ** (self.power - 39) * k
            reach = reach + off / ((self.W + 16) * 2.0 ** -24)
        return out, lse, size, reach


@pytest.mark.parametrize("power", [10, 24, 30])
@pytest.mark.parametrize("e4m3", [False, True])
def test_decode_query_with_one_large_element(env, e4m3, power):  # noqa: F811
    """An element of q far above the others that meets zeros: what the others give is as exact as
    without it (down to 2^-31 of it in f16)."""
    torch, ssd, dev = env
    for H in (16, 64):
        d = _Scaled(env, [70, 5000], [1, 2], H, e4m3=e4m3)
        d.power = power
        raw = d.cache.view(torch.uint8) if e4m3 else d.cache.view(torch.int16)
        raw[..., 3] = 0
        d.q[:, :, 3] = 2.0 ** power
        d.run()
        d.check()


@pytest.mark.parametrize("H", [16, 64])
def test_decode_not_finite_in_an_e4m3_cache(env, H):  # noqa: F811
    """A NaN makes the rows that see it NaN, in a stage that all rows see and in one that some do not;
    the rows before it keep their bits."""
    torch, ssd, dev = env
    for L, at in ((200, 70), (200, 198), (200, 197), (9000, 8998), (9000, 5000)):
        d = _Decode(env, [L], [4], H, page=8, e4m3=True)
        d.run()
        clean, clean_lse = d.out[:4].clone(), d.lse[:4].clone()
        d.cache.view(torch.uint8)[int(d.table[0, at // 8]), at % 8, 5] = 0x7f
        d.run()
        assert ssd.dec_sync_status() == ssd.DEC_OK
        for i in range(4):
            if L - 4 + i < at:
                assert torch.equal(d.out[i], clean[i]) and torch.equal(d.lse[i], clean_lse[i])
            else:
                assert bool(d.out[i].isnan().all()) and bool(d.lse[i].isnan().all())


@pytest.mark.parametrize("H", [2, 160])
def test_prompt_infinite_query_beside_large_ones(env, H):  # noqa: F811
    torch, ssd, dev = env
    p = _Prompt(env, [300], [700], H)
    p.k.abs_()
    p.k[..., 1] = 1.0
    p.run()
    want, want_lse = p.out.clone(), p.lse.clone()
    p.q[200, :] = 1e15
    p.q[200, :, 1] = -math.inf
    p.run()
    assert ssd.dec_sync_status() == ssd.DEC_OK
    assert not p.out[200].any() and bool((p.lse[200] == -math.inf).all())
    want[200], want_lse[200] = p.out[200], p.lse[200]
    assert torch.equal(p.out, want) and torch.equal(p.lse, want_lse)


# ------------------------------------------------ elements past 2^31 of rows and outputs ----

def test_prompt_and_decode_of_very_many_rows(env):  # noqa: F811
    torch, ssd, dev = env
    import latent_ref
    S, n, H, W, R = 8192, 8, 128, 320, 256
    T = S * n
    g = torch.Generator(device=dev).manual_seed(3)
    starts = torch.arange(S + 1, dtype=torch.int32, device=dev) * n
    some = torch.randn((64, W), generator=g, device=dev).to(torch.bfloat16)
    q = torch.empty((T, H, W), dtype=torch.bfloat16, device=dev)
    last = torch.randn((3 * n, H, W), generator=g, device=dev).to(torch.bfloat16)
    q[:-3 * n] = 0
    q[-3 * n:] = last
    out = torch.empty((T, H, R), dtype=torch.bfloat16, device=dev)
    ws = ssd.workspace(ssd.latent_decode_workspace_bytes(S, T, H, R, W - R), dev)
    table = torch.zeros((S, 1), dtype=torch.int32, device=dev)
    ssd.latent_decode(q, some.view(1, 64, W), table, torch.full((S,), 40, dtype=torch.int32, device=dev), out, ws,
                      0.06, q_start=starts)
    assert ssd.dec_sync_status() == ssd.DEC_OK
    keys = some[:40].double()[None]
    pos = torch.arange(n, device=dev) + 40 - n
    for s in range(3):
        at = slice(T - 3 * n + s * n, T - 3 * n + (s + 1) * n)
        want, _, size, reach = latent_ref.attend(q[at].double(), keys, keys[..., :R], pos, 0.06)
        score = (W + 16) * 2.0 ** -24 * reach + 2.0 ** -18
        _within(out[at], want, U * want.abs() + (U + 2 * score[..., None]) * size, "decode")
    # q of zeros weighs alike
    mean = torch.stack([keys[0, :40 - n + i + 1, :R].mean(0) for i in range(n)])
    size = torch.stack([keys[0, :40 - n + i + 1, :R].abs().mean(0) for i in range(n)])
    far = T // 2 // n * n
    for h in (0, H - 1):
        _within(out[far:far + n, h], mean, U * mean.abs() + (U + 2.0 ** -17) * size, "decode of zeros")
    del out, q, ws
    N, P, V = 128, 64, 128
    T = 2 ** 17
    S = 1024
    n = T // S
    starts = torch.arange(S + 1, dtype=torch.int32, device=dev) * n
    q = torch.zeros((T, H, N + P), dtype=torch.bfloat16, device=dev)
    kv = torch.zeros((T, H, N + V), dtype=torch.bfloat16, device=dev)
    r = torch.randn((T, P), generator=g, device=dev).to(torch.bfloat16)
    for x in (q, kv):
        x[-n:] = torch.randn(x[-n:].shape, generator=g, device=dev).to(torch.bfloat16)
    out = torch.full((T, H, V), 5.0, dtype=torch.bfloat16, device=dev)
    ssd.latent_prompt(q, kv[..., :N], r, kv[..., N:], starts, out, 0.07)
    assert ssd.dec_sync_status() == ssd.DEC_OK
    assert not out[:-n].any()
    k = torch.cat([kv[-n:, :, :N].double(), r[-n:, None].double().expand(n, H, P)], -1).transpose(0, 1)
    want, _, size, reach = latent_ref.attend(q[-n:].double(), k, kv[-n:, :, N:].double().transpose(0, 1),
                                             torch.arange(n, device=dev), 0.07)
    score = (N + P + 16) * 2.0 ** -24 * reach + 2.0 ** -18
    _within(out[-n:], want, U * want.abs() + (U + 2 * score[..., None]) * size, "prompt")


def test_append_and_project_of_very_many_rows(env):  # noqa: F811
    torch, ssd, dev = env
    T, H, R, P = 2 ** 20, 40, 64, 64
    g = torch.Generator(device=dev).manual_seed(4)
    q = torch.empty((T, H, P), dtype=torch.bfloat16, device=dev)
    q[:] = torch.randn((1, H, P), generator=g, device=dev).to(torch.bfloat16)
    c, r = (torch.randn((T, d), generator=g, device=dev).to(torch.bfloat16) for d in (R, P))
    cache = torch.zeros((T // 64, 64, R + P), dtype=torch.bfloat16, device=dev)
    slots = torch.arange(T, dtype=torch.int32, device=dev).flip(0).contiguous()
    positions = torch.zeros(T, dtype=torch.int32, device=dev)  # nothing turns
    inv, _ = ssd.rope_frequencies(P, device=dev)
    out = torch.zeros_like(q)
    ssd.latent_append(c, r, positions, slots, inv, cache, q_rope=q, q_out=out)
    assert ssd.dec_sync_status() == ssd.DEC_OK
    assert torch.equal(out, q)
    assert torch.equal(cache.view(T, -1).flip(0), torch.cat([c, r], -1))
    del q, out, cache
    T, H, K, N = 70000, 64, 64, 512
    x = torch.zeros((T, H, K), dtype=torch.bfloat16, device=dev)
    x[-200:] = torch.randn((200, H, K), generator=g, device=dev).to(torch.bfloat16)
    w = torch.randn((H, N, K), generator=g, device=dev).to(torch.bfloat16)
    y = torch.full((T, H, N), 5.0, dtype=torch.bfloat16, device=dev)
    ssd.latent_project(x, w, y)
    assert ssd.dec_sync_status() == ssd.DEC_OK
    assert not y[:-200].any()
    want = torch.einsum("thk,hnk->thn", x[-200:].double(), w.double())
    size = torch.einsum("thk,hnk->thn", x[-200:].double().abs(), w.double().abs())
    _within(y[-200:], want, U * want.abs() + (K + 2) * 2.0 ** -24 * size, "y")


def test_append_wants_a_place_for_the_queries(env):  # noqa: F811
    torch, ssd, dev = env
    c, r = torch.zeros((2, 576), dtype=torch.bfloat16, device=dev).split([512, 64], 1)
    cache = torch.ones((1, 8, 576), dtype=torch.bfloat16, device=dev)
    at = torch.arange(2, dtype=torch.int32, device=dev)
    q = torch.zeros((2, 4, 64), dtype=torch.bfloat16, device=dev)
    with pytest.raises(ValueError, match="q_out"):
        ssd.latent_append(c, r, at, at, torch.ones(32, device=dev), cache, q_rope=q)
    assert bool((cache == 1).all())

"""GPU parity of latent_append, latent_project, latent_decode and latent_prompt with plain 64-bit
forms.

Tolerances, derived from the arithmetic (u = 2^-8 is bf16's unit roundoff):
  - latent_append: u |y| for the rounding, plus 2^-18 |y| for a fp32 norm (a sum of squares in
    chains of 15 additions, a reciprocal root, two products), or 2^-20 (|x0| + |x1|) for a fp32
    rotation; e4m3: unit roundoff 2^-4, half of the smallest step 2^-10.
  - latent_project: u |y| plus (K + 2) 2^-24 sum_k |x_k W_k| for fp32 sums.
  - latent_decode, latent_prompt: u |out| for the last rounding; u sum_j w_j |v_j| for weights
    that round to 16 bits before the product; and twice the relative error of the weights, which
    is the absolute error of a fp32 score, (D + 16) 2^-24 scale sum_d |q_d k_d|, plus 2^-18 for
    exponentials and sums. lse: the score's error, 2^-18, and 2^-22 |lse|.
"""
import math

import pytest

pytestmark = pytest.mark.gpu
U = 2.0 ** -8


@pytest.fixture(scope="module")
def env():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import split_switched_decode_gb300 as ssd
    ssd.build()
    dev = torch.device("cuda:0")
    torch.cuda.set_device(dev)
    return torch, ssd, dev


def _gen(torch, dev, seed):
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    return g


def _randn(torch, dev, g, *shape):
    return torch.randn(shape, generator=g, device=dev).to(torch.bfloat16)


def _i32(torch, x, dev):
    return torch.tensor(list(x), dtype=torch.int32, device=dev)


def _starts(counts):
    at = [0]
    for n in counts:
        at.append(at[-1] + n)
    return at


def _within(got, want, bound, what):
    err = (got.double() - want).abs()
    ok = (err <= bound) | ((got.double() == want) & want.isinf()) | (got.isnan() & want.isnan())
    assert bool(ok.all()), (what, int((~ok).sum()), ok.numel(),
                            float((err / bound.clamp(min=1e-300))[~ok].max()))


# ----------------------------------------------------------------- append ----

def _append(env, T, H, R, P, rot, interleaved, e4m3, page, rows, norm=True, seed=0, max_pos=131072,
            pad=0):
    torch, ssd, dev = env
    import latent_ref
    g = _gen(torch, dev, 100 + seed + T + R)
    down = _randn(torch, dev, g, T, R + P + pad)
    up = _randn(torch, dev, g, T, max(H, 1), 32 + P)
    c, k_rope = down[:, :R], down[:, R:R + P] if P else None
    q_rope = up[..., 32:] if H and P else None
    pages = -(-T // page) + 1
    dtype = torch.float8_e4m3fn if e4m3 else torch.bfloat16
    cache = torch.zeros((pages, page, R + P), device=dev).to(dtype)
    scale = torch.full((1,), 0.0173, device=dev) if e4m3 else None
    weight = (torch.rand(R, generator=g, device=dev) + 0.5).to(torch.bfloat16) if norm else None
    positions = torch.randint(0, max_pos, (T,), generator=g, device=dev, dtype=torch.int32)
    slots = torch.randperm(pages * page, generator=g, device=dev)[:T].to(torch.int32)
    skipped = T > 2
    if skipped:
        slots[1], slots[2] = -1, pages * page  # neither is written
    inv, mag = ssd.rope_frequencies(rot, device=dev) if rot else (None, 1.0)
    mag = 1.25 if rot else 1.0
    q = torch.full((T, max(H, 1), R + P), 7.0, device=dev).to(torch.bfloat16)
    kept = torch.full((T, R + P), 7.0, device=dev).to(torch.bfloat16) if rows else None
    ssd.latent_append(c, k_rope, positions, slots, inv, cache, weight=weight, eps=1e-5,
                      q_rope=q_rope, q_out=q[..., R:] if q_rope is not None else None, rows=kept,
                      interleaved=interleaved, magnitude=mag, cache_scale=scale)
    torch.cuda.synchronize()
    want = latent_ref.normed(c, weight, 1e-5) if norm else c.double()
    size = want.abs() * 2.0 ** -18
    freq = inv if inv is not None else torch.zeros(0, device=dev)
    if P:
        r, rs = latent_ref.rotate(k_rope.double(), positions, freq, mag, interleaved)
        want, size = torch.cat([want, r], -1), torch.cat([size, rs * 2.0 ** -20], -1)
    if rows:
        _within(kept, want, U * want.abs() + size + 1e-38, "rows")
    flat = cache.float().double().view(-1, R + P)
    held = want / scale.double() if e4m3 else want
    size = size / scale.double() if e4m3 else size
    if e4m3:
        held = held.clamp(-448, 448)
    unit, least = (2.0 ** -4, 2.0 ** -10) if e4m3 else (U, 1e-38)
    live = torch.ones(T, dtype=torch.bool, device=dev)
    if skipped:
        live[1:3] = False
    at = slots[live].long()
    _within(flat[at], held[live], unit * held[live].abs() + size[live] + least, "cache")
    rest = torch.ones(flat.shape[0], dtype=torch.bool, device=dev)
    rest[at] = False
    assert bool((flat[rest] == 0).all())
    if q_rope is not None:
        w, s = latent_ref.rotate(q_rope.double(), positions, freq, mag, interleaved)
        _within(q[..., R:], w, U * w.abs() + s * 2.0 ** -20 + 1e-38, "q")
        assert bool((q[..., :R] == 7.0).all())


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("T,H,R,P,rot,page", [
    (1, 64, 512, 64, 64, 16), (1, 1, 64, 64, 32, 1), (3, 16, 512, 64, 64, 7), (37, 128, 256, 64, 48, 16),
    (303, 5, 448, 128, 128, 64), (304, 8, 512, 64, 16, 16), (700, 16, 192, 64, 0, 48),
    (2432, 3, 192, 128, 64, 16), (3001, 20, 512, 64, 64, 48),  # (with many rows: another form)
])
def test_append(env, T, H, R, P, rot, page, interleaved, e4m3):
    _append(env, T, H, R, P, rot, interleaved, e4m3, page, rows=T % 2 == 1, pad=16 * (T % 3))


def test_append_no_rotary_part_no_queries_no_norm(env):
    _append(env, 5, 0, 512, 0, 0, False, False, 16, rows=True)
    _append(env, 5, 0, 512, 64, 64, True, True, 16, rows=True, norm=False)
    _append(env, 2000, 0, 512, 64, 64, False, False, 16, rows=False)


def test_append_far_positions_and_in_place(env):
    torch, ssd, dev = env
    import latent_ref
    g = _gen(torch, dev, 5)
    T, H = 9, 12
    c, r, q = (_randn(torch, dev, g, *s) for s in ((T, 512), (T, 64), (T, H, 192)))
    positions = _i32(torch, [0, 1, 2 ** 31 - 1, 2 ** 30 + 1, 999999937, 131071, 17, 2 ** 24 + 1, 5], dev)
    inv, _ = ssd.rope_frequencies(64, device=dev)
    cache = torch.zeros((2, 8, 576), device=dev).to(torch.bfloat16)
    for interleaved in (False, True):
        x = q.clone()
        ssd.latent_append(c, r, positions, torch.arange(T, dtype=torch.int32, device=dev), inv, cache,
                          q_rope=x[..., 128:], q_out=x[..., 128:], interleaved=interleaved)
        w, s = latent_ref.rotate(q[..., 128:].double(), positions, inv, 1.0, interleaved)
        _within(x[..., 128:], w, U * w.abs() + s * 2.0 ** -20, "q")
        assert torch.equal(x[..., :128], q[..., :128])
        assert torch.equal(cache.view(-1, 576)[:T, :512], c)


# ---------------------------------------------------------------- project ----

def _project(env, T, H, K, N, x_pad=0, y_pad=0, heads_first=False, seed=0):
    torch, ssd, dev = env
    g = _gen(torch, dev, 200 + seed + T + K + N)
    x = _randn(torch, dev, g, T, H, K + x_pad)[..., x_pad:]
    w = _randn(torch, dev, g, H, N, K)
    whole = torch.full((H, T, N + y_pad) if heads_first else (T, H, N + y_pad), 3.0, device=dev) \
        .to(torch.bfloat16)
    y = (whole.transpose(0, 1) if heads_first else whole)[..., :N]
    ssd.latent_project(x, w, y)
    torch.cuda.synchronize()
    want = torch.einsum("thk,hnk->thn", x.double(), w.double())
    size = torch.einsum("thk,hnk->thn", x.double().abs(), w.double().abs())
    _within(y, want, U * want.abs() + (K + 2) * 2.0 ** -24 * size, "y")
    if y_pad:
        assert bool((whole[..., N:] == 3.0).all())


@pytest.mark.parametrize("T,H,K,N", [
    (1, 64, 128, 512), (1, 1, 8, 8), (2, 3, 512, 128), (17, 16, 72, 200), (63, 5, 512, 128),
    (64, 64, 512, 128), (65, 4, 128, 512), (127, 3, 192, 256), (128, 2, 64, 64), (129, 7, 136, 264),
    (300, 16, 128, 512), (1000, 2, 512, 136), (513, 1, 1024, 8), (33, 2, 4096, 64),
])
def test_project(env, T, H, K, N):
    _project(env, T, H, K, N)


@pytest.mark.parametrize("T", [1, 50, 200])
def test_project_strides(env, T):
    _project(env, T, 6, 128, 512, x_pad=64, y_pad=64)
    _project(env, T, 6, 512, 128, y_pad=8, heads_first=True)
    _project(env, T, 1, 128, 256, x_pad=8, y_pad=16)


# ----------------------------------------------------------------- decode ----

def _cache_of(torch, dev, g, tokens, e4m3, scale):
    x = torch.randn(tokens, generator=g, device=dev)
    if not e4m3:
        return x.to(torch.bfloat16)
    return (x / scale).clamp(-448, 448).to(torch.float8_e4m3fn)


def _values(torch, cache):
    return cache.float().double()


class _Decode:
    """One batch: ragged lengths and rows over a paged cache, and its reference."""

    def __init__(self, env, lens, rows, H, R=512, P=64, page=16, e4m3=False, window=0, scale=0.06,
                 seed=0, pad=0, grow=0.0, poison=False, drop=()):
        torch, ssd, dev = env
        self.env, self.H, self.R, self.W, self.page = env, H, R, R + P, page
        self.lens, self.rows, self.window, self.scale = list(lens), list(rows), window, scale
        g = _gen(torch, dev, 300 + seed + sum(lens) + H)
        used = [-(-n // page) for n in lens]
        total = sum(used) + 3
        width = max(1, max(used)) + 1
        self.c_scale = torch.full((1,), 0.013, device=dev) if e4m3 else None
        store = _cache_of(torch, dev, g, (total, page, self.W + pad), e4m3, 0.013)
        self.cache = store[..., :self.W]
        ids = torch.randperm(total, generator=g, device=dev).to(torch.int32)
        table = torch.full((len(lens), width), -1, dtype=torch.int32, device=dev)
        at = 0
        for s, n in enumerate(used):
            table[s, :n] = ids[at:at + n]
            at += n
        if grow:  # later tokens score higher and higher
            q_dir = torch.randn(self.W, generator=g, device=dev)
            for s, n in enumerate(lens):
                for i in range(used[s]):
                    p = int(table[s, i])
                    j = torch.arange(i * page, (i + 1) * page, device=dev)
                    x = self.cache[p].float() * 0.1 + q_dir * (grow * j[:, None])
                    self.cache[p] = x.to(store.dtype)
        self.exists = []
        for s, n in enumerate(lens):
            e = torch.ones(n, dtype=torch.bool, device=dev)
            for i in range(used[s]):
                if (s, i) in drop:
                    table[s, i] = -1 if i % 2 else total
                    e[i * page:(i + 1) * page] = False
            self.exists.append(e)
        if poison:  # everything that no row sees
            mark = torch.zeros((total, page), dtype=torch.bool, device=dev)
            for s, n in enumerate(lens):
                first = max(0, n - rows[s] - window + 1) if window else 0
                for j in range(first, n):
                    p = int(table[s, j // page])
                    if 0 <= p < total:
                        mark[p, j % page] = True
            raw = store.view(torch.uint8) if e4m3 else store.view(torch.int16)
            raw[~mark] = 0x7f if e4m3 else 0x7fc0
        self.table = table
        T = sum(rows)
        self.T = T
        self.q = _randn(torch, dev, g, T + 2, H, self.W)
        if grow:
            self.q = (self.q.float() * 0.1 + q_dir).to(torch.bfloat16)
        self.seq_len = _i32(torch, lens, dev)
        self.q_start = _i32(torch, _starts(rows), dev)
        self.out = torch.full((T + 2, H, R), 5.0, device=dev).to(torch.bfloat16)
        self.lse = torch.full((T + 2, H), 5.0, device=dev)
        self.ws = ssd.workspace(ssd.latent_decode_workspace_bytes(len(lens), T + 2, H, R, P), dev)

    def run(self, stream=None):
        self.env[1].latent_decode(self.q, self.cache, self.table, self.seq_len, self.out, self.ws,
                                  self.scale, q_start=self.q_start, window=self.window,
                                  lse=self.lse, cache_scale=self.c_scale, stream=stream)

    def reference(self):
        torch, ssd, dev = self.env
        import latent_ref
        parts = []
        t = 0
        for s, (n, r) in enumerate(zip(self.lens, self.rows)):
            pages = self.table[s, :-(-n // self.page)].long()
            ok = (pages >= 0) & (pages < self.cache.shape[0])
            raw = self.cache.contiguous()
            raw = raw.view(torch.uint8)[pages.clamp(0, raw.shape[0] - 1)].view(raw.dtype)
            keys = _values(torch, raw).reshape(-1, self.W)[:n]
            if self.c_scale is not None:
                keys = keys * self.c_scale.double()
            keys = torch.where(self.exists[s][:, None], keys, torch.zeros_like(keys))
            first = max(0, n - r - self.window + 1) if self.window else 0
            keys[:first] = keys[:first].nan_to_num(0.0)  # seen by no row
            pos = torch.arange(r, device=dev) + n - r
            parts.append(latent_ref.attend(self.q[t:t + r].double(), keys[None], keys[None, :, :self.R],
                                           pos, self.scale, self.window, self.exists[s]))
            t += r
        return [torch.cat(x) for x in zip(*parts)]

    def check(self):
        torch = self.env[0]
        torch.cuda.synchronize()
        out, lse, size, reach = self.reference()
        T = self.T
        score = (self.W + 16) * 2.0 ** -24 * reach + 2.0 ** -18
        bound = U * out.abs() + (U + 2 * score[..., None]) * size + 1e-30
        _within(self.out[:T], out, bound, "out")
        _within(self.lse[:T], lse, score + 2.0 ** -22 * lse.abs().nan_to_num(0, 0, 0), "lse")
        assert bool((self.out[T:] == 5.0).all()) and bool((self.lse[T:] == 5.0).all())


LENS = [1, 63, 64, 65, 777, 0, 128, 300]


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("H", [1, 16, 20, 32, 64, 128])
def test_decode_heads(env, H, e4m3):
    d = _Decode(env, LENS, [1] * len(LENS), H, e4m3=e4m3)
    d.run()
    d.check()


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("R,P", [(64, 0), (64, 64), (192, 0), (256, 64), (320, 64), (448, 128), (512, 0),
                                 (512, 64)])
def test_decode_widths(env, R, P, e4m3):
    for H in (16, 40):
        d = _Decode(env, [5, 200, 1000], [1, 1, 2], H, R=R, P=P, e4m3=e4m3)
        d.run()
        d.check()


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("page", [1, 7, 8, 13, 24, 48, 128, 1000])
def test_decode_pages(env, page, e4m3):
    for H in (16, 64):
        d = _Decode(env, [3, 129, 500, 1024], [1, 2, 1, 3], H, page=page, e4m3=e4m3, pad=64)
        d.run()
        d.check()


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("rows", [[1, 2, 3, 4], [8, 8, 8, 8], [9, 0, 70, 1], [40, 5, 2, 30]])
def test_decode_rows(env, rows, e4m3):
    for H in (8, 24):
        d = _Decode(env, [40, 7, 300, 29], rows, H, e4m3=e4m3, poison=True)  # rows before the first key too
        d.run()
        d.check()


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("window", [1, 5, 64, 100, 4096])
def test_decode_window(env, window, e4m3):
    d = _Decode(env, [1, 64, 333, 900], [1, 2, 5, 3], 16, window=window, e4m3=e4m3, poison=True)
    d.run()
    d.check()


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("H", [16, 32, 64])
def test_decode_long(env, H, e4m3):
    d = _Decode(env, [40000, 3, 9001], [1, 1, 2], H, page=64, e4m3=e4m3)
    for _ in range(2):  # the counters are back at zero
        d.run()
        d.check()


# (the last: elements past 448 that are cast to e4m3 are NaN, and so is the row that sees them)
@pytest.mark.parametrize("e4m3,grow", [(False, 0.004), (True, 0.09), (True, 0.15)])
@pytest.mark.parametrize("H", [16, 64])
def test_decode_growing_scores(env, H, e4m3, grow):
    d = _Decode(env, [700, 90], [1, 2], H, grow=grow, e4m3=e4m3)
    d.run()
    d.check()
    d.scale = -d.scale
    d.run()
    d.check()


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("page", [7, 16])
def test_decode_missing_pages(env, page, e4m3):
    d = _Decode(env, [100, 64, 200], [1, 2, 1], 16, page=page, e4m3=e4m3, poison=True,
                drop={(0, 0), (0, 3), (1, 0), (1, 1), (1, 2), (1, 3), (1, 4), (1, 5), (1, 6), (1, 7),
                      (1, 8), (1, 9), (2, 5)})
    d.run()
    d.check()


def test_decode_not_finite(env):
    """An infinity or NaN makes the rows that see it NaN, in a stage that all rows see and in
    one that some do not; the rows before it stay."""
    torch, ssd, dev = env
    for at, value in ((70, math.nan), (198, math.nan), (197, math.inf), (198, -math.inf), (10, math.inf)):
        d = _Decode(env, [200], [4], 16, page=8)
        p, o = int(d.table[0, at // 8]), at % 8
        d.run()
        clean = d.out[:4].clone()
        d.cache[p, o, 5] = value
        d.run()
        torch.cuda.synchronize()
        for i in range(4):
            if 196 + i < at:
                assert torch.equal(d.out[i], clean[i])
                continue
            for h in range(16):
                score = float(d.q[i, h, 5]) * value
                if math.isnan(score) or score > 0:
                    assert bool(d.out[i, h].isnan().all()) and math.isnan(float(d.lse[i, h]))
                else:  # a score of -infinity
                    keep = [e for e in range(512) if e != 5]
                    assert bool(d.out[i, h, keep].isfinite().all())


def test_decode_queries_with_large_elements(env):
    """e4m3: a large element of q beside small ones that decide the scores."""
    torch, ssd, dev = env
    d = _Decode(env, [300], [1], 16, e4m3=True)
    zero = d.cache.view(torch.uint8)
    zero[..., 3] = 0
    d.q[:, :, 3] = 2.0 ** 18
    d.run()
    d.check()


def test_decode_one_row_each_by_default_and_lse_optional(env):
    torch, ssd, dev = env
    d = _Decode(env, LENS, [1] * len(LENS), 16)
    d.run()
    out = torch.empty_like(d.out[:d.T])
    ssd.latent_decode(d.q[:d.T], d.cache, d.table, d.seq_len, out, d.ws, d.scale)
    assert torch.equal(out, d.out[:d.T])


def test_decode_same_bits_every_time_and_on_another_stream(env):
    torch, ssd, dev = env
    d = _Decode(env, [9000, 40, 3000], [2, 1, 4], 32)
    d.run()
    first = d.out.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        d.out.fill_(5.0)
        side.wait_stream(torch.cuda.current_stream())
        d.run(stream=side)
        torch.cuda.current_stream().wait_stream(side)
        assert torch.equal(first, d.out)


def test_decode_strided_rows(env):
    torch, ssd, dev = env
    d = _Decode(env, [100, 30], [2, 1], 8)
    q = torch.zeros((d.T, 8 * 576 + 64), dtype=torch.bfloat16, device=dev)
    out = torch.zeros((d.T, 8 * 512 + 8), dtype=torch.bfloat16, device=dev)
    q[:, 64:] = d.q[:d.T].reshape(d.T, -1)
    d.run()
    ssd.latent_decode(q[:, 64:].unflatten(1, (8, 576)), d.cache,
                      d.table, d.seq_len, out[:, :4096].unflatten(1, (8, 512)), d.ws, d.scale,
                      q_start=d.q_start)
    assert torch.equal(out[:, :4096], d.out[:d.T].reshape(d.T, -1))
    assert bool((out[:, 4096:] == 0).all())


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("H", [8, 64])
def test_decode_rows_of_no_sequence_and_a_used_workspace(env, H, e4m3):
    """Rows before the first sequence and behind the last stay, sequences without rows are passed over,
    and nothing is expected of what the workspace holds."""
    torch, ssd, dev = env
    lens = [0] * 45 + [700] + [90] * 4
    rows = [0] * 45 + [2] + [1, 0, 3, 0]
    d = _Decode(env, lens, rows, H, e4m3=e4m3)
    d.ws.fill_(255)
    d.run()
    d.check()
    q, starts = torch.empty_like(d.q[:d.T + 1]), d.q_start + 1
    q[0], q[1:] = 1.0, d.q[:d.T]
    out = torch.full((d.T + 1, H, 512), 5.0, device=dev).to(torch.bfloat16)
    lse = torch.full((d.T + 1, H), 5.0, device=dev)
    d.ws.random_(0, 256)
    ssd.latent_decode(q, d.cache, d.table, d.seq_len, out, d.ws, d.scale, q_start=starts, lse=lse,
                      cache_scale=d.c_scale)
    assert torch.equal(out[1:], d.out[:d.T]) and torch.equal(lse[1:], d.lse[:d.T])
    assert bool((out[0] == 5.0).all()) and bool((lse[0] == 5.0).all())


def test_decode_two_graphs_share_a_workspace(env):
    torch, ssd, dev = env
    a, b = (_Decode(env, lens, [1] * 3, 16) for lens in ([5000, 3, 800], [64, 9000, 200]))
    ws = a.ws if a.ws.numel() >= b.ws.numel() else b.ws
    a.ws = b.ws = ws
    want = []
    for d in (a, b):
        d.run()
        want.append((d.out.clone(), d.lse.clone()))
    graphs = []
    for d in (a, b):
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            d.run()
        graphs.append(g)
    for _ in range(3):
        for d, g, (out, lse) in zip((a, b), graphs, want):
            d.out.fill_(5.0)
            d.lse.fill_(5.0)
            g.replay()
            assert torch.equal(d.out, out) and torch.equal(d.lse, lse)


def test_decode_pages_far_apart(env):
    """Pages whose elements lie past 2^31."""
    torch, ssd, dev = env
    store = torch.zeros((5, 1 << 29), dtype=torch.bfloat16, device=dev)
    cache = store[:, :16 * 576].unflatten(1, (16, 576))
    g = _gen(torch, dev, 9)
    cache.copy_(_randn(torch, dev, g, 5, 16, 576))
    table = _i32(torch, [4, 0, 3], dev).view(1, 3)
    q = _randn(torch, dev, g, 1, 16, 576)
    ws = ssd.workspace(ssd.latent_decode_workspace_bytes(1, 1, 16, 512, 64), dev)
    outs = []
    for c in (cache, cache.contiguous()):
        out = torch.empty((1, 16, 512), dtype=torch.bfloat16, device=dev)
        ssd.latent_decode(q, c, table, _i32(torch, [45], dev), out, ws, 0.06)
        outs.append(out)
    assert torch.equal(*outs)
    # and the write
    c = _randn(torch, dev, g, 2, 512)
    r = _randn(torch, dev, g, 2, 64)
    ssd.latent_append(c, r, _i32(torch, [1, 2], dev), _i32(torch, [4 * 16 + 3, 16], dev), None, cache)
    assert torch.equal(cache[4, 3], torch.cat([c[0], r[0]])) and torch.equal(cache[1, 0],
                                                                             torch.cat([c[1], r[1]]))


def test_decode_wait_that_runs_out(env):
    """A wait that nothing ends gives a status, and the context goes on."""
    torch, ssd, dev = env
    for e4m3 in (False, True):
        d = _Decode(env, [9000, 40], [1, 2], 16, e4m3=e4m3)
        ssd.dec_set_wait_limit_ns(2_000_000)
        ssd.dec_debug_attn_timeout(True)
        try:
            d.run()
            assert ssd.dec_sync_status() == ssd.DEC_ERR_TIMEOUT
        finally:
            ssd.dec_debug_attn_timeout(False)
            ssd.dec_set_wait_limit_ns(2_000_000_000)
        d.ws.zero_()
        d.out.fill_(5.0)
        d.lse.fill_(5.0)
        d.run()
        assert ssd.dec_sync_status() == ssd.DEC_OK
        d.check()


# ----------------------------------------------------------------- prompt ----

class _Prompt:
    def __init__(self, env, rows, keys, H, N=128, P=64, V=128, scale=0.09, seed=0, joint=True, extra=1):
        torch, ssd, dev = env
        self.env, self.rows, self.keys, self.H = env, list(rows), list(keys), H
        self.N, self.P, self.V, self.scale = N, P, V, scale
        g = _gen(torch, dev, 400 + seed + sum(keys) + H)
        self.T, self.Tk = sum(rows), sum(keys)
        T, Tk = self.T + extra, self.Tk + extra
        self.q = _randn(torch, dev, g, T, H, N + P)
        if joint:
            kv = _randn(torch, dev, g, Tk, H, N + V)
            self.k, self.v = kv[..., :N], kv[..., N:]
        else:
            self.k = _randn(torch, dev, g, H, Tk, N).transpose(0, 1)
            self.v = _randn(torch, dev, g, Tk, H, V + 8)[..., :V]
        self.r = _randn(torch, dev, g, Tk, P + 16)[:, :P] if P else None
        self.q_start = _i32(torch, _starts(rows), dev)
        self.k_start = _i32(torch, _starts(keys), dev)
        self.out = torch.full((T, H, V), 5.0, device=dev).to(torch.bfloat16)
        self.lse = torch.full((T, H), 5.0, device=dev)

    def run(self, **kw):
        self.env[1].latent_prompt(self.q, self.k, self.r, self.v, self.q_start, self.out, self.scale,
                                  k_start=self.k_start, lse=self.lse, **kw)

    def check(self):
        torch, ssd, dev = self.env
        import latent_ref
        torch.cuda.synchronize()
        t = j = 0
        for s, (n, L) in enumerate(zip(self.rows, self.keys)):
            k = self.k[j:j + L].double().transpose(0, 1)
            if self.P:
                k = torch.cat([k, self.r[j:j + L].double()[None].expand(self.H, L, self.P)], -1)
            v = self.v[j:j + L].double().transpose(0, 1)
            pos = torch.arange(n, device=dev) + L - n
            if n:
                out, lse, size, reach = latent_ref.attend(self.q[t:t + n].double(), k, v, pos, self.scale)
                score = (self.N + self.P + 16) * 2.0 ** -24 * reach + 2.0 ** -18
                bound = U * out.abs() + (U + 2 * score[..., None]) * size + 1e-30
                _within(self.out[t:t + n], out, bound, f"out {s}")
                _within(self.lse[t:t + n], lse, score + 2.0 ** -22 * lse.abs().nan_to_num(0, 0, 0),
                        f"lse {s}")
            t, j = t + n, j + L
        assert bool((self.out[t:] == 5.0).all()) and bool((self.lse[t:] == 5.0).all())


@pytest.mark.parametrize("rows,keys", [
    ([1], [1]), ([1], [500]), ([127], [127]), ([128], [128]), ([129], [129]), ([255, 256, 257], [255, 256, 257]),
    ([777], [777]), ([5, 0, 300], [5, 40, 300]), ([130, 3], [400, 1000]), ([60, 200], [10, 150]),
    ([40, 7], [0, 0]), ([513], [1200]),
])
def test_prompt(env, rows, keys):
    for H in (1, 5):
        p = _Prompt(env, rows, keys, H)
        p.run()
        p.check()


@pytest.mark.parametrize("rows,keys", [
    ([1], [500]), ([129], [129]), ([255, 256, 257], [255, 256, 257]), ([777], [777]), ([130, 3], [400, 1000]),
    ([60, 200], [10, 150]), ([40, 7], [0, 0]), ([513], [1200]),
])
def test_prompt_many_heads(env, rows, keys):
    p = _Prompt(env, rows, keys, 160)
    p.run()
    p.check()


@pytest.mark.parametrize("N,P,V", [(64, 64, 64), (64, 0, 64), (128, 0, 128), (128, 64, 64), (64, 64, 128),
                                   (64, 0, 128)])
def test_prompt_widths(env, N, P, V):
    for joint in (True, False):
        for H, rows, keys in ((3, [300, 20], [300, 220]), (1, [30], [1900]), (80, [300, 20], [300, 220])):
            p = _Prompt(env, rows, keys, H, N, P, V, joint=joint)
            p.run()
            p.check()


def test_prompt_many_sequences(env):
    rows = [(7 * i) % 5 for i in range(900)]
    p = _Prompt(env, rows, [n + (i % 3) for i, n in enumerate(rows)], 2)
    p.run()
    p.check()


@pytest.mark.parametrize("rows,H", [([4096], 64), ([777], 16), ([1000], 3)])
def test_prompt_many_calls(env, rows, H):
    """The same bits and no wait that runs out over up to a thousand blocks of rows, 300 times."""
    torch, ssd, dev = env
    p = _Prompt(env, rows, rows, H, extra=0)
    p.run()
    first = p.out.clone()
    for _ in range(300):
        p.run()
    assert ssd.dec_sync_status() == ssd.DEC_OK
    assert torch.equal(first, p.out)


def test_prompt_keys_by_default(env):
    torch, ssd, dev = env
    p = _Prompt(env, [200, 77], [200, 77], 4, extra=0)
    p.run()
    out = torch.empty_like(p.out)
    ssd.latent_prompt(p.q, p.k, p.r, p.v, p.q_start, out, p.scale)
    assert torch.equal(out, p.out)


# (a CTA takes 128 rows where there are few, 256 rows with many heads)
@pytest.mark.parametrize("H", [2, 160])
def test_prompt_growing_scores(env, H):
    torch, ssd, dev = env
    p = _Prompt(env, [600], [600], H)
    ramp = torch.linspace(0, 2, p.Tk + 1, device=dev)[:, None, None]
    p.k.copy_((p.k.float() * 0.1 + ramp).to(torch.bfloat16))
    p.q.copy_((p.q.float() * 0.1 + 0.5).to(torch.bfloat16))
    for scale in (0.09, -0.09, 1.5):
        p.scale = scale
        p.run()
        p.check()


@pytest.mark.parametrize("H", [2, 160])
def test_prompt_scores_that_jump(env, H):
    """Scores that grow by far more than what moves the maximum at once, within a tile's halves and from
    tile to tile, for some rows only."""
    torch, ssd, dev = env
    p = _Prompt(env, [700], [700], H)
    for j, size in ((3, 1.0), (70, 8.0), (100, 20.0), (127, 30.0), (200, 45.0), (330, 60.0), (331, 61.0),
                    (500, 90.0), (640, 130.0)):
        p.k[j] = 0
        p.k[j, :, 5] = size
    p.q[:, :, 5] = 4.0
    p.q[::3, :, 5] = -4.0
    for scale in (0.09, 1.0, -1.0):
        p.scale = scale
        p.run()
        assert ssd.dec_sync_status() == ssd.DEC_OK
        p.check()


@pytest.mark.parametrize("H", [2, 160])
def test_prompt_not_finite_where_not_seen(env, H):
    """NaN in keys and values of later tokens and of other sequences does not reach a row; a value
    that is seen makes its element what the sum makes it."""
    torch, ssd, dev = env
    for at in (150, 40, 299, 128, 255, 100, 70, 200):
        p = _Prompt(env, [300, 90], [300, 90], H)
        p.run()
        clean = p.out.clone()
        p.k[300:] = math.nan
        p.v[300:] = math.nan
        p.run()
        assert torch.equal(p.out[:300], clean[:300])
        p = _Prompt(env, [300, 90], [300, 90], H)
        p.v[at, 1, 17] = math.inf
        p.v[at, 1, 18] = math.nan
        p.run()
        torch.cuda.synchronize()
        want = clean.clone()
        got = p.out
        rows = slice(at, 300)
        assert bool((got[rows, 1, 17] == math.inf).all()), at
        assert bool(got[rows, 1, 18].isnan().all()), at
        got[rows, 1, 17:19] = want[rows, 1, 17:19]
        # rows that see it hold its weight in the sum all the same: the others' elements stay
        assert bool((got.float() - want.float()).abs().max() <= 2.0 ** -7 * want.float().abs().max())
        assert torch.equal(got[:at], want[:at]) and torch.equal(got[300:], want[300:])
        p = _Prompt(env, [300, 90], [300, 90], H)
        p.k[at, 0, 3] = math.nan
        p.run()
        assert bool(p.out[at:300, 0].isnan().all()) and torch.equal(p.out[:at], clean[:at])


# ------------------------------------------------------------ used together ----

def _layer(env, prompt, steps, H=16, R=512, N=128, P=64, V=128, page=16, e4m3=False, graph=True):
    """A prompt in the expanded form, then single tokens in the absorbed one from a captured
    graph: both against plain attention over the same latent vectors."""
    torch, ssd, dev = env
    import latent_ref
    g = _gen(torch, dev, 77)
    S, total = len(prompt), sum(prompt)
    longest = max(prompt) + steps
    max_pages = -(-longest // page)
    w_uk = (_randn(torch, dev, g, H, R, N).float() * N ** -0.5).to(torch.bfloat16)   # into latent
    w_uv = (_randn(torch, dev, g, H, V, R).float() * R ** -0.5).to(torch.bfloat16)   # back
    weight = torch.ones(R, device=dev).to(torch.bfloat16)
    inv, mag = ssd.rope_frequencies(P, device=dev)
    scale = (N + P) ** -0.5
    dtype = torch.float8_e4m3fn if e4m3 else torch.bfloat16
    cache = torch.zeros((S * max_pages + 1, page, R + P), device=dev).to(dtype)
    c_scale = torch.full((1,), 0.02, device=dev) if e4m3 else None
    table = torch.full((S, max_pages), -1, dtype=torch.int32, device=dev)
    free = torch.randperm(S * max_pages, generator=g, device=dev).to(torch.int32)
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32, device=dev)

    # the prompt
    down, up = _randn(torch, dev, g, total, R + P), _randn(torch, dev, g, total, H, N + P)
    kv_len, summary = i32(S), i32(4)
    q_start, pos, slots = i32(S + 1), i32(total), i32(total)
    ssd.kv_plan(kv_len, _i32(torch, prompt, dev), table, free, summary[1:2], page, kv_len, q_start, pos,
                slots, summary)
    q, rows = up.clone(), torch.empty_like(down)
    ssd.latent_append(down[:, :R], down[:, R:], pos, slots, inv, cache, weight=weight, q_rope=q[..., N:],
                      q_out=q[..., N:], rows=rows, cache_scale=c_scale)
    # keys and values of every head from the latent vectors: one matrix a head
    k, v = (torch.empty((total, H, d), dtype=torch.bfloat16, device=dev) for d in (N, V))
    lat = rows[:, None, :R].expand(total, H, R).contiguous()
    ssd.latent_project(lat, w_uk.transpose(1, 2).contiguous(), k)
    ssd.latent_project(lat, w_uv, v)
    out = torch.empty((total, H, V), dtype=torch.bfloat16, device=dev)
    ssd.latent_prompt(q, k, rows[:, R:], v, q_start, out, scale)
    torch.cuda.synchronize()
    x = rows[:, :R].double()
    for got, w in ((k, w_uk.transpose(1, 2)), (v, w_uv)):
        w = w.double()
        _within(got, torch.einsum("jr,hdr->jhd", x, w),
                U * torch.einsum("jr,hdr->jhd", x, w).abs()
                + (R + 2) * 2.0 ** -24 * torch.einsum("jr,hdr->jhd", x.abs(), w.abs()), "expanded")

    def near(got, query, keys, values, at, lse=None):
        want, _, size, reach = latent_ref.attend(query.double(), keys, values, at, scale)
        score = (query.shape[-1] + 16) * 2.0 ** -24 * reach + 2.0 ** -18
        _within(got, want, U * want.abs() + (U + 2 * score[..., None]) * size + 1e-30, "attention")

    t = 0
    for s, n in enumerate(prompt):
        kk = torch.cat([k[t:t + n].double(), rows[t:t + n, None, R:].double().expand(n, H, P)], -1)
        near(out[t:t + n], q[t:t + n], kk.transpose(0, 1), v[t:t + n].double().transpose(0, 1),
             torch.arange(n, device=dev))
        t += n

    # single tokens
    new_down, new_up = _randn(torch, dev, g, S, R + P), _randn(torch, dev, g, S, H, N + P)
    q_lat = torch.empty((S, H, R + P), dtype=torch.bfloat16, device=dev)
    o_lat = torch.empty((S, H, R), dtype=torch.bfloat16, device=dev)
    o = torch.empty((S, H, V), dtype=torch.bfloat16, device=dev)
    kept = torch.empty_like(new_down)
    q_start, pos, slots = i32(S + 1), i32(S), i32(S)
    ws = ssd.workspace(ssd.latent_decode_workspace_bytes(S, S, H, R, P), dev)
    w_in = w_uk  # [H, R, N]: q[t, h] . (U_h c) = (U_h^T q) . c

    def step():
        ssd.kv_plan(kv_len, None, table, free, summary[1:2], page, kv_len, q_start, pos, slots, summary)
        ssd.latent_append(new_down[:, :R], new_down[:, R:], pos, slots, inv, cache, weight=weight,
                          q_rope=new_up[..., N:], q_out=q_lat[..., R:], rows=kept, cache_scale=c_scale)
        ssd.latent_project(new_up[..., :N], w_in, q_lat[..., :R])
        ssd.latent_decode(q_lat, cache, table, kv_len, o_lat, ws, scale, q_start=q_start,
                          cache_scale=c_scale)
        ssd.latent_project(o_lat, w_uv, o)

    cg = None
    for i in range(steps):
        new_down.copy_(_randn(torch, dev, g, S, R + P))
        new_up.copy_(_randn(torch, dev, g, S, H, N + P))
        if graph and i == 1:
            torch.cuda.synchronize()
            cg = torch.cuda.CUDAGraph()
            with torch.cuda.graph(cg):
                step()
        cg.replay() if cg is not None else step()
        torch.cuda.synchronize()
        held = cache.float().double() * (c_scale.double() if e4m3 else 1.0)
        for s, n in enumerate(prompt):
            n += i + 1
            h = held[table[s, :-(-n // page)].long()].reshape(-1, R + P)[:n]
            assert bool((h.abs().sum(-1) > 0).all())
            err = (h[-1] - kept[s].double()).abs()
            assert bool((err <= (2.0 ** -4 * h[-1].abs() + 2.0 ** -9 if e4m3 else 0)).all())
            near(o_lat[s:s + 1], q_lat[s:s + 1], h[None], h[None, :, :R],
                 torch.full((1,), n - 1, device=dev))
        w = w_uv.double()
        back = torch.einsum("shr,hvr->shv", o_lat.double(), w)
        size = torch.einsum("shr,hvr->shv", o_lat.double().abs(), w.abs())
        _within(o, back, U * back.abs() + (R + 2) * 2.0 ** -24 * size, "back")
    assert kv_len.tolist() == [n + steps for n in prompt]


@pytest.mark.parametrize("e4m3", [False, True])
def test_layer_prompt_then_tokens(env, e4m3):
    _layer(env, [70, 1, 300, 15], 20, e4m3=e4m3)


def test_layer_many_heads(env):
    _layer(env, [33, 130], 5, H=128)


# ------------------------------------------------- batches and calls at the edges ----

@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("count", [32, 33, 400])
def test_decode_many_sequences(env, count, e4m3):
    lens = [(37 * i) % 150 for i in range(count)]
    rows = [(i * 5) % 3 for i in range(count)]
    lens[count // 2], rows[count // 2] = 5000, 2
    for H, page in ((8, 16), (64, 13)):
        d = _Decode(env, lens, rows, H, page=page, e4m3=e4m3)
        d.run()
        d.check()


@pytest.mark.parametrize("e4m3", [False, True])
def test_decode_as_many_sequences_as_there_can_be(env, e4m3):
    torch, ssd, dev = env
    S, H, R, W, page = 8192, 4, 64, 128, 16
    g = _gen(torch, dev, 77)
    cache = _cache_of(torch, dev, g, (S, page, W), e4m3, 0.013)
    c_scale = torch.full((1,), 0.013, device=dev) if e4m3 else None
    table = torch.randperm(S, generator=g, device=dev).to(torch.int32).view(S, 1)
    lens = torch.randint(0, page + 1, (S,), generator=g, device=dev, dtype=torch.int32)
    q = _randn(torch, dev, g, S, H, W)
    out = torch.empty((S, H, R), dtype=torch.bfloat16, device=dev)
    ws = ssd.workspace(ssd.latent_decode_workspace_bytes(S, S, H, R, W - R), dev)
    ssd.latent_decode(q, cache, table, lens, out, ws, 0.1, cache_scale=c_scale)
    torch.cuda.synchronize()
    keys = _values(torch, cache)[table[:, 0].long()] * (c_scale.double() if e4m3 else 1.0)
    seen = torch.arange(page, device=dev)[None, None] < lens[:, None, None]
    z = (0.1 * q.double() @ keys.transpose(1, 2)).masked_fill(~seen, float("-inf"))
    reach = (0.1 * q.double().abs() @ keys.abs().transpose(1, 2)).masked_fill(~seen, 0).amax(-1)
    w = z.softmax(-1).nan_to_num(0.0)
    want, size = w @ keys[..., :R], w @ keys[..., :R].abs()
    score = (W + 16) * 2.0 ** -24 * reach + 2.0 ** -18  # as in _Decode.check
    _within(out, want, U * want.abs() + (U + 2 * score[..., None]) * size + 1e-30, "out")


@pytest.mark.parametrize("page", [1 << 16, (1 << 16) - 3])
@pytest.mark.parametrize("e4m3", [False, True])
def test_decode_far_tokens_of_a_window(env, e4m3, page):
    """Token numbers up to the last that an int32 length allows, all pages of a sequence in one place."""
    torch, ssd, dev = env
    import latent_ref
    H, R, W, n, window = 8, 128, 192, 0x7ffffe25, 100
    g = _gen(torch, dev, 78)
    cache = _cache_of(torch, dev, g, (1, page, W), e4m3, 0.013)
    c_scale = torch.full((1,), 0.013, device=dev) if e4m3 else None
    table = torch.zeros((1, (1 << 31) // page + 1), dtype=torch.int32, device=dev)
    q = _randn(torch, dev, g, 2, H, W)
    out = torch.empty((2, H, R), dtype=torch.bfloat16, device=dev)
    lse = torch.empty((2, H), device=dev)
    ws = ssd.workspace(ssd.latent_decode_workspace_bytes(1, 2, H, R, W - R), dev)
    ssd.latent_decode(q, cache, table, _i32(torch, [n], dev), out, ws, 0.06, window=window, lse=lse,
                      q_start=_i32(torch, [0, 2], dev), cache_scale=c_scale)
    torch.cuda.synchronize()
    at = torch.arange(n - window - 1, n, device=dev) % page
    keys = _values(torch, cache[0])[at] * (c_scale.double() if e4m3 else 1.0)
    pos = torch.arange(2, device=dev) + window - 1
    want, want_lse, size, reach = latent_ref.attend(q.double(), keys[None], keys[None, :, :R], pos, 0.06,
                                                    window)
    score = (W + 16) * 2.0 ** -24 * reach + 2.0 ** -18  # as in _Decode.check
    _within(out, want, U * want.abs() + (U + 2 * score[..., None]) * size + 1e-30, "out")
    _within(lse, want_lse, score + 2.0 ** -22 * want_lse.abs(), "lse")


@pytest.mark.parametrize("scale", [0.0, -0.06])
def test_scales_of_zero_and_below(env, scale):
    for e4m3 in (False, True):
        d = _Decode(env, [1, 70, 600, 0], [1, 2, 3, 1], 16, e4m3=e4m3, scale=scale)
        d.run()
        d.check()
    p = _Prompt(env, [300, 20], [300, 220], 3, scale=scale)
    p.run()
    p.check()


def test_prompt_scale_of_zero_with_large_scores(env):
    """Equal weights, whatever the scores are (about 1e30 here)."""
    torch, ssd, dev = env
    p = _Prompt(env, [200], [200], 2, scale=0.0)
    p.q.mul_(1e14)
    p.k.mul_(1e14)
    p.run()
    torch.cuda.synchronize()
    n = torch.arange(1, 201, device=dev).double()[:, None]
    v = p.v[:200].double()
    mean, size = v.cumsum(0) / n[..., None], v.abs().cumsum(0) / n[..., None]
    _within(p.out[:200], mean, U * mean.abs() + (U + 2.0 ** -17) * size, "out")
    _within(p.lse[:200], n.log().expand(200, 2), 2.0 ** -18 + 2.0 ** -22 * n.log(), "lse")


def test_calls_at_once_on_two_streams(env):
    torch, ssd, dev = env
    a = _Decode(env, [9000, 40, 3000], [2, 1, 4], 64)
    b = _Decode(env, [5000, 300], [1, 3], 16, e4m3=True)
    p = _Prompt(env, [700, 3], [900, 3], 8)
    each = (a, b, p)
    for x in each:
        x.run()
    torch.cuda.synchronize()
    want = [(x.out.clone(), x.lse.clone()) for x in each]
    streams = [torch.cuda.Stream() for _ in each]
    for _ in range(20):
        for x in each:
            x.out.fill_(5.0)
            x.lse.fill_(5.0)
        for x, s in zip(each, streams):
            s.wait_stream(torch.cuda.current_stream())
            x.run(stream=s)
        for s in streams:
            torch.cuda.current_stream().wait_stream(s)
        for x, (out, lse) in zip(each, want):
            assert torch.equal(x.out, out) and torch.equal(x.lse, lse)
    assert ssd.dec_sync_status() == ssd.DEC_OK


def test_prompt_replayed_with_other_lengths(env):
    """One captured graph serves every division of its rows and keys."""
    torch, ssd, dev = env
    p = _Prompt(env, [300, 20, 100], [300, 220, 100], 4)
    p.run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        p.run()
    for rows, keys in (([300, 20, 100], [300, 220, 100]), ([0, 400, 20], [10, 500, 110]),
                       ([1, 1, 418], [200, 1, 419]), ([0, 0, 0], [5, 5, 5])):
        p.rows, p.keys = rows, keys
        p.q_start.copy_(_i32(torch, _starts(rows), dev))
        p.k_start.copy_(_i32(torch, _starts(keys), dev))
        p.out.fill_(5.0)
        p.lse.fill_(5.0)
        graph.replay()
        p.check()


def test_binding_refuses_what_is_elsewhere_or_of_another_size(env):
    torch, ssd, dev = env
    d = _Decode(env, [100, 30], [1, 1], 8)
    q, out = d.q[:2], d.out[:2]
    good = dict(table=d.table, lens=d.seq_len, q_start=d.q_start, lse=d.lse[:2], ws=d.ws)

    def run(**kw):
        a = dict(good, **kw)
        ssd.latent_decode(q, d.cache, a["table"], a["lens"], out, a["ws"], 0.06, q_start=a["q_start"],
                          lse=a["lse"])

    run()
    for name in good:
        with pytest.raises(TypeError):
            run(**{name: good[name].cpu()})
    for name in ("lens", "q_start", "lse"):
        with pytest.raises(ValueError):
            run(**{name: good[name][:1]})
    for name in ("table", "lens", "q_start"):
        with pytest.raises(TypeError):
            run(**{name: good[name].long()})
    c, r = _randn(torch, dev, _gen(torch, dev, 5), 2, 576).split([512, 64], 1)
    at = _i32(torch, [0, 1], dev)
    freq = torch.ones(32, device=dev)
    ssd.latent_append(c, r, at, at, freq, d.cache)
    for args in ((at.cpu(), at, freq), (at, at.cpu(), freq), (at, at, freq.cpu()), (at, at, freq.double())):
        with pytest.raises(TypeError):
            ssd.latent_append(c, r, *args, d.cache)
    with pytest.raises(ValueError):
        ssd.latent_append(c, r, at[:1], at, freq, d.cache)
    with pytest.raises(TypeError):
        ssd.latent_append(c.cpu(), r, at, at, freq, d.cache)
    p = _Prompt(env, [30], [30], 2)
    p.run()
    for name in ("q_start", "k_start", "lse", "r", "v"):
        was = getattr(p, name)
        setattr(p, name, was.cpu())
        with pytest.raises(TypeError):
            p.run()
        setattr(p, name, was)
    assert ssd.dec_sync_status() == ssd.DEC_OK

"""GPU parity of kv_plan, rope_append and attn_decode with plain 64-bit forms.

Tolerances, derived from the arithmetic (u = 2^-8 is bf16's unit roundoff):
  - the planner's outputs are whole numbers: equal.
  - rope_append: one rounding of a fp32 rotation, u |y| plus 2^-20 (|x0| + |x1|) for the
    sine, the cosine and three fp32 operations; e4m3: unit roundoff 2^-4, smallest step
    2^-9, and the same 2^-20 share of the unscaled size.
  - attn_decode: u |out| for the last rounding; u sum_j w_j |v_j| for weights that round to
    bf16 before the product with V; and twice the relative error of the weights, which is
    the absolute error of a fp32 score, (D + 16) 2^-24 scale sum_d |q_d k_d|, plus 2^-18
    for exponentials and sums.
"""
import math

import numpy as np
import pytest

import attn_ref

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


def _f64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def _i32(torch, x, dev):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device=dev)


# ------------------------------------------------------------------ kv_plan ----

def _plan(env, kv, new, table, free, used, page, max_tokens, alias=False):
    torch, ssd, dev = env
    S = len(kv)
    kv_t = _i32(torch, kv, dev)
    new_t = None if new is None else _i32(torch, new, dev)
    tab_t = _i32(torch, table, dev)
    summary = torch.full((4,), -9, dtype=torch.int32, device=dev)
    summary[1] = used
    used_t = summary[1:2] if alias else _i32(torch, [used], dev)
    seq = kv_t if alias else torch.full((S,), -9, dtype=torch.int32, device=dev)
    qs = torch.full((S + 1,), -9, dtype=torch.int32, device=dev)
    pos = torch.full((max_tokens,), -9, dtype=torch.int32, device=dev)
    slots = torch.full((max_tokens,), -9, dtype=torch.int32, device=dev)
    ssd.kv_plan(kv_t, new_t, tab_t, _i32(torch, free, dev), used_t, page, seq, qs, pos, slots,
                summary)
    torch.cuda.synchronize()
    return [x.cpu().numpy() for x in (tab_t, seq, qs, pos, slots, summary)]


def _check_plan(env, kv, new, table, free, used, page, max_tokens, alias=False):
    got = _plan(env, kv, new, table, free, used, page, max_tokens, alias)
    want = attn_ref.kv_plan(kv, [1] * len(kv) if new is None else new, table, free, used, page,
                            max_tokens)
    for g, w, name in zip(got, want, ("table", "seq_len", "q_start", "positions", "slots",
                                      "summary")):
        assert np.array_equal(g, w), name


def _plan_case(seed, S, page, max_len, max_new, spare=0):
    rng = np.random.default_rng(seed)
    kv = rng.integers(0, max_len + 1, S)
    new = rng.integers(0, max_new + 1, S)
    have = -(-kv // page)
    width = int((-(-(kv + new) // page)).max()) + 1
    wanted = int((-(-(kv + new) // page) - have).sum())
    ids = rng.permutation(int(have.sum()) + wanted + 7)
    table = np.full((S, width), -1)
    at = 0
    for s in range(S):
        table[s, :have[s]] = ids[at:at + have[s]]
        at += have[s]
    return kv, new, table, ids[at:at + max(0, wanted + spare)]


@pytest.mark.parametrize("alias", [False, True])
@pytest.mark.parametrize("S,page,max_len,max_new", [
    (1, 1, 0, 1), (1, 16, 100, 1), (2, 3, 5, 40), (64, 16, 8192, 8), (33, 48, 500, 3),
    (1023, 16, 64, 2), (1024, 8, 64, 2), (1025, 7, 64, 3), (4, 64, 3000, 9000),
    (8192, 16, 32, 2),
])
def test_plan(env, S, page, max_len, max_new, alias):
    kv, new, table, free = _plan_case(S + page, S, page, max_len, max_new)
    T = max(1, int(new.sum()))
    _check_plan(env, kv, new, table, free, 0, page, T, alias)
    _check_plan(env, kv, new, table, free, 0, page, T + 77, alias)   # padded rows


def test_plan_one_token_each_by_default(env):
    kv, _, table, free = _plan_case(5, 50, 16, 200, 1, spare=50)
    table = np.concatenate([table, np.full((50, 1), -1)], 1)
    _check_plan(env, kv, None, table, free, 0, 16, 50)


def test_plan_shortages(env):
    """Rows beyond max_tokens, a free list that runs out, a list partly used, a table that is
    too narrow, lengths below zero, pages that a sequence lacks."""
    kv, new, table, free = _plan_case(6, 40, 4, 50, 9, spare=20)
    T = int(new.sum())
    _check_plan(env, kv, new, table, free, 0, 4, T // 2)
    _check_plan(env, kv, new, table, free[:11], 0, 4, T)
    _check_plan(env, kv, new, table, free, 5, 4, T)
    _check_plan(env, kv, new, table, free, len(free), 4, T)
    _check_plan(env, kv, new, table, free, len(free) + 3, 4, T)
    _check_plan(env, kv, new, table, free, -3, 4, T)
    _check_plan(env, kv, new, table, free[:0], 0, 4, T)
    _check_plan(env, kv, new, np.ascontiguousarray(table[:, :5]), free, 0, 4, T)
    kv2, new2 = kv.copy(), new.copy()
    kv2[::7], new2[::5] = -4, -1
    _check_plan(env, kv2, new2, table, free, 0, 4, T)
    table2 = table.copy()
    table2[:, 0] = -1
    _check_plan(env, kv, new, table2, free, 0, 4, T)


def test_plan_large_numbers(env):
    """Sums past 2^31 and slots past int32 saturate or are dropped, they do not wrap."""
    big = 2 ** 30
    table = np.full((4, 2), 2 ** 31 - 5)
    _check_plan(env, [1, 2, 3, 16], [big, big, big, big], table, [2 ** 31 - 1] * 8, 0, 16, 100)


def test_plan_carries_its_state_in_a_graph(env):
    """seq_len in place of kv_len and the free count in summary[1]: one captured call, step
    after step, as a plain loop gives."""
    torch, ssd, dev = env
    S, page, width, steps = 5, 4, 12, 30
    table = torch.full((S, width), -1, dtype=torch.int32, device=dev)
    length = _i32(torch, [0, 3, 4, 9, 1], dev)
    want_len = length.cpu().numpy().astype(np.int64)
    free = _i32(torch, np.random.default_rng(1).permutation(S * width), dev)
    want_tab, used = table.cpu().numpy().astype(np.int64), 0
    for s in range(S):
        n = -(-want_len[s] // page)
        want_tab[s, :n] = free.cpu().numpy()[used:used + n]
        used += n
    table.copy_(_i32(torch, want_tab, dev))
    summary = _i32(torch, [0, used, 0, 0], dev)
    qs = torch.zeros(S + 1, dtype=torch.int32, device=dev)
    pos, slots = (torch.zeros(S, dtype=torch.int32, device=dev) for _ in range(2))

    def call():
        ssd.kv_plan(length, None, table, free, summary[1:2], page, length, qs, pos, slots, summary)
    g = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    with torch.cuda.graph(g, stream=side):
        call()
    for _ in range(steps):
        g.replay()
        torch.cuda.synchronize()
        want_tab, want_len, _, wp, ws, wsum = attn_ref.kv_plan(
            want_len, [1] * S, want_tab, free.cpu().numpy(), used, page, S)
        used = int(wsum[1])
        for got, want in ((table, want_tab), (length, want_len), (pos, wp), (slots, ws),
                          (summary, wsum)):
            assert np.array_equal(got.cpu().numpy(), want)


# -------------------------------------------------------------- rope_append ----

def _caches(torch, dev, pages, Hkv, page, D, e4m3, layout="heads", fill=0):
    """Two [pages, Hkv, page, D] caches: by heads, by tokens, or as halves of one array."""
    byte = torch.uint8 if e4m3 else torch.int16
    if layout == "heads":
        k, v = (torch.full((pages, Hkv, page, D), fill, dtype=byte, device=dev) for _ in range(2))
    elif layout == "tokens":
        k, v = (torch.full((pages, page, Hkv, D), fill, dtype=byte, device=dev).transpose(1, 2)
                for _ in range(2))
    else:
        both = torch.full((pages, 2, Hkv, page, D), fill, dtype=byte, device=dev)
        k, v = both[:, 0], both[:, 1]
    dt = torch.float8_e4m3fn if e4m3 else torch.bfloat16
    return k.view(dt), v.view(dt)


def _cache_f64(torch, c):
    return _f64(c.contiguous())


def _e4m3_ok(got, want, size, scale):
    """got: stored values; want: unrounded value / scale."""
    want = np.clip(want, -448.0, 448.0)
    return np.abs(got - want) <= 2.0 ** -4 * np.abs(want) + 2.0 ** -10 + 2.0 ** -20 * size / scale


@pytest.mark.parametrize("layout", ["heads", "tokens", "halves"])
@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("T,Hq,Hkv,D,rot", [
    (1, 1, 1, 16, 16), (1, 64, 8, 128, 128), (3, 7, 1, 64, 32), (5, 6, 2, 80, 80),
    (4, 4, 4, 96, 2), (9, 12, 3, 256, 256), (2, 5, 5, 48, 0), (17, 8, 2, 112, 42),
    (2, 3, 3, 256, 250), (130, 16, 2, 128, 64),
])
def test_rope_append(env, T, Hq, Hkv, D, rot, interleaved, e4m3, layout):
    torch, ssd, dev = env
    g = torch.Generator(device=dev).manual_seed(T * 131 + D + rot)
    rows = torch.randn((T, (Hq + 2 * Hkv) * D), generator=g, device=dev).to(torch.bfloat16)
    q = rows[:, :Hq * D].view(T, Hq, D)
    k = rows[:, Hq * D:(Hq + Hkv) * D].view(T, Hkv, D)
    v = rows[:, (Hq + Hkv) * D:].view(T, Hkv, D)
    page = 5
    pages = T // page + 3
    rng = np.random.default_rng(D + T)
    slots = rng.permutation(pages * page)[:T]
    pos = rng.integers(0, 200000, T)
    pos[0] = 0
    if T > 3:
        slots[1], slots[2] = -1, pages * page   # not cached: no place, and one past the end
        pos[3] = 2 ** 31 - 1
    inv, mag = (None, 1.0) if rot == 0 else ssd.rope_frequencies(rot, 10000.0, ssd.ROPE_PARTS, 4.0,
                                                                device=dev)
    kc, vc = _caches(torch, dev, pages, Hkv, page, D, e4m3, layout)
    ks = vs = None
    if e4m3:
        ks = torch.rand(Hkv, generator=g, device=dev) * 0.1 + 0.005
        vs = torch.rand(Hkv, generator=g, device=dev) * 0.1 + 0.002   # some values saturate
    out = torch.full_like(q.contiguous(), float("nan"))
    ssd.rope_append(q, k, v, _i32(torch, pos, dev), _i32(torch, slots, dev), inv, out, kc, vc,
                    interleaved=interleaved, magnitude=mag, k_scale=ks, v_scale=vs)
    torch.cuda.synchronize()
    qn, kn, vn, on = _f64(q), _f64(k), _f64(v), _f64(out)
    kcn, vcn = _cache_f64(torch, kc), _cache_f64(torch, vc)
    invn = [] if inv is None else inv.cpu().numpy()
    touched = np.zeros((pages, page), bool)
    for t in range(T):
        y, size = attn_ref.rotate(qn[t], pos[t], invn, mag, interleaved)
        assert np.all(np.abs(on[t] - y) <= U * np.abs(y) + 2.0 ** -20 * size), t
        if not 0 <= slots[t] < pages * page:
            continue
        at, o = slots[t] // page, slots[t] % page
        touched[at, o] = True
        y, size = attn_ref.rotate(kn[t], pos[t], invn, mag, interleaved)
        gk, gv = kcn[at, :, o], vcn[at, :, o]
        if e4m3:
            s = _f64(ks)[:, None]
            assert np.all(_e4m3_ok(gk, y / s, size, s))
            s = _f64(vs)[:, None]
            assert np.all(_e4m3_ok(gv, vn[t] / s, np.abs(vn[t]), s))
        else:
            assert np.all(np.abs(gk - y) <= U * np.abs(y) + 2.0 ** -20 * size)
            assert np.array_equal(gv, vn[t])
    # everything else in the cache stays as it was
    assert not kcn.transpose(0, 2, 1, 3)[~touched].any()
    assert not vcn.transpose(0, 2, 1, 3)[~touched].any()


@pytest.mark.parametrize("rot,interleaved", [(128, False), (128, True), (64, False), (42, False),
                                             (30, True)])
def test_rope_append_in_place(env, rot, interleaved):
    """q_out = q gives the bits of a separate q_out, inside a projection's rows."""
    torch, ssd, dev = env
    T, Hq, Hkv, D, page = 33, 8, 2, 128, 16
    g = torch.Generator(device=dev).manual_seed(3)
    rows = torch.randn((T, (Hq + 2 * Hkv) * D), generator=g, device=dev).to(torch.bfloat16)
    q = rows[:, :Hq * D].view(T, Hq, D)
    k = rows[:, Hq * D:(Hq + Hkv) * D].view(T, Hkv, D)
    v = rows[:, (Hq + Hkv) * D:].view(T, Hkv, D)
    pos = torch.arange(T, dtype=torch.int32, device=dev) * 7
    inv, _ = ssd.rope_frequencies(rot, device=dev)
    out = torch.empty((T, Hq, D), dtype=torch.bfloat16, device=dev)
    kc, vc = _caches(torch, dev, 4, Hkv, page, D, False)
    tail = rows[:, Hq * D:].clone()
    ssd.rope_append(q, k, v, pos, pos % 64, inv, out, kc, vc, interleaved=interleaved)
    ssd.rope_append(q, k, v, pos, pos % 64, inv, q, kc, vc, interleaved=interleaved)
    torch.cuda.synchronize()
    assert torch.equal(q, out) and torch.equal(rows[:, Hq * D:], tail)


def test_rope_append_infinite_and_nan_values(env):
    torch, ssd, dev = env
    T, H, D = 2, 1, 64
    x = torch.ones((T, H, D), dtype=torch.bfloat16, device=dev)
    v = torch.ones_like(x)
    v[0, 0, :3] = torch.tensor([float("inf"), float("-inf"), float("nan")])
    for e4m3 in (False, True):
        kc, vc = _caches(torch, dev, 1, H, 4, D, e4m3)
        inv, _ = ssd.rope_frequencies(D, device=dev)
        pos = torch.zeros(T, dtype=torch.int32, device=dev)
        ssd.rope_append(x, x, v, pos, _i32(torch, [2, 0], dev), inv, torch.empty_like(x), kc, vc)
        torch.cuda.synchronize()
        got = _f64(vc)[0, 0, 2, :4]
        top = 448.0 if e4m3 else np.inf
        assert got[0] == top and got[1] == -top and np.isnan(got[2]) and got[3] == 1.0
        assert np.all(_f64(vc)[0, 0, 0] == 1.0)


# -------------------------------------------------------------- attn_decode ----

class _Case:
    """Random sequences in a paged cache, with NaN at every place that no row may read."""

    def __init__(self, env, lengths, rows, Hq, Hkv, D, page, e4m3=False, layout="heads", seed=0,
                 spread=1.5, width=None, q_start=True):
        torch, ssd, dev = env
        self.env, self.lengths, self.rows = env, list(lengths), list(rows)
        self.Hq, self.Hkv, self.D, self.page, self.e4m3 = Hq, Hkv, D, page, e4m3
        S, T = len(self.lengths), sum(self.rows)
        used = [attn_ref.pages_of(n, page) for n in self.lengths]
        total = sum(used) + 3
        rng = np.random.default_rng(seed)
        ids = rng.permutation(total)
        width = max(1, max(used)) + 1 if width is None else width
        # entries past a sequence's pages are garbage: out of range, or other pages
        self.table = rng.integers(-2 ** 31, 2 ** 31, (S, width))
        self.table[:, ::2] = rng.integers(0, total, (S, (width + 1) // 2))
        at = 0
        nan = 0x7f if e4m3 else 0x7fc0
        self.kc, self.vc = _caches(torch, dev, total, Hkv, page, D, e4m3, layout, nan)
        self.k, self.v = [], []
        g = torch.Generator(device=dev).manual_seed(seed)
        self.ks = self.vs = None
        if e4m3:
            self.ks = torch.rand(Hkv, generator=g, device=dev) * 0.02 + 0.01
            self.vs = torch.rand(Hkv, generator=g, device=dev) * 0.02 + 0.01
        for s, n in enumerate(self.lengths):
            for c, scale, keep in ((self.kc, self.ks, self.k), (self.vc, self.vs, self.v)):
                x = torch.randn((n, Hkv, D), generator=g, device=dev)
                if e4m3:
                    x = (x / scale[:, None]).clamp(-448, 448).to(torch.float8_e4m3fn)
                    keep.append(_f64(x) * _f64(scale)[:, None])
                else:
                    x = x.to(torch.bfloat16)
                    keep.append(_f64(x))
                for i in range(used[s]):
                    part = x[i * page:(i + 1) * page]
                    dst = c[int(ids[at + i]), :, :part.shape[0]]
                    kind = torch.uint8 if e4m3 else torch.int16
                    dst.view(kind).copy_(part.transpose(0, 1).contiguous().view(kind))
            m = min(used[s], width)
            self.table[s, :m] = ids[at:at + m]
            at += used[s]
        self.q = torch.randn((T, Hq, D), generator=g, device=dev).to(torch.bfloat16)
        self.scale = spread / math.sqrt(D)
        self.q_start = np.concatenate([[0], np.cumsum(self.rows)]) if q_start else None
        self.ws = ssd.workspace(ssd.attn_decode_workspace_bytes(S, T, Hq, Hkv, D))

    def run(self, window=0, lse=True, q=None, out=None, stream=None):
        torch, ssd, dev = self.env
        T = sum(self.rows)
        out = torch.full((T, self.Hq, self.D), 77.0, dtype=torch.bfloat16, device=dev) \
            if out is None else out
        l = torch.full((T, self.Hq), 77.0, dtype=torch.float32, device=dev) if lse else None
        ssd.attn_decode(self.q if q is None else q, self.kc, self.vc,
                        _i32(torch, self.table, dev), _i32(torch, self.lengths, dev), out, self.ws,
                        q_start=None if self.q_start is None else _i32(torch, self.q_start, dev),
                        scale=self.scale, window=window, lse=l, k_scale=self.ks,
                        v_scale=self.vs, stream=stream)
        torch.cuda.synchronize()
        return out, l

    def visible(self, s):
        torch, ssd, dev = self.env
        pages = self.kc.shape[0]
        ok = [j // self.page < self.table.shape[1]
              and 0 <= self.table[s, j // self.page] < pages for j in range(self.lengths[s])]
        return np.array(ok, bool)

    def check(self, window=0, **kw):
        out, lse = self.run(window, **kw)
        o, t = _f64(out), 0
        l = None if lse is None else lse.cpu().numpy().astype(np.float64)
        q = _f64(self.q)
        for s, n in enumerate(self.lengths):
            r = self.rows[s]
            width = self.table.shape[1] * self.page
            k, v, ok = self.k[s][:width], self.v[s][:width], self.visible(s)[:width]
            want, wl, size, reach = attn_ref.attention(q[t:t + r], k, v, ok, self.scale, window)
            score = (self.D + 16) * 2.0 ** -24 * reach
            bound = U * np.abs(want) + (U + 2 * score[..., None] + 2.0 ** -18) * size
            err = np.abs(o[t:t + r] - want)
            assert np.all(err <= bound), (s, float((err / np.maximum(bound, 1e-300)).max()))
            if l is not None:
                empty = np.isinf(wl)
                assert np.array_equal(l[t:t + r][empty], wl[empty])
                d = np.abs(l[t:t + r][~empty] - wl[~empty])
                assert np.all(d <= score[~empty] + 2.0 ** -20 * (1 + np.abs(wl[~empty])))
            t += r
        return out, lse


LAYOUTS = ["heads", "tokens", "halves"]


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("D", [16, 48, 64, 80, 128, 144, 192, 256])
@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (3, 3), (8, 1), (14, 2), (16, 1), (20, 1)])
def test_attn_heads_and_sizes(env, Hq, Hkv, D, e4m3):
    c = _Case(env, [1, 0, 17, 300, 64, 33], [1] * 6, Hq, Hkv, D, 16, e4m3, seed=D + Hq)
    c.check()


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("page", [1, 3, 16, 48, 64, 100, 256])
def test_attn_pages_and_layouts(env, page, layout, e4m3):
    c = _Case(env, [1, 31, 32, 33, 255, 257, 500], [1, 2, 1, 3, 1, 1, 2], 8, 2, 64, page, e4m3,
              layout, seed=page)
    c.check()


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("rows", [1, 2, 3, 4, 5, 8, 9, 16, 17, 40])
@pytest.mark.parametrize("Hq,Hkv,D", [(8, 1, 128), (7, 1, 64), (4, 4, 96), (2, 1, 256),
                                      (24, 2, 128)])
def test_attn_several_rows(env, rows, Hq, Hkv, D, e4m3):
    """Verification rows, causal among themselves; also more rows than tokens (the first
    rows then see nothing)."""
    c = _Case(env, [rows, 130, 0, 77, max(0, rows - 2)], [rows, rows, rows, 1, rows], Hq, Hkv, D,
              16, e4m3, seed=rows)
    out, lse = c.check()
    if rows > 2:
        t = sum(c.rows[:4])
        assert not out[t:t + 2].any() and bool((lse[t:t + 2] == -math.inf).all())


@pytest.mark.parametrize("rows", [1, 3])
@pytest.mark.parametrize("window", [1, 2, 15, 16, 17, 100, 1000])
def test_attn_window(env, window, rows):
    c = _Case(env, [1, 16, 90, 1001, 0, 333], [rows] * 6, 8, 2, 64, 16, seed=window)
    c.check(window)


def test_attn_missing_pages(env):
    """Pages outside the cache are not seen; a row all of whose pages are missing is empty."""
    c = _Case(env, [64, 40, 200], [1, 2, 1], 4, 2, 64, 16, seed=9)
    c.table[0, 1] = -1
    c.table[1, :] = 10 ** 6
    c.table[2, 4:9] = -2 ** 31
    c.check()
    c.check(window=30)


def test_attn_table_narrower_than_the_length(env):
    """A length past the table's pages is taken as what the table holds."""
    c = _Case(env, [100, 50], [1, 1], 4, 2, 64, 16, seed=10, width=3)
    held = [min(n, 48) for n in c.lengths]
    c.k, c.v = [x[:n] for x, n in zip(c.k, held)], [x[:n] for x, n in zip(c.v, held)]
    full, c.lengths = c.lengths, held
    want, _ = c.check()
    c.lengths = full
    got, _ = c.run()
    assert c.env[0].equal(got, want)


@pytest.mark.parametrize("e4m3", [False, True])
def test_attn_nan_and_infinity_in_unseen_places(env, e4m3):
    """Values of later tokens of the same call (a later draft token gone wrong) do not reach
    earlier rows; a row that sees them gets what the definition gives."""
    torch, ssd, dev = env
    c = _Case(env, [50, 200], [6, 3], 8, 2, 64, 16, e4m3, seed=11)
    want, want_lse = c.check()
    bad = float("nan") if e4m3 else float("inf")
    for s, j in ((0, 47), (1, 199)):
        page = int(c.table[s, j // 16])
        kind = torch.uint8 if e4m3 else torch.int16
        for cache, value in ((c.kc, float("nan")), (c.vc, bad)):
            cell = torch.full((2, 64), value, device=dev).to(cache.dtype)
            cache[page, :, j % 16].view(kind).copy_(cell.view(kind))
    got, lse = c.run()
    for t, clean in enumerate([True] * 3 + [False] * 3 + [True, True, False]):
        if clean:  # rows of sequence 0 at 44, 45, 46; of sequence 1 at 197, 198
            assert torch.equal(got[t], want[t]) and torch.equal(lse[t], want_lse[t]), t
        else:
            assert bool(torch.isnan(got[t].float()).all()) and bool(torch.isnan(lse[t]).all()), t


def test_attn_infinite_values_alone(env):
    """An infinite value (finite keys) reaches the rows that see it, in its element only."""
    torch, ssd, dev = env
    c = _Case(env, [40], [4], 4, 1, 64, 16, seed=12)
    want, want_lse = c.check()
    c.vc[int(c.table[0, 38 // 16]), 0, 38 % 16, 5] = float("inf")
    got, lse = c.run()
    assert torch.equal(lse, want_lse) and torch.equal(got[:2], want[:2])
    assert bool((got[2:, :, 5] == math.inf).all())
    keep = [d for d in range(64) if d != 5]
    assert torch.equal(got[2:, :, keep], want[2:, :, keep])


@pytest.mark.parametrize("e4m3", [False, True])
def test_attn_large_scores(env, e4m3):
    """Scores in the hundreds: the running maximum keeps every exponential in range."""
    c = _Case(env, [300, 1, 47], [2, 1, 1], 8, 2, 128, 16, e4m3, seed=13, spread=150.0)
    c.check()


def test_attn_small_and_large_queries_e4m3(env):
    """Query rows far outside the 16-bit range of the 8-bit path's operands."""
    c = _Case(env, [300, 65], [1, 2], 8, 2, 64, 16, True, seed=14)
    c.q[0] *= 1e30
    c.q[1] *= 1e-30
    c.scale *= 1e-28
    c.check()


def test_attn_scores_of_minus_infinity(env):
    torch, ssd, dev = env
    c = _Case(env, [20], [1], 2, 1, 64, 16, seed=15)
    c.q.fill_(1.0)
    c.kc[int(c.table[0, 0])] = float("-inf")
    got, lse = c.run()  # only the last four tokens count
    want, wl, size, _ = attn_ref.attention(_f64(c.q), c.k[0][16:], c.v[0][16:],
                                           np.ones(4, bool), c.scale, 0)
    assert np.all(np.abs(_f64(got) - want) <= U * np.abs(want) + (U + 2.0 ** -12) * size)
    c.kc[int(c.table[0, 1])] = float("-inf")
    got, lse = c.run()
    assert not got.any() and bool((lse == -math.inf).all())


def test_attn_without_lse_and_q_start_and_with_strides(env):
    torch, ssd, dev = env
    c = _Case(env, [100, 3, 257], [1, 1, 1], 8, 2, 64, 16, seed=16, q_start=False)
    want, _ = c.check()
    assert torch.equal(c.run(lse=False)[0], want)
    wide = torch.full((3, 24 * 64), 5.0, dtype=torch.bfloat16, device=dev)
    wide[:, :8 * 64] = c.q.view(3, -1)
    o = torch.full((3, 10 * 64), 5.0, dtype=torch.bfloat16, device=dev)
    got, _ = c.run(q=wide[:, :8 * 64].view(3, 8, 64), out=o[:, 64:9 * 64].view(3, 8, 64))
    assert torch.equal(got, want)
    assert bool((o[:, :64] == 5.0).all()) and bool((o[:, 9 * 64:] == 5.0).all())


def test_attn_rows_of_no_sequence_are_left(env):
    torch, ssd, dev = env
    c = _Case(env, [30, 60, 9], [2, 3, 2], 4, 2, 64, 16, seed=17)
    want, want_lse = c.check()
    c.q_start = np.array([0, 2, 2, 4])     # the second sequence has no rows now
    c.q[2:4] = c.q[5:7].clone()
    got, lse = c.run()
    assert torch.equal(got[:2], want[:2]) and torch.equal(got[2:4], want[5:7])
    assert torch.equal(lse[2:4], want_lse[5:7])
    assert bool((got[4:] == 77.0).all()) and bool((lse[4:] == 77.0).all())


def test_attn_row_starts_out_of_range(env):
    """Row starts are read within 0..T and never lead out of the arrays."""
    torch, ssd, dev = env
    c = _Case(env, [30, 60, 9], [2, 3, 2], 4, 2, 64, 16, seed=18)
    for bad in ([0, 2, 5, 2 ** 31 - 1], [-2 ** 31, 2, 5, 7], [7, 5, 2, 0]):
        c.q_start = np.array(bad)
        c.run()
    c.q_start = np.array([0, 2, 5, 7])
    c.check()
    n = c.lengths
    c.lengths = [-5, 2 ** 31 - 1, 9]
    c.run()
    c.lengths = n
    c.check()


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("lengths,rows,Hq,Hkv,D", [
    ([20011], 1, 8, 1, 128), ([5000, 1, 9000, 130], 1, 8, 2, 64), ([4099], 8, 8, 1, 128),
    ([7001, 3000], 16, 8, 1, 64), ([2500], 3, 4, 1, 256), ([40000], 1, 1, 1, 64),
])
def test_attn_long_and_deterministic(env, lengths, rows, Hq, Hkv, D, e4m3):
    """Lengths that many workers share; the same bits every time, on the same workspace."""
    torch, ssd, dev = env
    c = _Case(env, lengths, [rows] * len(lengths), Hq, Hkv, D, 16, e4m3, seed=19)
    out, lse = c.check()
    for _ in range(3):
        o, l = c.run()
        assert torch.equal(o, out) and torch.equal(l, lse)


def test_attn_many_sequences(env):
    rng = np.random.default_rng(20)
    lengths = rng.integers(0, 40, 700)
    rows = rng.integers(1, 4, 700)
    c = _Case(env, lengths, rows, 4, 2, 32, 8, seed=20)
    c.check()


def test_attn_cache_beyond_32_bit_offsets(env):
    """Element offsets past 2^32 in both caches (9 GB of pages, two of them used)."""
    torch, ssd, dev = env
    Hkv, page, D = 2, 64, 128
    pages = (1 << 32) // (Hkv * page * D) + 40
    kc = torch.empty((pages, Hkv, page, D), dtype=torch.bfloat16, device=dev)
    vc = torch.empty_like(kc)
    g = torch.Generator(device=dev).manual_seed(21)
    table = np.array([[pages - 1, 0, pages - 7]])
    n = 150
    k = torch.randn((n, Hkv, D), generator=g, device=dev).to(torch.bfloat16)
    v = torch.randn((n, Hkv, D), generator=g, device=dev).to(torch.bfloat16)
    q = torch.randn((1, 4, D), generator=g, device=dev).to(torch.bfloat16)
    slots = [int(table[0, j // page]) * page + j % page for j in range(n)]
    qo = torch.empty((n, 4, D), dtype=torch.bfloat16, device=dev)
    ssd.rope_append(q.expand(n, 4, D).contiguous(), k, v,
                    torch.zeros(n, dtype=torch.int32, device=dev), _i32(torch, slots, dev), None,
                    qo, kc, vc)
    out = torch.empty_like(q)
    ws = ssd.workspace(ssd.attn_decode_workspace_bytes(1, 1, 4, Hkv, D))
    ssd.attn_decode(q, kc, vc, _i32(torch, table, dev), _i32(torch, [n], dev), out, ws)
    torch.cuda.synchronize()
    want, _, size, _ = attn_ref.attention(_f64(q), _f64(k), _f64(v), np.ones(n, bool),
                                          D ** -0.5, 0)
    assert np.all(np.abs(_f64(out) - want) <= U * np.abs(want) + (U + 2.0 ** -12) * size)


def test_attn_on_another_stream_and_in_a_graph(env):
    """The three operators chained on a side stream, and captured: the same bits."""
    torch, ssd, dev = env
    c = _Case(env, [500, 80], [1, 1], 8, 2, 64, 16, seed=22)
    want, _ = c.check()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got, _ = c.run(stream=side)
    assert torch.equal(got, want)
    args = (_i32(torch, c.table, dev), _i32(torch, c.lengths, dev))
    qs = _i32(torch, c.q_start, dev)
    out = torch.empty_like(want)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        ssd.attn_decode(c.q, c.kc, c.vc, *args, out, c.ws, q_start=qs, scale=c.scale)
    for _ in range(2):
        out.fill_(9.0)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)


# Many rows a kv head (verification rows, wide groups) on a bf16 cache with pages of whole
# 8-token blocks run on their own kernel, with items of 32, 64 or 128 rows.

@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("rows,Hq,Hkv,D,page", [
    (8, 3, 1, 64, 8), (9, 2, 1, 16, 16), (5, 10, 2, 128, 24), (8, 8, 1, 128, 32),
    (16, 16, 2, 96, 64), (3, 64, 2, 256, 16), (17, 7, 1, 144, 40), (40, 8, 1, 64, 128),
    (20, 20, 1, 48, 16), (4, 8, 1, 80, 16),
])
def test_attn_many_rows(env, rows, Hq, Hkv, D, page, layout):
    c = _Case(env, [rows, 63, 64, 65, 0, 700, 1, 130], [rows, rows, rows, rows, rows, rows, 1, 2],
              Hq, Hkv, D, page, layout=layout, seed=rows + D)
    c.check()


@pytest.mark.parametrize("window", [1, 7, 64, 65, 200])
def test_attn_many_rows_window(env, window):
    c = _Case(env, [9, 64, 300, 1001, 0], [9, 9, 9, 9, 9], 8, 2, 128, 16, seed=window)
    c.check(window)


@pytest.mark.parametrize("rows", [1, 8])
@pytest.mark.parametrize("e4m3", [False, True])
def test_attn_scores_that_keep_growing(env, rows, e4m3):
    """Scores in the hundreds over many stages: the running maximum moves again and again, and
    with it what has been summed."""
    c = _Case(env, [1500, 700], [rows, rows], 8, 1, 128, 16, e4m3, seed=31, spread=150.0)
    c.check()


@pytest.mark.parametrize("scale", [-0.3, 0.0])
@pytest.mark.parametrize("rows", [1, 8])
@pytest.mark.parametrize("e4m3", [False, True])
def test_attn_negative_and_zero_scale(env, scale, rows, e4m3):
    c = _Case(env, [200, 70, 0], [rows] * 3, 8, 1, 64, 16, e4m3, seed=32)
    c.scale = scale
    c.check()


@pytest.mark.parametrize("lengths,rows", [([40, 700], 6), ([64, 130], 9), ([66, 200], 20)])
def test_attn_many_rows_nan_in_unseen_places(env, lengths, rows):
    """The newest token's key and value gone wrong: only the row that sees it is affected,
    whether the token lies in the item's first stage or a later one."""
    torch, ssd, dev = env
    c = _Case(env, lengths, [rows, rows], 8, 1, 128, 16, seed=33 + rows)
    want, want_lse = c.check()
    for value in (float("nan"), float("inf")):
        for s, n in enumerate(lengths):
            page = int(c.table[s, (n - 1) // 16])
            c.kc[page, :, (n - 1) % 16] = float("nan")
            c.vc[page, :, (n - 1) % 16] = value
        got, lse = c.run()
        for s in range(2):
            a, b = s * rows, (s + 1) * rows - 1
            assert torch.equal(got[a:b], want[a:b]) and torch.equal(lse[a:b], want_lse[a:b])
            assert bool(torch.isnan(got[b].float()).all()) and bool(torch.isnan(lse[b]).all())


def test_attn_many_rows_missing_pages(env):
    """Missing pages inside, at the end and everywhere."""
    c = _Case(env, [200, 40, 500, 300], [9, 9, 9, 9], 8, 2, 128, 16, seed=34)
    c.table[0, 3:5] = -1
    c.table[1, :] = 10 ** 6
    c.table[2, 31] = -2 ** 31
    c.table[3, :12] = -1
    c.check()
    c.check(window=100)


def test_attn_one_workspace_for_all(env):
    """Calls with few and with many rows, of both cache types, in turn on one workspace: each
    finds its counters at zero."""
    torch, ssd, dev = env
    cases = [_Case(env, [9000, 100], [rows] * 2, Hq, 1, 128, 16, e4m3, seed=35)
             for rows, Hq, e4m3 in ((1, 8, False), (8, 8, False), (8, 8, True), (16, 8, False))]
    ws = max((c.ws for c in cases), key=lambda t: t.numel())
    for c in cases:
        c.ws = ws
    wants = [c.check() for c in cases]
    for _ in range(2):
        for c, (out, lse) in zip(cases, wants):
            got, l = c.run()
            assert torch.equal(got, out) and torch.equal(l, lse)
    assert ssd.dec_sync_status() == ssd.DEC_OK


# ----------------------------------------------------------------- refusals ----

def test_binding_refusals(env):
    torch, ssd, dev = env
    c = _Case(env, [40], [1], 4, 2, 64, 16, seed=23)
    tab, n = _i32(torch, c.table, dev), _i32(torch, c.lengths, dev)
    out = torch.full_like(c.q, 3.0)
    ok = dict(q=c.q, k_cache=c.kc, v_cache=c.vc, block_table=tab, seq_len=n, out=out, ws=c.ws)

    def refused(exc, **kw):
        with pytest.raises(exc):
            ssd.attn_decode(**{**ok, **kw})
    refused(TypeError, q=c.q.float())
    refused(ValueError, q=c.q.transpose(0, 1))  # 4 rows of one head: out does not fit
    refused(TypeError, k_cache=c.kc.float(), v_cache=c.vc.float())
    refused(TypeError, seq_len=n.long())
    refused(TypeError, block_table=tab[0])
    refused(ValueError, v_cache=c.vc[:1])
    refused(ValueError, out=out[:, :2])
    refused(ValueError, seq_len=n.repeat(2))
    refused(TypeError, k_scale=torch.ones(1, device=dev))
    refused(TypeError, lse=torch.ones((1, 2), device=dev))
    refused(ssd.DecError, out=c.q)
    small = torch.zeros(8, dtype=torch.uint8, device=dev)
    with pytest.raises(ssd.DecError) as e:
        ssd.attn_decode(**{**ok, "ws": small})
    assert e.value.status == ssd.DEC_ERR_WORKSPACE_TOO_SMALL
    ssd.dec_set_fault_inject(1)
    with pytest.raises(ssd.DecError) as e:
        ssd.attn_decode(**ok)
    assert e.value.status == ssd.DEC_ERR_CUDA
    torch.cuda.synchronize()
    assert bool((out == 3.0).all()), "a refused call must not write its output"
    ssd.attn_decode(**ok)


# The same on an e4m3 cache, whose elements are widened to f16 on the way.

@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("rows,Hq,Hkv,D,page", [
    (8, 3, 1, 64, 8), (9, 2, 1, 16, 16), (5, 10, 2, 128, 24), (8, 8, 1, 128, 32),
    (16, 16, 2, 96, 64), (3, 64, 2, 256, 16), (17, 7, 1, 144, 40), (40, 8, 1, 64, 128),
    (20, 20, 1, 48, 16), (4, 8, 1, 80, 16), (10, 8, 1, 256, 64),
])
def test_attn_many_rows_e4m3(env, rows, Hq, Hkv, D, page, layout):
    c = _Case(env, [rows, 63, 64, 65, 0, 700, 1, 130], [rows, rows, rows, rows, rows, rows, 1, 2],
              Hq, Hkv, D, page, True, layout=layout, seed=rows + D)
    c.check()


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("window", [1, 64, 200])
def test_attn_many_rows_e4m3_window_and_missing_pages(env, window, D):
    c = _Case(env, [9, 64, 300, 1001, 0, 500], [9] * 6, 8, 2, D, 16, True, seed=window)
    c.check(window)
    c.table[2, 3:5] = -1
    c.table[1, :] = 10 ** 6
    c.table[5, :12] = -1
    c.check(window)
    c.check()


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("lengths,rows", [([40, 700], 6), ([66, 200], 20), ([9000, 100], 8)])
def test_attn_many_rows_e4m3_nan_in_unseen_places(env, lengths, rows, D):
    torch, ssd, dev = env
    c = _Case(env, lengths, [rows, rows], 8, 1, D, 16, True, seed=36 + rows)
    want, want_lse = c.check()
    for s, n in enumerate(lengths):
        page = int(c.table[s, (n - 1) // 16])
        c.kc.view(torch.uint8)[page, :, (n - 1) % 16] = 0x7f  # NaN
        c.vc.view(torch.uint8)[page, :, (n - 1) % 16] = 0x7f
    got, lse = c.run()
    for s in range(2):
        a, b = s * rows, (s + 1) * rows - 1
        assert torch.equal(got[a:b], want[a:b]) and torch.equal(lse[a:b], want_lse[a:b])
        assert bool(torch.isnan(got[b].float()).all()) and bool(torch.isnan(lse[b]).all())
    assert ssd.dec_sync_status() == ssd.DEC_OK

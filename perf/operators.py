"""Cases of the attention operators of the decode path: the page planner of the key-value
cache (kv_plan), rotary positions with the write into the cache (rope_append) and attention
of new tokens over the paged cache (attn_decode).

``run`` computes a case in plain torch where ``own`` is false and through
``split_switched_decode_gb300`` where it is true; ``exact`` computes it in 64 bits.
"""
from __future__ import annotations

import math
import random

import torch

own = False

F8_MAX = 448.0  # largest finite e4m3 value


# ------------------------------------------------------------------- cases ----

def listed():
    """Twelve cases over the three operators, from one token to long contexts."""
    return [
        # one decode step of a full batch: 64 sequences get one new token each
        dict(name="plan_decode_64", op="plan", S=64, new=1, ragged=False, max_len=8192,
             page=16, mix=1),
        # speculative verification: up to 8 rows for each of 64 sequences
        dict(name="plan_verify_64x8", op="plan", S=64, new=8, ragged=True, max_len=32768,
             page=64, mix=2),
        # prompt chunks arriving for many requests at once (about 65 thousand tokens)
        dict(name="plan_prompts_512", op="plan", S=512, new=255, ragged=True, max_len=4096,
             page=16, mix=3),
        # batch 1 decode: the row of a 64-head projection with 8 key/value heads
        dict(name="rope_one_row", op="rope", T=1, Hq=64, Hkv=8, D=128, rot=128,
             interleaved=False, e4m3=False, page=16, max_pos=8192, factor=1.0),
        # verification rows, rotary on half of the head, interleaved pairs, 8-bit cache
        dict(name="rope_verify_512_e4m3", op="rope", T=512, Hq=32, Hkv=4, D=128, rot=64,
             interleaved=True, e4m3=True, page=64, max_pos=32768, factor=1.0),
        # a prompt chunk at long positions, frequencies scaled for a longer context
        dict(name="rope_prompt_8192", op="rope", T=8192, Hq=64, Hkv=8, D=128, rot=128,
             interleaved=False, e4m3=False, page=16, max_pos=131072, factor=4.0),
        # the smallest call: one sequence, one new token, a short odd context
        dict(name="attn_one_short", op="attn", S=1, new=1, ragged=False, min_len=777,
             max_len=777, Hq=16, Hkv=2, D=128, page=16, e4m3=False, window=0, mix=4),
        # one user, a long document
        dict(name="attn_one_128k", op="attn", S=1, new=1, ragged=False, min_len=131072,
             max_len=131072, Hq=64, Hkv=8, D=128, page=16, e4m3=False, window=0, mix=5),
        # a full decode batch with ragged contexts, one slot of the batch unused
        dict(name="attn_batch_64", op="attn", S=64, new=1, ragged=True, min_len=0,
             max_len=8192, Hq=64, Hkv=8, D=128, page=16, e4m3=False, window=0, mix=6),
        # the same with an 8-bit cache and longer contexts
        dict(name="attn_batch_64_e4m3", op="attn", S=64, new=1, ragged=True, min_len=1024,
             max_len=16384, Hq=64, Hkv=8, D=128, page=64, e4m3=True, window=0, mix=7),
        # speculative verification: 8 new rows per sequence, causal among themselves
        dict(name="attn_verify_64x8", op="attn", S=64, new=8, ragged=False, min_len=512,
             max_len=8192, Hq=64, Hkv=8, D=128, page=32, e4m3=False, window=0, mix=8),
        # odd sizes: 7 heads a group, a head of 80, pages of 48, a sliding window
        dict(name="attn_window_odd", op="attn", S=33, new=3, ragged=True, min_len=1,
             max_len=6001, Hq=28, Hkv=4, D=80, page=48, e4m3=False, window=1000, mix=9),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    """One more case of the ranges above; sizes over their logarithm, odd ones among them."""
    op = rng.choice(["plan", "rope", "attn", "attn", "attn"])
    page = rng.choice([8, 16, 16, 32, 48, 64, 128, rng.randint(1, 100)])
    if op == "plan":
        S = _log_int(rng, 1, 512)
        return dict(op="plan", S=S, new=_log_int(rng, 1, max(1, min(2048, 65536 // S))),
                    ragged=rng.random() < 0.7, max_len=_log_int(rng, 16, 32768), page=page,
                    mix=rng.randint(100, 1 << 30))
    Hkv = rng.choice([1, 2, 3, 4, 8, 8, 16])
    Hq = Hkv * rng.choice([1, 2, 4, 5, 7, 8, 8, 12, 16])
    D = rng.choice([64, 128, 128, 128, 256, 16 * rng.randint(2, 16)])
    e4m3 = rng.random() < 0.35
    if op == "rope":
        T = _log_int(rng, 1, max(1, min(8192, (1 << 26) // ((Hq + 2 * Hkv) * D))))
        rot = rng.choice([D, D, D // 2, 2 * rng.randint(1, D // 2)])
        return dict(op="rope", T=T, Hq=Hq, Hkv=Hkv, D=D, rot=rot,
                    interleaved=rng.random() < 0.5, e4m3=e4m3, page=page,
                    max_pos=_log_int(rng, 64, 131072), factor=rng.choice([1.0, 1.0, 2.0, 8.0]))
    S = _log_int(rng, 1, 96)
    new = rng.choice([1, 1, 1, 2, 4, 8, rng.randint(1, 12)])
    per_token = 2 * Hkv * D * (1 if e4m3 else 2)
    max_len = _log_int(rng, 16, max(16, min(131072, int(8e8) // (per_token * S),
                                            int(1.5e8) // (S * Hq * new))))
    return dict(op="attn", S=S, new=new, ragged=rng.random() < 0.7,
                min_len=rng.randint(0, max_len), max_len=max_len, Hq=Hq, Hkv=Hkv, D=D,
                page=page, e4m3=e4m3,
                window=rng.choice([0, 0, 0, _log_int(rng, 1, 4096)]),
                mix=rng.randint(100, 1 << 30))


def _plan_lengths(case):
    """(kv_len, new_len) of a planner case: lengths of the case, not of the seed."""
    r = random.Random(case["mix"])
    kv = [r.randint(0, case["max_len"]) for _ in range(case["S"])]
    new = [r.randint(0, case["new"]) if case["ragged"] else case["new"]
           for _ in range(case["S"])]
    return kv, new


def _attn_lengths(case):
    """(seq_len, rows) of an attention case: cached tokens with the new ones, new rows."""
    r = random.Random(case["mix"])
    S = case["S"]
    length = [r.randint(case["min_len"], case["max_len"]) for _ in range(S)]
    rows = [r.randint(1, case["new"]) if case["ragged"] else case["new"] for _ in range(S)]
    if case["min_len"] == 0 and S > 1:
        length[S // 2] = 0  # an unused slot of the batch
    return length, rows


def _pages(tokens, page):
    return (tokens + page - 1) // page


# ------------------------------------------------------------------ inputs ----

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _frequencies(rot, factor, device):
    """Inverse frequencies of base 10000 and the magnitude, scaled by parts for factor > 1:
    the slow dimensions are interpolated, the fast ones kept, a ramp between."""
    i = torch.arange(0, rot, 2, dtype=torch.float64)
    inv = 10000.0 ** (-i / rot)
    if factor == 1.0:
        return inv.to(torch.float32).to(device), 1.0

    def index(turns):
        return rot * math.log(4096 / (turns * 2 * math.pi)) / (2 * math.log(10000.0))
    lo = max(math.floor(index(32.0)), 0)
    hi = min(math.ceil(index(1.0)), rot - 1)
    ramp = ((i / 2 - lo) / max(hi - lo, 1e-3)).clamp(0, 1)
    inv = inv / factor * ramp + inv * (1 - ramp)
    return inv.to(torch.float32).to(device), 0.1 * math.log(factor) + 1.0


def _random_cache(shape, scale, g):
    """Keys or values ~ N(0, 1) in bf16, or as e4m3 with a scale for each head."""
    x = torch.randn(shape, generator=g, device="cuda", dtype=torch.bfloat16)
    if scale is None:
        return x
    x /= scale.view(1, -1, 1, 1).to(torch.bfloat16)
    return x.clamp_(-F8_MAX, F8_MAX).to(torch.float8_e4m3fn)


def _head_scales(H, g):
    return torch.rand(H, generator=g, device="cuda") * 0.02 + 0.01


def prepare(case, seed):
    """A program's state before the call: tensors on the GPU and, for the framework's
    kernels, the buffers and the workspace that a serving loop keeps."""
    g = _gen(seed)
    st = _PREPARE[case["op"]](case, g)
    st["case"] = case
    return st


def _prepare_plan(case, g):
    S, page = case["S"], case["page"]
    kv, new = _plan_lengths(case)
    total = [a + b for a, b in zip(kv, new)]
    max_pages = max(1, max(_pages(t, page) for t in total))
    held = sum(_pages(a, page) for a in kv)
    wanted = sum(_pages(t, page) for t in total) - held
    ids = torch.randperm(held + wanted + 8, generator=g, device="cuda").to(torch.int32)
    kv_t = torch.tensor(kv, dtype=torch.int32, device="cuda")
    have = (kv_t + page - 1) // page
    cols = torch.arange(max_pages, device="cuda")
    table = torch.full((S, max_pages), -1, dtype=torch.int32, device="cuda")
    table[cols[None, :] < have[:, None]] = ids[:held]
    st = dict(
        kv_len=kv_t, new_len=torch.tensor(new, dtype=torch.int32, device="cuda"),
        table=table, free=ids[held:].clone(),
        used=torch.zeros(1, dtype=torch.int32, device="cuda"), max_tokens=max(1, sum(new)))
    if own:
        T = st["max_tokens"]
        st["out"] = [torch.empty(n, dtype=torch.int32, device="cuda")
                     for n in (S, S + 1, T, T, 4)]
    return st


def _prepare_rope(case, g):
    T, Hq, Hkv, D = (case[k] for k in ("T", "Hq", "Hkv", "D"))
    page = case["page"]
    rows = torch.randn((T, (Hq + 2 * Hkv) * D), generator=g, device="cuda").to(torch.bfloat16)
    pages = _pages(T, page) + 2
    dtype = torch.float8_e4m3fn if case["e4m3"] else torch.bfloat16
    inv, magnitude = _frequencies(case["rot"], case["factor"], "cuda")
    st = dict(
        rows=rows, inv_freq=inv, magnitude=magnitude,
        q=rows[:, :Hq * D].view(T, Hq, D),
        k=rows[:, Hq * D:(Hq + Hkv) * D].view(T, Hkv, D),
        v=rows[:, (Hq + Hkv) * D:].view(T, Hkv, D),
        positions=torch.randint(0, case["max_pos"], (T,), generator=g, device="cuda",
                                dtype=torch.int32),
        slots=torch.randperm(pages * page, generator=g, device="cuda")[:T].to(torch.int32),
        k_cache=torch.zeros((pages, Hkv, page, D), device="cuda").to(dtype),
        v_cache=torch.zeros((pages, Hkv, page, D), device="cuda").to(dtype),
        k_scale=_head_scales(Hkv, g) if case["e4m3"] else None,
        v_scale=_head_scales(Hkv, g) if case["e4m3"] else None)
    if own:
        st["q_out"] = torch.empty((T, Hq, D), dtype=torch.bfloat16, device="cuda")
    return st


def _prepare_attn(case, g):
    S, Hq, Hkv, D, page = (case[k] for k in ("S", "Hq", "Hkv", "D", "page"))
    length, rows = _attn_lengths(case)
    used = [_pages(n, page) for n in length]
    max_pages = max(1, max(used))
    total = sum(used) + 4
    ids = torch.randperm(total, generator=g, device="cuda").to(torch.int32)
    len_t = torch.tensor(length, dtype=torch.int32, device="cuda")
    cols = torch.arange(max_pages, device="cuda")
    table = torch.full((S, max_pages), -1, dtype=torch.int32, device="cuda")
    table[cols[None, :] < ((len_t + page - 1) // page)[:, None]] = ids[:sum(used)]
    k_scale = _head_scales(Hkv, g) if case["e4m3"] else None
    v_scale = _head_scales(Hkv, g) if case["e4m3"] else None
    start = [0]
    for n in rows:
        start.append(start[-1] + n)
    T = start[-1]
    st = dict(
        q=torch.randn((T, Hq, D), generator=g, device="cuda").to(torch.bfloat16),
        k_cache=_random_cache((total, Hkv, page, D), k_scale, g),
        v_cache=_random_cache((total, Hkv, page, D), v_scale, g),
        k_scale=k_scale, v_scale=v_scale, table=table, seq_len=len_t,
        q_start=torch.tensor(start, dtype=torch.int32, device="cuda"),
        max_rows=max(rows), scale=1.5 / math.sqrt(D))
    if own:
        import split_switched_decode_gb300 as ssd
        st["out"] = torch.zeros((T, Hq, D), dtype=torch.bfloat16, device="cuda")
        st["lse"] = torch.zeros((T, Hq), dtype=torch.float32, device="cuda")
        st["ws"] = ssd.workspace(ssd.attn_decode_workspace_bytes(S, T, Hq, Hkv, D))
    return st


_PREPARE = {"plan": _prepare_plan, "rope": _prepare_rope, "attn": _prepare_attn}


# --------------------------------------------------------------------- run ----

def run(state):
    """One pass: the plain form, or the framework's call."""
    return (_OWN if own else _PLAIN)[state["case"]["op"]](state)


def _own_plan(st):
    import split_switched_decode_gb300 as ssd
    seq_len, q_start, positions, slots, summary = st["out"]
    ssd.kv_plan(st["kv_len"], st["new_len"], st["table"], st["free"], st["used"],
                st["case"]["page"], seq_len, q_start, positions, slots, summary)
    return dict(table=st["table"], seq_len=seq_len, q_start=q_start, positions=positions,
                slots=slots, summary=summary)


def _own_rope(st):
    import split_switched_decode_gb300 as ssd
    c = st["case"]
    ssd.rope_append(st["q"], st["k"], st["v"], st["positions"], st["slots"], st["inv_freq"],
                    st["q_out"], st["k_cache"], st["v_cache"], interleaved=c["interleaved"],
                    magnitude=st["magnitude"], k_scale=st["k_scale"], v_scale=st["v_scale"])
    return dict(q=st["q_out"], k_cache=st["k_cache"], v_cache=st["v_cache"])


def _own_attn(st):
    import split_switched_decode_gb300 as ssd
    ssd.attn_decode(st["q"], st["k_cache"], st["v_cache"], st["table"], st["seq_len"],
                    st["out"], st["ws"], q_start=st["q_start"], scale=st["scale"],
                    window=st["case"]["window"], lse=st["lse"], k_scale=st["k_scale"],
                    v_scale=st["v_scale"])
    return dict(out=st["out"], lse=st["lse"])


def _plain_plan(st):
    page, T = st["case"]["page"], st["max_tokens"]
    kv, new, table, free = st["kv_len"], st["new_len"], st["table"], st["free"]
    S, max_pages = table.shape
    q_start = torch.zeros(S + 1, dtype=torch.int32, device=kv.device)
    q_start[1:] = torch.cumsum(new, 0, dtype=torch.int32).clamp(max=T)
    seq_len = kv + q_start[1:] - q_start[:-1]
    have = (kv + page - 1) // page
    take = (seq_len + page - 1) // page - have
    first = torch.cumsum(take, 0, dtype=torch.int32) - take + st["used"]
    cols = torch.arange(max_pages, device=kv.device, dtype=torch.int32)[None, :]
    fresh = (cols >= have[:, None]) & (cols < (have + take)[:, None])
    rank = first[:, None] + cols - have[:, None]
    got = free[rank.clamp(0, free.numel() - 1).long()]
    got = torch.where(rank < free.numel(), got, torch.full_like(got, -1))
    table = torch.where(fresh, got, table)
    t = torch.arange(T, device=kv.device, dtype=torch.int32)
    s = torch.searchsorted(q_start, t, right=True) - 1
    live = t < q_start[-1]
    s = torch.where(live, s, torch.zeros_like(s))
    pos = kv[s] + t - q_start[s]
    entry = table[s, (pos // page).clamp(max=max_pages - 1).long()]
    slots = torch.where(live & (entry >= 0), entry * page + pos % page, torch.full_like(pos, -1))
    positions = torch.where(live, pos, torch.zeros_like(pos))
    wanted = take.sum()
    after = (st["used"][0] + wanted).clamp(max=free.numel())
    summary = torch.stack([q_start[-1], after, new.sum() - q_start[-1],
                           wanted - (after - st["used"][0])]).to(torch.int32)
    return dict(table=table, seq_len=seq_len, q_start=q_start, positions=positions,
                slots=slots, summary=summary)


def _plain_rotate(x, cos, sin, rot, interleaved):
    x = x.float()
    r, rest = x[..., :rot], x[..., rot:]
    if interleaved:
        a, b = r[..., 0::2], r[..., 1::2]
        r = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = r[..., :rot // 2], r[..., rot // 2:]
        r = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([r, rest], -1)


def _plain_rope(st):
    c = st["case"]
    page = c["page"]
    angle = st["positions"].float()[:, None, None] * st["inv_freq"]
    cos, sin = angle.cos() * st["magnitude"], angle.sin() * st["magnitude"]
    q = _plain_rotate(st["q"], cos, sin, c["rot"], c["interleaved"]).to(torch.bfloat16)
    k = _plain_rotate(st["k"], cos, sin, c["rot"], c["interleaved"])
    v = st["v"].float()
    if c["e4m3"]:
        k = (k / st["k_scale"][:, None]).clamp(-F8_MAX, F8_MAX)
        v = (v / st["v_scale"][:, None]).clamp(-F8_MAX, F8_MAX)
    slots = st["slots"].long()
    at, off = slots // page, slots % page
    for cache, x in ((st["k_cache"], k), (st["v_cache"], v)):
        x = x.to(cache.dtype)
        if c["e4m3"]:  # indexed as bytes
            cache, x = cache.view(torch.uint8), x.view(torch.uint8)
        cache[at, :, off] = x
    return dict(q=q, k_cache=st["k_cache"], v_cache=st["v_cache"])


def _plain_attn(st):
    c = st["case"]
    S, Hq, Hkv, D, page = (c[k] for k in ("S", "Hq", "Hkv", "D", "page"))
    G, n = Hq // Hkv, st["max_rows"]
    table, length, q_start = st["table"], st["seq_len"], st["q_start"]
    L = table.shape[1] * page
    at = table.clamp(min=0).long()

    def gathered(cache, scale):
        x = cache.view(torch.uint8) if c["e4m3"] else cache
        x = x[at].permute(0, 2, 1, 3, 4).reshape(S, Hkv, L, D)
        x = (x.view(torch.float8_e4m3fn) if c["e4m3"] else x).float()
        return x if scale is None else x * scale[:, None, None]

    keys, values = gathered(st["k_cache"], st["k_scale"]), gathered(st["v_cache"], st["v_scale"])
    rows = q_start[1:] - q_start[:-1]
    i = torch.arange(n, device=table.device)
    row = (q_start[:-1, None] + i).clamp(max=st["q"].shape[0] - 1).long()     # [S, n]
    q = st["q"].float()[row].view(S, n, Hkv, G, D).permute(0, 2, 1, 3, 4).reshape(S, Hkv, n * G, D)
    score = (q @ keys.transpose(-1, -2)).view(S, Hkv, n, G, L) * st["scale"]
    pos = (length - rows)[:, None] + i                                        # [S, n]
    j = torch.arange(L, device=table.device)
    seen = j <= pos[..., None]
    if c["window"]:
        seen &= j > pos[..., None] - c["window"]
    score = score.masked_fill(~seen[:, None, :, None], -math.inf)
    top = score.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    p = (score - top).exp()
    total = p.sum(-1, keepdim=True)
    out = (p.view(S, Hkv, n * G, L) @ values).view(S, Hkv, n, G, D)
    out = torch.where(total > 0, out / total, torch.zeros_like(out))
    lse = (total.log() + top).squeeze(-1)
    # back from padded rows to the packed ones
    t = torch.arange(st["q"].shape[0], device=table.device, dtype=torch.int32)
    s = torch.searchsorted(q_start, t, right=True) - 1
    k = (t - q_start[s]).long()
    out = out.permute(0, 2, 1, 3, 4).reshape(S, n, Hq, D)[s, k].to(torch.bfloat16)
    return dict(out=out, lse=lse.permute(0, 2, 1, 3).reshape(S, n, Hq)[s, k])


_OWN = {"plan": _own_plan, "rope": _own_rope, "attn": _own_attn}
_PLAIN = {"plan": _plain_plan, "rope": _plain_rope, "attn": _plain_attn}


# -------------------------------------------------------------------- work ----

def work(case):
    """Bytes and operations that one pass cannot do without."""
    if case["op"] == "plan":
        kv, new = _plan_lengths(case)
        fresh = sum(_pages(a + b, case["page"]) - _pages(a, case["page"])
                    for a, b in zip(kv, new))
        return {"bytes": 4 * (4 * case["S"] + 6) + 8 * sum(new) + 8 * fresh, "flops": 0}
    Hq, Hkv, D = case["Hq"], case["Hkv"], case["D"]
    each = 1 if case["e4m3"] else 2
    if case["op"] == "rope":
        T = case["T"]
        return {"bytes": T * ((Hq + 2 * Hkv) * D * 2 + Hq * D * 2 + 2 * Hkv * D * each + 8)
                + 2 * case["rot"],
                "flops": T * (Hq + Hkv) * case["rot"] * 3}
    length, rows = _attn_lengths(case)
    read = pairs = 0
    for n, r in zip(length, rows):
        first = max(0, n - r - case["window"] + 1) if case["window"] else 0
        read += n - first
        for i in range(r):
            pos = n - r + i
            pairs += max(0, min(pos + 1, case["window"] or pos + 1))
    T = sum(rows)
    return {"bytes": read * 2 * Hkv * D * each + T * Hq * (4 * D + 4)
            + 4 * sum(_pages(n, case["page"]) for n in length) + 8 * case["S"],
            "flops": 4 * D * Hq * pairs}


# ------------------------------------------------------------------- exact ----

def exact(case, seed):
    """What run() returns, from the definition in 64 bits; None where outputs are whole
    numbers."""
    if case["op"] == "plan":
        return None
    st = prepare(case, seed)
    return _exact_rope(case, st) if case["op"] == "rope" else _exact_attn(case, st)


def _exact_rope(case, st):
    T, D, rot, page = case["T"], case["D"], case["rot"], case["page"]
    half = rot // 2
    turn = torch.outer(st["positions"].double(), st["inv_freq"].double())
    wave = torch.polar(torch.full_like(turn, st["magnitude"]), turn)[:, None, :]

    def rotated(x):
        y = x.double()
        if case["interleaved"]:
            z = torch.view_as_complex(y[..., :rot].reshape(*y.shape[:-1], half, 2)) * wave
            y[..., :rot] = torch.view_as_real(z).reshape(*y.shape[:-1], rot)
        else:
            z = torch.complex(y[..., :half].contiguous(), y[..., half:rot].contiguous()) * wave
            y[..., :half], y[..., half:rot] = z.real, z.imag
        return y

    caches = {}
    for name, x, scale in (("k_cache", rotated(st["k"]), st["k_scale"]),
                           ("v_cache", st["v"].double(), st["v_scale"])):
        if scale is not None:
            x = (x / scale.double().view(1, -1, 1)).clamp(-F8_MAX, F8_MAX)
        pages, Hkv = st[name].shape[:2]
        flat = torch.zeros((pages * page, Hkv, D), dtype=torch.float64, device="cuda")
        flat[st["slots"].long()] = x
        caches[name] = flat.view(pages, page, Hkv, D).transpose(1, 2).contiguous()
    return dict(q=rotated(st["q"]), **caches)


def _exact_attn(case, st):
    Hq, Hkv, D, page = (case[k] for k in ("Hq", "Hkv", "D", "page"))
    G = Hq // Hkv
    length, rows = _attn_lengths(case)
    table = st["table"].cpu()
    out = torch.zeros((sum(rows), Hq, D), dtype=torch.float64, device="cuda")
    lse = torch.full((sum(rows), Hq), -math.inf, dtype=torch.float64, device="cuda")
    t = 0
    for s, (n, r) in enumerate(zip(length, rows)):
        ids = table[s, :_pages(n, page)].long().cuda()
        for h in range(Hkv if n else 0):
            k = st["k_cache"][:, h][ids] if not case["e4m3"] else \
                st["k_cache"].view(torch.uint8)[:, h][ids].view(torch.float8_e4m3fn)
            v = st["v_cache"][:, h][ids] if not case["e4m3"] else \
                st["v_cache"].view(torch.uint8)[:, h][ids].view(torch.float8_e4m3fn)
            k, v = k.double().view(-1, D)[:n], v.double().view(-1, D)[:n]
            if case["e4m3"]:
                k, v = k * st["k_scale"][h].double(), v * st["v_scale"][h].double()
            for i in range(r):
                end = n - r + i + 1
                begin = max(0, end - case["window"]) if case["window"] else 0
                if end <= 0:
                    continue
                heads = slice(h * G, (h + 1) * G)
                z = st["scale"] * (st["q"][t + i, heads].double() @ k[begin:end].T)
                lse[t + i, heads] = z.logsumexp(-1)
                out[t + i, heads] = z.softmax(-1) @ v[begin:end]
        t += r
    return dict(out=out, lse=lse)

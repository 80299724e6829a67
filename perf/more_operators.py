"""Cases of the latent attention operators of the decode path, whose keys and values come from
one shared latent vector a token: norm, rotary positions and the write into the latent cache
(latent_append), the per-head products into and out of the latent space (latent_project),
attention of new tokens over the paged latent cache (latent_decode) and of whole prompts over
expanded keys and values (latent_prompt).

``run`` computes a case in plain torch where ``own`` is false and through
``split_switched_decode_gb300`` where it is true; ``exact`` computes it in 64 bits.
"""
from __future__ import annotations

import math
import random

import torch

own = False

F8_MAX = 448.0  # largest finite e4m3 value
EPS = 1e-6


# ------------------------------------------------------------------- cases ----

def listed():
    """Twelve cases over the four operators, from one token to long contexts."""
    return [
        # batch 1 decode: one row of the projections before a 64-head layer
        dict(name="append_one_row", op="append", T=1, H=64, R=512, P=64, interleaved=True,
             e4m3=False, rows=False, page=16, max_pos=8192, factor=1.0),
        # verification rows of many sequences into an 8-bit cache
        dict(name="append_verify_512_e4m3", op="append", T=512, H=16, R=512, P=64,
             interleaved=False, e4m3=True, rows=False, page=64, max_pos=32768, factor=1.0),
        # a prompt chunk, frequencies scaled for a longer context, rows kept for the expansion
        dict(name="append_prompt_8192", op="append", T=8192, H=64, R=512, P=64,
             interleaved=True, e4m3=False, rows=True, page=16, max_pos=131072, factor=4.0),
        # batch 1 decode: 64 heads of 128 elements into the latent space
        dict(name="project_in_one_row", op="project", T=1, H=64, K=128, N=512),
        # a decode batch: latent outputs back to heads of 128 elements
        dict(name="project_out_64", op="project", T=64, H=64, K=512, N=128),
        # a prompt chunk into the latent space
        dict(name="project_in_4096", op="project", T=4096, H=64, K=128, N=512),
        # the smallest attention: one sequence, one new token, 16 heads, a short odd context
        dict(name="decode_one_short", op="decode", S=1, new=1, ragged=False, min_len=777,
             max_len=777, H=16, R=512, P=64, page=16, e4m3=False, window=0, mix=11),
        # one user, a long document
        dict(name="decode_one_128k", op="decode", S=1, new=1, ragged=False, min_len=131072,
             max_len=131072, H=64, R=512, P=64, page=64, e4m3=False, window=0, mix=12),
        # a full decode batch with ragged contexts, one slot of the batch unused
        dict(name="decode_batch_64", op="decode", S=64, new=1, ragged=True, min_len=0,
             max_len=16384, H=64, R=512, P=64, page=16, e4m3=False, window=0, mix=13),
        # speculative verification: 8 new rows a sequence, 16 heads, an 8-bit cache
        dict(name="decode_verify_32x8_e4m3", op="decode", S=32, new=8, ragged=False,
             min_len=1024, max_len=16384, H=16, R=512, P=64, page=32, e4m3=True, window=0,
             mix=14),
        # a short prompt of odd length, 16 heads
        dict(name="prompt_one_777", op="prompt", S=1, max_new=777, ragged=False, max_old=0,
             H=16, N=128, P=64, V=128, mix=15),
        # prompts of many lengths arriving together, some behind a cached prefix
        dict(name="prompt_ragged_6", op="prompt", S=6, max_new=4096, ragged=True,
             max_old=2048, H=32, N=128, P=64, V=128, mix=16),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    """One more case of the ranges above; sizes over their logarithm, odd ones among them."""
    op = rng.choice(["append", "project", "project", "decode", "decode", "decode", "prompt",
                     "prompt"])
    H = rng.choice([1, 8, 16, 16, 32, 64, 64, 128, rng.randint(1, 128)])
    R = rng.choice([512, 512, 512, 256, 64 * rng.randint(1, 8)])
    P = rng.choice([64, 64, 64, 0]) if R > 64 else 64
    page = rng.choice([8, 16, 16, 32, 48, 64, 128, rng.randint(1, 100)])
    mix = rng.randint(100, 1 << 30)
    if op == "append":
        return dict(op="append", T=_log_int(rng, 1, max(1, min(8192, (1 << 25) // (H * 64)))),
                    H=H, R=R, P=64, interleaved=rng.random() < 0.5,
                    e4m3=rng.random() < 0.35, rows=rng.random() < 0.5, page=page,
                    max_pos=_log_int(rng, 64, 131072), factor=rng.choice([1.0, 1.0, 2.0, 8.0]))
    if op == "project":
        small = rng.choice([64, 128, 128, 192, 16 * rng.randint(2, 16)])
        K, N = rng.choice([(small, R), (R, small)])
        return dict(op="project", T=_log_int(rng, 1, max(1, min(4096, (1 << 27) // (H * (K + N))))),
                    H=H, K=K, N=N)
    if op == "prompt":
        S = _log_int(rng, 1, 12)
        most = max(16, min(4096, int(math.sqrt(2e8 / (S * H)))))
        return dict(op="prompt", S=S, max_new=_log_int(rng, 16, most),
                    ragged=rng.random() < 0.7, max_old=rng.choice([0, 0, most // 2]), H=H,
                    N=rng.choice([128, 128, 64]), P=64, V=rng.choice([128, 128, 64]), mix=mix)
    S = _log_int(rng, 1, 96)
    new = rng.choice([1, 1, 1, 2, 4, 8, rng.randint(1, 12)])
    e4m3 = rng.random() < 0.35
    max_len = _log_int(rng, 16, max(16, min(131072, int(5e8) // (2 * (R + P) * S),
                                            int(6e7) // (S * H * new))))
    return dict(op="decode", S=S, new=new, ragged=rng.random() < 0.7,
                min_len=rng.randint(0, max_len), max_len=max_len, H=H, R=R, P=P, page=page,
                e4m3=e4m3, window=rng.choice([0, 0, 0, 0, _log_int(rng, 1, 4096)]), mix=mix)


def _decode_lengths(case):
    """(seq_len, rows) of a decode case: cached tokens with the new ones, new rows."""
    r = random.Random(case["mix"])
    S = case["S"]
    length = [r.randint(case["min_len"], case["max_len"]) for _ in range(S)]
    rows = [r.randint(1, case["new"]) if case["ragged"] else case["new"] for _ in range(S)]
    if case["min_len"] == 0 and S > 1:
        length[S // 2] = 0  # an unused slot of the batch
    return length, rows


def _prompt_lengths(case):
    """(rows, keys) of a prompt case: new tokens, and with them those cached before."""
    r = random.Random(case["mix"])
    rows = [r.randint(1, case["max_new"]) if case["ragged"] else case["max_new"]
            for _ in range(case["S"])]
    old = [r.choice([0, r.randint(0, case["max_old"])]) for _ in rows]
    return rows, [a + b for a, b in zip(rows, old)]


def _pages(tokens, page):
    return (tokens + page - 1) // page


def _starts(counts):
    at = [0]
    for n in counts:
        at.append(at[-1] + n)
    return at


# ------------------------------------------------------------------ inputs ----

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _normal(shape, g, scale=1.0):
    x = torch.randn(shape, generator=g, device="cuda", dtype=torch.bfloat16)
    return x if scale == 1.0 else x.mul_(scale)


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


def prepare(case, seed):
    """A program's state before the call: tensors on the GPU and, for the framework's
    kernels, the buffers and the workspace that a serving loop keeps."""
    g = _gen(seed)
    st = _PREPARE[case["op"]](case, g)
    st["case"] = case
    return st


def _prepare_append(case, g):
    T, H, R, P, page = (case[k] for k in ("T", "H", "R", "P", "page"))
    down = _normal((T, R + P), g)                       # the row of the down projection
    up = _normal((T, H, 128 + P), g)                    # the row of the query projection
    pages = _pages(T, page) + 2
    dtype = torch.float8_e4m3fn if case["e4m3"] else torch.bfloat16
    inv, magnitude = _frequencies(P, case["factor"], "cuda")
    st = dict(
        c=down[:, :R], k_rope=down[:, R:], q_rope=up[..., 128:], inv_freq=inv,
        magnitude=magnitude,
        weight=(torch.rand(R, generator=g, device="cuda") + 0.5).to(torch.bfloat16),
        positions=torch.randint(0, case["max_pos"], (T,), generator=g, device="cuda",
                                dtype=torch.int32),
        slots=torch.randperm(pages * page, generator=g, device="cuda")[:T].to(torch.int32),
        cache=torch.zeros((pages, page, R + P), device="cuda").to(dtype),
        scale=torch.rand(1, generator=g, device="cuda") * 0.02 + 0.01 if case["e4m3"] else None)
    if own:
        q = torch.empty((T, H, R + P), dtype=torch.bfloat16, device="cuda")
        st["q_out"] = q[..., R:]                        # beside the absorbed part
        st["rows"] = torch.empty((T, R + P), dtype=torch.bfloat16, device="cuda") \
            if case["rows"] else None
    return st


def _prepare_project(case, g):
    T, H, K, N = (case[k] for k in ("T", "H", "K", "N"))
    st = dict(x=_normal((T, H, K), g), w=_normal((H, N, K), g, K ** -0.5))
    if own:
        st["y"] = torch.empty((T, H, N), dtype=torch.bfloat16, device="cuda")
    return st


def _prepare_decode(case, g):
    S, H, R, P, page = (case[k] for k in ("S", "H", "R", "P", "page"))
    length, rows = _decode_lengths(case)
    used = [_pages(n, page) for n in length]
    max_pages = max(1, max(used))
    total = sum(used) + 4
    ids = torch.randperm(total, generator=g, device="cuda").to(torch.int32)
    len_t = torch.tensor(length, dtype=torch.int32, device="cuda")
    cols = torch.arange(max_pages, device="cuda")
    table = torch.full((S, max_pages), -1, dtype=torch.int32, device="cuda")
    table[cols[None, :] < ((len_t + page - 1) // page)[:, None]] = ids[:sum(used)]
    cache = _normal((total, page, R + P), g)
    scale = None
    if case["e4m3"]:
        scale = torch.rand(1, generator=g, device="cuda") * 0.02 + 0.01
        cache = (cache / scale.to(torch.bfloat16)).clamp_(-F8_MAX, F8_MAX) \
            .to(torch.float8_e4m3fn)
    T = sum(rows)
    st = dict(
        q=_normal((T, H, R + P), g), cache=cache, cache_scale=scale, table=table,
        seq_len=len_t, max_rows=max(rows), scale=1.5 / math.sqrt(R + P),
        q_start=torch.tensor(_starts(rows), dtype=torch.int32, device="cuda"))
    if own:
        import split_switched_decode_gb300 as ssd
        st["out"] = torch.zeros((T, H, R), dtype=torch.bfloat16, device="cuda")
        st["lse"] = torch.zeros((T, H), dtype=torch.float32, device="cuda")
        st["ws"] = ssd.workspace(ssd.latent_decode_workspace_bytes(S, T, H, R, P))
    return st


def _prepare_prompt(case, g):
    H, N, P, V = (case[k] for k in ("H", "N", "P", "V"))
    rows, keys = _prompt_lengths(case)
    T, Tk = sum(rows), sum(keys)
    kv = _normal((Tk, H, N + V), g)                     # the row of the up projection
    st = dict(
        q=_normal((T, H, N + P), g), k_nope=kv[..., :N], v=kv[..., N:],
        k_rope=_normal((Tk, P), g), scale=1.5 / math.sqrt(N + P),
        q_start=torch.tensor(_starts(rows), dtype=torch.int32, device="cuda"),
        k_start=torch.tensor(_starts(keys), dtype=torch.int32, device="cuda"))
    if own:
        st["out"] = torch.zeros((T, H, V), dtype=torch.bfloat16, device="cuda")
        st["lse"] = torch.zeros((T, H), dtype=torch.float32, device="cuda")
    return st


_PREPARE = {"append": _prepare_append, "project": _prepare_project,
            "decode": _prepare_decode, "prompt": _prepare_prompt}


# --------------------------------------------------------------------- run ----

def run(state):
    """One pass: the plain form, or the framework's call."""
    return (_OWN if own else _PLAIN)[state["case"]["op"]](state)


def _own_append(st):
    import split_switched_decode_gb300 as ssd
    ssd.latent_append(st["c"], st["k_rope"], st["positions"], st["slots"], st["inv_freq"],
                      st["cache"], weight=st["weight"], eps=EPS, q_rope=st["q_rope"],
                      q_out=st["q_out"], rows=st["rows"],
                      interleaved=st["case"]["interleaved"], magnitude=st["magnitude"],
                      cache_scale=st["scale"])
    out = dict(q=st["q_out"], cache=st["cache"])
    return out if st["rows"] is None else dict(out, rows=st["rows"])


def _own_project(st):
    import split_switched_decode_gb300 as ssd
    ssd.latent_project(st["x"], st["w"], st["y"])
    return st["y"]


def _own_decode(st):
    import split_switched_decode_gb300 as ssd
    ssd.latent_decode(st["q"], st["cache"], st["table"], st["seq_len"], st["out"], st["ws"],
                      st["scale"], q_start=st["q_start"], window=st["case"]["window"],
                      lse=st["lse"], cache_scale=st["cache_scale"])
    return dict(out=st["out"], lse=st["lse"])


def _own_prompt(st):
    import split_switched_decode_gb300 as ssd
    ssd.latent_prompt(st["q"], st["k_nope"], st["k_rope"], st["v"], st["q_start"], st["out"],
                      st["scale"], k_start=st["k_start"], lse=st["lse"])
    return dict(out=st["out"], lse=st["lse"])


def _plain_rotate(x, cos, sin, interleaved):
    x = x.float()
    half = x.shape[-1] // 2
    if interleaved:
        a, b = x[..., 0::2], x[..., 1::2]
        return torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    a, b = x[..., :half], x[..., half:]
    return torch.cat([a * cos - b * sin, b * cos + a * sin], -1)


def _plain_append(st):
    c = st["case"]
    angle = st["positions"].double()[:, None] * st["inv_freq"].double()
    cos = (angle.cos() * st["magnitude"]).float()
    sin = (angle.sin() * st["magnitude"]).float()
    q = _plain_rotate(st["q_rope"], cos[:, None], sin[:, None], c["interleaved"])
    x = st["c"].float()
    y = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * st["weight"].float()
    row = torch.cat([y, _plain_rotate(st["k_rope"], cos, sin, c["interleaved"])], -1)
    slots = st["slots"].long()
    at, off = slots // c["page"], slots % c["page"]
    if c["e4m3"]:  # indexed as bytes
        held = (row / st["scale"]).clamp(-F8_MAX, F8_MAX).to(torch.float8_e4m3fn)
        st["cache"].view(torch.uint8)[at, off] = held.view(torch.uint8)
    else:
        st["cache"][at, off] = row.to(torch.bfloat16)
    out = dict(q=q.to(torch.bfloat16), cache=st["cache"])
    return dict(out, rows=row.to(torch.bfloat16)) if c["rows"] else out


def _plain_project(st):
    x, w = st["x"].float().transpose(0, 1), st["w"].float()
    return (x @ w.transpose(1, 2)).transpose(0, 1).to(torch.bfloat16).contiguous()


def _plain_decode(st):
    c = st["case"]
    S, H, R, P, page = (c[k] for k in ("S", "H", "R", "P", "page"))
    n, W = st["max_rows"], R + P
    table, length, q_start = st["table"], st["seq_len"], st["q_start"]
    L = table.shape[1] * page
    x = st["cache"].view(torch.uint8) if c["e4m3"] else st["cache"]
    x = x[table.clamp(min=0).long()].reshape(S, L, W)
    keys = x.view(torch.float8_e4m3fn).float() * st["cache_scale"] if c["e4m3"] else x.float()
    rows = q_start[1:] - q_start[:-1]
    i = torch.arange(n, device=table.device)
    row = (q_start[:-1, None] + i).clamp(max=st["q"].shape[0] - 1).long()     # [S, n]
    q = st["q"].float()[row].view(S, n * H, W)
    score = (q @ keys.transpose(-1, -2)).view(S, n, H, L) * st["scale"]
    pos = (length - rows)[:, None] + i                                        # [S, n]
    j = torch.arange(L, device=table.device)
    seen = j <= pos[..., None]
    if c["window"]:
        seen &= j > pos[..., None] - c["window"]
    score = score.masked_fill(~seen[:, :, None], -math.inf)
    top = score.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    p = (score - top).exp()
    total = p.sum(-1, keepdim=True)
    out = (p.view(S, n * H, L) @ keys[..., :R]).view(S, n, H, R)
    out = torch.where(total > 0, out / total, torch.zeros_like(out))
    lse = (total.log() + top).squeeze(-1)
    # back from padded rows to the packed ones
    t = torch.arange(st["q"].shape[0], device=table.device, dtype=torch.int32)
    s = torch.searchsorted(q_start, t, right=True) - 1
    k = (t - q_start[s]).long()
    return dict(out=out[s, k].to(torch.bfloat16), lse=lse[s, k])


def _plain_prompt(st):
    c = st["case"]
    rows, keys = _prompt_lengths(c)
    N, qs, ks = c["N"], _starts(rows), _starts(keys)
    outs, lses = [], []
    for s in range(c["S"]):
        q = st["q"][qs[s]:qs[s + 1]].float().transpose(0, 1)                  # [H, n, N+P]
        k = st["k_nope"][ks[s]:ks[s + 1]].float().permute(1, 2, 0)            # [H, N, L]
        r = st["k_rope"][ks[s]:ks[s + 1]].float().T                           # [P, L]
        score = (q[..., :N] @ k + q[..., N:] @ r) * st["scale"]
        pos = torch.arange(rows[s], device=q.device) + keys[s] - rows[s]
        hidden = torch.arange(keys[s], device=q.device) > pos[:, None]
        score = score.masked_fill(hidden, -math.inf)
        top = score.amax(-1, keepdim=True)
        p = (score - top).exp()
        total = p.sum(-1, keepdim=True)
        v = st["v"][ks[s]:ks[s + 1]].float().transpose(0, 1)
        outs.append(((p @ v) / total).transpose(0, 1).to(torch.bfloat16))
        lses.append((total.log() + top).squeeze(-1).T)
    return dict(out=torch.cat(outs), lse=torch.cat(lses))


_OWN = {"append": _own_append, "project": _own_project, "decode": _own_decode,
        "prompt": _own_prompt}
_PLAIN = {"append": _plain_append, "project": _plain_project, "decode": _plain_decode,
          "prompt": _plain_prompt}


# -------------------------------------------------------------------- work ----

def work(case):
    """Bytes and operations that one pass cannot do without."""
    H = case["H"]
    if case["op"] == "append":
        T, R, P = case["T"], case["R"], case["P"]
        out = (1 if case["e4m3"] else 2) + (2 if case["rows"] else 0)
        return {"bytes": T * ((R + P) * (2 + out) + 4 * H * P + 8) + 2 * R + 2 * P,
                "flops": T * (4 * R + 3 * (H + 1) * P)}
    if case["op"] == "project":
        T, K, N = case["T"], case["K"], case["N"]
        return {"bytes": 2 * H * (T * (K + N) + K * N), "flops": 2 * T * H * K * N}
    if case["op"] == "prompt":
        N, P, V = case["N"], case["P"], case["V"]
        rows, keys = _prompt_lengths(case)
        pairs = sum(n * (2 * L - n + 1) // 2 for n, L in zip(rows, keys))
        return {"bytes": 2 * sum(rows) * H * (N + P + V + 2) + 2 * sum(keys) * (H * (N + V) + P)
                + 8 * case["S"], "flops": 2 * (N + P + V) * H * pairs}
    R, W = case["R"], case["R"] + case["P"]
    length, rows = _decode_lengths(case)
    read = pairs = 0
    for n, r in zip(length, rows):
        first = max(0, n - r - case["window"] + 1) if case["window"] else 0
        read += n - first
        for i in range(r):
            pos = n - r + i
            pairs += max(0, min(pos + 1, case["window"] or pos + 1))
    return {"bytes": read * W * (1 if case["e4m3"] else 2) + sum(rows) * H * (2 * W + 2 * R + 4)
            + 4 * sum(_pages(n, case["page"]) for n in length) + 8 * case["S"],
            "flops": 2 * (W + R) * H * pairs}


# ------------------------------------------------------------------- exact ----

def exact(case, seed):
    """What run() returns, from the definition in 64 bits."""
    return _EXACT[case["op"]](case, prepare(case, seed))


def _exact_append(case, st):
    R, P, page = case["R"], case["P"], case["page"]
    turn = torch.outer(st["positions"].double(), st["inv_freq"].double())
    wave = torch.polar(torch.full_like(turn, st["magnitude"]), turn)

    def rotated(x, w):
        y = x.double()
        if case["interleaved"]:
            z = torch.view_as_complex(y.reshape(*y.shape[:-1], P // 2, 2).contiguous()) * w
            return torch.view_as_real(z).flatten(-2)
        z = torch.complex(y[..., :P // 2].contiguous(), y[..., P // 2:].contiguous()) * w
        return torch.cat([z.real, z.imag], -1)

    c = st["c"].double()
    mean = torch.linalg.vector_norm(c, dim=-1, keepdim=True).square() / R
    row = torch.empty((case["T"], R + P), dtype=torch.float64, device="cuda")
    row[:, :R] = c / (mean + EPS).sqrt() * st["weight"].double()
    row[:, R:] = rotated(st["k_rope"], wave)
    flat = torch.zeros((st["cache"].shape[0] * page, R + P), dtype=torch.float64, device="cuda")
    held = row if st["scale"] is None else \
        (row / st["scale"].double()).clamp(-F8_MAX, F8_MAX)
    flat[st["slots"].long()] = held
    out = dict(q=rotated(st["q_rope"], wave[:, None]), cache=flat.view(-1, page, R + P))
    return dict(out, rows=row) if case["rows"] else out


def _exact_project(case, st):
    y = torch.empty((case["T"], case["H"], case["N"]), dtype=torch.float64, device="cuda")
    for h in range(case["H"]):
        y[:, h] = st["x"][:, h].double() @ st["w"][h].double().T
    return y


def _exact_decode(case, st):
    H, R, W, page = case["H"], case["R"], case["R"] + case["P"], case["page"]
    length, rows = _decode_lengths(case)
    table = st["table"].cpu()
    out = torch.zeros((sum(rows), H, R), dtype=torch.float64, device="cuda")
    lse = torch.full((sum(rows), H), -math.inf, dtype=torch.float64, device="cuda")
    t = 0
    for s, (n, r) in enumerate(zip(length, rows)):
        if n:
            ids = table[s, :_pages(n, page)].long().cuda()
            if case["e4m3"]:
                c = st["cache"].view(torch.uint8)[ids].view(torch.float8_e4m3fn).double()
                c = c * st["cache_scale"].double()
            else:
                c = st["cache"][ids].double()
            c = c.view(-1, W)[:n]
        for i in range(r):
            end = n - r + i + 1
            begin = max(0, end - case["window"]) if case["window"] else 0
            if end > 0:
                z = st["scale"] * (st["q"][t + i].double() @ c[begin:end].T)
                lse[t + i] = z.logsumexp(-1)
                out[t + i] = z.softmax(-1) @ c[begin:end, :R]
        t += r
    return dict(out=out, lse=lse)


def _exact_prompt(case, st):
    rows, keys = _prompt_lengths(case)
    H, T = case["H"], sum(rows)
    out = torch.zeros((T, H, case["V"]), dtype=torch.float64, device="cuda")
    lse = torch.zeros((T, H), dtype=torch.float64, device="cuda")
    t = j = 0
    for n, L in zip(rows, keys):
        later = torch.ones((n, L), dtype=torch.bool, device="cuda").triu(L - n + 1)
        for h in range(H):
            k = torch.cat([st["k_nope"][j:j + L, h], st["k_rope"][j:j + L]], -1).double()
            z = st["scale"] * (st["q"][t:t + n, h].double() @ k.T)
            z[later] = -math.inf
            lse[t:t + n, h] = z.logsumexp(-1)
            out[t:t + n, h] = z.softmax(-1) @ st["v"][j:j + L, h].double()
        t, j = t + n, j + L
    return dict(out=out, lse=lse)


_EXACT = {"append": _exact_append, "project": _exact_project, "decode": _exact_decode,
          "prompt": _exact_prompt}

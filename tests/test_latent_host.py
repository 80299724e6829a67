"""Latent attention without a GPU: refusals of the C entry points and of the binding, workspace
sizes, what the kernels do about waits that run out (read from their sources), and the plain
forms of the GPU tests by hand."""
import ctypes
import math
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "split_switched_decode_gb300", "csrc")


@pytest.fixture(scope="module")
def ssd():
    import split_switched_decode_gb300 as m
    m.build()
    return m


A = ctypes.c_void_p(0x10000)  # never dereferenced: every call below fails its checks
B = ctypes.c_void_p(0x20000)
U = ctypes.c_void_p(0x10002)  # misaligned for everything
U4 = ctypes.c_void_p(0x10004)  # misaligned for rows


def _check(ssd, fn, names, good, cases):
    for changes, status in cases:
        args = dict(good, **changes)
        assert fn(*[args[n] for n in names]) == getattr(ssd, status), changes


INVALID, SHAPE, ALIGN = "DEC_ERR_INVALID_ARG", "DEC_ERR_UNSUPPORTED_SHAPE", "DEC_ERR_MISALIGNED"
BIG = 1 << 39


def test_append_refusals(ssd):
    names = ("c cs weight eps kr ks qr qs qh pos slots inv mag T H R P rot inter qo os oh rows rs "
             "cache kind scale pages page pstride tstride s").split()
    good = dict(c=A, cs=576, weight=A, eps=1e-6, kr=A, ks=576, qr=A, qs=8 * 64, qh=64, pos=A, slots=A,
                inv=A, mag=1.0, T=4, H=8, R=512, P=64, rot=64, inter=0, qo=B, os=8 * 64, oh=64, rows=A,
                rs=576, cache=A, kind=0, scale=None, pages=3, page=16, pstride=16 * 576, tstride=576,
                s=None)
    _check(ssd, ssd.lib().latent_append, names, good, [
        (dict(c=None), INVALID), (dict(pos=None), INVALID), (dict(slots=None), INVALID),
        (dict(cache=None), INVALID), (dict(T=0), INVALID), (dict(H=-1), INVALID),
        (dict(inter=2), INVALID), (dict(rot=66), INVALID), (dict(rot=-2), INVALID),
        (dict(rot=65), INVALID), (dict(inv=None), INVALID), (dict(kr=None), INVALID),
        (dict(qr=None), INVALID), (dict(qo=None), INVALID), (dict(eps=-1.0), INVALID),
        (dict(eps=float("nan")), INVALID), (dict(kind=2), INVALID), (dict(pages=0), INVALID),
        (dict(page=0), INVALID), (dict(R=0), INVALID), (dict(P=-64), INVALID),
        (dict(pstride=-8), INVALID), (dict(cs=-576), INVALID), (dict(cs=504), INVALID),
        (dict(ks=56), INVALID), (dict(qh=56), INVALID), (dict(os=256, oh=64), INVALID),
        (dict(rs=512), INVALID),
        (dict(qo=A, os=1024), INVALID), (dict(tstride=512), INVALID),
        (dict(R=500), SHAPE), (dict(R=576, P=0), SHAPE), (dict(P=32), SHAPE), (dict(P=128), SHAPE),
        (dict(rot=24), SHAPE), (dict(T=(1 << 20) + 1), SHAPE), (dict(H=1025), SHAPE),
        (dict(pages=1 << 20, page=1 << 12), SHAPE), (dict(cs=BIG), SHAPE), (dict(tstride=BIG), SHAPE),
        (dict(c=U), ALIGN), (dict(kr=U), ALIGN), (dict(qr=U), ALIGN), (dict(qo=U), ALIGN),
        (dict(rows=U), ALIGN), (dict(weight=U), ALIGN), (dict(pos=U), ALIGN), (dict(slots=U), ALIGN),
        (dict(inv=U), ALIGN), (dict(cache=U), ALIGN), (dict(cs=580), ALIGN), (dict(qs=516), ALIGN),
        (dict(tstride=580), ALIGN), (dict(kind=1, tstride=584, pstride=16 * 584), ALIGN),
    ])


def test_project_refusals(ssd):
    names = "x xs xh w y ys yh T H K N s".split()
    good = dict(x=A, xs=8 * 128, xh=128, w=A, y=B, ys=8 * 512, yh=512, T=4, H=8, K=128, N=512, s=None)
    _check(ssd, ssd.lib().latent_project, names, good, [
        (dict(x=None), INVALID), (dict(w=None), INVALID), (dict(y=None), INVALID), (dict(T=0), INVALID),
        (dict(H=0), INVALID), (dict(K=0), INVALID), (dict(N=0), INVALID), (dict(xh=120), INVALID),
        (dict(xs=-8), INVALID), (dict(xh=0), INVALID), (dict(ys=1024, yh=512), INVALID),
        (dict(y=A), INVALID), (dict(x=B), INVALID),
        (dict(K=132), SHAPE), (dict(N=516), SHAPE), (dict(K=4104), SHAPE), (dict(N=4104), SHAPE),
        (dict(T=(1 << 20) + 1), SHAPE), (dict(H=1025), SHAPE), (dict(xs=BIG), SHAPE),
        (dict(x=U), ALIGN), (dict(w=U4), ALIGN), (dict(y=U), ALIGN), (dict(xs=1028), ALIGN),
        (dict(yh=516), ALIGN),
    ])


def test_decode_refusals(ssd):
    names = ("q qs cache kind scale pages page pstride tstride table width lens starts S T H R P scl window "
             "out os lse ws nws s").split()
    good = dict(q=A, qs=8 * 576, cache=A, kind=0, scale=None, pages=3, page=16, pstride=16 * 576,
                tstride=576, table=A, width=4, lens=A, starts=A, S=2, T=4, H=8, R=512, P=64, scl=0.1,
                window=0, out=B, os=8 * 512, lse=None, ws=A, nws=0, s=None)
    _check(ssd, ssd.lib().latent_decode, names, good, [
        (dict(q=None), INVALID), (dict(cache=None), INVALID), (dict(table=None), INVALID),
        (dict(lens=None), INVALID), (dict(out=None), INVALID), (dict(ws=None), INVALID),
        (dict(S=0), INVALID), (dict(T=0), INVALID), (dict(H=0), INVALID), (dict(width=0), INVALID),
        (dict(window=-1), INVALID), (dict(starts=None), INVALID), (dict(kind=3), INVALID),
        (dict(os=4088), INVALID), (dict(qs=-8), INVALID), (dict(out=A), INVALID),
        (dict(R=520), SHAPE), (dict(R=576, P=64), SHAPE), (dict(P=32), SHAPE), (dict(S=8193), SHAPE),
        (dict(T=65537), SHAPE), (dict(H=1025), SHAPE), (dict(qs=BIG), SHAPE),
        (dict(q=U), ALIGN), (dict(out=U), ALIGN), (dict(table=U), ALIGN), (dict(lens=U), ALIGN),
        (dict(starts=U), ALIGN), (dict(lse=U), ALIGN), (dict(ws=U), ALIGN), (dict(qs=4612), ALIGN),
        (dict(tstride=580), ALIGN),
    ])
    for shape in ((0, 1, 1, 512, 64), (1, 0, 1, 512, 64), (1, 1, 0, 512, 64), (1, 1, 1, 500, 64),
                  (1, 1, 1, 512, 65), (1, 1, 1, 576, 0), (1, 1, 1, 512, 128), (8193, 8193, 1, 512, 64),
                  (1, 65537, 1, 512, 64), (1, 1, 1025, 512, 64)):
        assert ssd.latent_decode_workspace_bytes(*shape) == 0


def test_prompt_refusals(ssd):
    names = "q qs k ks kh r rs v vs vh qst kst S T Tk H N P V scl out os lse s".split()
    good = dict(q=A, qs=8 * 192, k=A, ks=8 * 256, kh=256, r=A, rs=64, v=A, vs=8 * 256, vh=256, qst=A, kst=A,
                S=2, T=300, Tk=400, H=8, N=128, P=64, V=128, scl=0.1, out=B, os=8 * 128, lse=None, s=None)
    _check(ssd, ssd.lib().latent_prompt, names, good, [
        (dict(q=None), INVALID), (dict(k=None), INVALID), (dict(r=None), INVALID), (dict(v=None), INVALID),
        (dict(qst=None), INVALID), (dict(out=None), INVALID), (dict(S=0), INVALID), (dict(T=0), INVALID),
        (dict(Tk=0), INVALID), (dict(H=0), INVALID), (dict(kst=None), INVALID), (dict(qs=1528), INVALID),
        (dict(kh=120), INVALID), (dict(vs=-8), INVALID), (dict(rs=56), INVALID), (dict(os=1016), INVALID),
        (dict(out=A), INVALID),
        (dict(N=96), SHAPE), (dict(P=32), SHAPE), (dict(V=256), SHAPE), (dict(S=8193), SHAPE),
        (dict(T=(1 << 20) + 1), SHAPE), (dict(Tk=(1 << 20) + 1), SHAPE), (dict(H=1025), SHAPE),
        (dict(ks=BIG), SHAPE),
        (dict(q=U), ALIGN), (dict(k=U), ALIGN), (dict(r=U), ALIGN), (dict(v=U), ALIGN), (dict(out=U), ALIGN),
        (dict(qst=U), ALIGN), (dict(kst=U), ALIGN), (dict(lse=U), ALIGN), (dict(qs=1540), ALIGN),
        (dict(vh=260), ALIGN),
    ])


def test_calls_in_slots_are_the_calls(ssd):
    """Arguments in slots reach the same checks: each refusal above that concerns one argument."""
    import struct
    lib = ssd.lib()
    call = lib.dec_latent_call
    assert call(4, b"\0" * 512) == ssd.DEC_ERR_INVALID_ARG and call(-1, b"\0" * 512) == ssd.DEC_ERR_INVALID_ARG
    assert call(0, None) == ssd.DEC_ERR_INVALID_ARG
    good = [0x10000, 576, 0x10000, 1e-6, 0x10000, 576, 0x10000, 512, 64, 0x10000, 0x10000, 0x10000, 1.0, 4, 8,
            512, 64, 64, 0, 0x20000, 512, 64, 0x10000, 576, 0x10000, 0, 0, 3, 16, 16 * 576, 576, 0]
    form = "<" + "".join("d" if isinstance(x, float) else "q" for x in good)
    bad = [(0, 0, 1), (0, 0x10002, 3), (1, 504, 1), (3, -1.0, 1), (5, 56, 1), (8, 56, 1), (11, 0, 1),
           (13, 0, 1), (13, 1 << 40, 2), (14, 1 << 33, 2), (15, 500, 2), (16, 32, 2), (17, 24, 2), (18, 2, 1),
           (20, 516, 3), (22, 0x10002, 3), (25, 5, 1), (28, 0, 1), (30, 580, 3)]
    status = {1: ssd.DEC_ERR_INVALID_ARG, 2: ssd.DEC_ERR_UNSUPPORTED_SHAPE, 3: ssd.DEC_ERR_MISALIGNED}
    for i, value, want in bad:
        args = list(good)
        args[i] = value
        assert call(0, struct.pack(form, *args)) == status[want], (i, value)
    good = [0x10000, 1024, 128, 0x10000, 0x20000, 4096, 512, 4, 8, 128, 512, 0]
    for i, value, want in [(0, 0, 1), (2, 120, 1), (3, 0x10004, 3), (6, 516, 3), (7, 0, 1), (9, 132, 2),
                           (10, 516, 2), (9, (1 << 32) + 128, 2)]:
        args = list(good)
        args[i] = value
        assert call(1, struct.pack("<12q", *args)) == status[want], (i, value)
    good = [0x10000, 4608, 0x10000, 0, 0, 3, 16, 9216, 576, 0x10000, 4, 0x10000, 0x10000, 2, 4, 8, 512, 64, 0.1, 0,
            0x20000, 4096, 0, 0x10000, 0, 0]
    for i, value, want in [(2, 0, 1), (3, 7, 1), (8, 580, 3), (10, 0, 1), (12, 0, 1), (13, 8193, 2), (16, 520, 2),
                           (19, -1, 1), (20, 0x10000, 1), (21, 4088, 1), (22, 0x10002, 3), (23, 0, 1)]:
        args = list(good)
        args[i] = value
        assert call(2, struct.pack("<18qd7q", *args)) == status[want], (i, value)
    good = [0x10000, 1536, 0x10000, 2048, 256, 0x10000, 64, 0x10000, 2048, 256, 0x10000, 0x10000, 2, 300, 400, 8, 128,
            64, 128, 0.1, 0x20000, 1024, 0, 0]
    for i, value, want in [(5, 0, 1), (6, 56, 1), (9, 260, 3), (11, 0, 1), (14, 0, 1), (16, 96, 2), (18, 256, 2),
                           (20, 0x10000, 1), (21, 1016, 1), (22, 0x10002, 3)]:
        args = list(good)
        args[i] = value
        assert call(3, struct.pack("<19qd4q", *args)) == status[want], (i, value)


def test_binding_wants_cuda_tensors(ssd):
    torch = pytest.importorskip("torch")
    x = torch.zeros((2, 3, 64), dtype=torch.bfloat16)
    i = torch.zeros(3, dtype=torch.int32)
    with pytest.raises(TypeError, match="x must be a bfloat16 CUDA tensor"):
        ssd.latent_project(x, x, x)
    with pytest.raises(TypeError, match="q must be a bfloat16 CUDA tensor"):
        ssd.latent_prompt(x, x, None, x, i, x, 1.0)
    with pytest.raises(TypeError, match="cache must be"):
        ssd.latent_append(x[0], None, i, i, None, x)
    with pytest.raises(TypeError, match="cache must be"):
        ssd.latent_decode(x, x, i, i, x, x, 1.0)


FLAG = "*static_cast<volatile int *>(&abort_flag)"


@pytest.mark.parametrize("file", ["latent_decode.cuh", "latent_prompt.cu", "latent_project.cu"])
def test_in_flight_work_is_waited_for_before_tensor_memory_goes(file):
    """Whether a wait ran out is looked at once no role can wait any more; products and copies
    are drained before tensor memory is released; the CTA leaves early only as a whole, before
    it allocates."""
    with open(os.path.join(CSRC, file)) as f:
        text = re.sub(r"//[^\n]*", "", f.read())
    at = text.index("extern __shared__")
    body = text[at:text.index("tmem_dealloc(", at)]
    flag = body.rindex(FLAG)
    met = body.rindex("__syncthreads();", 0, flag)
    assert "wait(" not in body[met:flag].replace("mbar_wait_drain(", "")
    assert body.index("tc_commit(", flag) < body.index("mbar_wait_drain(", flag)
    assert body.index("__syncthreads();", flag) > body.rindex("mbar_wait_drain(")
    alloc = body.index("tmem_alloc(")
    assert "return;" not in body[alloc:] and "__trap" not in body


# ------------------------------------------------- the plain forms themselves ----

def test_plain_attention_by_hand():
    torch = pytest.importorskip("torch")
    import latent_ref
    q = torch.zeros((2, 2, 4), dtype=torch.float64)
    k = torch.ones((1, 3, 4), dtype=torch.float64)
    v = torch.arange(12, dtype=torch.float64).reshape(1, 3, 4)
    pos = torch.tensor([1, 2])
    out, lse, _, _ = latent_ref.attend(q, k, v, pos, 1.0)
    assert torch.allclose(out[0, 0], v[0, :2].mean(0)) and torch.allclose(out[1, 1], v[0].mean(0))
    assert torch.allclose(lse[:, 0], torch.tensor([math.log(2), math.log(3)], dtype=torch.float64))
    out, lse, _, _ = latent_ref.attend(q, k, v, pos, 1.0, window=1)
    assert torch.allclose(out[:, 0], v[0, 1:]) and float(lse.abs().max()) < 1e-12
    out, lse, _, _ = latent_ref.attend(q, k, v, pos, 1.0, exists=torch.zeros(3, dtype=torch.bool))
    assert not out.any() and bool((lse == -math.inf).all())
    out, lse, _, _ = latent_ref.attend(q, k, v, torch.tensor([-1, 0]), 1.0)
    assert not out[0].any() and torch.allclose(out[1, 0], v[0, 0])


def test_plain_rotation_and_norm_by_hand():
    torch = pytest.importorskip("torch")
    import latent_ref
    x = torch.tensor([[1.0, 2.0, 3.0, 4.0]], dtype=torch.float64)
    one, quarter = torch.tensor([1]), torch.tensor([math.pi / 2], dtype=torch.float64)
    y, _ = latent_ref.rotate(x, one, quarter, 2.0, False)
    assert torch.allclose(y, torch.tensor([[-4.0, 2.0, 3.0, 4.0]], dtype=torch.float64))
    y, _ = latent_ref.rotate(x, one, quarter.repeat(2), 1.0, True)
    assert torch.allclose(y, torch.tensor([[-2.0, 1.0, -4.0, 3.0]], dtype=torch.float64))
    c = torch.tensor([[3.0, 4.0]], dtype=torch.float64)
    y = latent_ref.normed(c, torch.tensor([1.0, 2.0]), 0.0)
    assert torch.allclose(y, torch.tensor([[3.0, 8.0]], dtype=torch.float64) / math.sqrt(12.5))

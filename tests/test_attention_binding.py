"""What the attention calls of the Python binding hand to the library, seen on the CPU: tensors
and library are stand-ins, so nothing is launched and no address is used."""
import pytest


class _Tensor:
    """As much of a contiguous CUDA tensor as the binding looks at."""

    def __init__(self, dtype, shape, size, cuda=True, contiguous=True):
        self.dtype, self.shape, self.is_cuda, self._contiguous = dtype, shape, cuda, contiguous
        self.nbytes = self.numel() * size

    def numel(self):
        n = 1
        for d in self.shape:
            n *= d
        return n

    def stride(self):
        out, n = [], 1
        for d in reversed(self.shape):
            out.append(n)
            n *= d
        return tuple(reversed(out))

    def dim(self):
        return len(self.shape)

    def is_contiguous(self):
        return self._contiguous

    def data_ptr(self):
        return 0x1000


class _Library:
    def __init__(self):
        self.calls = []

    def attn_decode(self, *args):
        self.calls.append(args)
        return 0


class _Stream:
    cuda_stream = 0


@pytest.fixture
def call(monkeypatch):
    torch = pytest.importorskip("torch")
    import split_switched_decode_gb300 as ssd
    ssd.build()
    ssd._attention_lib()  # looks torch's types up
    lib = _Library()
    monkeypatch.setattr(ssd, "_attention_lib", lambda: lib)
    bf16, i32, u8 = torch.bfloat16, torch.int32, torch.uint8
    ok = dict(q=_Tensor(bf16, (2, 4, 64), 2), k_cache=_Tensor(bf16, (3, 2, 16, 64), 2),
              v_cache=_Tensor(bf16, (3, 2, 16, 64), 2), block_table=_Tensor(i32, (2, 3), 4),
              seq_len=_Tensor(i32, (2,), 4), out=_Tensor(bf16, (2, 4, 64), 2),
              ws=_Tensor(u8, (4096,), 1), stream=_Stream())

    def attn_decode(**changes):
        ssd.attn_decode(**{**ok, **changes})
        return lib.calls[-1]
    attn_decode.lib, attn_decode.u8 = lib, u8
    return attn_decode


def test_attn_decode_hands_over_the_workspace(call):
    args = call()
    assert args[-3:] == (0x1000, 4096, 0)


@pytest.mark.parametrize("where", [dict(cuda=False), dict(contiguous=False)])
def test_attn_decode_wants_its_workspace_on_the_device(call, where):
    """The kernel writes there: an address of the host must not reach it."""
    with pytest.raises(TypeError, match="ws"):
        call(ws=_Tensor(call.u8, (4096,), 1, **where))
    assert not call.lib.calls

"""The attention part of a decode layer as the example runs it: prompts in chunks, then single
tokens through a captured graph, against a plain dense computation in 64 bits on the layer's
own projected rows, and the output projection on the layer's own mixed rows."""
import importlib.util
import os

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
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                        "decode_attention.py")
    spec = importlib.util.spec_from_file_location("decode_attention", path)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    torch.cuda.set_device(0)
    return torch, ssd, example


def _f64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


@pytest.mark.parametrize("e4m3", [False, True])
def test_prompts_then_steps_match_dense(env, e4m3):
    torch, ssd, example = env
    from split_switched_decode_gb300 import inputs
    S, H, G, D = 4, 16, 2, 64
    layer = example.AttentionLayer(seqs=S, e4m3=e4m3, max_len=128)
    hidden = layer.w_in.shape[1]
    history = [[] for _ in range(S)]  # (k, v) rows in 64 bits, k before the rotation
    inv = layer.inv_freq.cpu().numpy()
    step_scale = 0.05 if e4m3 else None

    def follow(x, out, new):
        """The layer's rows are known (its q was rotated in place): project again."""
        T = x.shape[0]
        rows = torch.empty((T, (H + 2 * G) * D), dtype=torch.bfloat16, device="cuda")
        ws = ssd.workspace(ssd.dec_linear_workspace_bytes(T, rows.shape[1], hidden))
        ssd.dec_linear(x, layer.w_in, None, rows, ws)
        torch.cuda.synchronize()
        r, t = _f64(rows), 0
        mixed = _f64(layer.mixed[:T]).reshape(T, H, D)
        for s, n in enumerate(new):
            at = len(history[s])
            qs = []
            for i in range(n):
                row = r[t + i]
                q, _ = attn_ref.rotate(row[:H * D].reshape(H, D), at + i, inv, 1.0, False)
                k, _ = attn_ref.rotate(row[H * D:(H + G) * D].reshape(G, D), at + i, inv, 1.0,
                                       False)
                history[s].append((k, row[(H + G) * D:].reshape(G, D)))
                qs.append(q)
            if n:
                k = np.stack([h[0] for h in history[s]])
                v = np.stack([h[1] for h in history[s]])
                want, _, size, reach = attn_ref.attention(np.stack(qs), k, v,
                                                          np.ones(len(k), bool), D ** -0.5, 0)
                # one rounding each of q, k, v, the weights and the output: bf16, or e4m3 (unit
                # roundoff 2^-4, half a smallest step 2^-10 of the scale) for k and v. A score
                # is off by (u_q + u_k) reach and its weight by that share (times itself, and
                # once more through the sum)
                uk = 2.0 ** -4 if e4m3 else U
                score = (U + uk) * reach[..., None]
                if e4m3:
                    score = score + D ** -0.5 * 2.0 ** -10 * step_scale * \
                        np.abs(np.stack(qs)).sum(-1, keepdims=True)
                    size = size + 2.0 ** -10 * step_scale
                bound = U * np.abs(want) + (uk + U + 2 * np.expm1(score) + 2.0 ** -12) * size
                assert np.all(np.abs(mixed[t:t + n] - want) <= bound), s
            t += n
        # the output projection on the layer's own mixed rows, as dec_linear's own tests bound it
        y = mixed.reshape(T, H * D) @ _f64(layer.w_out).T + _f64(x)
        rms = np.sqrt(np.mean(y ** 2))
        assert np.all(np.abs(_f64(out) - y) <= 1e-2 * (np.abs(y) + rms))

    for chunk, new in enumerate(([7, 1, 20, 3], [0, 33, 1, 16])):
        x = inputs.activations(sum(new), hidden, "cuda", chunk, "prompt")
        out = torch.empty_like(x)
        layer.step(x, out, torch.tensor(new, dtype=torch.int32, device="cuda"))
        torch.cuda.synchronize()
        follow(x, out, new)
    assert layer.length.tolist() == [7, 34, 21, 19]
    x = inputs.activations(S, hidden, "cuda", 9, "token")
    out = torch.empty_like(x)
    graph = layer.capture(x, out)
    for i in range(12):
        x.copy_(inputs.activations(S, hidden, "cuda", 20 + i, "token"))
        graph.replay()
        torch.cuda.synchronize()
        follow(x, out, [1] * S)
    assert layer.length.tolist() == [19, 46, 33, 31]
    # every page in a table is a different one, and as many are used as the lengths need
    need = sum(-(-n // layer.page) for n in layer.length.tolist())
    assert int(layer.summary[1]) == need
    held = [layer.table[s, :-(-n // layer.page)].tolist()
            for s, n in enumerate(layer.length.tolist())]
    assert len({p for row in held for p in row}) == need
    assert ssd.dec_sync_status() == ssd.DEC_OK


def test_example_runs(env, capsys):
    torch, ssd, example = env
    layer, out = example.main(["--steps", "5", "--seqs", "3"])
    assert "us a step" in capsys.readouterr().out and bool(torch.isfinite(out.float()).all())
    assert ssd.dec_sync_status() == ssd.DEC_OK

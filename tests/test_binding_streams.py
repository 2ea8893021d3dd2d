"""Where the binding's fresh memory comes from when a call is given a stream: that stream's pool.
Checked without a GPU, on stand-ins for torch's streams and the library."""
import ast
import contextlib
import inspect

import pytest
import torch

from quantized_weight_streaming_q4k_gb300 import ops

Q4_0 = ops.Q4_0


def test_every_allocation_of_the_binding_is_told_its_stream():
    tree = ast.parse(inspect.getsource(ops))
    for fn in [n for n in tree.body if isinstance(n, ast.FunctionDef)]:
        if fn.name == "_empty":
            continue
        names = {ast.unparse(c.func) for c in ast.walk(fn) if isinstance(c, ast.Call)}
        assert not names & {"torch.empty", "torch.zeros", "torch.full", "torch.empty_like",
                            "torch.zeros_like"}, fn.name
        for c in ast.walk(fn):
            if isinstance(c, ast.Call) and ast.unparse(c.func) in ("_empty", "_out", "_xq_out",
                                                                   "_workspace"):
                assert "stream" in {ast.unparse(a) for a in c.args}, (fn.name, ast.unparse(c))


class Stream:
    cuda_stream = 1234


class Lib:
    """Every function returns 0, every workspace is 4096 bytes; the launches' streams are kept."""
    def __init__(self):
        self.launched = []

    def __getattr__(self, name):
        if name.endswith("workspace_bytes"):
            return lambda *a: 4096
        return lambda *a: self.launched.append((name, a[-1])) or 0


@pytest.fixture
def fakes(monkeypatch):
    """CPU tensors pass for the current device's (whose number get_device() gives: -1)."""
    now, made, lib = [None], [], Lib()

    @contextlib.contextmanager
    def on(stream):
        now.append(stream)
        yield
        now.pop()

    empty = torch.empty

    def fake_empty(shape, dtype, device):
        made.append((now[-1], dtype))
        return empty(shape, dtype=dtype)

    monkeypatch.setattr(torch.cuda, "current_device", lambda: -1)
    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(ops, "_here", lambda t, name, dev: None)
    monkeypatch.setattr(ops, "_dev", lambda t, name, dtype=None: t.data_ptr())
    monkeypatch.setattr(ops, "lib", lambda: lib)
    monkeypatch.setattr(ops, "stream_handle", lambda s=None: s.cuda_stream if s else 0)
    q, k = torch.zeros(9, 4, 64), torch.zeros(9, 2, 64)
    kp, kc = torch.zeros(2, 9, 64), torch.zeros(9, 2, 5, 64)
    pos, x = torch.arange(9), torch.zeros(256)
    W = torch.zeros(256 * 144, dtype=torch.uint8)
    monkeypatch.setattr(torch, "empty", fake_empty)
    calls = {                                            # outputs and workspaces of each
        "embed_tokens": (1, lambda s: ops.embed_tokens(Q4_0, W, pos, 9, 64, stream=s)),
        "qk_norm_rope": (2, lambda s: ops.qk_norm_rope(q, k, pos, 64, 1e4, stream=s)),
        "prompt_attention": (2, lambda s: ops.prompt_attention(q, k, k, [0, 9], 1.0, stream=s)),
        "prefix_attention": (2, lambda s: ops.prefix_attention(q, kp, kp, 9, kc, kc, [5] * 9, 1.0,
                                                               stream=s)),
        "q4k_matvec": (1, lambda s: ops.q4k_matvec(W, x, 256, 256, stream=s)),
        "q4k_prefill_matmul": (2, lambda s: ops.q4k_prefill_matmul(W, x, 256, 256, 1, stream=s)),
        "kv_attention": (2, lambda s: ops.kv_attention(q, kp, kp, 4, 2, 64, 9, 9, 1.0, stream=s)),
        "quantize_q8_0": (1, lambda s: ops.quantize_q8_0(x, 256, stream=s)),
        "rms_norm_q8": (1, lambda s: ops.rms_norm_q8(x, x, 1e-6, 256, stream=s)),
        "q4k_qkv_proj": (3, lambda s: ops.q4k_qkv_proj(W, W, W, x, 256, 256, 256, stream=s)),
        "q4k_ffn_gate_up_geglu_down": (2, lambda s: ops.q4k_ffn_gate_up_geglu_down(
            W, W, W, ops.Q4_K, x, 256, 256, stream=s)),
        "rms_norm": (1, lambda s: ops.rms_norm(x, x, 1e-6, stream=s)),
        "decode_chain": (1, lambda s: ops.decode_chain([], x, dict(
            hidden=256, inter=256, n_q_heads=4, n_kv_heads=2, head_dim=64, eps=1e-6,
            post_norms=1), stream=s)),
    }
    return made, lib, calls


@pytest.mark.parametrize("name", ["embed_tokens", "qk_norm_rope", "prompt_attention",
                                  "prefix_attention", "q4k_matvec", "q4k_prefill_matmul",
                                  "kv_attention", "quantize_q8_0", "rms_norm_q8", "q4k_qkv_proj",
                                  "q4k_ffn_gate_up_geglu_down", "rms_norm", "decode_chain"])
def test_fresh_memory_belongs_to_the_call_s_stream(fakes, name):
    made, lib, calls = fakes
    count, call = calls[name]
    side = Stream()
    call(side)
    assert lib.launched and all(s == side.cuda_stream for _, s in lib.launched)
    assert len(made) == count and all(s is side for s, _ in made), made
    made.clear()
    call(None)
    assert len(made) == count and all(s is None for s, _ in made), made

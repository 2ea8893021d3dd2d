"""Calls on another stream while the current one still works on memory that was freed in Python."""
import pytest
import torch

from quantized_weight_streaming_q4k_gb300 import build, ops, synth

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()
    torch.cuda.set_device(0)
    yield
    assert ops.device_error() == 0


def calls():
    g = torch.Generator(device="cuda")
    g.manual_seed(83000)

    def normal(*shape):
        return torch.randn(shape, device="cuda", generator=g)

    n, nq, nkv, hd = 700, 4, 2, 128
    q, k, v = normal(n, nq, hd), normal(n, nkv, hd), normal(n, nkv, hd)
    kp, kc, pos = normal(nkv, 2000, hd), normal(n, nkv, 3, hd)[:6], torch.arange(n, device="cuda")
    W = torch.from_numpy(synth.q4_k_matrix(synth.rng(83, 1), 512, 512)).cuda()
    x, tok = normal(n, 512), pos % 512
    return {
        "embed_tokens": lambda s: ops.embed_tokens(ops.Q4_K, W, tok, 512, 512, stream=s),
        "qk_norm_rope": lambda s: ops.qk_norm_rope(q, k, pos, hd, 1e4, stream=s)[0],
        "prompt_attention": lambda s: ops.prompt_attention(q, k, v, [0, n], 0.1, stream=s),
        "prefix_attention": lambda s: ops.prefix_attention(q[:6], kp, kp, 2000, kc, kc, [3] * 6,
                                                           0.1, stream=s),
        "q4k_prefill_matmul": lambda s: ops.q4k_prefill_matmul(W, x, 512, 512, n, stream=s),
        "kv_attention": lambda s: ops.kv_attention(q[0], kp, kp, nq, nkv, hd, 2000, 2000, 0.1,
                                                   stream=s),
    }


@pytest.mark.parametrize("name", ["embed_tokens", "qk_norm_rope", "prompt_attention",
                                  "prefix_attention", "q4k_prefill_matmul", "kv_attention"])
def test_memory_that_the_current_stream_still_uses(name):
    call = calls()[name]
    want = call(None).clone()
    side = torch.cuda.Stream()
    call(side)                                             # both pools have been used
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    # work that is queued behind a pause of some 50 ms: fills and reads blocks of the sizes that
    # the call asks for, which are free in Python by then
    torch.cuda._sleep(100_000_000)
    ok = []
    for size in [want.numel() * 4] * 4 + [1 << 20, 4 << 20, 16 << 20]:
        t = torch.empty(size, dtype=torch.uint8, device="cuda").fill_(7)
        ok.append((t == 7).all())
        del t
    got = call(side)
    torch.cuda.synchronize()
    assert all(bool(t) for t in ok)
    assert torch.equal(got, want)


def test_outputs_may_be_freed_while_the_current_stream_reads_them():
    call, side = calls()["prompt_attention"], torch.cuda.Stream()
    want = call(None).clone()
    torch.cuda.synchronize()
    for _ in range(5):
        got = call(side)
        torch.cuda.current_stream().wait_stream(side)
        torch.cuda._sleep(20_000_000)
        same = (got == want).all()
        del got
        more = [call(side) for _ in range(3)]              # would take the block again
        assert bool(same)
        del more


@pytest.mark.parametrize("name", ["qk_norm_rope", "prompt_attention", "prefix_attention"])
def test_a_side_stream_inside_a_captured_graph(name):
    call, side = calls()[name], torch.cuda.Stream()
    want = call(None).clone()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        here = torch.cuda.current_stream()
        side.wait_stream(here)
        a = call(side)                                     # both at once, each its memory
        b = call(None)
        here.wait_stream(side)
        c = a + b
    for _ in range(3):
        c.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(a, want) and torch.equal(b, want) and torch.equal(c, want * 2)

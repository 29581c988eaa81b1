"""Decodes and prefill on a stream that is not the current one, with workspace
and outputs left to the binding."""
import pytest
import torch

import mla_decode_attention_paged_gb300 as mla
from mla_decode_attention_paged_gb300 import workloads as W
from test_gpu_fp4 import SCALE, _args, _decode_inputs

pytestmark = pytest.mark.gpu


def _stream_of(t):
    """Handle of the stream whose memory the allocator took a tensor from."""
    for seg in torch.cuda.memory_snapshot():
        if seg["address"] <= t.data_ptr() < seg["address"] + seg["total_size"]:
            return seg["stream"]
    raise AssertionError("not the allocator's")


def _calls(H):
    """{name: (call(stream), workspace bytes)} over one FP4 cache."""
    x, g, B, T, K = _decode_inputs(H, 64, [900, 33, 2048], seed=61), W.generator(62), 3, 4, 100
    d, qn, qp, cache, sz, table, lens = _args(x)
    uk, uv = x["W_UK"].cuda(), x["W_UV"].cuda()
    qtn, qtp = W.draw_bf16((B, T, H, 128), 2.0, g).cuda(), W.draw_bf16((B, T, H, 64), 2.0, g).cuda()
    c, k = W.draw_bf16((B, T, 512), 1.0, g).cuda(), W.draw_bf16((B, T, 64), 1.0, g).cuda()
    index = torch.full((B, K), -1, dtype=torch.int32)
    for b, n in enumerate(x["lens"]):
        index[b, :min(n, K)] = torch.randperm(n, generator=g)[:K].to(torch.int32)
    index = index.cuda()
    return {
        # first: it writes the rows that the others read (the same ones each time)
        "prefill": (lambda s: mla.prefill(d, cache, sz, table, lens, c, k, qtn, qtp, uk, uv, SCALE, stream=s),
                    mla.prefill_workspace_size(d, B, T)),
        "decode": (lambda s: mla.decode(d, qn, qp, cache, sz, table, lens, uk, uv, SCALE, stream=s),
                   mla.decode_workspace_size(d, B)),
        "decode_multi": (lambda s: mla.decode_multi(d, qtn, qtp, cache, sz, table, lens, uk, uv, SCALE, stream=s),
                         mla.decode_multi_workspace_size(d, B, T)),
        "decode_sparse": (lambda s: mla.decode_sparse(d, qn, qp, cache, sz, table, lens, index, uk, uv, SCALE, stream=s),
                          mla.decode_sparse_workspace_size(d, B, K)),
        "decode_no_alloc": (lambda s: mla.decode_no_alloc(d, qn, qp, cache, sz, table, lens, uk, uv, SCALE, num_splits=4,
                                                          stream=s), 1 << 20),
    }


@pytest.mark.parametrize("as_handle", [False, True])
@pytest.mark.parametrize("H", [16, 32])
def test_tensors_made_for_another_stream(cuda_lib, H, as_handle):
    """They are that stream's memory: what the current stream allocates and fills
    while the call waits and runs there does not meet them."""
    calls = _calls(H)
    want = {name: call(None) for name, (call, _) in calls.items()}
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for name, (call, size) in calls.items():
        with torch.cuda.stream(s):
            torch.cuda._sleep(4_000_000)  # the call waits for about 2 ms
        got = call(s.cuda_stream if as_handle else s)
        for _ in range(50):
            torch.empty(size, dtype=torch.uint8, device="cuda").fill_(0xFF)
        torch.cuda.synchronize()
        for a, b in zip(got, want[name]):
            if b is not None:
                assert _stream_of(a) == s.cuda_stream and torch.equal(a, b), name


@pytest.mark.parametrize("named", ["current", "stream", "handle"])
def test_captured_without_buffers(cuda_lib, named):
    """A call captured with workspace and outputs left to the binding: they are the
    graph's memory, and each replay gives the eager bits whatever is allocated and
    filled outside it in between."""
    calls = _calls(16)
    want = {name: call(None) for name, (call, _) in calls.items()}
    torch.cuda.synchronize()
    for name, (call, size) in calls.items():
        s = torch.cuda.Stream()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            got = call({"current": None, "stream": s, "handle": s.cuda_stream}[named])
        for _ in range(3):
            for t in got:
                if t is not None:
                    t.fill_(float("nan"))
            for _ in range(20):
                torch.empty(size, dtype=torch.uint8, device="cuda").fill_(0xFF)
            graph.replay()
            torch.cuda.synchronize()
            for a, b in zip(got, want[name]):
                assert b is None or torch.equal(a, b), name

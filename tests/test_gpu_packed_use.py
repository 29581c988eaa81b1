"""How programs use the packed-prompt operators: captured into a graph and
replayed, on several streams at once, with offsets past 32 bits, with
arguments the binding refuses, and with a wait that runs out."""
import numpy as np
import pytest
import torch

import mla_decode_attention_paged_gb300 as mla
from mla_decode_attention_paged_gb300 import workloads as W
import packed_reference as R

pytestmark = pytest.mark.gpu

SCALE = 0.0721
H, P = 16, 64


def _cu(lens):
    return torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32).cuda()


def _step(seed, q_lens=(40, 300, 1), k_lens=(900, 300, 2100)):
    """A chunk step: read the cache back, expand it, attend.  Returns (run(stream), outputs)."""
    g = W.generator(seed)
    lens = torch.tensor(k_lens, dtype=torch.int32)
    table, npg = W.draw_page_table(lens, P, True, g)
    codes, sc = W.draw_fp8_cache(npg, P, g)
    d = mla.dims(H, P, fp8=True)
    x = dict(cache=codes.cuda(), sc=(sc * 0.5).cuda(), table=table.cuda(), cu_q=_cu(q_lens), cu_k=_cu(k_lens),
             uk=W.draw_bf16((H, 128, 512), 0.02, g).cuda(), uv=W.draw_bf16((H, 128, 512), 0.02, g).cuda(),
             qn=W.draw_bf16((sum(q_lens), H, 128), 1.0, g).cuda(), qp=W.draw_bf16((sum(q_lens), H, 64), 1.0, g).cuda())
    nk, nq = sum(k_lens), sum(q_lens)
    bf16 = lambda *s: torch.empty(s, dtype=torch.bfloat16, device="cuda")
    c, pe, k, v, out = bf16(nk, 512), bf16(nk, 64), bf16(nk, H, 128), bf16(nk, H, 128), bf16(nq, H, 128)
    lse = torch.empty((nq, H), device="cuda")
    ws = torch.empty(mla.prompt_attention_workspace_size(d, len(q_lens), nq), dtype=torch.uint8, device="cuda")

    def run(stream=None):
        mla.cache_read(d, x["cache"], x["sc"], x["table"], x["cu_k"], c_kv=c, k_pe=pe, stream=stream)
        mla.expand_kv(d, c, x["uk"], x["uv"], k_nope=k, v=v, stream=stream)
        mla.prompt_attention(d, x["qn"], x["qp"], k, pe, v, x["cu_q"], x["cu_k"], SCALE, workspace=ws, out=out,
                             lse_out=lse, stream=stream)

    return run, (c, pe, k, v, out, lse), ws, x


def test_graph_replay_matches_eager(cuda_lib):
    run, outs, ws, x = _step(1)
    run()
    torch.cuda.synchronize()
    ref = [t.clone() for t in outs]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        run(s)
    for _ in range(3):
        for t in outs:
            t.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        for t, r in zip(outs, ref):
            assert torch.equal(t, r)
    # new contents of the same tensors: other lengths, other queries
    x["qn"].mul_(0.5)
    x["cu_q"].copy_(_cu((341, 0, 0)))
    x["cu_k"].copy_(_cu((1500, 800, 1000)))
    x["table"].copy_(x["table"].flip(0).contiguous())  # rows past a shorter table entry are -1: read as bad pages
    graph.replay()
    torch.cuda.synchronize()
    got = [t.clone() for t in outs]
    run()
    torch.cuda.synchronize()
    for t, r in zip(outs[4:], got[4:]):
        assert torch.equal(t, r)


def test_two_graphs_share_a_workspace(cuda_lib):
    """Captured one after another on one stream, calls of different sizes may share their workspace."""
    a, b = _step(2), _step(3, (17,), (4000,))
    big = torch.empty(max(a[2].numel(), b[2].numel()), dtype=torch.uint8, device="cuda")
    refs = []
    for run, outs, _, _ in (a, b):
        run()
        torch.cuda.synchronize()
        refs.append([t.clone() for t in outs])
    d = mla.dims(H, P)

    def attend(t):
        _, (c, pe, k, v, out, lse), _, x = t
        mla.prompt_attention(d, x["qn"], x["qp"], k, pe, v, x["cu_q"], x["cu_k"], SCALE, workspace=big, out=out,
                             lse_out=lse, stream=s)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graphs = []
    for t in (a, b):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            attend(t)
        graphs.append(g)
    for order in ((0, 1), (1, 0), (0, 0), (1, 1)):
        for i in order:
            graphs[i].replay()
        torch.cuda.synchronize()
        for t, ref in zip((a, b), refs):
            assert torch.equal(t[1][4], ref[4]) and torch.equal(t[1][5], ref[5])


def test_streams_side_by_side(cuda_lib):
    """Four streams, each with its own tensors and workspace, give what each gives alone."""
    steps = [_step(10 + i, (60 + i, 200, 3), (1000, 200 + i, 1500)) for i in range(4)]
    refs = []
    for run, outs, _, _ in steps:
        run()
        torch.cuda.synchronize()
        refs.append([t.clone() for t in outs])
    streams = [torch.cuda.Stream() for _ in steps]
    torch.cuda.synchronize()
    for _ in range(3):
        for (run, _, _, _), s in zip(steps, streams):
            run(s)
    torch.cuda.synchronize()
    for (_, outs, ws, _), ref in zip(steps, refs):
        assert mla.read_device_status(ws) == mla.MLA_OK
        for t, r in zip(outs, ref):
            assert torch.equal(t, r)
    with torch.cuda.stream(streams[0]):  # the binding takes the current stream
        steps[0][0]()
    streams[0].synchronize()
    assert torch.equal(steps[0][1][4], refs[0][4])


@pytest.mark.parametrize("as_handle", [False, True])
def test_tensors_made_for_another_stream(cuda_lib, as_handle):
    """Workspace and outputs that the binding allocates belong to the stream of
    the call: what the current stream allocates meanwhile does not meet them."""
    run, outs, _, x = _step(30)
    run()
    torch.cuda.synchronize()
    ref = [t.clone() for t in outs]
    d = mla.dims(H, P, fp8=True)
    s = torch.cuda.Stream()
    on = s.cuda_stream if as_handle else s
    nk = x["cu_k"][-1].item()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        torch.cuda._sleep(20_000_000)  # the calls below wait for about 10 ms
    c, pe = mla.cache_read(d, x["cache"], x["sc"], x["table"], x["cu_k"], n_rows=nk, stream=on)
    k, v = mla.expand_kv(d, c, x["uk"], x["uv"], stream=on)
    out, lse = mla.prompt_attention(d, x["qn"], x["qp"], k, pe, v, x["cu_q"], x["cu_k"], SCALE, stream=on)
    size = mla.prompt_attention_workspace_size(d, 3, x["qn"].shape[0])
    for _ in range(4):
        torch.empty(size, dtype=torch.uint8, device="cuda").fill_(1)
    torch.cuda.synchronize()
    for t, r in zip((c, pe, k, v, out, lse), ref):
        assert torch.equal(t, r)


def test_offsets_past_32_bits(cuda_lib):
    """Query, key and output rows whose element offsets do not fit 31 bits."""
    heads, big = 128, 140000  # 140,000 x 128 heads x 128 = 2.3e9 elements
    g = torch.Generator(device="cuda").manual_seed(1)
    rnd = lambda *s: torch.randn(s, generator=g, device="cuda").to(torch.bfloat16)
    q_lens, k_lens = [big - 50, 0, 50], [0, big - 300, 300]
    q = torch.zeros((big, heads, 128), dtype=torch.bfloat16, device="cuda")
    qp = torch.zeros((big, heads, 64), dtype=torch.bfloat16, device="cuda")
    k, v, kp = torch.zeros_like(q), torch.zeros_like(q), torch.zeros((big, 64), dtype=torch.bfloat16, device="cuda")
    q[-50:], qp[-50:], k[-300:], v[-300:], kp[-300:] = (rnd(50, heads, 128), rnd(50, heads, 64), rnd(300, heads, 128),
                                                        rnd(300, heads, 128), rnd(300, 64))
    out, lse = mla.prompt_attention(mla.dims(heads, 64), q, qp, k, kp, v, _cu(q_lens), _cu(k_lens), SCALE)
    ref, lref, tol, ltol = R.attention(q[-50:].cpu(), qp[-50:].cpu(), k[-300:].cpu(), kp[-300:].cpu(), v[-300:].cpu(),
                                       [50], [300], SCALE)
    assert R.worst(out[-50:], ref, tol) <= 1.0 and R.worst(lse[-50:], lref, ltol) <= 1.0
    assert not out[:-50].any() and torch.isneginf(lse[:-50]).all()
    del q, qp, k, v, out, lse
    # the expansion of as many rows, and its last rows alone
    c = rnd(big, 512)
    uk, uv = rnd(heads, 128, 512), rnd(heads, 128, 512)
    k, v = mla.expand_kv(mla.dims(heads, 64), c, uk, uv)
    k1, v1 = mla.expand_kv(mla.dims(heads, 64), c[-200:].contiguous(), uk, uv)
    assert torch.equal(k[-200:], k1) and torch.equal(v[-200:], v1)
    ref, tol = R.expand(c[-3:].cpu(), uk.cpu())
    assert R.worst(k[-3:], ref, tol) <= 1.0
    del k, v, k1, v1, c
    # a cache of 4 million rows (4.8 GB), the rows at its end
    pages = 1 << 16
    cache = torch.zeros((pages, P, 576), dtype=torch.bfloat16, device="cuda")
    cache[-2:] = rnd(2, P, 576)
    table = torch.tensor([[0, pages - 2, pages - 1]], dtype=torch.int32, device="cuda")
    c, kp = mla.cache_read(mla.dims(H, P), cache, None, table, _cu([100]),
                           starts=torch.tensor([P + 7], dtype=torch.int32, device="cuda"), n_rows=100)
    rows = cache[-2:].flatten(0, 1)[7:107]
    assert torch.equal(c, rows[:, :512]) and torch.equal(kp, rows[:, 512:])


def test_binding_refusals(cuda_lib):
    d = mla.dims(H, P)
    bf16 = lambda *s: torch.zeros(s, dtype=torch.bfloat16, device="cuda")
    a = dict(q_nope=bf16(8, H, 128), q_pe=bf16(8, H, 64), k_nope=bf16(9, 4, 128), k_pe=bf16(9, 64), v=bf16(9, 4, 128),
             cu_q=_cu([8]), cu_k=_cu([9]))
    run = lambda **kw: mla.prompt_attention(d, *{**a, **kw}.values(), SCALE)
    run()
    for kw in (dict(q_pe=bf16(8, H, 128)), dict(v=bf16(9, H, 128)), dict(k_pe=bf16(8, 64)), dict(cu_k=_cu([4, 5])),
               dict(q_nope=bf16(8, 32, 128)), dict(v=bf16(4, 9, 128).transpose(0, 1)), dict(q_pe=a["q_pe"].cpu())):
        with pytest.raises(ValueError):
            run(**kw)
    for kw in (dict(q_pe=a["q_pe"].float()), dict(cu_q=a["cu_q"].long()), dict(v=None)):
        with pytest.raises(TypeError):
            run(**kw)
    with pytest.raises(mla.MLAError):  # 3 does not divide 16
        run(k_nope=bf16(9, 3, 128), v=bf16(9, 3, 128))
    with pytest.raises(ValueError):
        mla.expand_kv(d, bf16(4, 512), bf16(H, 128, 512), bf16(H, 64, 512))
    with pytest.raises(TypeError):
        mla.cache_read(mla.dims(H, P, int8=True), bf16(2, P, 576), None, _cu([1])[None], _cu([5]), n_rows=5)
    with pytest.raises(TypeError):  # an INT8 cache without its scales
        mla.cache_read(mla.dims(H, P, int8=True), bf16(2, P, 576).to(torch.int8), None, _cu([1])[None], _cu([5]), n_rows=5)
    with pytest.raises(ValueError):
        mla.cache_read(d, bf16(2, P, 576), None, _cu([1])[None], _cu([5]))  # no output, no n_rows


def test_no_rows(cuda_lib):
    d = mla.dims(H, P)
    bf16 = lambda *s: torch.zeros(s, dtype=torch.bfloat16, device="cuda")
    k, v = mla.expand_kv(d, bf16(0, 512), bf16(H, 128, 512), bf16(H, 128, 512))
    assert k.shape == (0, H, 128) and v.shape == (0, H, 128)
    out, lse = mla.prompt_attention(d, bf16(0, H, 128), bf16(0, H, 64), bf16(5, H, 128), bf16(5, 64), bf16(5, H, 128),
                                    _cu([0]), _cu([5]), SCALE)
    assert out.shape == (0, H, 128) and lse.shape == (0, H)
    c, pe = mla.cache_read(d, bf16(2, P, 576), None, _cu([1])[None], _cu([0]), n_rows=0)
    assert c.shape == (0, 512) and pe.shape == (0, 64)
    torch.cuda.synchronize()


def test_wait_timeout_is_reported(cuda_lib):
    """A copy that never completes: the waits run out, the status says so, and the next calls are right."""
    run, outs, ws, x = _step(20)
    run()
    torch.cuda.synchronize()
    ref = [t.clone() for t in outs]
    d = mla.dims(H, P)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    try:
        mla.test_inject_wait_timeout(True)
        mla.expand_kv(d, outs[0], x["uk"], x["uv"], k_nope=torch.empty_like(outs[2]), v=torch.empty_like(outs[3]),
                      device_status=status)
        assert mla.read_status_word(status) == mla.MLA_ERR_DEVICE_TIMEOUT
        mla.prompt_attention(d, x["qn"], x["qp"], outs[2], outs[1], outs[3], x["cu_q"], x["cu_k"], SCALE, workspace=ws)
        assert mla.read_device_status(ws) == mla.MLA_ERR_DEVICE_TIMEOUT
    finally:
        mla.test_inject_wait_timeout(False)
    run()
    torch.cuda.synchronize()
    assert mla.read_device_status(ws) == mla.MLA_OK
    for t, r in zip(outs, ref):
        assert torch.equal(t, r)

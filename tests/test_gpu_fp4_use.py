"""The FP4 cache as it is used: a prompt written, read back and attended in
both forms, steps inside CUDA graphs and on several streams, many short
sequences, random configurations, and a wait that runs out."""
import numpy as np
import pytest
import torch

import fp4_reference as F
import mla_decode_attention_paged_gb300 as mla
import packed_reference as R
from harness import assert_parity, f64
from mla_decode_attention_paged_gb300 import workloads as W
from test_gpu_fp4 import SCALE, _args, _check, _decode_inputs, _lens, _reference, _run

pytestmark = pytest.mark.gpu


def test_prompt_written_read_and_attended(cuda_lib):
    """Packed prompts appended, read back, expanded and attended un-absorbed;
    the last chunk of the same prompts by prefill (absorbed); then a decode step.
    Each against the 64-bit definition on the rows that the append left."""
    H, P, chunk, theta = 16, 64, 20, 10000.0
    lens = [150, 20, 333]
    x = _decode_inputs(H, P, lens, seed=3, T=chunk)
    d, g, n = x["d"], W.generator(4), sum(lens)
    c, k = W.draw_bf16((n, 512), 1.0, g), W.draw_bf16((n, 64), 1.0, g)
    ids = torch.repeat_interleave(torch.arange(3, dtype=torch.int32), _lens(lens).long())
    pos = torch.cat([torch.arange(m, dtype=torch.int32) for m in lens])
    cu_k, cu_q = _lens(np.concatenate([[0], np.cumsum(lens)])), _lens([0, chunk, 2 * chunk, 3 * chunk])
    cache, table = torch.zeros_like(x["cache"]).cuda(), x["table"].cuda()
    mla.cache_append(d, cache, None, table, ids.cuda(), pos.cuda(), c.cuda(), k.cuda(), theta)
    x["cache"] = cache.cpu()
    rows = [F.gathered(x["cache"].numpy(), x["table"].numpy(), b, m, P) for b, m in enumerate(lens)]
    rc, rk = mla.cache_read(d, cache, None, table, cu_k.cuda(), n_rows=n)
    assert np.array_equal(f64(torch.cat([rc, rk], -1)), np.concatenate(rows))
    kn, v = mla.expand_kv(d, rc, x["W_UK"].cuda(), x["W_UV"].cuda())
    qn, qp = x["q_nope"].view(3 * chunk, H, 128), x["q_pe"].view(3 * chunk, H, 64)
    out, lse = mla.prompt_attention(d, qn.cuda(), qp.cuda(), kn, rk, v, cu_q.cuda(), cu_k.cuda(), SCALE)
    ref, lref, tol, ltol = R.attention(qn, qp, kn.cpu(), rk.cpu(), v.cpu(), [chunk] * 3, lens, SCALE)
    assert R.worst(out.cpu(), ref, tol) <= 1.0 and R.worst(lse.cpu(), lref, ltol) <= 1.0
    # absorbed: the same chunk by prefill, which writes the same rows again
    new = [slice(int(cu_k[b + 1]) - chunk, int(cu_k[b + 1])) for b in range(3)]
    cc, kk = torch.stack([c[s] for s in new]), torch.stack([k[s] for s in new])
    out2, lse2 = mla.prefill(d, cache, None, table, _lens(lens).cuda(), cc.cuda(), kk.cuda(), x["q_nope"].cuda(),
                             x["q_pe"].cuda(), x["W_UK"].cuda(), x["W_UV"].cuda(), SCALE, theta)
    assert torch.equal(cache.cpu(), x["cache"])
    uk, uv = f64(x["W_UK"]), f64(x["W_UV"])
    want = [F.attend(f64(x["q_nope"])[b, t], f64(x["q_pe"])[b, t], rows[b][:lens[b] - chunk + t + 1], uk, uv, SCALE)
            for b in range(3) for t in range(chunk)]
    o, l = np.stack([w[0] for w in want]), np.stack([w[1] for w in want])
    pairs = [(i, h) for i in range(3 * chunk) for h in range(H)]
    assert_parity(out2.view(-1, H, 128), lse2.view(-1, H), o, l, pairs)
    assert_parity(out, lse, o, l, pairs)
    _check(dict(x, T=1, q_nope=x["q_nope"][:, -1].contiguous(), q_pe=x["q_pe"][:, -1].contiguous()))


@pytest.mark.parametrize("H,T", [(16, 1), (16, 3), (128, 1)])
def test_graph_replay(cuda_lib, H, T):
    """An append and a decode captured on a side stream give the eager bits."""
    x = _decode_inputs(H, 64, [700, 129, 2000, 64], seed=5, T=T)
    d, g, B = x["d"], W.generator(6), 4
    q_nope, q_pe, cache, table, lens = x["q_nope"].cuda(), x["q_pe"].cuda(), x["cache"].cuda(), x["table"].cuda(), _lens(x["lens"]).cuda()
    c, k = W.draw_bf16((B * T, 512), 1.0, g).cuda(), W.draw_bf16((B * T, 64), 1.0, g).cuda()
    ids = torch.arange(B, dtype=torch.int32, device="cuda").repeat_interleave(T)
    pos = (lens.repeat_interleave(T) - T + torch.arange(T, dtype=torch.int32, device="cuda").repeat(B)).int()
    uk, uv = x["W_UK"].cuda(), x["W_UV"].cuda()
    ws = torch.empty(mla.decode_multi_workspace_size(d, B, T), dtype=torch.uint8, device="cuda")
    out, lse = torch.empty_like(q_nope), torch.empty(q_nope.shape[:-1], dtype=torch.float32, device="cuda")
    start = cache.clone()

    def step(stream):
        mla.cache_append(d, cache, None, table, ids, pos, c, k, 10000.0, stream=stream)
        (mla.decode if T == 1 else mla.decode_multi)(d, q_nope, q_pe, cache, None, table, lens, uk, uv, SCALE,
                                                     workspace=ws, out=out, lse_out=lse, stream=stream)

    step(None)
    torch.cuda.synchronize()
    want = (out.clone(), lse.clone(), cache.clone())
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        step(s)
    for _ in range(3):
        out.zero_()
        cache.copy_(start)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1]) and torch.equal(cache, want[2])
    assert mla.read_device_status(ws) == mla.MLA_OK


def test_two_calls_at_once(cuda_lib):
    """Decodes on two streams, each with its own workspace, over one cache."""
    a, b = _decode_inputs(16, 64, [5000, 77, 900], seed=7), _decode_inputs(32, 64, [5000, 77, 900], seed=7)
    b["cache"], b["table"] = a["cache"], a["table"]
    want = [_run(x)[:2] for x in (a, b)]
    cache, table = a["cache"].cuda(), a["table"].cuda()
    streams = [torch.cuda.Stream() for _ in range(2)]
    jobs = []
    for x in (a, b):
        ws = torch.empty(mla.decode_workspace_size(x["d"], 3), dtype=torch.uint8, device="cuda")
        out = torch.empty((3, x["H"], 128), dtype=torch.bfloat16, device="cuda")
        lse = torch.empty((3, x["H"]), dtype=torch.float32, device="cuda")
        jobs.append((x["d"], x["q_nope"].cuda(), x["q_pe"].cuda(), cache, None, table, _lens(x["lens"]).cuda(),
                     x["W_UK"].cuda(), x["W_UV"].cuda(), ws, out, lse))
    torch.cuda.synchronize()
    for _ in range(10):
        for job, s in zip(jobs, streams):
            mla.decode(*job[:9], SCALE, workspace=job[9], out=job[10], lse_out=job[11], stream=s)
        torch.cuda.synchronize()
        for job, (o, l) in zip(jobs, want):
            assert torch.equal(job[10], o) and torch.equal(job[11], l)
            job[10].zero_()


@pytest.mark.parametrize("H", [16, 32])
def test_many_short_sequences(cuda_lib, H):
    g = W.generator(8)
    _check(_decode_inputs(H, 16, [int(n) for n in torch.randint(0, 4, (700,), generator=g)], seed=9))


@pytest.mark.parametrize("H,B,splits", [(16, 33, 0), (16, 1057, 1), (16, 1057, 5000), (32, 1100, 0)])
def test_many_empty_sequences(cuda_lib, H, B, splits):
    """Runs of empty sequences between full ones: where each CTA starts is searched
    for among 32, 32 x 32 and more."""
    g = W.generator(10)
    some = torch.rand(B, generator=g) < 0.1
    some[0], some[-1] = False, False
    lens = torch.where(some, torch.randint(1, 400, (B,), generator=g), torch.zeros(B, dtype=torch.int64))
    x = _decode_inputs(H, 32, [int(n) for n in lens], seed=11)
    out, lse = _check(x, splits)
    assert not out[~some.cuda()].any() and torch.isneginf(lse[~some.cuda()]).all()


@pytest.mark.parametrize("seed", range(12))
def test_random_configuration(cuda_lib, seed):
    g = W.generator(1000 + seed)
    pick = lambda v: v[int(torch.randint(0, len(v), (1,), generator=g))]
    H, P = pick([16, 16, 32, 64, 96, 128]), pick([16, 32, 64, 128])
    T = pick([1, 1, 2, 3, 5, 8])
    B = 1 + int(torch.randint(0, 6, (1,), generator=g))
    lens = [int(torch.randint(0, pick([20, 300, 1500]), (1,), generator=g)) for _ in range(B)]
    spread = pick([0.0, 0.5, 3.0])
    x, splits = _decode_inputs(H, P, lens, seed=seed, T=T, spread=spread, q_std=pick([0.3, 2.0])), pick([0, 0, 1, 3, 40])
    if spread < 3.0:
        _check(x, splits)
    else:
        _check_large_scores(x, splits)


def _check_large_scores(x, splits):
    """Rows whose blocks differ by factors of e^3 and more make scores of tens of
    thousands, where the rounding of the queries shows: as fp16 (2^-11 of a value)
    and two E4M3 terms (2^-4 of a value twice: 2^-8).  With sums of 576 products in
    fp32 a score is off by at most d = (2^-8 + 2^-11 + 576 2^-23) scale sum |q c|, the
    log-sum-exp by the largest d, a weight by a factor e^(2 d), and an output by
    min(e^(2 d) - 1, 2) of the largest value that it averages, besides the usual."""
    out, lse, st = _run(x, splits)
    assert st == mla.MLA_OK
    ref, lref = _reference(x)
    B, rows = lref.shape
    H, T = x["H"], x["T"]
    out, lse = f64(out.view(B, rows, 128).cpu()), lse.view(B, rows).double().cpu().numpy()
    qn, qp = f64(x["q_nope"]).reshape(B, T, H, 128), f64(x["q_pe"]).reshape(B, T, H, 64)
    uk, uv = f64(x["W_UK"]), f64(x["W_UV"])
    for b, n in enumerate(x["lens"]):
        c = F.gathered(x["cache"].numpy(), x["table"].numpy(), b, n, x["P"])
        for r in range(rows):
            t, h = divmod(r, H)
            seen = c[:max(0, n - T + t + 1)]
            if len(seen) == 0:
                assert not out[b, r].any() and np.isneginf(lse[b, r])
                continue
            q = np.concatenate([uk[h].T @ qn[b, t, h], qp[b, t, h]])
            d = (2.0 ** -8 + 2.0 ** -11 + 576 * 2.0 ** -23) * SCALE * (np.abs(seen) @ np.abs(q)).max()
            assert abs(lse[b, r] - lref[b, r]) <= 2e-2 + d
            largest = np.abs(seen[:, :512] @ uv[h].T).max(axis=0)
            tol = 2e-2 + 1e-2 * np.abs(ref[b, r]).max() + min(np.expm1(min(2 * d, 10.0)), 2.0) * largest
            assert np.all(np.abs(out[b, r] - ref[b, r]) <= tol)


@pytest.mark.parametrize("H", [16, 32])
def test_a_wait_that_runs_out_is_reported(cuda_lib, H):
    """The test hook's extra arrival never comes: the status says so, and the
    next decode is as the one before."""
    x = _decode_inputs(H, 64, [300, 64], seed=11)
    a, la, st = _run(x)
    assert st == mla.MLA_OK
    mla.test_inject_wait_timeout(True)
    try:
        assert _run(x)[2] == mla.MLA_ERR_DEVICE_TIMEOUT
    finally:
        mla.test_inject_wait_timeout(False)
    b, lb, st = _run(x)
    assert st == mla.MLA_OK and torch.equal(a, b) and torch.equal(la, lb)


def test_refusals_on_the_gpu(cuda_lib):
    x = _decode_inputs(16, 64, [10], seed=13)
    d, qn, qp, cache, _, table, lens = _args(x)
    uk, uv = x["W_UK"].cuda(), x["W_UV"].cuda()
    for bad in (cache[:, :, :288].contiguous(), cache.view(-1, 32, 320), cache.view(-1, 320)):
        with pytest.raises((ValueError, IndexError)):
            mla.decode(d, qn, qp, bad, None, table, lens, uk, uv, SCALE)
    with pytest.raises(TypeError):
        mla.decode(d, qn, qp, cache.view(torch.int8), None, table, lens, uk, uv, SCALE)
    with pytest.raises(ValueError):
        mla.decode(d, qn, qp, cache[:, ::2], None, table, lens, uk, uv, SCALE)
    with pytest.raises(TypeError):
        mla.decode(d, qn.float(), qp, cache, None, table, lens, uk, uv, SCALE)
    with pytest.raises((TypeError, ValueError)):
        mla.decode(d, qn, qp, cache, None, table.cpu(), lens, uk, uv, SCALE)
    with pytest.raises(mla.MLAError) as e:
        mla.decode(d, qn, qp, cache, None, table, lens, uk, uv, SCALE, workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))
    assert e.value.status == mla.MLA_ERR_WORKSPACE
    with pytest.raises(mla.MLAError):
        mla.decode(d, qn, qp, cache, None, table, lens, uk, uv, -1.0)

"""GPU parity of the packed-prompt operators -- mla_cache_read, mla_expand_kv
and mla_prompt_attention -- against plain 64-bit implementations, through the
C ABI, and of a run of them together against the fp64 oracle's prefill."""
import numpy as np
import pytest
import torch

import oracle as O
import mla_decode_attention_paged_gb300 as mla
from mla_decode_attention_paged_gb300 import workloads as W
from harness import assert_parity, f64
import packed_reference as R

pytestmark = pytest.mark.gpu

SCALE = 1.0 / np.sqrt(192.0)


def _cu(lens, first=0):
    return torch.tensor(np.concatenate([[first], first + np.cumsum(lens)]), dtype=torch.int32)


# ----- mla_cache_read -----------------------------------------------------------
def _cache(fmt, npg, P, g):
    if fmt == "bf16":
        return W.draw_bf16((npg, P, 576), 1.0, g), None
    return W.draw_int8_cache(npg, P, g) if fmt == "int8" else W.draw_fp8_cache(npg, P, g)


def _dims(fmt, P, H=16):
    return mla.dims(H, P, int8=fmt == "int8", fp8=fmt == "fp8")


@pytest.mark.parametrize("fmt", ["bf16", "int8", "fp8"])
@pytest.mark.parametrize("P,lens,starts", [
    (16, (1,), None),
    (64, (37, 0, 1, 300, 0), (5, 0, 63, 64, 7)),
    (128, (129, 128, 127, 2), (0, 1, 200, 127)),
    (32, (0, 0, 5000), (0, 3, 31)),
])
def test_cache_read(cuda_lib, fmt, P, lens, starts):
    g = W.generator(sum(lens) + P)
    ends = [n + (starts[b] if starts else 0) for b, n in enumerate(lens)]
    table, npg = W.draw_page_table(torch.tensor(ends, dtype=torch.int32), P, True, g, spare_pages=2)
    cache, sz = _cache(fmt, npg, P, g)
    first, n = 3, 3 + sum(lens) + 9  # rows of no sequence before and behind
    cu = _cu(lens, first)
    c = torch.full((n, 512), 7.0, dtype=torch.bfloat16, device="cuda")
    k = torch.full((n, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    st = torch.tensor(starts, dtype=torch.int32).cuda() if starts else None
    mla.cache_read(_dims(fmt, P), cache.cuda(), None if sz is None else sz.cuda(), table.cuda(), cu.cuda(), starts=st,
                   c_kv=c, k_pe=k, device_status=status)
    assert mla.read_status_word(status) == mla.MLA_OK
    got = torch.cat([c, k], dim=-1).cpu()
    ref = R.read_rows(fmt, cache, sz, table, cu.tolist(), starts, P)
    body = got[first:first + len(ref)]
    if fmt == "bf16":
        assert torch.equal(body.double(), ref)
    else:  # two roundings: the product to fp32, then to bf16
        assert R.worst(body, ref, (R.BF16 + R.FP32) * ref.abs()) <= 1.0
    assert torch.all(got[:first] == 7.0) and torch.all(got[first + len(ref):] == 7.0)


@pytest.mark.parametrize("fmt", ["bf16", "int8", "fp8"])
def test_cache_read_gives_back_what_was_appended(cuda_lib, fmt):
    """Append, then read: bf16 bit for bit, INT8 within half a step of the
    row's scale plus a bf16 rounding, FP8 within half an E4M3 step."""
    g = W.generator(3)
    P, lens = 64, torch.tensor([200, 1, 65], dtype=torch.int32)
    table, npg = W.draw_page_table(lens, P, True, g)
    n = int(lens.sum())
    c, k = W.draw_bf16((n, 512), 1.0, g).cuda(), W.draw_bf16((n, 64), 1.0, g).cuda()
    cache = torch.zeros((npg, P, 576), dtype={"bf16": torch.bfloat16, "int8": torch.int8, "fp8": torch.uint8}[fmt],
                        device="cuda")
    sz = {"bf16": None, "int8": torch.zeros((npg, P, 2), device="cuda"), "fp8": torch.zeros((npg, P), device="cuda")}[fmt]
    ids = torch.repeat_interleave(torch.arange(3, dtype=torch.int32), lens.long()).cuda()
    pos = torch.cat([torch.arange(int(m), dtype=torch.int32) for m in lens]).cuda()
    d = _dims(fmt, P)
    mla.cache_append(d, cache, sz, table.cuda(), ids, pos, c, k, 0.0)
    c2, k2 = mla.cache_read(d, cache, sz, table.cuda(), _cu(lens.tolist()).cuda(), n_rows=n)
    x, y = torch.cat([c, k], -1).double().cpu(), torch.cat([c2, k2], -1).double().cpu()
    if fmt == "bf16":
        assert torch.equal(x, y)
    elif fmt == "int8":
        step = (x.amax(-1).clamp_min(0) - x.amin(-1).clamp_max(0)) / 255
        assert ((x - y).abs() <= 0.5001 * step[:, None] + 2 * R.BF16 * x.abs().amax(-1, keepdim=True)).all()
    else:  # half a step of E4M3 is 2^-4 of a normal value, 2^-10 of the scale below
        s = x.abs().amax(-1, keepdim=True) / 448
        assert ((x - y).abs() <= (2.0 ** -4 + 2 * R.BF16) * x.abs() + 2.0 ** -10 * s).all()


def test_cache_read_bad_entries(cuda_lib):
    """Bad pages, positions past the table and bad offsets are reported and
    their rows left as they were; the other rows are read."""
    g = W.generator(4)
    P = 16
    table, npg = W.draw_page_table(torch.tensor([64, 40], dtype=torch.int32), P, True, g)
    cache, _ = _cache("bf16", npg, P, g)
    d = _dims("bf16", P)
    ref = R.read_rows("bf16", cache, None, table, [0, 64, 104], None, P)

    def read(tab, cu, starts=None):
        c = torch.full((104, 512), 7.0, dtype=torch.bfloat16, device="cuda")
        k = torch.full((104, 64), 7.0, dtype=torch.bfloat16, device="cuda")
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        mla.cache_read(d, cache.cuda(), None, tab.cuda(), torch.tensor(cu, dtype=torch.int32).cuda(),
                       starts=None if starts is None else torch.tensor(starts, dtype=torch.int32).cuda(), c_kv=c, k_pe=k,
                       device_status=status)
        return torch.cat([c, k], -1).double().cpu(), mla.read_status_word(status)

    for bad in (-1, npg, 2 ** 31 - 1):
        t = table.clone()
        t[0, 1] = bad
        got, st = read(t, [0, 64, 104])
        assert st == mla.MLA_ERR_DEVICE_BOUNDS
        assert torch.all(got[16:32] == 7.0)
        assert torch.equal(got[:16], ref[:16]) and torch.equal(got[32:], ref[32:])
    for starts in ([0, 2 ** 31 - 1], [0, -50]):  # positions past the table, below 0
        got, st = read(table, [0, 64, 104], starts)
        assert st == mla.MLA_ERR_DEVICE_BOUNDS
        assert torch.equal(got[:64], ref[:64]) and torch.all(got[64:] == 7.0)
    for cu in ([0, 64, 40], [0, 64, 200], [-4, 60, 104]):
        _, st = read(table, cu)
        assert st == mla.MLA_ERR_DEVICE_BOUNDS


# ----- mla_expand_kv --------------------------------------------------------------
@pytest.mark.parametrize("n,H", [(1, 16), (16, 16), (77, 32), (128, 16), (129, 64), (257, 16), (1000, 16), (300, 128)])
def test_expand(cuda_lib, n, H):
    g = W.generator(n + H)
    c, uk, uv = W.draw_bf16((n, 512), 1.0, g), W.draw_bf16((H, 128, 512), 0.02, g), W.draw_bf16((H, 128, 512), 0.02, g)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    k_out = torch.full((n + 1, H, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    v_out = torch.full((n + 1, H, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    k, v = mla.expand_kv(mla.dims(H, 64), c.cuda(), uk.cuda(), uv.cuda(), k_nope=k_out[:n], v=v_out[:n],
                         device_status=status)
    assert mla.read_status_word(status) == mla.MLA_OK
    for got, w in ((k, uk), (v, uv)):
        ref, tol = R.expand(c, w)
        assert R.worst(got, ref, tol) <= 1.0
    assert torch.all(k_out[n] == 7.0) and torch.all(v_out[n] == 7.0)  # nothing past the last row


def test_expand_rows_do_not_mix(cuda_lib):
    """A NaN latent row makes its own outputs NaN and no other's."""
    g = W.generator(9)
    c, uk, uv = W.draw_bf16((200, 512), 1.0, g), W.draw_bf16((16, 128, 512), 0.02, g), W.draw_bf16((16, 128, 512), 0.02, g)
    c[77, 3] = float("nan")
    k, v = mla.expand_kv(mla.dims(16, 64), c.cuda(), uk.cuda(), uv.cuda())
    for t in (k, v):
        nan = torch.isnan(t).flatten(1)
        assert nan[77].all() and not nan[:77].any() and not nan[78:].any()


# ----- mla_prompt_attention ---------------------------------------------------------
def _prompt(q_lens, k_lens, H=16, kv=16, seed=0, q_std=1.5, pad=0):
    g = W.generator(seed + sum(q_lens) + H)
    nq, nk = sum(q_lens) + pad, sum(k_lens) + pad
    return dict(q_nope=W.draw_bf16((nq, H, 128), q_std, g), q_pe=W.draw_bf16((nq, H, 64), q_std, g),
                k_nope=W.draw_bf16((nk, kv, 128), 1.0, g), k_pe=W.draw_bf16((nk, 64), 1.0, g),
                v=W.draw_bf16((nk, kv, 128), 1.0, g), q_lens=list(q_lens), k_lens=list(k_lens), H=H)


def _gpu(x, cu_q=None, cu_k=None, scale=SCALE, **kw):
    cu_q = _cu(x["q_lens"]) if cu_q is None else cu_q
    cu_k = _cu(x["k_lens"]) if cu_k is None else cu_k
    d = mla.dims(x["H"], 64)
    ws = torch.empty(mla.prompt_attention_workspace_size(d, len(cu_q) - 1, x["q_nope"].shape[0]), dtype=torch.uint8,
                     device="cuda")
    out, lse = mla.prompt_attention(d, *(x[n].cuda() for n in ("q_nope", "q_pe", "k_nope", "k_pe", "v")), cu_q.cuda(),
                                    cu_k.cuda(), scale, workspace=ws, **kw)
    torch.cuda.synchronize()
    return out, lse, mla.read_device_status(ws)


def _check(x, scale=SCALE):
    out, lse, st = _gpu(x, scale=scale)
    assert st == mla.MLA_OK
    n = sum(x["q_lens"])
    ref, lref, tol, ltol = R.attention(x["q_nope"], x["q_pe"], x["k_nope"], x["k_pe"], x["v"], x["q_lens"], x["k_lens"],
                                       scale)
    dead = torch.isinf(lref)
    out, lse = out[:n].cpu(), lse[:n].cpu()
    assert torch.all(out[dead] == 0) and torch.all(torch.isneginf(lse[dead]))
    assert R.worst(out[~dead], ref[~dead], tol[~dead]) <= 1.0
    assert R.worst(lse[~dead], lref[~dead], ltol[~dead]) <= 1.0


@pytest.mark.parametrize("n", [1, 2, 15, 16, 17, 127, 128, 129, 255, 256, 257, 384, 700])
def test_prompt_one_sequence(cuda_lib, n):
    _check(_prompt([n], [n], seed=1))


@pytest.mark.parametrize("q_lens,k_lens", [
    ((1, 1, 1, 1), (1, 128, 129, 700)),             # single tokens behind histories
    ((40, 0, 300, 1, 0), (40, 17, 300, 1, 0)),      # empty sequences, one with keys only
    ((128, 256, 130), (400, 257, 1000)),            # chunks behind histories
    ((300, 5, 200), (100, 0, 199)),                 # rows that see no key
    ((260, 513, 129, 3), (260, 513, 129, 3)),
])
def test_prompt_packed(cuda_lib, q_lens, k_lens):
    _check(_prompt(q_lens, k_lens, seed=2))


@pytest.mark.parametrize("H,kv", [(16, 1), (16, 4), (32, 32), (32, 2), (128, 8), (64, 1)])
def test_prompt_grouped_heads(cuda_lib, H, kv):
    _check(_prompt((150, 33, 270), (150, 200, 270), H=H, kv=kv, seed=3))


@pytest.mark.parametrize("H,kv,q_lens,k_lens", [
    (96, 3, (5, 130), (77, 130)),                 # 32 heads of a group in the rows
    (96, 32, (100, 9), (100, 300)),               # groups of 3: none
    (96, 16, (100, 9), (100, 300)),               # groups of 6: two at a time
    (128, 1, (1, 2, 3, 17), (1, 500, 3, 40)),     # 128: a block of two tokens
    (128, 1, (9,), (2100,)),                      # packed and split
    (16, 2, (1, 1, 0, 1, 33), (3000, 1, 5, 129, 33)),
    (32, 4, (300, 5, 200), (100, 0, 199)),        # rows that see no key
])
def test_prompt_packed_heads(cuda_lib, H, kv, q_lens, k_lens):
    _check(_prompt(q_lens, k_lens, H=H, kv=kv, seed=13))


@pytest.mark.parametrize("q_std,scale", [(0.01, SCALE), (20.0, SCALE), (1.0, 1.0), (1.0, 1e-3)])
def test_prompt_flat_and_peaked_scores(cuda_lib, q_std, scale):
    _check(_prompt((520,), (520,), q_std=q_std, seed=4), scale=scale)


def test_prompt_rising_scores(cuda_lib):
    """Scores that climb by hundreds along the keys: every tile raises the running maximum."""
    x = _prompt((300,), (1300,), seed=5)
    x["k_pe"] = (x["k_pe"].float() + torch.arange(1300)[:, None] * 0.05).to(torch.bfloat16)
    x["q_pe"] = x["q_pe"].abs()
    _check(x)


def test_prompt_rows_of_no_sequence(cuda_lib):
    """Rows before the first and behind the last sequence stay as they were,
    and what they and the neighbouring sequences hold reaches no result."""
    x = _prompt((100, 70, 30), (100, 190, 30), seed=6, pad=40)
    out0, lse0, st = _gpu(x)
    assert st == mla.MLA_OK
    y = {k: (v.clone() if torch.is_tensor(v) else v) for k, v in x.items()}
    for name, lens in (("q_nope", x["q_lens"]), ("q_pe", x["q_lens"]), ("k_nope", x["k_lens"]), ("k_pe", x["k_lens"]),
                       ("v", x["k_lens"])):
        y[name][lens[0]:lens[0] + lens[1]] = float("nan")  # the middle sequence
        y[name][sum(lens):] = float("inf")                 # the rows behind the last
    n = sum(x["q_lens"])
    out = torch.full((n + 40, 16, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((n + 40, 16), 7.0, device="cuda")
    _, _, st = _gpu(y, out=out, lse_out=lse)
    assert st == mla.MLA_OK
    keep = torch.cat([torch.arange(100), torch.arange(170, 200)])
    assert torch.equal(out[keep], out0[keep]) and torch.equal(lse[keep], lse0[keep])
    assert torch.all(out[n:] == 7.0) and torch.all(lse[n:] == 7.0)
    assert torch.isnan(out[100:170]).all()
    # the same rows behind a gap at the start
    x2 = {k: (v.clone() if torch.is_tensor(v) else v) for k, v in x.items()}
    for name in ("q_nope", "q_pe", "k_nope", "k_pe", "v"):
        x2[name] = torch.cat([x[name][-40:], x[name][:-40]])
        x2[name][:40] = float("nan")
    out2 = torch.full((n + 40, 16, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    _gpu(x2, cu_q=_cu(x["q_lens"], 40), cu_k=_cu(x["k_lens"], 40), out=out2)
    assert torch.equal(out2[40:], out0[:n]) and torch.all(out2[:40] == 7.0)


def test_prompt_nan_key_reaches_only_its_viewers(cuda_lib):
    x = _prompt((300,), (300,), seed=7)
    out0, lse0, _ = _gpu(x)
    x["k_nope"][200, 5, 17] = float("nan")
    out, lse, _ = _gpu(x)
    assert torch.equal(out[:200], out0[:200]) and torch.equal(lse[:200], lse0[:200])
    assert torch.isnan(out[200:, 5]).all() and torch.isnan(lse[200:, 5]).all()
    other = [h for h in range(16) if h != 5]
    assert torch.equal(out[:, other], out0[:, other])


def test_prompt_bad_offsets(cuda_lib):
    """A sequence with bad offsets and those after it are skipped and reported."""
    x = _prompt((50, 60, 40), (50, 60, 40), seed=8)
    out0, _, _ = _gpu(x)
    for cu_q, cu_k in (([0, 50, 40, 150], [0, 50, 110, 150]), ([0, 50, 110, 150], [0, 50, 30, 150]),
                       ([0, 50, 151, 150], [0, 50, 110, 150]), ([0, 50, 110, 150], [0, 50, 2000, 2100])):
        out = torch.full((150, 16, 128), 7.0, dtype=torch.bfloat16, device="cuda")
        _, _, st = _gpu(x, cu_q=torch.tensor(cu_q, dtype=torch.int32), cu_k=torch.tensor(cu_k, dtype=torch.int32), out=out)
        assert st == mla.MLA_ERR_DEVICE_BOUNDS
        assert torch.equal(out[:50], out0[:50]) and torch.all(out[50:] == 7.0)
    out = torch.full((150, 16, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    _, _, st = _gpu(x, cu_q=torch.tensor([-1, 50, 110, 150], dtype=torch.int32), out=out)
    assert st == mla.MLA_ERR_DEVICE_BOUNDS and torch.all(out == 7.0)


@pytest.mark.parametrize("good,last", [
    ((50,), 2000),                    # keys to split
    (tuple(range(40)), 40),           # more sequences than are listed without a plan
    ((3000,), 40),                    # more units than are split
])
def test_prompt_bad_offsets_in_a_plan(cuda_lib, good, last):
    """As test_prompt_bad_offsets, for calls whose work a plan lists: the good sequences before are computed."""
    q = list(good) + [60, 40]
    k = list(good) + [60, last]
    x = _prompt(q, k, seed=18)
    out0, lse0, st = _gpu(x)
    assert st == mla.MLA_OK
    cu_q, cu_k = _cu(q), _cu(k)
    n, m = len(good) + 1, sum(good)  # the offset to break, and the rows before it
    for name, at, value in (("q", n, m - 1), ("k", n, m - 1), ("q", n, sum(q) + 1), ("k", n, sum(k) + 1),
                            ("q", n, 2**31 - 1), ("k", n, -(2**31))):
        bad_q, bad_k = cu_q.clone(), cu_k.clone()
        (bad_q if name == "q" else bad_k)[at] = value
        out = torch.full_like(out0, 7.0)
        lse = torch.full_like(lse0, 7.0)
        _, _, st = _gpu(x, cu_q=bad_q, cu_k=bad_k, out=out, lse_out=lse)
        assert st == mla.MLA_ERR_DEVICE_BOUNDS
        # which pieces a block is cut into may differ without the last sequences: compare to the formula's bounds
        y = {**x, "q_lens": list(good), "k_lens": list(good)}
        ref, lref, tol, ltol = R.attention(x["q_nope"], x["q_pe"], x["k_nope"], x["k_pe"], x["v"], y["q_lens"],
                                           y["k_lens"], SCALE)
        assert R.worst(out[:m].cpu(), ref, tol) <= 1.0 and R.worst(lse[:m].cpu(), lref, ltol) <= 1.0
        assert torch.all(out[m:] == 7.0) and torch.all(lse[m:] == 7.0)


@pytest.mark.parametrize("q_lens,k_lens", [
    ((100, 70, 30), (1500, 1900, 30)),                     # split keys
    ((3000, 70, 600), (3000, 1900, 700)),                  # whole blocks
    (tuple(range(1, 40)), tuple(range(3, 42))),            # many sequences
])
def test_prompt_rows_of_no_sequence_in_a_plan(cuda_lib, q_lens, k_lens):
    """As test_prompt_rows_of_no_sequence, for calls whose work a plan lists."""
    x = _prompt(q_lens, k_lens, seed=19, pad=40)
    out0, lse0, st = _gpu(x)
    assert st == mla.MLA_OK
    y = {k: (v.clone() if torch.is_tensor(v) else v) for k, v in x.items()}
    for name, lens in (("q_nope", q_lens), ("q_pe", q_lens), ("k_nope", k_lens), ("k_pe", k_lens), ("v", k_lens)):
        y[name][lens[0]:lens[0] + lens[1]] = float("nan")  # the second sequence
        y[name][sum(lens):] = float("inf")                 # the rows behind the last
    n = sum(q_lens)
    out, lse = torch.full_like(out0, 7.0), torch.full_like(lse0, 7.0)
    _, _, st = _gpu(y, out=out, lse_out=lse)
    assert st == mla.MLA_OK
    keep = torch.cat([torch.arange(q_lens[0]), torch.arange(q_lens[0] + q_lens[1], n)])
    assert torch.equal(out[keep], out0[keep]) and torch.equal(lse[keep], lse0[keep])
    assert torch.all(out[n:] == 7.0) and torch.all(lse[n:] == 7.0)
    assert torch.isnan(out[q_lens[0]:q_lens[0] + q_lens[1]]).all()


def test_prompt_no_keys_no_lse(cuda_lib):
    x = _prompt((5, 7), (0, 0), seed=9)
    out, lse, st = _gpu(x)
    assert st == mla.MLA_OK and torch.all(out == 0) and torch.all(torch.isneginf(lse))
    x = _prompt((130,), (130,), seed=9)
    out0, _, _ = _gpu(x)
    out, lse, _ = _gpu(x, want_lse=False)
    assert lse is None and torch.equal(out, out0)


@pytest.mark.parametrize("q_lens,k_lens,H,kv", [
    ((1,), (5000,), 16, 16),                  # one token: keys split over the SMs
    ((19, 7), (9000, 5011), 16, 16),
    ((300,), (300,), 16, 4),                  # short: split or not, the same result within the bounds
    ((2048,), (2048,), 16, 2),                # the longest blocks of one prompt
    ((129, 40), (3000, 17), 16, 16),          # a split block beside one with rows that see no key
    ((1, 1, 1), (4097, 128, 2600), 32, 1),
])
def test_prompt_split_keys(cuda_lib, q_lens, k_lens, H, kv):
    x = _prompt(q_lens, k_lens, H=H, kv=kv, seed=12)
    _check(x)
    a, b = _gpu(x), _gpu(x)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("H,kv,n", [(16, 1, 200), (64, 1, 128), (32, 2, 129)])
def test_prompt_many_single_tokens(cuda_lib, H, kv, n):
    """Single tokens behind contexts of which a few are long enough to split; one
    block to a sequence, in plans of either size, with and without a bad end."""
    k_lens = [(37 * i) % 300 for i in range(n)]
    k_lens[n // 3], k_lens[n - 2], k_lens[5] = 3001, 2048, 1409
    x = _prompt([1] * n, k_lens, H=H, kv=kv, seed=21)
    _check(x)
    a, b = _gpu(x), _gpu(x)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    cu_k = _cu(k_lens)
    cu_k[-1] = sum(k_lens) + 1
    out = torch.full_like(a[0], 7.0)
    _, _, st = _gpu(x, cu_k=cu_k, out=out)
    assert st == mla.MLA_ERR_DEVICE_BOUNDS and torch.all(out[n - 1:] == 7.0) and not torch.any(out[:n - 1] == 7.0)


def test_prompt_many_sequences(cuda_lib):
    """More sequences than the plan's CTA has threads, mostly empty."""
    g = torch.Generator().manual_seed(5)
    lens = torch.randint(0, 4, (2500,), generator=g).tolist()
    lens[1700] = 300
    _check(_prompt(lens, lens, seed=10, H=16, kv=2))


def test_prompt_repeats_bit_identical(cuda_lib):
    x = _prompt((700, 33, 1200), (900, 33, 1200), seed=11)
    a = _gpu(x)
    for _ in range(3):
        b = _gpu(x)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


# ----- together ------------------------------------------------------------------------
@pytest.mark.parametrize("fmt", ["bf16", "int8", "fp8"])
def test_chunk_through_the_cache_matches_the_oracle(cuda_lib, fmt):
    """A chunk of every sequence the un-absorbed way -- append the chunk, read
    the whole history back, expand it, attend -- against the oracle's prefill
    over the same cache; the same call as mla_prefill for equal chunks."""
    g = W.generator(31)
    H, P, T = 16, 64, 24
    lens = torch.tensor([124, 24, 700], dtype=torch.int32)
    table, npg = W.draw_page_table(lens, P, True, g)
    cache, sz = _cache(fmt, npg, P, g)
    if fmt != "bf16":
        sz = sz * (0.3 if fmt == "int8" else 0.5)
    c_kv, k_pe = W.draw_bf16((3, T, 512), 1.0, g), W.draw_bf16((3, T, 64), 1.0, g)
    qn, qp = W.draw_bf16((3, T, H, 128), 1.0, g), W.draw_bf16((3, T, H, 64), 1.0, g)
    uk, uv = W.draw_bf16((H, 128, 512), 0.02, g), W.draw_bf16((H, 128, 512), 0.02, g)
    cache_o = (W.bf16_to_bits(cache) if fmt == "bf16" else cache.numpy()).copy()
    sz_o = None if sz is None else sz.numpy().copy()
    ref_o, ref_l = O.prefill_chunk(cache_o, sz_o, table.numpy(), lens.numpy(), W.bf16_to_bits(c_kv), W.bf16_to_bits(k_pe),
                                   10000.0, f64(qn), f64(qp), f64(uk), f64(uv), SCALE, P, fmt == "int8",
                                   **({"fp8": True} if fmt == "fp8" else {}))
    d = _dims(fmt, P)
    cache, sz, table = cache.cuda(), None if sz is None else sz.cuda(), table.cuda()
    ids = torch.arange(3, dtype=torch.int32).repeat_interleave(T).cuda()
    pos = (lens[:, None] - T + torch.arange(T, dtype=torch.int32)[None]).flatten().int().cuda()
    mla.cache_append(d, cache, sz, table, ids, pos, c_kv.view(-1, 512).cuda(), k_pe.view(-1, 64).cuda(), 10000.0)
    cu_k = _cu(lens.tolist()).cuda()
    c_all, pe_all = mla.cache_read(d, cache, sz, table, cu_k, n_rows=int(lens.sum()))
    k_all, v_all = mla.expand_kv(d, c_all, uk.cuda(), uv.cuda())
    out, lse = mla.prompt_attention(d, qn.view(-1, H, 128).cuda(), qp.view(-1, H, 64).cuda(), k_all, pe_all, v_all,
                                    _cu([T] * 3).cuda(), cu_k, float(SCALE))
    torch.cuda.synchronize()
    ref_o, ref_l = ref_o.reshape(3 * T, H, 128), ref_l.reshape(3 * T, H)
    assert_parity(out, lse, ref_o, ref_l, [(b, h) for b in range(3 * T) for h in range(H)], "packed chunk")

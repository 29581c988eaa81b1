"""GPU tests of the FP4 cache: append, read-back and every decode over it, each
against the plain 64-bit implementation in fp4_reference.

Decodes are held to the library's tolerances (2e-2 absolute, 1e-2 of a row's
largest value, 2e-2 for the log-sum-exp); appended bytes, rows read back and
outputs of a single token, which involve no softmax, to what their roundings
allow."""
import numpy as np
import pytest
import torch

import fp4_reference as F
import mla_decode_attention_paged_gb300 as mla
from harness import assert_parity, f64
from mla_decode_attention_paged_gb300 import workloads as W

pytestmark = pytest.mark.gpu

SCALE = 1.0 / np.sqrt(192.0)
BF16 = 2.0 ** -8  # a rounding to bf16, relative


def _lens(lens):
    return torch.tensor(lens, dtype=torch.int32)


def _rows(n, g, spread=0.0):
    """Values [n, 576] of bf16 rows, blocks of different size where spread > 0."""
    x = torch.randn((n, 18, 32), generator=g)
    if spread:
        x *= torch.exp(spread * torch.randn((n, 18, 1), generator=g))
    return x.view(n, 576).to(torch.bfloat16)


def _cache(npg, P, g, spread=0.0):
    """uint8 [npg, P, 320] of encoded rows: a few hundred different ones, drawn from."""
    some = torch.from_numpy(F.encode(_rows(min(npg * P, 300), g, spread).double().numpy()))
    pick = torch.randint(0, len(some), (npg * P,), generator=g)
    return some[pick].view(npg, P, 320)


def _decode_inputs(H, P, lens, seed, T=1, spread=0.3, q_std=2.0):
    g = W.generator(seed)
    table, npg = W.draw_page_table(_lens([max(n, 1) for n in lens]), P, True, g, spare_pages=2)
    B = len(lens)
    q = (B, H) if T == 1 else (B, T, H)
    return dict(d=mla.dims(H, P, fp4=True), P=P, H=H, T=T, lens=lens, table=table, cache=_cache(npg, P, g, spread),
                q_nope=W.draw_bf16(q + (128,), q_std, g), q_pe=W.draw_bf16(q + (64,), q_std, g),
                W_UK=W.draw_bf16((H, 128, 512), 0.02, g), W_UV=W.draw_bf16((H, 128, 512), 0.02, g))


def _args(x):
    return (x["d"], x["q_nope"].cuda(), x["q_pe"].cuda(), x["cache"].cuda(), None, x["table"].cuda(),
            _lens(x["lens"]).cuda())


def _run(x, splits=0, **kw):
    fn, size = (mla.decode, mla.decode_workspace_size) if x["T"] == 1 else (mla.decode_multi, None)
    B = len(x["lens"])
    n = (mla.decode_workspace_size(x["d"], B, splits) if x["T"] == 1
         else mla.decode_multi_workspace_size(x["d"], B, x["T"], splits))
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    out, lse = fn(*_args(x), x["W_UK"].cuda(), x["W_UV"].cuda(), SCALE, num_splits=splits, workspace=ws, **kw)
    torch.cuda.synchronize()
    return out, lse, mla.read_device_status(ws)


def _reference(x):
    H, T, B = x["H"], x["T"], len(x["lens"])
    qn, qp = f64(x["q_nope"]).reshape(B, T, H, 128), f64(x["q_pe"]).reshape(B, T, H, 64)
    out, lse = np.zeros((B, T * H, 128)), np.zeros((B, T * H))
    uk, uv = f64(x["W_UK"]), f64(x["W_UV"])
    for b, n in enumerate(x["lens"]):
        rows = F.gathered(x["cache"].numpy(), x["table"].numpy(), b, n, x["P"])
        for t in range(T):
            o, l = F.attend(qn[b, t], qp[b, t], rows[:max(0, n - T + t + 1)], uk, uv, SCALE)
            out[b, t * H:(t + 1) * H], lse[b, t * H:(t + 1) * H] = o, l
    return out, lse


def _check(x, splits=0):
    out, lse, st = _run(x, splits)
    assert st == mla.MLA_OK
    ref, lref = _reference(x)
    B, R = lref.shape
    assert_parity(out.view(B, R, 128), lse.view(B, R), ref, lref, [(b, r) for b in range(B) for r in range(R)])
    return out, lse


# ----- append -------------------------------------------------------------------
def _append(P, lens, starts, c, k, theta, dirty=0xAB, **change):
    """Appends the packed tokens; returns (cache, status, expected cache)."""
    g = W.generator(7)
    table, npg = W.draw_page_table(_lens([s + n for s, n in zip(starts, lens)]), P, True, g, spare_pages=1)
    ids = np.repeat(np.arange(len(lens)), lens).astype(np.int32)
    pos = np.concatenate([np.arange(s, s + n) for s, n in zip(starts, lens)]).astype(np.int32)
    cache = torch.full((npg, P, 320), dirty, dtype=torch.uint8)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    dev = cache.cuda()
    mla.cache_append(mla.dims(16, P, fp4=True), dev, None, table.cuda(), torch.from_numpy(ids).cuda(),
                     torch.from_numpy(pos).cuda(), c.cuda(), k.cuda(), theta, device_status=status)
    want = F.appended(cache.numpy(), table.numpy(), ids, pos, f64(c), f64(k), theta, P)
    return dev.cpu().numpy(), mla.read_status_word(status), want


@pytest.mark.parametrize("P,lens,starts,theta", [
    (16, (1,), (0,), 10000.0),
    (64, (33, 1, 200), (0, 63, 4090), 10000.0),
    (128, (129, 7), (1000000, 131071), 10000.0),
    (32, (50, 3), (31, 0), 0.0),           # not rotated
    (16, (40,), (12345,), 500000.0),
    (16, (9,), (77,), 0.5),                # frequencies above one
    (64, (2500,), (100,), 10000.0),        # more than one warp to a block
])
def test_append_bytes(cuda_lib, P, lens, starts, theta):
    """Every byte of every row, and nothing else in the pool."""
    g = W.generator(sum(lens))
    n = sum(lens)
    got, st, want = _append(P, lens, starts, W.draw_bf16((n, 512), 1.0, g), W.draw_bf16((n, 64), 3.0, g), theta)
    assert st == mla.MLA_OK
    assert np.array_equal(got, want)


def test_append_special_values(cuda_lib):
    """Zeros of both signs, ties, subnormals, the largest values, and blocks
    that hold an infinity or a NaN (their neighbours stay as they are)."""
    g = W.generator(1)
    c, k = W.draw_bf16((12, 512), 1.0, g), W.draw_bf16((12, 64), 1.0, g)
    c[0], k[0] = 0.0, -0.0
    ties = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0])
    c[1] = torch.cat([ties, -ties] * 32).to(torch.bfloat16)
    k[1] = (torch.cat([ties, -ties] * 4) * 2.0 ** 100).to(torch.bfloat16)
    c[2] = (c[2].float() * 2.0 ** -126).to(torch.bfloat16)
    c[3] = (c[3].float() * 2.0 ** -132).to(torch.bfloat16)
    c[4] = torch.sign(c[4].float()).to(torch.bfloat16) * torch.finfo(torch.bfloat16).max
    c[5, 70], c[6, 200], c[7, 511], k[8, 0], k[9, 63] = (float("inf"), float("nan"), float("-inf"), float("nan"),
                                                          float("inf"))
    c[10] = (c[10].float().view(16, 32) * 2.0 ** torch.arange(-60.0, 100.0, 10.0)[:, None]).view(512).to(torch.bfloat16)
    c[11, ::32] = 6.03125
    got, st, want = _append(16, (12,), (0,), c, k, 0.0)
    assert st == mla.MLA_OK
    assert np.array_equal(got, want)


def test_append_far_position(cuda_lib):
    """Positions past a billion.  The fp64 angle itself is off there by up to
    pos 2^-53 radians, so the keys' codes may differ where a value is that near
    a border; the latents may not."""
    P, pos = 128, (1 << 30) + 77
    table = torch.full((1, pos // P + 1), -1, dtype=torch.int32, device="cuda")
    table[0, pos // P] = 1
    g = W.generator(2)
    c, k = W.draw_bf16((1, 512), 1.0, g), W.draw_bf16((1, 64), 1.0, g)
    cache = torch.zeros((2, P, 320), dtype=torch.uint8, device="cuda")
    one = torch.tensor([pos], dtype=torch.int32, device="cuda")
    mla.cache_append(mla.dims(16, P, fp4=True), cache, None, table, torch.zeros_like(one), one, c.cuda(), k.cuda(), 1e4)
    want = F.encode(np.concatenate([f64(c), F.rotated(f64(k), [pos], 1e4)], axis=1))[0]
    got = cache[1, pos % P].cpu().numpy()
    assert np.array_equal(got[:256], want[:256]) and np.array_equal(got[288:], want[288:])
    a, b = F.decode_rows(got[None])[0, 512:], F.decode_rows(want[None])[0, 512:]
    assert np.mean(a != b) <= 1 / 64
    cache[1, pos % P] = 0
    assert not cache.any()


def test_append_skips_bad_tokens(cuda_lib):
    P, g = 16, W.generator(3)
    table = torch.tensor([[0, 1], [2, 9], [-1, 3]], dtype=torch.int32)  # pool of 5 pages: entries 9 and -1 are bad
    ids = torch.tensor([0, 3, -1, 0, 0, 1, 2, 2], dtype=torch.int32)
    pos = torch.tensor([17, 0, 0, 32, -1, 20, 5, 16], dtype=torch.int32)
    c, k = W.draw_bf16((8, 512), 1.0, g), W.draw_bf16((8, 64), 1.0, g)
    cache = torch.zeros((5, P, 320), dtype=torch.uint8, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    mla.cache_append(mla.dims(16, P, fp4=True), cache, None, table.cuda(), ids.cuda(), pos.cuda(), c.cuda(), k.cuda(),
                     1e4, device_status=status)
    assert mla.read_status_word(status) == mla.MLA_ERR_DEVICE_BOUNDS
    good = [0, 7]
    want = F.appended(np.zeros((5, P, 320), np.uint8), table.numpy(), ids.numpy()[good], pos.numpy()[good], f64(c)[good],
                      f64(k)[good], 1e4, P)
    assert np.array_equal(cache.cpu().numpy(), want)


@pytest.mark.parametrize("n", [2047, 2048, 2049, 13001, 50000, 194560, 194561])
def test_append_many_tokens(cuda_lib, n):
    """Every length of a warp's run of tokens, some of them out of range: rows from
    400 different ones (not rotated), and nothing behind or between them."""
    P, g = 64, W.generator(n)
    pages = (n + P - 1) // P
    some = _rows(400, g, 0.5)
    pick = torch.randint(0, 400, (n,), generator=g)
    pos = torch.arange(n, dtype=torch.int32)
    bad = torch.rand(n, generator=g) < 0.01
    bad[-1] = True
    table = torch.randperm(pages, generator=g).to(torch.int32)
    values = some[pick].cuda()
    cache = torch.full((pages, P, 320), 0xAB, dtype=torch.uint8, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    mla.cache_append(mla.dims(16, P, fp4=True), cache, None, table.view(1, -1).cuda(),
                     torch.zeros(n, dtype=torch.int32, device="cuda"), torch.where(bad, -1 - pos, pos).cuda(),
                     values[:, :512].contiguous(), values[:, 512:].contiguous(), 0.0, device_status=status)
    assert mla.read_status_word(status) == mla.MLA_ERR_DEVICE_BOUNDS
    rows = torch.from_numpy(F.encode(some.double().numpy()))[pick]
    rows[bad] = 0xAB
    want = torch.full((pages * P, 320), 0xAB, dtype=torch.uint8)
    want[table[pos // P].long() * P + pos % P] = rows
    assert torch.equal(cache.cpu().view(-1, 320), want)


# ----- read-back -------------------------------------------------------------------
@pytest.mark.parametrize("P,lens,starts", [
    (16, (1,), None),
    (64, (37, 0, 1, 300, 0), (5, 0, 63, 64, 7)),
    (128, (129, 128, 127, 2), (0, 1, 200, 127)),
    (32, (0, 0, 9000), (0, 3, 31)),
])
def test_read(cuda_lib, P, lens, starts):
    """Rows come back exactly (every FP4 value is a bf16 value); rows of no
    sequence stay as they are."""
    g = W.generator(sum(lens) + P)
    ends = [n + (starts[b] if starts else 0) for b, n in enumerate(lens)]
    table, npg = W.draw_page_table(_lens(ends), P, True, g, spare_pages=2)
    cache = _cache(npg, P, g, spread=8.0)
    cache[..., 306:] = 0xEE  # not read
    first, n = 3, 3 + sum(lens) + 9
    cu = torch.tensor(np.concatenate([[first], first + np.cumsum(lens)]), dtype=torch.int32)
    c = torch.full((n, 512), 7.0, dtype=torch.bfloat16, device="cuda")
    k = torch.full((n, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    mla.cache_read(mla.dims(16, P, fp4=True), cache.cuda(), None, table.cuda(), cu.cuda(),
                   starts=None if starts is None else _lens(starts).cuda(), c_kv=c, k_pe=k, device_status=status)
    assert mla.read_status_word(status) == mla.MLA_OK
    got = torch.cat([c, k], dim=-1).cpu()
    at = [(b, (starts[b] if starts else 0) + t) for b in range(len(lens)) for t in range(lens[b])]
    rows = np.stack([cache.numpy()[table.numpy()[b, p // P], p % P] for b, p in at])
    assert np.array_equal(f64(got[first:first + len(at)]), F.decode_rows(rows))
    assert torch.all(got[:first] == 7.0) and torch.all(got[first + len(at):] == 7.0)


def test_read_every_scale(cuda_lib):
    """All 256 scale bytes: subnormal results, NaN blocks, and values past
    bf16's largest (infinity)."""
    g = W.generator(11)
    cache = torch.randint(0, 256, (16, 16, 320), generator=g).to(torch.uint8)
    cache[..., 288:306] = torch.arange(256).view(16, 16, 1).to(torch.uint8)
    table = torch.arange(16, dtype=torch.int32).view(1, 16)
    c, k = mla.cache_read(mla.dims(16, 16, fp4=True), cache.cuda(), None, table.cuda(), _lens([0, 256]).cuda(), n_rows=256)
    want = torch.from_numpy(F.decode_rows(cache.view(256, 320).numpy())).to(torch.bfloat16)
    got = torch.cat([c, k], -1).cpu()
    nan = torch.isnan(want)
    assert torch.equal(torch.isnan(got), nan) and nan[255].all() and not nan[:255].any()
    assert torch.equal(got[~nan], want[~nan])


# ----- decode -------------------------------------------------------------------------
@pytest.mark.parametrize("H", [16, 32, 64, 96, 128, 256])
@pytest.mark.parametrize("P", [16, 128])
def test_decode_heads_and_pages(cuda_lib, H, P):
    _check(_decode_inputs(H, P, [1, 0, 63, 64, 65, 127, 128, 129, 300], seed=H + P))


@pytest.mark.parametrize("P", [32, 64])
@pytest.mark.parametrize("splits", [1, 2, 7, 152, 1000])
def test_decode_splits(cuda_lib, P, splits):
    _check(_decode_inputs(16, P, [777, 1, 2049, 130, 0, 1024], seed=splits), splits)


@pytest.mark.parametrize("H,T", [(16, 2), (16, 3), (16, 4), (16, 8), (32, 2), (32, 5), (64, 2), (128, 3)])
def test_decode_multi(cuda_lib, H, T):
    """Several tokens per sequence, causal among themselves; sequences shorter
    than that, and ones whose last tokens begin a tile."""
    _check(_decode_inputs(H, 64, [T, 1, 128 + T - 1, 127, 129, 520, 0], seed=H + T, T=T))


@pytest.mark.parametrize("H,T", [(16, 1), (32, 1), (16, 2)])
def test_decode_all_empty(cuda_lib, H, T):
    """A batch of nothing: zeros and minus infinity, written."""
    x = _decode_inputs(H, 64, [0, 0, 0], seed=1, T=T)
    q = x["q_nope"].shape[:-1]
    out = torch.full(q + (128,), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full(q, 7.0, device="cuda")
    _, _, st = _run(x, out=out, lse_out=lse)
    assert st == mla.MLA_OK and not out.any() and torch.isneginf(lse).all()


def test_decode_long(cuda_lib):
    x = _decode_inputs(16, 64, [20011, 5000], seed=4)
    a, la = _check(x)
    b, lb = _check(x)
    assert torch.equal(a, b) and torch.equal(la, lb)  # bit-identical run to run


@pytest.mark.parametrize("H", [16, 32, 128])
@pytest.mark.parametrize("order", ["rising", "falling", "one large", "large first"])
def test_decode_running_maximum(cuda_lib, H, order):
    """Scores that keep raising the maximum by more than the exponential's
    range, scores that fall, one token above thousands and thousands of tokens
    below one."""
    n = 700
    x = _decode_inputs(H, 64, [n], seed=17, q_std=0.0)
    x["q_pe"][..., 0] = 1.0
    rows = np.zeros((n, 576))
    g = W.generator(5)
    rows[:, :512] = f64(_rows(n, g))[:, :512]
    ramp = np.linspace(0, 6000, n)
    level = {"rising": ramp, "falling": ramp[::-1], "one large": np.where(np.arange(n) == 400, 400.0, 4.0),
             "large first": np.where(np.arange(n) == 0, 230.0, 4.0)}[order]
    rows[:, 512] = f64(torch.tensor(level.copy()).to(torch.bfloat16))
    enc = F.encode(rows)
    flat = x["cache"].view(-1, 320)
    for t in range(n):
        flat[int(x["table"][0, t // 64]) * 64 + t % 64] = torch.from_numpy(enc[t])
    _check(x)
    _check(x, splits=5)


@pytest.mark.parametrize("H", [16, 32, 128])
def test_decode_one_token_is_its_value(cuda_lib, H):
    """One cached token: out = W^UV c, whatever its score: block scales over
    all that the decode reads exactly, below it (rounded) and above (saturated)."""
    exps = list(range(-19, 17)) + [-100, 100]
    x = _decode_inputs(H, 16, [1] * len(exps), seed=23, q_std=0.01)
    for b, e in enumerate(exps):
        x["cache"][x["table"][b, 0], 0, 288:306] = 127 + e
        x["cache"][x["table"][b, 0], 0, 304:306] = 127 - 3
    out, lse, st = _run(x)
    assert st == mla.MLA_OK
    uv = f64(x["W_UV"])
    for b in range(len(exps)):
        c = F.gathered(x["cache"].numpy(), x["table"].numpy(), b, 1, 16)[0, :512]
        ref, mag = uv @ c, np.abs(uv) @ np.abs(c)
        # bf16 rounding of the result; the latent as two bf16 terms (2^-16), sums of 512 products in fp32
        tol = BF16 * np.abs(ref) + (2.0 ** -16 + 512 * 2.0 ** -23) * mag + 1e-38
        assert np.all(np.abs(f64(out[b].cpu()) - ref) <= tol), exps[b]


def test_decode_tails_do_not_matter(cuda_lib):
    """Rows past a sequence's end and the unread bytes of every row may hold
    anything, NaN scales included; rows before the end with a NaN block make
    their own sequence NaN and no other."""
    for H in (16, 32, 128):
        x = _decode_inputs(H, 64, [70, 129, 1, 500], seed=31)
        a, la, _ = _run(x)
        y = dict(x, cache=x["cache"].clone())
        used = torch.zeros(x["cache"].shape[:2], dtype=torch.bool)
        for b, n in enumerate(x["lens"]):
            for t in range(n):
                used[x["table"][b, t // 64], t % 64] = True
        y["cache"][~used] = 0xFF
        y["cache"][..., 306:] = 0xFF
        b_, lb, _ = _run(y)
        assert torch.equal(a, b_) and torch.equal(la, lb)
        y["cache"][y["table"][1, 1], 3, 290] = 255  # token 67 of sequence 1
        c, lc, st = _run(y)
        assert st == mla.MLA_OK and torch.isnan(c[1]).all() and torch.isnan(lc[1]).all()
        for b in (0, 2, 3):
            assert torch.equal(a[b], c[b]) and torch.equal(la[b], lc[b])


@pytest.mark.parametrize("H", [16, 32, 96])
@pytest.mark.parametrize("value", [float("inf"), float("-inf"), 1e30, float("nan")])
def test_decode_infinite_query(cuda_lib, H, value):
    """A query value past fp16, infinite or NaN makes its own head NaN; the heads
    that share its scale keep their results."""
    x = _decode_inputs(H, 32, [200, 1, 517], seed=31)
    ref, lref = _reference(x)
    x["q_pe"][0, 5, 9] = x["q_pe"][2, H - 1, 63] = value
    out, lse, st = _run(x)
    assert st == mla.MLA_OK
    bad = torch.zeros((3, H), dtype=torch.bool)
    bad[0, 5] = bad[2, H - 1] = True
    assert torch.isnan(out[bad]).all() and torch.isnan(lse[bad]).all()
    assert_parity(out, lse, ref, lref, [(b, h) for b in range(3) for h in range(H) if not bad[b, h]])


@pytest.mark.parametrize("H", [16, 32, 64])
def test_decode_heads_far_apart(cuda_lib, H):
    """Heads share the scale of their query terms: sizes from 1 to 2^-15 of the largest."""
    x = _decode_inputs(H, 64, [300, 77], seed=32)
    size = 2.0 ** -(torch.arange(H) % 16).view(1, H, 1)
    x["q_nope"], x["q_pe"] = x["q_nope"] * size.to(torch.bfloat16), x["q_pe"] * size.to(torch.bfloat16)
    _check(x)


@pytest.mark.parametrize("H,T,where", [(16, 2, "latent"), (16, 3, "latent"), (32, 2, "latent"), (16, 8, "both"),
                                       (128, 2, "latent"), (32, 4, "rope")])
def test_hidden_nan_rows(cuda_lib, H, T, where):
    """A NaN block reaches the query tokens that see its row and no others."""
    lens = [300, 128 + T, 2 * T + 1]
    x = _decode_inputs(H, 64, lens, seed=33, T=T)
    ref, lref = _reference(x)
    blocks = {"latent": [288 + 3], "rope": [288 + 17], "both": list(range(288, 306))}[where]
    for b, n in enumerate(lens):  # the last query token's row
        page = int(x["table"][b, (n - 1) // 64])
        x["cache"][page, (n - 1) % 64, blocks] = 255
    out, lse, st = _run(x)
    assert st == mla.MLA_OK
    assert torch.isnan(out[:, T - 1]).all() and torch.isnan(lse[:, T - 1]).all()
    R = (T - 1) * H
    assert_parity(out.view(3, T * H, 128), lse.view(3, T * H), ref, lref, [(b, r) for b in range(3) for r in range(R)])


def test_prefill_hidden_nan(cuda_lib):
    """A NaN in a chunk's token 40: queries 0 .. 39 are as without it, 40 .. are NaN."""
    H, P, T, n = 16, 64, 90, 150
    x = _decode_inputs(H, P, [n], seed=34)
    g = W.generator(35)
    c, k = W.draw_bf16((1, T, 512), 1.0, g), W.draw_bf16((1, T, 64), 1.0, g)
    q, qp = W.draw_bf16((1, T, H, 128), 2.0, g).cuda(), W.draw_bf16((1, T, H, 64), 2.0, g).cuda()
    uk, uv = x["W_UK"].cuda(), x["W_UV"].cuda()

    def run(c):
        cache = x["cache"].cuda()
        ws = torch.empty(mla.prefill_workspace_size(x["d"], 1, T, 0), dtype=torch.uint8, device="cuda")
        out, lse = mla.prefill(x["d"], cache, None, x["table"].cuda(), _lens([n]).cuda(), c.cuda(), k.cuda(), q, qp,
                               uk, uv, SCALE, workspace=ws)
        assert mla.read_device_status(ws) == mla.MLA_OK
        return out[0], lse[0]

    clean, lclean = run(c)
    assert torch.isfinite(clean).all() and torch.isfinite(lclean).all()
    c[0, 40, 100] = float("nan")
    out, lse = run(c)
    assert torch.equal(out[:40], clean[:40]) and torch.equal(lse[:40], lclean[:40])
    assert torch.isnan(out[40:]).all() and torch.isnan(lse[40:]).all()


def test_decode_pages_shuffled(cuda_lib):
    """The same rows under another page table give the same bits."""
    x = _decode_inputs(16, 32, [900, 33, 260], seed=37)
    a, la, _ = _run(x)
    g = W.generator(1)
    npg = x["cache"].shape[0]
    perm = torch.randperm(npg, generator=g)
    cache = torch.empty_like(x["cache"])
    cache[perm] = x["cache"]
    table = torch.where(x["table"] >= 0, perm[x["table"].clamp_min(0).long()].to(torch.int32), x["table"])
    b, lb, _ = _run(dict(x, cache=cache, table=table))
    assert torch.equal(a, b) and torch.equal(la, lb)


def test_decode_reports_bad_entries(cuda_lib):
    for H in (16, 128):
        x = _decode_inputs(H, 64, [300, 100], seed=41)
        a, la, _ = _run(x)
        bad = dict(x, table=x["table"].clone())
        bad["table"][0, 2] = 1 << 30
        b, lb, st = _run(bad)
        assert st == mla.MLA_ERR_DEVICE_BOUNDS and torch.equal(a[1], b[1])
        for n in (-1, x["table"].shape[1] * 64 + 1):
            c, lc, st = _run(dict(x, lens=[n, 100]))
            assert st == mla.MLA_ERR_DEVICE_BOUNDS
            assert not c[0].any() and torch.isneginf(lc[0]).all() and torch.equal(a[1], c[1])


def test_decode_past_four_gigabytes(cuda_lib):
    """Pages behind byte 2^32 of the pool."""
    P = 128
    pages = (1 << 32) // (P * 320) + 300
    x = _decode_inputs(16, P, [300, 40], seed=43)
    npg = x["cache"].shape[0]
    pool = torch.zeros((pages, P, 320), dtype=torch.uint8, device="cuda")
    pool[-npg:] = x["cache"].cuda()
    shift = torch.where(x["table"] >= 0, x["table"] + pages - npg, x["table"]).to(torch.int32)
    for H in (16, 128):
        y = _decode_inputs(H, P, [300, 40], seed=43)
        a, la, _ = _run(dict(y, cache=x["cache"], table=x["table"]))
        z = dict(y, table=shift)
        out, lse = mla.decode(y["d"], y["q_nope"].cuda(), y["q_pe"].cuda(), pool, None, shift.cuda(),
                              _lens([300, 40]).cuda(), y["W_UK"].cuda(), y["W_UV"].cuda(), SCALE)
        assert torch.equal(a, out) and torch.equal(la, lse)
    c, k = mla.cache_read(x["d"], pool, None, shift.cuda(), _lens([0, 300, 340]).cuda(), n_rows=340)
    c2, k2 = mla.cache_read(x["d"], x["cache"].cuda(), None, x["table"].cuda(), _lens([0, 300, 340]).cuda(), n_rows=340)
    assert torch.equal(c, c2) and torch.equal(k, k2)


# ----- sparse, prefill, fixed scratch ------------------------------------------------
@pytest.mark.parametrize("H,P", [(16, 64), (32, 16), (128, 128)])
def test_decode_sparse(cuda_lib, H, P):
    """Listed rows only: short and long lists, one row twice, entries out of
    range, an empty list."""
    lens = [500, 3, 1000, 50]
    x = _decode_inputs(H, P, lens, seed=47)
    g = W.generator(3)
    idx = torch.full((4, 200), -1, dtype=torch.int32)
    idx[0] = torch.randperm(500, generator=g)[:200].to(torch.int32)
    idx[1, 5:8] = torch.tensor([2, 0, 2], dtype=torch.int32)
    idx[2, ::3] = torch.randperm(1000, generator=g)[:67].to(torch.int32)
    ws = torch.empty(mla.decode_sparse_workspace_size(x["d"], 4, 200), dtype=torch.uint8, device="cuda")

    def run(i):
        out, lse = mla.decode_sparse(*_args(x), i.cuda(), x["W_UK"].cuda(), x["W_UV"].cuda(), SCALE, workspace=ws)
        torch.cuda.synchronize()
        return out, lse, mla.read_device_status(ws)

    out, lse, st = run(idx)
    assert st == mla.MLA_OK
    ref, lref = np.zeros((4, H, 128)), np.zeros((4, H))
    for b in range(4):
        rows = F.gathered(x["cache"].numpy(), x["table"].numpy(), b, lens[b], P)
        sel = [i for i in idx[b].tolist() if i >= 0]
        ref[b], lref[b] = F.attend(f64(x["q_nope"])[b], f64(x["q_pe"])[b], rows[sel], f64(x["W_UK"]), f64(x["W_UV"]), SCALE)
    assert_parity(out, lse, ref, lref, [(b, h) for b in range(4) for h in range(H)])
    worse = idx.clone()
    worse[3, 0], worse[1, 0] = 50, -7
    out2, lse2, st = run(worse)
    assert st == mla.MLA_ERR_DEVICE_BOUNDS and torch.equal(out, out2) and torch.equal(lse, lse2)


@pytest.mark.parametrize("H,chunk,lens", [(16, 24, (124, 24, 300)), (16, 130, (130, 400)), (128, 40, (41, 200)), (32, 3, (3, 129))])
def test_prefill(cuda_lib, H, chunk, lens):
    """A chunk appended and attended, then a decode step over what it left."""
    P, theta, B = 64, 10000.0, len(lens)
    x = _decode_inputs(H, P, list(lens), seed=53, T=chunk)
    g = W.generator(9)
    c, k = W.draw_bf16((B, chunk, 512), 1.0, g), W.draw_bf16((B, chunk, 64), 1.0, g)
    cache = x["cache"].cuda()
    ws = torch.empty(mla.prefill_workspace_size(x["d"], B, chunk), dtype=torch.uint8, device="cuda")
    out, lse = mla.prefill(x["d"], cache, None, x["table"].cuda(), _lens(lens).cuda(), c.cuda(), k.cuda(),
                           x["q_nope"].cuda(), x["q_pe"].cuda(), x["W_UK"].cuda(), x["W_UV"].cuda(), SCALE, theta,
                           workspace=ws)
    torch.cuda.synchronize()
    assert mla.read_device_status(ws) == mla.MLA_OK
    ids = np.repeat(np.arange(B), chunk)
    pos = np.concatenate([np.arange(n - chunk, n) for n in lens])
    want = F.appended(x["cache"].numpy(), x["table"].numpy(), ids, pos, f64(c).reshape(-1, 512), f64(k).reshape(-1, 64),
                      theta, P)
    assert np.array_equal(cache.cpu().numpy(), want)
    x["cache"] = torch.from_numpy(want)
    ref, lref = _reference(x)
    R = chunk * H
    pairs = [(b, r) for b in range(B) for r in list(range(min(R, 64))) + list(range(max(0, R - 64), R))]
    assert_parity(out.view(B, R, 128), lse.view(B, R), ref, lref, pairs)
    _check(dict(x, T=1, q_nope=x["q_nope"][:, -1].contiguous(), q_pe=x["q_pe"][:, -1].contiguous()))


def test_decode_no_alloc(cuda_lib):
    x = _decode_inputs(16, 64, [300, 65], seed=59)
    a, la, _ = _run(x, splits=4)
    lse = torch.empty((2, 16), dtype=torch.float32, device="cuda")
    b, lb = mla.decode_no_alloc(*_args(x), x["W_UK"].cuda(), x["W_UV"].cuda(), SCALE, num_splits=4, lse_out=lse)
    torch.cuda.synchronize()
    assert torch.equal(a, b) and torch.equal(la, lb)

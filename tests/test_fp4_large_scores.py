"""Decodes over FP4 rows whose blocks differ by factors of e^3 and more, with
scores up to some hundreds, held to a bound that a wrong output does not meet.

Queries are chosen so that nothing of them is rounded away: q_nope has one
power of two, so q_lat is a row of W^UK (bf16 values: eight significant bits,
as q_pe), which fp16 holds to 2^-25 and the two E4M3 terms to 2^-21 of the
largest query value of their group.  What is left, for a score with sum |q c| its
products' magnitudes:
  score         d = scale ((2^-25 + 2^-21 top) sum |c| + 576 2^-23 sum |q c|), sums of 576
                products in fp32; and 16 fp32 roundings of the largest score
  weight        a factor e^(2 d'), d' the largest of those; fp16: 2^-11; multiples of
                2^-26 of the largest weight below
  output        the weights' errors over sum p |W^UV c|, the latent as two bf16 terms
                (2^-16) and sums of 512 products in fp32, a rounding to bf16 (2^-8)
  log-sum-exp   d', and the sum's terms to 2^-20
The softmax scale is set so that no score's sum |q c| passes 400: 2 d' < 0.1."""
import numpy as np
import pytest
import torch

import fp4_reference as F
import mla_decode_attention_paged_gb300 as mla
from harness import f64
from mla_decode_attention_paged_gb300 import workloads as W
from test_gpu_fp4 import _decode_inputs, _lens

LARGEST = 400.0
CASES = [(16, 1, 64, (122, 68, 17)), (16, 3, 32, (300, 5)), (32, 1, 16, (129, 260)), (32, 2, 64, (70, 200)),
         (64, 1, 128, (122, 68)), (64, 3, 32, (150,)), (96, 2, 16, (90, 131)), (128, 1, 64, (140, 40)), (128, 2, 64, (133,))]


def _inputs(H, T, P, lens, seed):
    x = _decode_inputs(H, P, list(lens), seed=seed, T=T, spread=3.0, q_std=0.16)
    g = W.generator(seed + 1)
    at = torch.randint(0, 128, x["q_nope"].shape[:-1] + (1,), generator=g)
    size = 2.0 ** torch.randint(1, 6, at.shape, generator=g).float()
    x["q_nope"] = torch.zeros(x["q_nope"].shape).scatter_(-1, at, size).to(torch.bfloat16)
    return x


def _expected(x):
    """(softmax scale, out [rows, 128], lse [rows], tolerances of both, the largest 2 d')
    of all query rows, [sequence][token][head] in order."""
    H, T, B = x["H"], x["T"], len(x["lens"])
    qn, qp = f64(x["q_nope"]).reshape(B, T, H, 128), f64(x["q_pe"]).reshape(B, T, H, 64)
    uk, uv = f64(x["W_UK"]), f64(x["W_UV"])
    rows = [F.gathered(x["cache"].numpy(), x["table"].numpy(), b, n, x["P"]) for b, n in enumerate(x["lens"])]
    q = np.concatenate([np.einsum("bthd,hdc->bthc", qn, uk), qp], axis=-1)
    scale = LARGEST / max(float((np.abs(rows[b]) @ np.abs(q[b, t, h])).max()) for b in range(B) for t in range(T) for h in range(H))
    scale = float(np.float32(scale))
    out, lse, tol, ltol, worst = [], [], [], [], 0.0
    for b, n in enumerate(x["lens"]):
        top = np.abs(q[b]).max()
        for t in range(T):
            c = rows[b][:n - T + t + 1]
            for h in range(H):
                s, big = scale * (c @ q[b, t, h]), scale * (np.abs(c) @ np.abs(q[b, t, h]))
                d = scale * (2.0 ** -25 + 2.0 ** -21 * top) * np.abs(c).sum(1) + 576 * 2.0 ** -23 * big
                d = (d + 16 * 2.0 ** -24 * big).max()
                m = s.max()
                p = np.exp(s - m)
                total = p.sum()
                p /= total
                v = c[:, :512] @ uv[h].T
                o = p @ v
                off = (np.expm1(2 * d) + 2.0 ** -11) * (p @ np.abs(v)) + len(c) * 2.0 ** -26 * np.abs(v).max(0)
                off += (2.0 ** -16 + 512 * 2.0 ** -23) * (p @ (np.abs(c[:, :512]) @ np.abs(uv[h]).T))
                out.append(o)
                lse.append(m + np.log(total))
                tol.append(off + 2.0 ** -8 * (np.abs(o) + off))
                ltol.append(d + 2.0 ** -20 * (1 + len(c)))
                worst = max(worst, 2 * d)
    return scale, np.array(out), np.array(lse), np.array(tol), np.array(ltol), worst


def _agree(out, lse, want):
    """Whether outputs [rows, 128] and log-sum-exps [rows] are within their bounds."""
    _, ref, lref, tol, ltol, _ = want
    return bool(np.all(np.abs(out - ref) <= tol) and np.all(np.abs(lse - lref) <= ltol))


@pytest.mark.parametrize("H,T,P,lens", CASES)
def test_the_bounds_refuse_wrong_outputs(H, T, P, lens):
    """The tolerances stay small, and outputs of zero, of the row before, without the
    last token or with a tenth of an output's change do not meet them."""
    x = _inputs(H, T, P, lens, 1000 + H + T)
    want = _expected(x)
    scale, ref, lref, tol, ltol, worst = want
    assert worst < 0.1 and ltol.max() < 0.1
    assert _agree(ref, lref, want)
    assert not _agree(np.zeros_like(ref), lref, want)
    assert not _agree(np.roll(ref, 1, axis=0), lref, want)
    assert not _agree(ref * 1.1, lref, want)
    assert not _agree(ref, lref + 0.1, want)
    # each row alone: half of the outputs, and more, tell a zero from the value
    assert np.all((np.abs(ref) > tol).mean(axis=1) > 0.5)
    assert np.all((np.abs(ref) * 0.1 > tol).any(axis=1))


@pytest.mark.gpu
@pytest.mark.parametrize("splits", [0, 5])
@pytest.mark.parametrize("H,T,P,lens", CASES)
def test_large_scores(cuda_lib, H, T, P, lens, splits):
    x = _inputs(H, T, P, lens, 1000 + H + T)
    want = _expected(x)
    B = len(lens)
    ws = torch.empty(mla.decode_multi_workspace_size(x["d"], B, T, splits), dtype=torch.uint8, device="cuda")
    out, lse = (mla.decode if T == 1 else mla.decode_multi)(
        x["d"], x["q_nope"].cuda(), x["q_pe"].cuda(), x["cache"].cuda(), None, x["table"].cuda(), _lens(x["lens"]).cuda(),
        x["W_UK"].cuda(), x["W_UV"].cuda(), want[0], num_splits=splits, workspace=ws)
    torch.cuda.synchronize()
    assert mla.read_device_status(ws) == mla.MLA_OK
    got, glse = f64(out.cpu()).reshape(-1, 128), lse.double().cpu().numpy().reshape(-1)
    _, ref, lref, tol, ltol, _ = want
    assert np.max(np.abs(got - ref) / tol) <= 1.0, np.max(np.abs(got - ref) / tol)
    assert np.max(np.abs(glse - lref) / ltol) <= 1.0, np.max(np.abs(glse - lref) / ltol)

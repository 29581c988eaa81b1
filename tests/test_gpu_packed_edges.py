"""Edges of the packed-prompt operators: rows that see no key beside values that
are not finite, long contexts among short ones, the expansion on both sides of
its change of form, default-stream handles, and waits that run out."""
import time

import numpy as np
import pytest
import torch

import mla_decode_attention_paged_gb300 as mla
from mla_decode_attention_paged_gb300 import workloads as W
import packed_reference as R

pytestmark = pytest.mark.gpu

SCALE = 1.0 / np.sqrt(192.0)
NAMES = ("q_nope", "q_pe", "k_nope", "k_pe", "v")


def _cu(lens):
    return torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32).cuda()


def _prompt(q_lens, k_lens, H=16, kv=16, seed=0, extra_q=0):
    """Random inputs; ``extra_q`` query rows of no sequence behind the last."""
    g = W.generator(seed + sum(q_lens) + sum(k_lens) + H)
    nq, nk = sum(q_lens) + extra_q, sum(k_lens)
    return dict(q_nope=W.draw_bf16((nq, H, 128), 1.5, g), q_pe=W.draw_bf16((nq, H, 64), 1.5, g),
                k_nope=W.draw_bf16((nk, kv, 128), 1.0, g), k_pe=W.draw_bf16((nk, 64), 1.0, g),
                v=W.draw_bf16((nk, kv, 128), 1.0, g), q_lens=list(q_lens), k_lens=list(k_lens), H=H)


def _attend(x):
    """(out, lse, the workspace's first five words): status, then, where a plan
    ran, its items, the units taken, the split blocks and their rows (else -1)."""
    d = mla.dims(x["H"], 64)
    ws = torch.full((mla.prompt_attention_workspace_size(d, len(x["q_lens"]), x["q_nope"].shape[0]),), 255,
                    dtype=torch.uint8, device="cuda")
    out, lse = mla.prompt_attention(d, *(x[n].cuda() for n in NAMES), _cu(x["q_lens"]), _cu(x["k_lens"]), SCALE,
                                    workspace=ws)
    torch.cuda.synchronize()
    return out, lse, ws[:20].view(torch.int32).tolist()


# ----- rows that see no key ---------------------------------------------------------
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("H,kv,q_lens,k_lens", [
    (16, 16, (300,), (100,)),            # the blocks listed without a plan
    (16, 1, (296,), (100,)),             # 16 heads of a token in the rows
    (16, 16, (300, 1), (100, 3000)),     # planned, beside a block whose keys are split
    (16, 16, (300, 4000), (100, 4000)),  # planned, whole blocks
])
def test_rows_without_keys_beside_bad_values(cuda_lib, H, kv, q_lens, k_lens, bad):
    """A row that sees no key gives 0 and -inf, whatever the values that other
    rows of its tile see hold."""
    x = _prompt(q_lens, k_lens, H=H, kv=kv, seed=1)
    out0, lse0, _ = _attend(x)
    none = q_lens[0] - k_lens[0]  # rows of the first sequence that see no key
    x["v"][3] = bad  # query none + 3 is the first to see it, and its tile has rows that see nothing
    out, lse, words = _attend(x)
    assert words[0] == mla.MLA_OK
    assert torch.all(out[:none] == 0) and torch.all(torch.isneginf(lse[:none]))
    assert not torch.isfinite(out[none + 3:q_lens[0]]).any()
    assert torch.equal(out[q_lens[0]:], out0[q_lens[0]:]) and torch.equal(lse, lse0)


def test_scores_of_minus_infinity(cuda_lib):
    """A row whose visible scores are all -inf has no weight to give: 0 and -inf, as a row that sees no key."""
    x = _prompt((200, 2), (200, 3000), seed=2)
    x["q_nope"][..., 0] = 1.0
    x["k_nope"][:70, 5, 0] = float("-inf")        # one head: rows 0 .. 69 see nothing else
    x["k_nope"][200:, 7, 0] = float("-inf")       # all keys of the second sequence, which are split
    out, lse, words = _attend(x)
    assert words[0] == mla.MLA_OK and words[3] > 0
    for rows, h in ((slice(0, 70), 5), (slice(200, 202), 7)):
        assert torch.all(out[rows, h] == 0) and torch.all(torch.isneginf(lse[rows, h]))
    assert torch.isfinite(out).all() and torch.isfinite(lse[70:200, 5]).all()


# ----- one long context among short ones ---------------------------------------------
def _close(x, out, lse):
    n = sum(x["q_lens"])
    ref, lref, tol, ltol = R.attention(*(x[k] for k in NAMES), x["q_lens"], x["k_lens"], SCALE)
    assert R.worst(out[:n].cpu(), ref, tol) <= 1.0 and R.worst(lse[:n].cpu(), lref, ltol) <= 1.0


@pytest.mark.parametrize("H,kv,n", [(16, 16, 7), (16, 16, 8), (16, 16, 9), (128, 8, 13), (128, 8, 19), (32, 32, 4)])
def test_long_context_among_short_is_split(cuda_lib, H, kv, n):
    """Single tokens whose units fill most of one round of SMs, one of them
    behind a long context: its keys are spread over the SMs."""
    k_lens = [100 + i for i in range(n)]
    k_lens[n // 2] = 20000
    x = _prompt([1] * n, k_lens, H=H, kv=kv, seed=3)
    out, lse, words = _attend(x)
    assert words[0] == mla.MLA_OK
    assert words[3] >= 1  # split blocks
    _close(x, out, lse)


def test_long_context_of_a_padded_batch_is_split(cuda_lib):
    """Query rows of no sequence do not hide that the few others stand behind a long context."""
    x = _prompt((5,), (20000,), seed=4, extra_q=2043)
    out, lse, words = _attend(x)
    assert words[0] == mla.MLA_OK and words[3] >= 1
    _close(x, out, lse)


# ----- the expansion on both sides of its change of form ------------------------------
def _worst_expand(got, c, w):
    """Largest error in units of its bound, all rows, in 64 bits on the GPU."""
    bad = 0.0
    wd, wa = w.double().flatten(0, 1).T, w.double().abs().flatten(0, 1).T
    for i in range(0, len(c), 4096):
        cd = c[i:i + 4096].double()
        ref, mag = cd @ wd, cd.abs() @ wa
        r = (got[i:i + 4096].double().flatten(1) - ref).abs() / (R.BF16 * ref.abs() + 512 * R.SUM * mag)
        bad = max(bad, float(torch.nan_to_num(r, nan=float("inf")).max()))
    return bad


@pytest.mark.parametrize("n,H", [
    (4096, 16), (4097, 16),      # weights resident up to 256 rows to a head, latents from there on
    (5003, 16), (34893, 16),     # an odd end; several resident tiles to a pair of SMs
    (8193, 32), (16461, 64), (32769, 128),
])
def test_expand_both_forms(cuda_lib, n, H):
    g = W.generator(n + H)
    c = W.draw_bf16((n, 512), 1.0, g).cuda()
    uk, uv = W.draw_bf16((H, 128, 512), 0.02, g).cuda(), W.draw_bf16((H, 128, 512), 0.02, g).cuda()
    d = mla.dims(H, 64)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    k_out = torch.full((n + 1, H, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    v_out = torch.full((n + 1, H, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    k, v = mla.expand_kv(d, c, uk, uv, k_nope=k_out[:n], v=v_out[:n], device_status=status)
    assert mla.read_status_word(status) == mla.MLA_OK
    assert _worst_expand(k, c, uk) <= 1.0 and _worst_expand(v, c, uv) <= 1.0
    assert torch.all(k_out[n] == 7.0) and torch.all(v_out[n] == 7.0)
    step = 200 * H + 7  # the same rows in calls with the weights resident: the same sums in the same order
    for i in range(0, n, step):
        k1, v1 = mla.expand_kv(d, c[i:i + step], uk, uv)
        assert torch.equal(k[i:i + step], k1) and torch.equal(v[i:i + step], v1)


# ----- streams --------------------------------------------------------------------------
def _stream_of(t):
    """Handle of the stream whose memory the allocator took a tensor from."""
    for seg in torch.cuda.memory_snapshot():
        if seg["address"] <= t.data_ptr() < seg["address"] + seg["total_size"]:
            return seg["stream"]
    raise AssertionError("not the allocator's")


def test_default_stream_by_handle(cuda_lib):
    """Handle 0 is the default stream: what the binding allocates for such a call
    is that stream's memory, also while another stream is current."""
    g = W.generator(5)
    c, w = W.draw_bf16((40, 512), 1.0, g).cuda(), W.draw_bf16((16, 128, 512), 0.02, g).cuda()
    torch.cuda.synchronize()
    with torch.cuda.stream(torch.cuda.Stream()):
        k, v = mla.expand_kv(mla.dims(16, 64), c, w, w, stream=0)
    torch.cuda.synchronize()
    assert _stream_of(k) == 0 and _stream_of(v) == 0


# ----- waits that run out -------------------------------------------------------------
class _Injected:
    """A copy that never completes in every call inside: waits run out after 2 s, and
    what is in flight is waited for half a second more."""

    def __enter__(self):
        torch.cuda.synchronize()
        mla.test_inject_wait_timeout(True)
        self.t0 = time.monotonic()

    def __exit__(self, *exc):
        mla.test_inject_wait_timeout(False)
        torch.cuda.synchronize()
        self.seconds = time.monotonic() - self.t0


@pytest.mark.parametrize("n,H", [(300, 16), (5003, 16), (40, 128)])  # either form; fewer units than pairs and more
def test_expand_waits_for_what_is_in_flight(cuda_lib, n, H):
    g = W.generator(n)
    c = W.draw_bf16((n, 512), 1.0, g).cuda()
    uk, uv = W.draw_bf16((H, 128, 512), 0.02, g).cuda(), W.draw_bf16((H, 128, 512), 0.02, g).cuda()
    d = mla.dims(H, 64)
    k0, v0 = mla.expand_kv(d, c, uk, uv)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    run = _Injected()
    with run:
        mla.expand_kv(d, c, uk, uv, device_status=status)
    assert run.seconds >= 2.45
    assert mla.read_status_word(status) == mla.MLA_ERR_DEVICE_TIMEOUT
    k, v = mla.expand_kv(d, c, uk, uv)
    assert torch.equal(k, k0) and torch.equal(v, v0)


@pytest.mark.parametrize("q_lens,k_lens", [
    ((93,), (93,)),              # no plan
    ((300, 2), (300, 3000)),     # planned, split
    ((3000,), (3000,)),          # planned, whole blocks
])
def test_prompt_waits_for_what_is_in_flight(cuda_lib, q_lens, k_lens):
    x = {k: v.cuda() if torch.is_tensor(v) else v for k, v in _prompt(q_lens, k_lens, seed=6).items()}
    out0, lse0, words = _attend(x)
    assert words[0] == mla.MLA_OK
    run = _Injected()
    with run:
        _, _, words = _attend(x)
    assert run.seconds >= 2.45
    assert words[0] == mla.MLA_ERR_DEVICE_TIMEOUT
    out, lse, words = _attend(x)
    assert words[0] == mla.MLA_OK and torch.equal(out, out0) and torch.equal(lse, lse0)

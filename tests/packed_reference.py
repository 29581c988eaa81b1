"""Plain 64-bit implementations of the packed-prompt operators (cache
read-back, latent expansion, causal attention over packed prompts) and the
error bounds that the library's arithmetic allows them.

The bounds count roundings: a rounding to bf16 is off by at most 2^-8 of the
value (half a step), one to fp32 by at most 2^-24; a sum of n products in fp32
by at most n 2^-23 of the sum of their magnitudes (the tensor cores may
truncate where IEEE rounds).
"""
import torch

BF16, FP32, SUM = 2.0 ** -8, 2.0 ** -24, 2.0 ** -23


def read_rows(fmt, cache, scale, table, cu, starts, page):
    """float64 [cu[-1] - cu[0], 576]: the rows of a packed batch, one at a time."""
    rows = []
    for b in range(len(cu) - 1):
        for t in range(cu[b + 1] - cu[b]):
            pos = (starts[b] if starts is not None else 0) + t
            pg, slot = int(table[b, pos // page]), pos % page
            x = cache[pg, slot]
            if fmt == "bf16":
                rows.append(x.double())
            elif fmt == "int8":
                rows.append(float(scale[pg, slot, 0]) * (x.double() - float(scale[pg, slot, 1])))
            else:
                rows.append(float(scale[pg, slot]) * x.view(torch.float8_e4m3fn).double())
    return torch.stack(rows) if rows else torch.zeros((0, 576), dtype=torch.float64)


def expand(c, w):
    """(float64 [n, H, 128], error bound) of one product, W [H, 128, 512]."""
    c, w = c.double(), w.double()
    ref = torch.einsum("nc,hdc->nhd", c, w)
    mag = torch.einsum("nc,hdc->nhd", c.abs(), w.abs())
    return ref, BF16 * ref.abs() + 512 * SUM * mag


def attention(q_nope, q_pe, k_nope, k_pe, v, q_lens, k_lens, scale):
    """(out float64 [n_q, H, 128], lse [n_q, H], bounds of both) over the rows
    of the sequences, packed without gaps.

    A score is a sum of 192 products in fp32, scaled: off by ds.  A weight
    then is off by a factor exp(2 ds) (its score and the maximum) times 2^-20
    (scaling, exponential, sum), and by 2^-8 where it is rounded to bf16 for
    the product with the values, itself a sum in fp32."""
    H, G = q_nope.shape[1], k_nope.shape[1]
    out = torch.zeros((sum(q_lens), H, 128), dtype=torch.float64)
    lse = torch.full((sum(q_lens), H), float("-inf"), dtype=torch.float64)
    out_tol, lse_tol = torch.zeros_like(out), torch.zeros_like(lse)
    q0 = k0 = 0
    for nq, nk in zip(q_lens, k_lens):
        for h in range(H):
            g = h // (H // G)
            q = torch.cat([q_nope[q0:q0 + nq, h], q_pe[q0:q0 + nq, h]], dim=-1).double()
            k = torch.cat([k_nope[k0:k0 + nk, g], k_pe[k0:k0 + nk]], dim=-1).double()
            val = v[k0:k0 + nk, g].double()
            sees = torch.arange(nk)[None, :] <= torch.arange(nq)[:, None] + (nk - nq)
            s = scale * (q @ k.T)
            ds = scale * 192 * SUM * torch.where(sees, q.abs() @ k.abs().T, torch.zeros(1, dtype=torch.float64))
            s = torch.where(sees, s, torch.full_like(s, float("-inf")))
            live = sees.any(dim=-1)
            if not live.any():
                continue
            ds = ds.amax(dim=-1)[live]
            sl = s[live]
            p = torch.softmax(sl, dim=-1)
            o, l = p @ val, torch.logsumexp(sl, dim=-1)
            idx = torch.arange(q0, q0 + nq)[live]
            out[idx, h], lse[idx, h] = o, l
            rel = torch.expm1(4 * ds) + 2.0 ** -20 + nk * SUM
            out_tol[idx, h] = (BF16 + rel)[:, None] * (p @ val.abs()) + BF16 * o.abs()
            lse_tol[idx, h] = 2 * ds + (nk + 8) * SUM + 2.0 ** -20 + 8 * FP32 * (l.abs() + sl.amax(dim=-1).abs())
        q0, k0 = q0 + nq, k0 + nk
    return out, lse, out_tol, lse_tol


def worst(got, ref, tol):
    """Largest error in units of its bound (NaN counts as infinite)."""
    r = (got.double().cpu() - ref).abs() / tol.clamp_min(1e-30)
    r = torch.where(torch.isnan(r), torch.full_like(r, float("inf")), r)
    return float(r.max()) if r.numel() else 0.0

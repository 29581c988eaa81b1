"""Cases of the packed-prompt operators: reading cached rows back
(cache_read), expanding latents to per-head keys and values (expand_kv) and
causal attention over packed prompts (prompt_attention).

``run`` computes a case in its plain form (elementary torch operations in
fp32, rounded once at the end) or, with ``own`` set, through the package's
entry points.  All inputs are seeded random draws.
"""
import math

import torch

own = False

LATENT, ROPE, NOPE, VDIM = 512, 64, 128, 128
SCALE = 1.0 / math.sqrt(NOPE + ROPE)


# ----- sequence lengths as text: "512*4" is four times 512, "1,93" is two ----
def _lens(text):
    out = []
    for part in text.split(","):
        n, _, times = part.partition("*")
        out += [int(n)] * (int(times) if times else 1)
    return out


def _text(lens):
    return ",".join(str(n) for n in lens)


def _cu(lens, device):
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    return torch.tensor(cu, dtype=torch.int32, device=device)


# ----- cases -------------------------------------------------------------------
def _read(name, fmt, page, lens, starts):
    return {"name": name, "op": "read", "format": fmt, "page": page, "lens": lens, "starts": starts}


def _expand(name, rows, heads):
    return {"name": name, "op": "expand", "rows": rows, "heads": heads}


def _attn(name, heads, kv_heads, q_lens, k_lens):
    return {"name": name, "op": "attn", "heads": heads, "kv_heads": kv_heads, "q_lens": q_lens, "k_lens": k_lens}


def listed():
    return [
        # the cached prefix of one short conversation, re-read before its next chunk
        _read("read_bf16_37rows", "bf16", 16, "37", "0"),
        # the histories of a ragged INT8 batch, read whole before a packed prompt step
        _read("read_int8_ragged", "int8", 64,
              "8192,1,5021,777,64,4095,8191,63,2049,6000,129,7313,1500,8000,17,3333,"
              "8192,4811,910,65,128,7777,2600,5555,31,6411,1023,4500,8100,2222,350,7000", "0*32"),
        # the last 4,000-odd rows of long FP8 contexts (a window of every sequence)
        _read("read_fp8_windows", "fp8", 128, "4001*24,4097*24", "28767*24,12291*24"),
        # one short prompt's new latents
        _expand("expand_h16_77rows", 77, 16),
        # four sequences of 8,192 cached and 512 new tokens
        _expand("expand_h16_34816rows", 34816, 16),
        # an odd row count at 128 heads
        _expand("expand_h128_5003rows", 5003, 128),
        # one short prompt: latency
        _attn("attn_h16_93", 16, 16, "93", "93"),
        # a packed batch of ragged prompts
        _attn("attn_h16_ragged", 16, 16,
              "1,2048,93,511,1300,128,17,1999,640,256,1024,350,77,1601,900,5,1750,129,420,2000,33,700,1111,255",
              "1,2048,93,511,1300,128,17,1999,640,256,1024,350,77,1601,900,5,1750,129,420,2000,33,700,1111,255"),
        # one long prompt
        _attn("attn_h16_16384", 16, 16, "16384", "16384"),
        # a 512-token chunk of four sequences after 8,192 cached tokens each
        _attn("attn_h16_chunk512", 16, 16, "512*4", "8704*4"),
        # 128 query heads over 8 key/value heads, odd lengths
        _attn("attn_h128_kv8", 128, 8, "4093,1027,2501,333", "4093,1027,2501,333"),
        # a few new tokens of two sequences behind long histories
        _attn("attn_h16_tail", 16, 16, "19,7", "32768,20011"),
    ]


def _log_uniform(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["read", "expand", "attn", "attn"])
    if op == "read":
        fmt, page = rng.choice(["bf16", "int8", "fp8"]), rng.choice([16, 32, 64, 128])
        batch = _log_uniform(rng, 1, 64)
        longest = max(1, min(8192, 180000 // batch))
        lens = [_log_uniform(rng, 1, longest) for _ in range(batch)]
        if rng.random() < 0.5:
            starts = [0] * batch
        else:
            starts = [rng.randrange(0, 4097) for _ in range(batch)]
        return _read("", fmt, page, _text(lens), _text(starts))
    if op == "expand":
        heads = rng.choice([16, 32, 64, 128])
        return _expand("", _log_uniform(rng, 1, 34816 * 16 // heads), heads)
    heads = rng.choice([16, 16, 32, 64, 128])
    kv_heads = heads // rng.choice([1, 1, 2, 4, 8, heads])
    batch = _log_uniform(rng, 1, 32)
    longest = max(16, int(16384 / math.sqrt(batch * heads / 16)))
    q_lens = [_log_uniform(rng, 1, longest) for _ in range(batch)]
    history = rng.choice(["none", "none", "short", "long"])
    if history == "none":
        k_lens = list(q_lens)
    else:
        top = 512 if history == "short" else min(2 * longest, max(64, (1 << 21) // (kv_heads * batch)))
        k_lens = [n + rng.randrange(0, top + 1) for n in q_lens]
    if history == "long":  # a chunk of each sequence, not its whole prompt
        short = [max(1, n // 8) for n in q_lens]
        k_lens = [k - n + s for k, n, s in zip(k_lens, q_lens, short)]
        q_lens = short
    return _attn("", heads, kv_heads, _text(q_lens), _text(k_lens))


def work(case):
    if case["op"] == "read":
        lens, starts = _lens(case["lens"]), _lens(case["starts"])
        rows, page = sum(lens), case["page"]
        stored = {"bf16": 1152, "int8": 584, "fp8": 580}[case["format"]]
        pages = sum((s + n - 1) // page - s // page + 1 for n, s in zip(lens, starts))
        return {"bytes": rows * (stored + 1152) + 4 * pages + 4 * (2 * len(lens) + 1),
                "flops": 0 if case["format"] == "bf16" else 2 * 576 * rows}
    if case["op"] == "expand":
        n, h = case["rows"], case["heads"]
        return {"bytes": 2 * (n * LATENT + h * (NOPE + VDIM) * LATENT + n * h * (NOPE + VDIM)),
                "flops": 2 * n * h * (NOPE + VDIM) * LATENT}
    q, k = _lens(case["q_lens"]), _lens(case["k_lens"])
    h, g = case["heads"], case["kv_heads"]
    # query i of a sequence sees i + 1 + (keys - queries) keys
    seen = sum(nq * (nk - nq) + nq * (nq + 1) // 2 for nq, nk in zip(q, k))
    nq, nk = sum(q), sum(k)
    return {"bytes": nq * h * (2 * (NOPE + ROPE + VDIM) + 4) + nk * (2 * g * (NOPE + VDIM) + 2 * ROPE)
            + 8 * (len(q) + 1),
            "flops": 2 * h * seen * (NOPE + ROPE + VDIM)}


# ----- inputs --------------------------------------------------------------------
def _bf16(shape, std, g):
    return (torch.randn(shape, generator=g, device="cuda", dtype=torch.float32) * std).to(torch.bfloat16)


def _inputs(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    if case["op"] == "read":
        lens, starts, page = _lens(case["lens"]), _lens(case["starts"]), case["page"]
        need = [(s + n + page - 1) // page for n, s in zip(lens, starts)]
        total = sum(need) + 3
        order = torch.randperm(total, generator=g, device="cuda").to(torch.int32)
        table = torch.full((len(lens), max(need)), -1, dtype=torch.int32, device="cuda")
        at = 0
        for b, n in enumerate(need):
            table[b, :n] = order[at:at + n]
            at += n
        s = {"case": case, "table": table, "cu": _cu(lens, "cuda"), "rows": sum(lens),
             "starts": torch.tensor(starts, dtype=torch.int32, device="cuda"), "scale": None}
        shape = (total, page, LATENT + ROPE)
        if case["format"] == "bf16":
            s["cache"] = _bf16(shape, 1.0, g)
        elif case["format"] == "int8":
            # codes of N(0, 1) rows: scales near 6.5 / 255, zero points near 0
            scale = torch.rand(shape[:2], generator=g, device="cuda") * 0.008 + 0.022
            zero = torch.randint(-12, 13, shape[:2], generator=g, device="cuda").float()
            x = torch.randn(shape, generator=g, device="cuda")
            x.div_(scale[..., None]).round_().add_(zero[..., None]).clamp_(-128, 127)
            s["cache"], s["scale"] = x.to(torch.int8), torch.stack([scale, zero], dim=-1).contiguous()
        else:
            # codes of N(0, 1) rows: the largest magnitude near 3.3 maps to 448
            scale = torch.rand(shape[:2], generator=g, device="cuda") * 0.0015 + 0.0066
            x = torch.randn(shape, generator=g, device="cuda")
            x.div_(scale[..., None]).clamp_(-448, 448)
            s["cache"], s["scale"] = x.to(torch.float8_e4m3fn).view(torch.uint8), scale
        return s
    if case["op"] == "expand":
        h = case["heads"]
        return {"case": case, "c_kv": _bf16((case["rows"], LATENT), 1.0, g),
                "W_UK": _bf16((h, NOPE, LATENT), 0.02, g), "W_UV": _bf16((h, VDIM, LATENT), 0.02, g)}
    q, k, h, kv = _lens(case["q_lens"]), _lens(case["k_lens"]), case["heads"], case["kv_heads"]
    nq, nk = sum(q), sum(k)
    # scores with a standard deviation of 1.5; values with a mean per head and
    # dimension, so that averages over long contexts do not vanish
    v = torch.randn((nk, kv, VDIM), generator=g, device="cuda")
    v += 0.5 * torch.randn((1, kv, VDIM), generator=g, device="cuda")
    return {"case": case, "q_lens": q, "k_lens": k, "cu_q": _cu(q, "cuda"), "cu_k": _cu(k, "cuda"),
            "q_nope": _bf16((nq, h, NOPE), 1.5, g), "q_pe": _bf16((nq, h, ROPE), 1.5, g),
            "k_nope": _bf16((nk, kv, NOPE), 1.0, g), "k_pe": _bf16((nk, ROPE), 1.0, g),
            "v": v.to(torch.bfloat16)}


def prepare(case, seed):
    s = _inputs(case, seed)
    if own:
        import mla_decode_attention_paged_gb300 as mla
        s["mla"] = mla
        if case["op"] == "read":
            s["dims"] = mla.dims(16, case["page"], int8=case["format"] == "int8", fp8=case["format"] == "fp8")
            s["c_kv"] = torch.empty((s["rows"], LATENT), dtype=torch.bfloat16, device="cuda")
            s["k_pe"] = torch.empty((s["rows"], ROPE), dtype=torch.bfloat16, device="cuda")
        elif case["op"] == "expand":
            s["dims"] = mla.dims(case["heads"], 64)
            s["k_nope"] = torch.empty((case["rows"], case["heads"], NOPE), dtype=torch.bfloat16, device="cuda")
            s["v"] = torch.empty((case["rows"], case["heads"], VDIM), dtype=torch.bfloat16, device="cuda")
        else:
            s["dims"] = mla.dims(case["heads"], 64)
            nq = s["q_nope"].shape[0]
            s["out"] = torch.empty((nq, case["heads"], VDIM), dtype=torch.bfloat16, device="cuda")
            s["lse"] = torch.empty((nq, case["heads"]), dtype=torch.float32, device="cuda")
            s["workspace"] = torch.empty(mla.prompt_attention_workspace_size(s["dims"], len(s["q_lens"]), nq),
                                         dtype=torch.uint8, device="cuda")
    return s


# ----- one pass --------------------------------------------------------------------
def run(state):
    op = state["case"]["op"]
    if op == "read":
        return _run_read(state)
    if op == "expand":
        return _run_expand(state)
    return _run_attn(state)


def _run_read(s):
    if own:
        return s["mla"].cache_read(s["dims"], s["cache"], s["scale"], s["table"], s["cu"], starts=s["starts"],
                                   c_kv=s["c_kv"], k_pe=s["k_pe"])
    page = s["case"]["page"]
    r = torch.arange(s["rows"], device="cuda", dtype=torch.int32)
    b = torch.searchsorted(s["cu"], r, right=True) - 1
    pos = s["starts"][b] + r - s["cu"][b]
    row = s["table"][b, (pos // page).long()].long() * page + pos % page
    x = s["cache"].view(-1, LATENT + ROPE)[row]
    if s["case"]["format"] == "int8":
        sz = s["scale"].view(-1, 2)[row]
        x = (sz[:, :1] * (x.float() - sz[:, 1:])).to(torch.bfloat16)
    elif s["case"]["format"] == "fp8":
        x = (s["scale"].view(-1, 1)[row] * x.view(torch.float8_e4m3fn).float()).to(torch.bfloat16)
    return x[:, :LATENT].contiguous(), x[:, LATENT:].contiguous()


def _run_expand(s):
    if own:
        return s["mla"].expand_kv(s["dims"], s["c_kv"], s["W_UK"], s["W_UV"], k_nope=s["k_nope"], v=s["v"])
    c, h = s["c_kv"].float(), s["case"]["heads"]
    k_nope = (c @ s["W_UK"].float().view(-1, LATENT).T).to(torch.bfloat16).view(-1, h, NOPE)
    v = (c @ s["W_UV"].float().view(-1, LATENT).T).to(torch.bfloat16).view(-1, h, VDIM)
    return k_nope, v


def _run_attn(s):
    if own:
        return s["mla"].prompt_attention(s["dims"], s["q_nope"], s["q_pe"], s["k_nope"], s["k_pe"], s["v"],
                                         s["cu_q"], s["cu_k"], SCALE, workspace=s["workspace"], out=s["out"],
                                         lse_out=s["lse"])
    h, kv = s["case"]["heads"], s["case"]["kv_heads"]
    group = h // kv
    out = torch.empty_like(s["q_nope"])
    lse = torch.empty(out.shape[:2], dtype=torch.float32, device="cuda")
    q0 = k0 = 0
    for nq, nk in zip(s["q_lens"], s["k_lens"]):
        step = max(1, (1 << 28) // (h * nk))  # query rows whose scores fit 1 GB
        for i in range(0, nq, step):
            m = min(step, nq - i)
            n = nk - nq + i + m  # keys that the last of these rows sees
            # [kv, group * m, .]: the query heads of a key/value head together
            qn = s["q_nope"][q0 + i:q0 + i + m].float().view(m, kv, group, NOPE).permute(1, 2, 0, 3).reshape(kv, -1, NOPE)
            qp = s["q_pe"][q0 + i:q0 + i + m].float().view(m, kv, group, ROPE).permute(1, 2, 0, 3).reshape(kv, -1, ROPE)
            kn = s["k_nope"][k0:k0 + n].float().permute(1, 2, 0)
            x = torch.matmul(qn, kn)
            x += torch.matmul(qp, s["k_pe"][k0:k0 + n].float().T)
            x *= SCALE
            sees = torch.arange(n, device="cuda") <= (torch.arange(m, device="cuda") + (nk - nq + i))[:, None]
            x.view(kv, group, m, n).masked_fill_(~sees, float("-inf"))
            top = x.amax(dim=-1, keepdim=True)
            x -= top
            x.exp_()
            total = x.sum(dim=-1, keepdim=True)
            o = torch.matmul(x, s["v"][k0:k0 + n].float().transpose(0, 1)) / total
            out[q0 + i:q0 + i + m] = o.view(kv, group, m, VDIM).permute(2, 0, 1, 3).reshape(m, h, VDIM).to(torch.bfloat16)
            lse[q0 + i:q0 + i + m] = (top + total.log()).view(kv, group, m).permute(2, 0, 1).reshape(m, h)
        q0, k0 = q0 + nq, k0 + nk
    return out, lse


# ----- the definitions in 64 bits ---------------------------------------------------
def exact(case, seed):
    s = _inputs(case, seed)
    if case["op"] == "read":
        parts, page = [], case["page"]
        for b, (n, start) in enumerate(zip(_lens(case["lens"]), _lens(case["starts"]))):
            pages = s["table"][b, start // page:(start + n + page - 1) // page].long()
            rows = s["cache"][pages].flatten(0, 1)[start % page:start % page + n]
            if case["format"] == "fp8":
                rows = rows.view(torch.float8_e4m3fn)
            rows = rows.double()
            if case["format"] != "bf16":
                p = s["scale"][pages].flatten(0, 1)[start % page:start % page + n].double()
                rows = (rows - p[:, 1:2]) * p[:, 0:1] if case["format"] == "int8" else rows * p[:, None]
            parts.append(rows)
        x = torch.cat(parts)
        return x[:, :LATENT], x[:, LATENT:]
    if case["op"] == "expand":
        c = s["c_kv"].double()
        return (torch.einsum("nc,hdc->nhd", c, s["W_UK"].double()),
                torch.einsum("nc,hdc->nhd", c, s["W_UV"].double()))
    h, kv = case["heads"], case["kv_heads"]
    if work(case)["flops"] > 4e12:  # past about ten seconds in 64 bits
        return None
    outs, lses, q0, k0 = [], [], 0, 0
    for nq, nk in zip(s["q_lens"], s["k_lens"]):
        out = torch.empty((nq, h, VDIM), dtype=torch.float64, device="cuda")
        lse = torch.empty((nq, h), dtype=torch.float64, device="cuda")
        q = torch.cat([s["q_nope"], s["q_pe"]], dim=-1)[q0:q0 + nq].double()
        pe = s["k_pe"][k0:k0 + nk].double()
        for head in range(h):
            g = head // (h // kv)
            k = torch.cat([s["k_nope"][k0:k0 + nk, g].double(), pe], dim=-1)
            value = s["v"][k0:k0 + nk, g].double()
            for i in range(0, nq, 4096):
                last = min(nq, i + 4096)
                n = nk - nq + last
                sc = SCALE * (q[i:last, head] @ k[:n].T)
                sc += torch.full_like(sc, float("-inf")).triu(nk - nq + i + 1)
                lse[i:last, head] = torch.logsumexp(sc, dim=-1)
                out[i:last, head] = torch.softmax(sc, dim=-1) @ value[:n]
        outs.append(out)
        lses.append(lse)
        q0, k0 = q0 + nq, k0 + nk
    return torch.cat(outs), torch.cat(lses)

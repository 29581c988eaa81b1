"""Cases of the 4-bit latent cache: writing tokens into it (cache_append, with
the position rotation and the quantisation on the way), reading rows back out
of it (cache_read) and decoding over it (decode, decode_multi, decode_sparse).

A cached row is 576 values -- the 512-wide latent and the rotated 64-wide RoPE
key -- as E2M1 codes (magnitudes 0, 0.5, 1, 1.5, 2, 3, 4, 6) with a
power-of-two scale for every 32 values, in 320 bytes:
  bytes 0 .. 287    72 little-endian words of 8 codes.  Word w, i in 0 .. 3:
                    value 8w + i has its magnitude's code in bits 4i .. 4i + 2
                    and its sign in bit 8i + 7; value 8w + 4 + i has them in
                    bits 16 + 4i .. 16 + 4i + 2 and in bit 8i + 3
  bytes 288 .. 305  the scales of values 32j .. 32j + 31: 2^(byte - 127)
  bytes 306 .. 319  zero
A block with largest magnitude a gets the smallest power of two s with
a <= 6 s, and each value the nearest code to x / s, ties to the even code.

``run`` computes a case in its plain form (elementary torch operations) or,
with ``own`` set, through the package's entry points.  All inputs are seeded
random draws.
"""
import math

import torch

own = False

LATENT, ROPE, NOPE, VDIM, ROW = 512, 64, 128, 128, 576
ROW_BYTES, CODE_BYTES, BLOCKS = 320, 288, 18
SCALE = 1.0 / math.sqrt(NOPE + ROPE)
THETA = 10000.0


# ----- lengths as text: "512*4" is four times 512, "1,93" is two --------------
def _lens(text):
    out = []
    for part in text.split(","):
        n, _, times = part.partition("*")
        out += [int(n)] * (int(times) if times else 1)
    return out


def _text(lens):
    return ",".join(str(n) for n in lens)


# ----- cases -------------------------------------------------------------------
def _store(name, page, lens, starts):
    return {"name": name, "op": "store", "page": page, "lens": lens, "starts": starts}


def _read(name, page, lens, starts):
    return {"name": name, "op": "read", "page": page, "lens": lens, "starts": starts}


def _decode(name, heads, page, lens, q_len=1, top_k=0):
    return {"name": name, "op": "decode", "heads": heads, "page": page, "lens": lens, "q_len": q_len, "top_k": top_k}


def listed():
    return [
        # one decode step's new tokens, and the rows they became
        _store("store_32_tokens", 64, "1*32", "32767*8,1,4095,63,64,20011,777,9000,131071,5,12290*15"),
        # a 512-token chunk of four sequences behind 8,192 cached tokens
        _store("store_4x512", 64, "512*4", "8192*4"),
        # whole prompts of odd lengths
        _store("store_prompts", 64, "8191,5003,4097,129,1,6001,3333,7919,143", "0*9"),
        # the histories of a ragged batch, read before a packed prompt step
        _read("read_ragged", 16,
              "8192,1,5021,777,64,4095,8191,63,2049,6000,129,7313,1500,8000,17,3333,"
              "8192,4811,910,65,128,7777,2600,5555,31,6411,1023,4500,8100,2222,350,7000", "0*32"),
        # the last 4,000-odd rows of long contexts
        _read("read_windows", 128, "4001*24,4097*24", "28767*24,12291*24"),
        # one short conversation: latency
        _decode("decode_h16_93", 16, 16, "93"),
        # a batch of 32 sequences of 32,768 tokens
        _decode("decode_h16_32x32768", 16, 64, "32768*32"),
        # two contexts of a million tokens
        _decode("decode_h16_2x1m", 16, 64, "1048576*2"),
        # odd lengths, short and long together, at 32 heads
        _decode("decode_h32_ragged", 32, 32,
                "1,40001,93,5111,13007,128,17,1999,6403,25601,10247,350,77,16011,900,50021,1751,129,42013,2000,33,700,11113,255"),
        # 128 heads over sequences of 8,192 tokens
        _decode("decode_h128_128x8192", 128, 64, "8192*128"),
        # four drafted tokens of each sequence verified at once
        _decode("decode_h16_4tokens", 16, 64, "32768*32", q_len=4),
        # 2,048 selected tokens of each sequence
        _decode("decode_h16_top2048", 16, 64, "32768*32", top_k=2048),
    ]


def _log_uniform(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["store", "read", "decode", "decode", "decode", "multi", "sparse"])
    page = rng.choice([16, 32, 64, 128])
    if op in ("store", "read"):
        batch = _log_uniform(rng, 1, 64)
        longest = max(1, min(8192, (34000 if op == "store" else 180000) // batch))
        lens = [_log_uniform(rng, 1, longest) for _ in range(batch)]
        starts = [0] * batch if rng.random() < 0.5 else [rng.randrange(0, 30001) for _ in range(batch)]
        return (_store if op == "store" else _read)("", page, _text(lens), _text(starts))
    heads = rng.choice([16, 16, 32, 64, 128])
    q_len = rng.randrange(2, 9) if op == "multi" else 1
    batch = _log_uniform(rng, 1, 128)
    # as many tokens as the largest listed case at 16 rows, fewer where every token meets more rows
    total = min(1 << 20, (1 << 27) // (heads * q_len))
    longest = max(q_len, total // batch)
    lens = [_log_uniform(rng, q_len, longest) for _ in range(batch)]
    top_k = _log_uniform(rng, 16, 4096) if op == "sparse" else 0
    return _decode("", heads, page, _text(lens), q_len, top_k)


def work(case):
    lens = _lens(case["lens"])
    if case["op"] != "decode":
        rows, page = sum(lens), case["page"]
        starts = _lens(case["starts"])
        pages = sum((s + n - 1) // page - s // page + 1 for n, s in zip(lens, starts))
        if case["op"] == "read":
            return {"bytes": rows * (CODE_BYTES + BLOCKS + 2 * ROW) + 4 * (pages + 2 * len(lens) + 1), "flops": ROW * rows}
        # the tokens in, the rows out; and the rows in, the values out
        return {"bytes": rows * (2 * ROW + 8 + CODE_BYTES + BLOCKS) + rows * (CODE_BYTES + BLOCKS + 2 * ROW)
                + 4 * (2 * pages + 2 * len(lens) + 1), "flops": 3 * ROW * rows}
    h, t, page, k = case["heads"], case["q_len"], case["page"], case["top_k"]
    read = [min(k, n) if k else n for n in lens]
    # query i of t sees the tokens up to its own position
    seen = sum(n if k else t * n - t * (t - 1) // 2 for n in read)
    rows = len(lens) * t * h
    index = 4 * k * len(lens) + 4 * sum(read) if k else 4 * sum((n + page - 1) // page for n in lens)
    return {"bytes": sum(read) * (CODE_BYTES + BLOCKS) + index + rows * 2 * (NOPE + ROPE + VDIM)
            + 2 * h * (NOPE + VDIM) * LATENT + 4 * len(lens),
            "flops": 2 * h * seen * (ROW + LATENT) + 2 * rows * (NOPE + VDIM) * LATENT}


# ----- the cached rows, plain -----------------------------------------------------
def _codes_of(x, s):
    """Codes 0 .. 7 of |x| / s (at most 6): the nearest magnitude, ties to the even code."""
    y = x.abs() / s
    code = (y > 0.25).to(torch.int32)
    for edge, tie_up in ((0.75, True), (1.25, False), (1.75, True), (2.5, False), (3.5, True), (5.0, False)):
        code += (y >= edge) if tie_up else (y > edge)
    return code


def _pack(x):
    """Rows [n, 576] of bf16 values (as fp32) to packed rows uint8 [n, 320]."""
    n = x.shape[0]
    x = x.view(n, BLOCKS, 32)
    top = x.abs().amax(dim=-1, keepdim=True)
    m, e = torch.frexp(top)  # top = m 2^e, m in [0.5, 1): the scale's exponent is e - 3, one more if m > 0.75
    e = (e - 3 + (m > 0.75)).clamp_(min=-127)
    e = torch.where(top > 0, e, torch.full_like(e, -127))
    code = _codes_of(x.double(), torch.exp2(e.double())).view(n, 72, 8)
    sign = torch.signbit(x).to(torch.int32).view(n, 72, 8)
    word = torch.zeros((n, 72), dtype=torch.int32, device=x.device)
    for i in range(8):
        word |= code[:, :, i] << (4 * i)
        word |= sign[:, :, i] << (8 * i + 7 if i < 4 else 8 * (i - 4) + 3)
    out = torch.zeros((n, ROW_BYTES), dtype=torch.uint8, device=x.device)
    out[:, :CODE_BYTES] = word.view(torch.uint8).view(n, CODE_BYTES)
    out[:, CODE_BYTES:CODE_BYTES + BLOCKS] = (e + 127).to(torch.uint8).view(n, BLOCKS)
    return out


def _values(rows):
    """Packed rows uint8 [n, 320] to fp32 values [n, 576]."""
    n = rows.shape[0]
    word = rows[:, :CODE_BYTES].contiguous().view(torch.int32)[:, :, None]
    i = torch.arange(8, dtype=torch.int32, device=rows.device)
    mag = (word >> (4 * i)) & 7
    negative = (word >> torch.where(i < 4, 8 * i + 7, 8 * i - 29)) & 1
    value = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], device=rows.device)[mag]
    value = torch.where(negative == 1, -value, value).view(n, BLOCKS, 32)
    scale = torch.exp2(rows[:, CODE_BYTES:CODE_BYTES + BLOCKS].double() - 127.0).float()
    return (value * scale[:, :, None]).view(n, ROW)


def _rotate(k_pe, positions):
    """RoPE on pairs (2j, 2j + 1) at the given positions, in 64 bits, rounded to bf16."""
    j = torch.arange(ROPE // 2, device=k_pe.device, dtype=torch.float64)
    angle = positions.double()[:, None] * torch.pow(THETA, -2.0 * j / ROPE)
    c, s = torch.cos(angle), torch.sin(angle)
    x, y = k_pe.double()[:, 0::2], k_pe.double()[:, 1::2]
    return torch.stack([x * c - y * s, x * s + y * c], dim=-1).view(-1, ROPE).to(torch.bfloat16)


# ----- inputs --------------------------------------------------------------------
def _bf16(shape, std, g):
    return (torch.randn(shape, generator=g, device="cuda", dtype=torch.float32) * std).to(torch.bfloat16)


def _table(ends, page, g):
    """Block table of sequences of these lengths over a shuffled pool, and the pool's pages."""
    need = [(n + page - 1) // page for n in ends]
    total = sum(need) + 3
    order = torch.randperm(total, generator=g, device="cuda").to(torch.int32)
    table = torch.full((len(ends), max(need)), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    return table, total


def _cache(pages, page, g):
    """A pool of rows of N(0, 1) values, each page's rows at a magnitude of their own."""
    cache = torch.empty((pages, page, ROW_BYTES), dtype=torch.uint8, device="cuda")
    step = max(1, (1 << 18) // page)
    for p in range(0, pages, step):
        n = min(step, pages - p)
        x = torch.randn((n, page, ROW), generator=g, device="cuda")
        x *= torch.rand((n, 1, 1), generator=g, device="cuda") * 0.4 + 0.8
        cache[p:p + n] = _pack(x.to(torch.bfloat16).float().view(-1, ROW)).view(n, page, ROW_BYTES)
    return cache


def _inputs(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    lens = _lens(case["lens"])
    s = {"case": case, "lens": lens}
    if case["op"] != "decode":
        starts = _lens(case["starts"])
        cu = [0]
        for n in lens:
            cu.append(cu[-1] + n)
        s["table"], pages = _table([a + n for a, n in zip(starts, lens)], case["page"], g)
        s["cu"] = torch.tensor(cu, dtype=torch.int32, device="cuda")
        s["starts"], s["rows"] = torch.tensor(starts, dtype=torch.int32, device="cuda"), cu[-1]
        if case["op"] == "read":
            s["cache"] = _cache(pages, case["page"], g)
            return s
        s["cache"] = torch.zeros((pages, case["page"], ROW_BYTES), dtype=torch.uint8, device="cuda")
        of = torch.repeat_interleave(torch.arange(len(lens), device="cuda"), torch.tensor(lens, device="cuda"))
        s["seq_ids"] = of.to(torch.int32)
        s["positions"] = torch.arange(cu[-1], device="cuda", dtype=torch.int32) - s["cu"][of] + s["starts"][of]
        # latents of unit size, keys of the rotation with a few large channels
        s["new_c_kv"] = _bf16((cu[-1], LATENT), 1.0, g)
        s["new_k_pe"] = (_bf16((cu[-1], ROPE), 1.0, g).float() * (1.0 + 3.0 * torch.rand(ROPE, generator=g, device="cuda"))).to(torch.bfloat16)
        return s
    h, t, b = case["heads"], case["q_len"], len(lens)
    s["table"], pages = _table(lens, case["page"], g)
    s["cache"] = _cache(pages, case["page"], g)
    s["seq_lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    s["W_UK"], s["W_UV"] = _bf16((h, NOPE, LATENT), 0.02, g), _bf16((h, VDIM, LATENT), 0.02, g)
    # scores with a standard deviation of 1.5
    tokens = (b, h) if t == 1 else (b, t, h)
    s["q_nope"], s["q_pe"] = _bf16(tokens + (NOPE,), 2.2, g), _bf16(tokens + (ROPE,), 2.2, g)
    if case["top_k"]:
        index = torch.full((b, case["top_k"]), -1, dtype=torch.int32, device="cuda")
        for i, n in enumerate(lens):
            pick = torch.randperm(n, generator=g, device="cuda")[:case["top_k"]]
            index[i, :pick.numel()] = pick.to(torch.int32)
        s["index"] = index
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    if own:
        import mla_decode_attention_paged_gb300 as mla
        s["mla"] = mla
        if case["op"] != "decode":
            s["dims"] = mla.dims(16, case["page"], fp4=True)
            s["c_kv"] = torch.empty((s["rows"], LATENT), dtype=torch.bfloat16, device="cuda")
            s["k_pe"] = torch.empty((s["rows"], ROPE), dtype=torch.bfloat16, device="cuda")
        else:
            d = s["dims"] = mla.dims(case["heads"], case["page"], fp4=True)
            b = len(s["lens"])
            size = (mla.decode_sparse_workspace_size(d, b, case["top_k"]) if case["top_k"]
                    else mla.decode_multi_workspace_size(d, b, case["q_len"]))
            s["workspace"] = torch.empty(size, dtype=torch.uint8, device="cuda")
            s["out"] = torch.empty(s["q_nope"].shape[:-1] + (VDIM,), dtype=torch.bfloat16, device="cuda")
    return s


# ----- one pass --------------------------------------------------------------------
def run(state):
    op = state["case"]["op"]
    if op == "decode":
        return _run_decode(state)
    return _run_store(state) if op == "store" else _run_read(state)


def _rows_of(s, b, pos):
    """Row in the pool of each position of sequences b."""
    page = s["case"]["page"]
    return s["table"][b, (pos // page).long()].long() * page + pos % page


def _run_read(s):
    if own:
        return s["mla"].cache_read(s["dims"], s["cache"], None, s["table"], s["cu"], starts=s["starts"],
                                   c_kv=s["c_kv"], k_pe=s["k_pe"])
    r = torch.arange(s["rows"], device="cuda", dtype=torch.int32)
    b = torch.searchsorted(s["cu"], r, right=True) - 1
    row = _rows_of(s, b, s["starts"][b] + r - s["cu"][b])
    x = _values(s["cache"].view(-1, ROW_BYTES)[row]).to(torch.bfloat16)
    return x[:, :LATENT].contiguous(), x[:, LATENT:].contiguous()


def _run_store(s):
    if own:
        s["mla"].cache_append(s["dims"], s["cache"], None, s["table"], s["seq_ids"], s["positions"], s["new_c_kv"],
                              s["new_k_pe"], THETA)
        return _run_read(s)
    x = torch.cat([s["new_c_kv"], _rotate(s["new_k_pe"], s["positions"])], dim=-1).float()
    s["cache"].view(-1, ROW_BYTES)[_rows_of(s, s["seq_ids"].long(), s["positions"])] = _pack(x)
    return _run_read(s)


def _run_decode(s):
    case, h, t = s["case"], s["case"]["heads"], s["case"]["q_len"]
    if own:
        mla, out = s["mla"], s["out"]
        args = (s["dims"], s["q_nope"], s["q_pe"], s["cache"], None, s["table"], s["seq_lens"])
        more = dict(workspace=s["workspace"], out=out, want_lse=False)
        if case["top_k"]:
            mla.decode_sparse(*args, s["index"], s["W_UK"], s["W_UV"], SCALE, **more)
        elif t > 1:
            mla.decode_multi(*args, s["W_UK"], s["W_UV"], SCALE, **more)
        else:
            mla.decode(*args, s["W_UK"], s["W_UV"], SCALE, **more)
        return out
    b = len(s["lens"])
    q_lat = torch.einsum("bthd,hdc->bthc", s["q_nope"].float().view(b, t, h, NOPE), s["W_UK"].float())
    q = torch.cat([q_lat, s["q_pe"].float().view(b, t, h, ROPE)], dim=-1).view(b, t * h, ROW)
    o_lat = torch.empty((b, t * h, LATENT), device="cuda")
    for i, n in enumerate(s["lens"]):
        pos = s["index"][i, :min(n, case["top_k"])] if case["top_k"] else torch.arange(n, device="cuda")
        x = _values(s["cache"].view(-1, ROW_BYTES)[_rows_of(s, i, pos)])
        score = (q[i] @ x.T) * SCALE
        if t > 1:  # query j stands at position n - t + j
            last = torch.arange(n - t, n, device="cuda")
            score.view(t, h, n).masked_fill_((pos > last[:, None])[:, None, :], float("-inf"))
        weight = (score - score.amax(dim=-1, keepdim=True)).exp_()
        o_lat[i] = (weight @ x[:, :LATENT]) / weight.sum(dim=-1, keepdim=True)
    out = torch.einsum("bthc,hdc->bthd", o_lat.view(b, t, h, LATENT), s["W_UV"].float())
    return out.to(torch.bfloat16).view(s["q_nope"].shape[:-1] + (VDIM,))


# ----- the definitions in 64 bits ---------------------------------------------------
def _unpack64(rows):
    """Packed rows to their values in 64 bits, nibble by nibble."""
    n = rows.shape[0]
    b = rows[:, :CODE_BYTES]
    nib = torch.stack([b & 15, b >> 4], dim=-1).view(n, 72, 8)
    order = torch.tensor([1, 3, 5, 7, 0, 2, 4, 6], device=rows.device)  # the nibble that has value i's sign
    mag, sign = (nib & 7).long(), (nib >> 3)[:, :, order].double()
    half = torch.tensor([0, 1, 2, 3, 4, 6, 8, 12], dtype=torch.float64, device=rows.device)[mag] * (0.5 - sign)
    scale = torch.exp2(rows[:, CODE_BYTES:CODE_BYTES + BLOCKS].double() - 127.0)
    return (half.view(n, BLOCKS, 32) * scale[:, :, None]).view(n, ROW)


def _exact_read(s):
    parts, page = [], s["case"]["page"]
    for b, (n, start) in enumerate(zip(s["lens"], _lens(s["case"]["starts"]))):
        pages = s["table"][b, start // page:(start + n + page - 1) // page].long()
        parts.append(s["cache"][pages].flatten(0, 1)[start % page:start % page + n])
    return _unpack64(torch.cat(parts))


def _exact_store(s):
    """What the rows stand for: the nearest code's value times the block's scale."""
    x = torch.empty((s["rows"], ROW), dtype=torch.float64, device="cuda")
    x[:, :LATENT] = s["new_c_kv"].double()
    z = torch.view_as_complex(s["new_k_pe"].double().view(-1, ROPE // 2, 2))
    freq = torch.exp(torch.arange(0, ROPE, 2, dtype=torch.float64, device="cuda") * (-math.log(THETA) / ROPE))
    turn = s["positions"].double()[:, None] * freq
    z = torch.view_as_real(z * torch.polar(torch.ones_like(turn), turn)).view(-1, ROPE)
    x[:, LATENT:] = z.to(torch.bfloat16).double()
    x = x.view(-1, BLOCKS, 32)
    scale = torch.exp2(torch.ceil(torch.log2(x.abs().amax(dim=-1, keepdim=True) / 6.0)).clamp_(min=-127.0))
    y = x / scale
    # the step between neighbours: a half below 2, one below 4, two above; round() takes ties to even multiples
    step = torch.where(y.abs() < 2.0, 0.5, torch.where(y.abs() < 4.0, 1.0, 2.0))
    return ((y / step).round() * step * scale).view(-1, ROW)


def exact(case, seed):
    s = _inputs(case, seed)
    if case["op"] != "decode":
        x = _exact_store(s) if case["op"] == "store" else _exact_read(s)
        return x[:, :LATENT], x[:, LATENT:]
    h, t, page, b = case["heads"], case["q_len"], case["page"], len(s["lens"])
    q_nope, q_pe = s["q_nope"].double().view(b, t, h, NOPE), s["q_pe"].double().view(b, t, h, ROPE)
    uk, uv = s["W_UK"].double(), s["W_UV"].double()
    out = torch.zeros((b, t, h, VDIM), dtype=torch.float64, device="cuda")
    for i, n in enumerate(s["lens"]):
        rows = s["cache"][s["table"][i, :(n + page - 1) // page].long()].flatten(0, 1)[:n]
        if case["top_k"]:
            listed_rows = s["index"][i]
            rows = rows[listed_rows[listed_rows >= 0].long()]
        x = _unpack64(rows)
        for j in range(t):
            y = x[:n - t + j + 1] if t > 1 else x
            q = torch.cat([torch.matmul(q_nope[i, j][:, None, :], uk)[:, 0], q_pe[i, j]], dim=-1)
            p = torch.softmax(SCALE * torch.matmul(q, y.T), dim=-1)
            out[i, j] = torch.matmul(uv, torch.matmul(p, y[:, :LATENT])[:, :, None])[:, :, 0]
    return out.view(s["q_nope"].shape[:-1] + (VDIM,))

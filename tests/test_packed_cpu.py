"""CPU-only checks of the packed-prompt entry points: bad arguments are refused
on the host before anything is launched, by the C ABI and by the binding, and
the 64-bit references the GPU tests compare with agree with the fp64 oracle."""
import ctypes

import numpy as np
import pytest
import torch

import mla_decode_attention_paged_gb300 as mla
import oracle as O
import packed_reference as R
from mla_decode_attention_paged_gb300 import build as mla_build
from mla_decode_attention_paged_gb300 import workloads as W

OK, INVALID, UNSUPPORTED, WORKSPACE = (mla.MLA_OK, mla.MLA_ERR_INVALID_ARG, mla.MLA_ERR_UNSUPPORTED,
                                       mla.MLA_ERR_WORKSPACE)
FAKE = ctypes.c_void_p(0x10000)  # never dereferenced: validation fails first


def _at(offset):
    return ctypes.c_void_p(0x10000 + offset)


@pytest.fixture(scope="module")
def lib():
    mla_build.build()
    return mla.load_library()


def _refused(fn, good, changes, status=INVALID):
    for i, value in changes:
        args = list(good)
        args[i] = value
        assert fn(*args) == status, (i, value)


def test_cache_read_refusals(lib):
    d = mla.dims(16, 64)
    #       0                1     2     3  4     5  6  7     8     9   10    11    12    13
    good = [ctypes.byref(d), FAKE, None, 4, FAKE, 2, 8, None, FAKE, 10, FAKE, FAKE, None, None]
    _refused(lib.mla_cache_read, good, [
        (0, None), (1, None), (3, 0), (4, None), (5, 0), (5, -1), (6, 0), (8, None), (9, -1), (10, None), (11, None),
        (1, _at(8)), (4, _at(2)), (7, _at(2)), (8, _at(2)), (10, _at(8)), (11, _at(8)), (12, _at(2))])
    bad = mla.dims(24, 64)
    _refused(lib.mla_cache_read, good, [(0, ctypes.byref(bad))], UNSUPPORTED)
    for kw in ({"int8": True}, {"fp8": True}):  # 1-byte caches need their scales
        _refused(lib.mla_cache_read, good, [(0, ctypes.byref(mla.dims(16, 64, **kw)))])
    none = list(good)
    none[9] = 0
    none[1] = none[10] = none[11] = None
    assert lib.mla_cache_read(*none) == OK  # no rows: nothing to do


def test_expand_refusals(lib):
    d = mla.dims(16, 64)
    #       0                1     2   3     4     5     6     7     8
    good = [ctypes.byref(d), FAKE, 10, FAKE, FAKE, FAKE, FAKE, None, None]
    _refused(lib.mla_expand_kv, good, [
        (0, None), (1, None), (2, -1), (3, None), (4, None), (5, None), (6, None), (1, _at(8)), (3, _at(8)), (4, _at(8)),
        (5, _at(16)), (6, _at(16)), (7, _at(1)), (2, (1 << 26) // 16 + 1)])
    none = [ctypes.byref(d), None, 0, None, None, None, None, None, None]
    assert lib.mla_expand_kv(*none) == OK


def test_prompt_attention_refusals(lib):
    d = mla.dims(16, 64)
    size = lib.mla_prompt_attention_workspace_size(ctypes.byref(d), 3, 100)
    assert size > 0
    #       0                1     2     3    4     5     6     7    8   9     10    11 12                   13
    good = [ctypes.byref(d), FAKE, FAKE, 100, FAKE, FAKE, FAKE, 100, 16, FAKE, FAKE, 3, ctypes.c_float(0.1), FAKE,
            ctypes.c_size_t(size), FAKE, None, None]
    _refused(lib.mla_prompt_attention, good, [
        (0, None), (1, None), (2, None), (3, -1), (4, None), (5, None), (6, None), (7, -1), (8, 0), (8, 3), (8, 32),
        (9, None), (10, None), (11, 0), (11, (1 << 20) + 1), (15, None), (3, (1 << 26) // 16 + 1),
        (7, (1 << 26) // 16 + 1), (1, _at(8)), (2, _at(8)), (4, _at(8)), (5, _at(8)), (6, _at(8)), (9, _at(1)),
        (10, _at(2)), (15, _at(16)), (16, _at(2)), (12, ctypes.c_float(0.0)), (12, ctypes.c_float(-1.0)),
        (12, ctypes.c_float(float("inf"))), (12, ctypes.c_float(float("nan")))])
    _refused(lib.mla_prompt_attention, good, [(13, None), (13, _at(64)), (14, ctypes.c_size_t(size - 1))], WORKSPACE)


def test_prompt_workspace_size(lib):
    d = mla.dims(16, 64)
    f = lib.mla_prompt_attention_workspace_size
    assert f(ctypes.byref(d), 1, 0) > 0
    assert f(ctypes.byref(d), 1, 1) <= f(ctypes.byref(d), 1, 5000) <= f(ctypes.byref(d), 9, 5000)
    assert f(ctypes.byref(d), 0, 10) == 0 and f(ctypes.byref(d), 1, -1) == 0 and f(None, 1, 10) == 0
    assert f(ctypes.byref(d), 1, (1 << 26) // 16 + 1) == 0
    with pytest.raises(mla.MLAError):
        mla.prompt_attention_workspace_size(d, 0, 10)


def test_binding_refuses_host_tensors(lib):
    d = mla.dims(16, 64)
    bf16 = lambda *s: torch.zeros(s, dtype=torch.bfloat16)
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        mla.cache_read(d, bf16(2, 64, 576), None, i32(1, 2), i32(2), n_rows=4)
    with pytest.raises(ValueError, match="CUDA"):
        mla.expand_kv(d, bf16(4, 512), bf16(16, 128, 512), bf16(16, 128, 512))
    with pytest.raises(ValueError, match="CUDA"):
        mla.prompt_attention(d, bf16(4, 16, 128), bf16(4, 16, 64), bf16(4, 16, 128), bf16(4, 64), bf16(4, 16, 128),
                             i32(2), i32(2), 0.1)
    with pytest.raises(TypeError):
        mla.expand_kv(d, [1.0], bf16(16, 128, 512), bf16(16, 128, 512))
    with pytest.raises(ValueError, match="dimensions"):
        mla.expand_kv(d, bf16(4, 8, 512), bf16(16, 128, 512), bf16(16, 128, 512))


@pytest.mark.parametrize("fmt", ["bf16", "int8", "fp8"])
def test_references_agree_with_the_oracle(fmt):
    """Reading, expanding and attending in the references gives the oracle's prefill."""
    g = W.generator(5)
    H, P, T = 16, 16, 5
    lens = torch.tensor([23, 5, 40], dtype=torch.int32)
    table, npg = W.draw_page_table(lens, P, True, g)
    cache, sz = ((W.draw_bf16((npg, P, 576), 1.0, g), None) if fmt == "bf16" else
                 W.draw_int8_cache(npg, P, g) if fmt == "int8" else W.draw_fp8_cache(npg, P, g))
    if sz is not None:
        sz = sz * 0.3
    c_kv, k_pe = W.draw_bf16((3, T, 512), 1.0, g), W.draw_bf16((3, T, 64), 1.0, g)
    qn, qp = W.draw_bf16((3, T, H, 128), 1.0, g), W.draw_bf16((3, T, H, 64), 1.0, g)
    uk, uv = W.draw_bf16((H, 128, 512), 0.02, g), W.draw_bf16((H, 128, 512), 0.02, g)
    f = lambda t: O.bf16_bits_to_f64(W.bf16_to_bits(t))
    cache_o = (W.bf16_to_bits(cache) if fmt == "bf16" else cache.numpy()).copy()
    sz_o = None if sz is None else sz.numpy().copy()
    ref_o, ref_l = O.prefill_chunk(cache_o, sz_o, table.numpy(), lens.numpy(), W.bf16_to_bits(c_kv),
                                   W.bf16_to_bits(k_pe), 10000.0, f(qn), f(qp), f(uk), f(uv), 0.0722, P, fmt == "int8",
                                   **({"fp8": True} if fmt == "fp8" else {}))
    # the cache as the oracle's append left it
    after = torch.from_numpy(cache_o.view(np.int16)).view(torch.bfloat16) if fmt == "bf16" else torch.from_numpy(cache_o)
    rows = R.read_rows(fmt, after, None if sz_o is None else torch.from_numpy(sz_o), table, [0, 23, 28, 68], None, P)
    k, _ = R.expand(rows[:, :512], uk)
    v, _ = R.expand(rows[:, :512], uv)
    out, lse, _, _ = R.attention(qn.view(-1, H, 128), qp.view(-1, H, 64), k, rows[:, 512:], v, [T] * 3, lens.tolist(),
                                 0.0722)
    assert np.abs(out.numpy() - ref_o.reshape(3 * T, H, 128)).max() < 1e-9
    assert np.abs(lse.numpy() - ref_l.reshape(3 * T, H)).max() < 1e-9

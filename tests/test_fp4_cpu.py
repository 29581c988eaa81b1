"""CPU checks of the FP4 cache: the format's plain implementation by hand-worked
rows and bounds, and what the entry points refuse."""
import ctypes

import numpy as np
import pytest
import torch

import fp4_reference as F
import mla_decode_attention_paged_gb300 as mla
from mla_decode_attention_paged_gb300 import build as mla_build

FAKE = ctypes.c_void_p(0x10000)  # never dereferenced: validation fails first


def _at(offset):
    return ctypes.c_void_p(0x10000 + offset)


@pytest.fixture(scope="module")
def lib():
    mla_build.build()
    return mla.load_library()


def _refused(fn, good, changes, status=mla.MLA_ERR_INVALID_ARG):
    for i, value in changes:
        args = list(good)
        args[i] = value
        assert fn(*args) == status, (i, value)


# ----- the format ---------------------------------------------------------------
def test_hand_worked_row():
    x = np.zeros((1, 576))
    x[0, :8] = [6, -6, 0.25, 0.75, -1.25, 1.75, -2.5, 3.5]  # block 0: scale 1; ties go to the even code
    x[0, 31] = -0.0
    x[0, 32:35] = [6.03125, 1, 5]                           # block 1: just above 6, scale 2
    x[0, 64] = 2.0 ** -133                                  # block 2: below the smallest scale's half step
    x[0, 96] = 3.3895313892515355e38                        # block 3: the largest bf16 value
    row = F.encode(x)[0]
    assert list(row[288:292]) == [127, 128, 0, 253] and not row[292:].any()
    word = int.from_bytes(row[:4].tobytes(), "little")
    assert [(word >> (4 * k)) & 7 for k in range(8)] == [7, 7, 0, 2, 2, 4, 4, 6]
    assert [(word >> (8 * k + 7)) & 1 for k in range(4)] == [0, 1, 0, 0]
    assert [(word >> (8 * k + 3)) & 1 for k in range(4)] == [1, 0, 1, 0]
    assert row[12:16].tolist() == [0, 0, 0, 1 << 3]         # value 31 = value 7 of word 3: sign in bit 27
    v = F.decode_rows(row[None])[0]
    assert list(v[:8]) == [6, -6, 0, 1, -1, 2, -2, 4] and list(v[32:35]) == [6, 1, 4]
    assert v[64] == 0 and v[96] == 4 * 2.0 ** 126


def test_error_bounds_and_nan_blocks():
    rng = np.random.default_rng(5)
    x = np.exp(rng.uniform(-20, 20, (4, 18, 1))) * rng.standard_normal((4, 18, 32))
    x = torch.tensor(x.reshape(4, 576)).to(torch.bfloat16).double().numpy()
    x[1, 70], x[2, 130] = np.nan, -np.inf
    rows = F.encode(x)
    y = F.decode_rows(rows)
    s = 2.0 ** (rows[:, 288:306].astype(float) - 127).repeat(32, axis=1)
    bad = np.zeros_like(x, bool)
    bad[1, 64:96] = bad[2, 128:160] = True
    assert np.isnan(y[bad]).all() and not np.isnan(y[~bad]).any()
    a = np.abs(x)
    step = np.where(a <= 2 * s, 0.25, np.where(a <= 4 * s, 0.5, 1.0)) * s  # half a step between neighbours
    assert (np.abs(x - y) <= step)[~bad].all()
    top = a.reshape(4, 18, 32).max(-1).repeat(32, axis=1)
    assert ((top <= 6 * s) & (top > 3 * s))[~bad].all()


def test_e5m2_reading_is_exact_in_its_range():
    codes = np.zeros((256, 320), np.uint8)
    codes[:, :4] = np.frombuffer((0x76543210).to_bytes(4, "little"), np.uint8)
    codes[:, 288] = np.arange(256)
    x = F.decode_rows(codes)
    y = F.through_e5m2(x)
    exact = (np.arange(256) >= 127 - 15) & (np.arange(256) <= 127 + 13)
    assert np.array_equal(x[exact], y[exact])
    t = torch.tensor(x[:255]).clamp(-57344, 57344).to(torch.float8_e5m2).double().numpy()
    assert np.array_equal(t, y[:255])


# ----- dims and refusals -----------------------------------------------------------
def test_dims(lib):
    for H, P in ((16, 16), (32, 32), (96, 64), (128, 128)):
        assert mla.check_dims(mla.dims(H, P, fp4=True)) == mla.MLA_OK
    assert mla.check_dims(mla.dims(24, 64, fp4=True)) == mla.MLA_ERR_UNSUPPORTED
    assert mla.check_dims(mla.dims(16, 48, fp4=True)) == mla.MLA_ERR_UNSUPPORTED
    for kw in ({"fp8": True}, {"int8": True}):
        with pytest.raises(ValueError):
            mla.dims(16, 64, fp4=True, **kw)


def test_append_refusals(lib):
    d = mla.dims(16, 64, fp4=True)
    #       0                1     2     3  4     5  6  7     8     9  10    11    12                    13    14
    good = [ctypes.byref(d), FAKE, None, 4, FAKE, 2, 8, FAKE, FAKE, 3, FAKE, FAKE, ctypes.c_double(1e4), None, None]
    _refused(lib.mla_cache_append, good, [
        (0, None), (1, None), (3, 0), (4, None), (5, 0), (6, 0), (7, None), (8, None), (9, -1), (10, None), (11, None),
        (1, _at(8)), (4, _at(2)), (7, _at(2)), (8, _at(2)), (10, _at(8)), (11, _at(2))])
    none = list(good)
    none[9] = 0
    assert lib.mla_cache_append(*none) == mla.MLA_OK  # no tokens


def test_read_refusals(lib):
    d = mla.dims(16, 64, fp4=True)
    good = [ctypes.byref(d), FAKE, None, 4, FAKE, 2, 8, None, FAKE, 10, FAKE, FAKE, None, None]
    _refused(lib.mla_cache_read, good, [
        (0, None), (1, None), (3, 0), (4, None), (5, 0), (6, 0), (8, None), (9, -1), (10, None), (11, None), (1, _at(8)),
        (4, _at(2)), (7, _at(2)), (8, _at(2)), (10, _at(16)), (11, _at(16)), (12, _at(2))])
    none = list(good)
    none[9] = 0
    assert lib.mla_cache_read(*none) == mla.MLA_OK


def test_decode_refusals(lib):
    d = mla.dims(16, 64, fp4=True)
    good = [ctypes.byref(d), FAKE, FAKE, FAKE, None, 4, FAKE, 8, FAKE, 2, FAKE, FAKE, ctypes.c_float(0.1), 4, FAKE,
            ctypes.c_size_t(1 << 30), FAKE, None, None]
    _refused(lib.mla_decode, good, [
        (0, None), (1, None), (2, None), (3, None), (5, 0), (6, None), (7, 0), (8, None), (9, 0), (10, None), (11, None),
        (12, ctypes.c_float(0.0)), (12, ctypes.c_float(float("inf"))), (12, ctypes.c_float(float("nan"))), (13, -1),
        (16, None), (3, _at(8)), (6, _at(2)), (8, _at(2)), (17, _at(2)), (5, 1 << 30), (7, 1 << 30)])
    _refused(lib.mla_decode, good, [(14, None), (14, _at(64)), (15, ctypes.c_size_t(64))], mla.MLA_ERR_WORKSPACE)


def test_binding_refuses_other_shapes_and_types(lib):
    """Checked before any pointer is passed on (CPU tensors never get that far)."""
    d = mla.dims(16, 64, fp4=True)
    ids = torch.zeros(1, dtype=torch.int32)
    args = (None, torch.zeros(1, 4, dtype=torch.int32), ids, ids, torch.zeros(1, 512, dtype=torch.bfloat16),
            torch.zeros(1, 64, dtype=torch.bfloat16))
    with pytest.raises(TypeError):
        mla.cache_append(d, torch.zeros(4, 64, 320, dtype=torch.int8), *args)
    with pytest.raises(ValueError):
        mla.cache_append(d, torch.zeros(4, 64, 320, dtype=torch.uint8), *args)  # not on the GPU

"""How far the two E4M3 terms of the FP4 decode's queries are from the value, at
every fp16 value, against the bounds that include/mla.h states."""
import os
import re

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _stated():
    with open(os.path.join(ROOT, "include", "mla.h")) as f:
        text = re.sub(r"[\s*]+", " ", f.read())
    m = re.search(r"off by at most 2\^-(\d+) of the value or 2\^-(\d+) of the largest of those heads", text)
    assert m, "the header states the bound"
    return 2.0 ** -int(m.group(1)), 2.0 ** -int(m.group(2))


def _terms(x):
    """fp16 values as hi + lo / 16, both E4M3 to nearest."""
    e4m3 = lambda t: t.float().to(torch.float8_e4m3fn).to(torch.float16)
    hi = e4m3(x)
    return hi.double() + e4m3((x - hi) * 16).double() / 16


@pytest.mark.parametrize("largest", [128.0, 191.875, 255.875])
def test_query_terms(largest):
    """A group's largest value is scaled into [128, 256): of the value, the error is the
    first bound or less, and near 0 the second of the largest; neither is stated larger
    than it is."""
    of_value, of_largest = _stated()
    x = torch.arange(0x7c00, dtype=torch.int32).to(torch.int16).view(torch.float16)
    x = x[x <= largest]
    err, x = (_terms(x) - x.double()).abs(), x.double()
    assert torch.all(err <= torch.maximum(of_value * x, torch.tensor(of_largest * 128)))
    small = x < 2.0 ** -6
    assert (err[small].max() / 128).item() > of_largest / 2
    assert (err[~small] / x[~small]).max().item() > of_value / 2
    # a bf16 value (eight significant bits) above 2^-12 of the largest is held exactly, any
    # other fp16 value there to 2^-9
    above = x >= 2.0 ** -5
    assert torch.all(err[above] <= 2.0 ** -9 * x[above])
    bf16 = above & (x.to(torch.bfloat16).double() == x)
    assert bf16.any() and not err[bf16].any()

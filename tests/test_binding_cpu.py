"""CPU checks of what the binding does around a call of the library: the memory
it allocates.  Nothing is launched (binding_calls)."""
import pytest
import torch

import binding_calls as C
import mla_decode_attention_paged_gb300 as mla

ENTRIES = ["cache_append", "decode", "decode_multi", "decode_sparse", "prefill", "decode_no_alloc", "combine"]
ALLOCATE = [e for e in ENTRIES if e != "cache_append"]


@pytest.fixture
def lib(monkeypatch):
    """The noting library, with what needs a driver taken out of the binding."""
    lib = C.Library()
    monkeypatch.setattr(mla, "_lib", lib)
    monkeypatch.setattr(mla, "_call_on", lambda dev, stream, fn, *args: fn(*args, stream))
    monkeypatch.setattr(mla, "_stream", lambda stream: stream)
    return lib


@pytest.mark.parametrize("entry", ALLOCATE)
def test_what_a_call_allocates_is_its_streams(lib, monkeypatch, entry):
    """Workspace and outputs that the caller leaves out come from the memory of the
    stream that the call names: the current stream would hand a workspace out again
    while the call's kernels still use it."""
    made = []

    def new(shape, dtype, dev, stream):
        made.append(stream)
        return C.gpu(*(shape if isinstance(shape, (tuple, list)) else (shape,)), dtype=dtype)

    monkeypatch.setattr(mla, "_new", new)
    d, calls = C.calls()
    tensors, buffers, rest = calls[entry]
    getattr(mla, entry)(d, **tensors, **rest, stream=77)
    # decode_no_alloc gives no log-sum-exp unless it gets the buffer
    assert made == [77] * (1 if entry == "decode_no_alloc" else len(buffers))
    assert lib.calls[-1][0] == "mla_" + entry and lib.calls[-1][1][-1] == 77

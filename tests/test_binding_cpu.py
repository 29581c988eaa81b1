"""CPU checks of what the binding does around a call of the library: the memory
it allocates, the tensors it refuses, and the device it calls on.  Nothing is launched (binding_calls)."""
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


SMALLER = {"cache_append": ["positions", "c_kv", "k_pe"],
           "combine": ["partial_o", "partial_lse"]}
DECODE = ["q_nope", "q_pe", "block_table", "seq_lens", "W_UK", "W_UV"]


@pytest.mark.parametrize("cache_format", ["bf16", "int8", "fp8", "fp4"])
@pytest.mark.parametrize("entry", ENTRIES)
def test_tensors_too_small_for_the_call_are_refused(lib, cache_format, entry):
    """Each tensor with less than the call reads or writes is refused before the
    launch; larger ones, and the same elements in another shape, are not."""
    d, calls = C.calls(cache_format)
    tensors, buffers, rest = calls[entry]
    given = {**tensors, **{k: v for k, v in buffers.items() if k != "workspace"}}
    call = lambda **kw: getattr(mla, entry)(d, **{**tensors, **buffers, **rest, **kw})
    call()
    assert [name for name, _ in lib.calls] == ["mla_" + entry]
    small = SMALLER.get(entry, DECODE + (["c_kv", "k_pe"] if entry == "prefill" else []))
    small = small + [k for k in buffers if k != "workspace"] + (["scale_zero"] if tensors.get("scale_zero") is not None else [])
    small = small + (["cache"] if "cache" in tensors else [])
    for name in small:
        t = given[name]
        # one row less, with the sizes that the call takes from this tensor as they were
        less = t.view(-1)[:t.numel() - 1]
        if name in ("q_nope", "partial_o", "cache", "block_table"):
            less = t[..., :-1].contiguous() if name != "block_table" else t[:-1]
        with pytest.raises(ValueError):
            call(**{name: less})
        if name in ("q_nope", "cache", "partial_o", "block_table"):
            continue
        call(**{name: torch.cat([t.view(-1), t.view(-1)])})
        call(**{name: t.view(-1)})
    assert not [name for name, _ in lib.calls if name != "mla_" + entry]


def test_sparse_lists_of_more_sequences_than_queries(lib):
    """The batch is the lists'; queries, lengths and outputs of fewer sequences are refused."""
    d, calls = C.calls()
    tensors, buffers, rest = calls["decode_sparse"]
    more = C.gpu(C.B + 1, C.TOP_K, dtype=torch.int32)
    with pytest.raises(ValueError):
        mla.decode_sparse(d, **{**tensors, **buffers, **rest, "token_indices": more})
    assert not lib.calls


@pytest.mark.parametrize("entry", ENTRIES + ["read_device_status", "read_status_word"])
def test_calls_run_on_their_tensors_device(lib, monkeypatch, entry):
    """With device 0 current, tensors of device 1: the call is made with device 1
    current, on that device's stream where none is named."""
    monkeypatch.setattr(C.OnGpu, "at", 1)
    on = []
    monkeypatch.setattr(mla, "_call_on", lambda dev, stream, fn, *args: on.append((dev, stream)) or fn(*args, stream))
    d, calls = C.calls()
    if entry in calls:
        tensors, buffers, rest = calls[entry]
        getattr(mla, entry)(d, **{**tensors, **buffers, **rest})
    else:
        getattr(mla, entry)(C.gpu(64, dtype=torch.int32))
    assert on == [(torch.device("cuda", 1), None)]
    assert [name for name, _ in lib.calls] == ["mla_" + entry]


@pytest.mark.parametrize("entry", ["read_device_status", "read_status_word"])
def test_a_status_is_read_from_a_tensor(lib, entry):
    for bad in (None, 7):
        with pytest.raises(TypeError):
            getattr(mla, entry)(bad)
    with pytest.raises(ValueError):
        getattr(mla, entry)(torch.zeros(4, dtype=torch.int32))
    assert not lib.calls

"""Calls of the binding without a GPU, for its CPU tests: tensors that say they
are on device 0, a library that notes what it is called with and launches
nothing, and one valid call of every entry point that takes tensors."""
import torch

import mla_decode_attention_paged_gb300 as mla

B, T, H, P, PAGES, TABLE, N, TOP_K, SPLITS = 2, 3, 16, 16, 4, 5, 7, 6, 4


class OnGpu(torch.Tensor):
    """A host tensor that says it is on CUDA device ``at``."""
    at = 0
    is_cuda = property(lambda self: True)
    device = property(lambda self: torch.device("cuda", self.at))

    def get_device(self):
        return self.at


def gpu(*shape, dtype=torch.bfloat16):
    return torch.zeros(shape, dtype=dtype).as_subclass(OnGpu)


class Library:
    """Every function returns MLA_OK (sizes: 4,096 bytes); ``calls`` has the names and arguments."""

    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def call(*args):
            self.calls.append((name, args))
            return 4096 if name.endswith("_workspace_size") else mla.MLA_OK
        return call


def calls(cache_format="bf16"):
    """{entry point: (required tensors, given buffers, other arguments)}, in the binding's names."""
    i32, f32, u8 = torch.int32, torch.float32, torch.uint8
    d = mla.dims(H, P, **({} if cache_format == "bf16" else {cache_format: True}))
    width = mla.FP4_ROW_BYTES if cache_format == "fp4" else 576
    cache = gpu(PAGES, P, width, dtype={"bf16": torch.bfloat16, "int8": torch.int8}.get(cache_format, u8))
    scale = {"int8": lambda: gpu(PAGES, P, 2, dtype=f32), "fp8": lambda: gpu(PAGES, P, dtype=f32)}.get(cache_format, lambda: None)()
    pool = {"cache": cache, "scale_zero": scale, "block_table": gpu(B, TABLE, dtype=i32)}
    weights = {"W_UK": gpu(H, 128, 512), "W_UV": gpu(H, 128, 512)}
    lens = {"seq_lens": gpu(B, dtype=i32)}

    def q(*tokens):
        return {"q_nope": gpu(B, *tokens, H, 128), "q_pe": gpu(B, *tokens, H, 64)}

    def made(*tokens):
        return {"out": gpu(B, *tokens, H, 128), "lse_out": gpu(B, *tokens, H, dtype=f32)}

    work = {"workspace": gpu(4096, dtype=u8)}
    rest = {"softmax_scale": 0.1, "num_splits": SPLITS}
    return d, {
        "cache_append": ({**pool, "seq_ids": gpu(N, dtype=i32), "positions": gpu(N, dtype=i32), "c_kv": gpu(N, 512),
                          "k_pe": gpu(N, 64)}, {}, {}),
        "decode": ({**q(), **pool, **lens, **weights}, {**made(), **work}, rest),
        "decode_multi": ({**q(T), **pool, **lens, **weights}, {**made(T), **work}, rest),
        "decode_sparse": ({**q(), **pool, **lens, "token_indices": gpu(B, TOP_K, dtype=i32), **weights},
                          {**made(), **work}, rest),
        "prefill": ({**pool, **lens, "c_kv": gpu(B, T, 512), "k_pe": gpu(B, T, 64), **q(T), **weights},
                    {**made(T), **work}, rest),
        "decode_no_alloc": ({**q(), **pool, **lens, **weights}, made(), rest),
        "combine": ({"partial_o": gpu(B, SPLITS, H, 512, dtype=f32), "partial_lse": gpu(B, SPLITS, H, dtype=f32)},
                    {"o_lat_out": gpu(B, H, 512, dtype=f32), "lse_out": gpu(B, H, dtype=f32)}, {}),
    }

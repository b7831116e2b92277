"""Sizes that reach the adapters' tiles of 128 tokens with fp32 outputs, and the form that a call takes."""
import ctypes

import torch

from ternary_weight_linear_02_gb300 import lora

KIND = {torch.float16: 0, torch.bfloat16: 1, torch.float32: 2}

# tokens, inputs, shards, rank, adapters.  fp32 outputs take tiles of 128 from 256 tokens an adapter (tokens without one count as
# one more) and tokens * inputs * rank * shards = 880e6 on.
MANY32 = [
    (2048, 2304, (264, 96, 104), 64, 3),        # three launches, eight blocks a tile
    (2304, 9552, (72,), 40, 4),                 # a rank that is no multiple of 16
    (2048, 26880, (40, 16), 8, 2),
    (1300, 10624, (64, 8, 72, 136), 16, 4),     # four shards in one launch
    (2100, 2304, (128, 40, 0, 24), 48, 5),      # a shard without columns
    (4500, 576, (40, 24, 32, 8, 16, 72, 48), 56, 2),  # seven launches; eight blocks a tile, nine steps of 64 inputs: three blocks have none
    (5900, 448, (40, 24, 32, 8, 16, 72), 56, 4),      # six blocks a tile, seven steps: two have none
    (9000, 1800, (72,), 56, 5),                 # four blocks a tile
    (16000, 904, (136, 8), 32, 4),              # two
    (20000, 1400, (72,), 32, 4),                # one
    (2100, 17600, (40,), 24, 2), (3000, 4608, (1000,), 64, 10)]


def tile(tokens, inputs, shards, rank, n, dtype, out_dtype, gated=False):
    """Tokens of a tile of lora_add (lora_silu_mul) for dense tensors of these sizes."""
    lib = lora._lib()
    at = 1 << 20
    cols = sum(shards)
    ad = lora._Adapters(at, at, None, inputs, (ctypes.c_int64 * 8)(*shards), len(shards), rank, n, KIND[dtype])
    return lib.ternary_test_lora_tile(ctypes.c_void_p(at), ctypes.c_int64(inputs), ctypes.byref(ad), ctypes.c_void_p(at), ctypes.c_void_p(at),
                                      ctypes.c_int64(cols), ctypes.c_void_p(2 * at), ctypes.c_int64(cols // 2 if gated else cols),
                                      KIND[out_dtype], ctypes.c_int64(tokens), int(gated))

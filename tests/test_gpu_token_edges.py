"""Token operators on the GPU at the borders of what their documentation allows."""
import math

import numpy as np
import pytest
import torch

from test_gpu_tokens import DT, ROT, Batch, assert_appended, assert_attended, attended, gen, half_step, pkv, randn, turned  # noqa: F401

pytestmark = pytest.mark.gpu


def bits(x):
    return x.view(torch.int16)


# ---------------------------------------------------------------- lengths past the table
@pytest.mark.parametrize("held,hkv,g,d,page,dtype,window", [
    (64, 2, 1, 64, 16, "bf16", 0), (64, 1, 9, 128, 16, "fp16", 0), (20000, 2, 2, 64, 32, "bf16", 0),
    (9000, 1, 4, 128, 1000, "fp16", 777)])
def test_a_step_past_the_table_writes_nothing(pkv, held, hkv, g, d, page, dtype, window):
    """A length that the table cannot hold: its new token has no slot. It is not written, and what is attended to are the
    tokens that the table names, as they are in the pool."""
    b = Batch(pkv, [held, 40, held], hkv, d, page, dtype, seed=31)
    q = randn((3, hkv * g, d), b.dtype, b.g)
    k, v = randn((3, hkv, d), b.dtype, b.g), randn((3, hkv, d), b.dtype, b.g)
    for long in (held + 1, 2**31 - 1):
        before = b.pool.clone()
        b.len_t.copy_(torch.tensor([long, 40, -1], dtype=torch.int32))
        out = b.cache.decode_append(k, v, q, window=window)
        with pytest.raises(pkv.KVError) as e:
            b.cache.check_device()
        assert e.value.name == "DEVICE_CHECK"
        b.lens = [0, 40, 0]                         # only the second one's token is written
        assert_appended(b, before, [1, 1, 1], k, v, None)
        b.lens = [held, 40, 0]
        assert_attended(out, b, q, window=window)

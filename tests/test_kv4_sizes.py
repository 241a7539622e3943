"""The binding of the 4-bit cache refuses sizes that the C interface's 32-bit arguments would cut.

Tensors of such sizes need no memory here: they are fake CUDA tensors (shapes, strides and device only), which a call
has to refuse before it asks for an address.
"""

import pytest
import torch
from torch._subclasses.fake_tensor import FakeTensorMode

import attention_tiled_attn_b200 as attn


def fake_cache(N=2, H=2, C=32, E=64, Ev=64):
    return tuple(torch.empty((N, H, C, w), dtype=torch.uint8, device="cuda") for w in (E // 2, E // 16, Ev // 2, Ev // 16))


@pytest.mark.parametrize("rows", [2 ** 31, 2 ** 32 + 16])
def test_more_new_rows_than_32_bits(rows):
    with FakeTensorMode():
        k = torch.empty((2, 2, 1, 64), dtype=torch.bfloat16, device="cuda").expand(2, 2, rows, 64)  # one row, repeated
        with pytest.raises(ValueError, match="32 bits"):
            attn.attn_kv4_write(fake_cache(), k, k)


@pytest.mark.parametrize("size", [dict(C=2 ** 32 + 16), dict(N=2 ** 32 + 2), dict(H=2 ** 32 + 2), dict(E=2 ** 32 + 64), dict(Ev=2 ** 32 + 64)])
def test_a_cache_of_more_than_32_bits(size):
    s = dict(N=2, H=2, C=32, E=64, Ev=64) | size
    with FakeTensorMode():
        cache = fake_cache(**s)
        k = torch.empty((s["N"], s["H"], 1, s["E"]), dtype=torch.bfloat16, device="cuda")
        v = torch.empty((s["N"], s["H"], 1, s["Ev"]), dtype=torch.bfloat16, device="cuda")
        for call in (lambda: attn.attn_kv4_write(cache, k, v), lambda: attn.attn_kv4_read(cache, 1),
                     lambda: attn.attn_decode_kv4(k, cache, scale=1.0)):
            with pytest.raises(ValueError, match="32 bits"):
                call()

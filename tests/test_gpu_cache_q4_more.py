"""The 4-bit cache: refusals of the block copy, and scales and codes of every bf16 magnitude."""
import numpy as np
import pytest
import torch

import operator_refs as ref
import paged_kv_cache_39_gb300 as kv
from operator_refs import BF16, dev
from test_gpu_cache_q4 import i32

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("record", [33, 32, 64, 300, 288 * 3 + 16])
@pytest.mark.parametrize("bulk", [False, True])
def test_block_copy_refuses_bytes_that_are_no_4_bit_cache(record, bulk):
    c = torch.zeros((2, 4, 2, record), dtype=torch.uint8, device=dev())
    with pytest.raises(ValueError, match="4-bit"):
        kv.kv_copy_blocks(c, c.clone(), i32([1]), i32([2]), bulk=bulk)

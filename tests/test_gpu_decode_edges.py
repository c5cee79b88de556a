"""nexus_append, nexus_quantize and nexus_attend where one call's parts meet: pieces that share a
block's memory, scales that differ within a slice, rows that are taken back. Tolerances as in
test_gpu_decode.py."""
import math

import numpy as np
import pytest
import torch

from decode_harness import DEV, Case, attend64
from streaming_kv_cache_step_gb300 import nexus
from test_gpu_decode import BF, F32, _check_attend, _image, _scale_at, _status  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("page", [0, 16])
@pytest.mark.parametrize("tokens", [9, 32])
def test_attend_pieces_of_one_block_follow_one_another(d, page, tokens):
    # one row tile per slice and several slices per thread block: a slice's outputs pass through
    # the shared memory that the next one's whole tiles of K and V are copied to
    rng = np.random.default_rng(tokens + page)
    c = Case(seqs=60, kv_heads=4, group=4, d=d, page=page, capacity=384,
             lens=rng.choice([64, 128, 192, 256, 320, 384], (60, 4)), seed=page)
    _check_attend(c, [tokens] * 60, uniform=True)

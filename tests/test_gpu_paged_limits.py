"""What a token sees of a paged quantized cache, and what reaches it of what it
does not see: batches padded in front, more new tokens than a call takes, norms
of very different sizes, norms that are not finite."""
import math

import numpy as np
import pytest
import torch

from tests.paged_reference import attend, unpack
from tests.test_gpu_paged import DT, Batch, check, quantizer, run_case, tq  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d,ip", [(64, False), (128, False), (64, True), (128, True)])
def test_fewer_keys_than_new_tokens(tq, d, ip):  # noqa: F811
    """256 new tokens, all in front of the first 128 or so without a key (a batch
    padded in front): whole blocks of rows whose first 128 see nothing, several
    to a run, and such blocks among others."""
    run_case(tq, d, 4, ip, 4, 8, 1, 16, [(256, 128)] * 64, "bf16", seed=d, many=True)
    seqs = [(256, (128, 1, 700, 129, 256, 127)[i % 6]) for i in range(12)] + [(300, 40), (65, 3), (320, 180)]
    run_case(tq, d, 4, ip, 3, 2, 1, 16, seqs, "bf16", seed=d + 1, many=True)
    run_case(tq, d, 3, ip, 4, 1, 4, 48, [(129, 20), (96, 96), (70, 64), (1, 5)], "f16", seed=d + 2, many=True)
    tq.tq_sync_check(quantizer(tq, d, 4, ip)[0])

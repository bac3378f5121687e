"""dweight and dbias of gdn_group_norm_backward by their norm, in every form of the kernel: a worst
case over all terms of a long sum would not notice a token left out, this bound does."""
import numpy as np
import pytest
import torch

from linear_attention_12_b200 import gdn
from oracle import norm as onorm
from tests.test_gpu_norm import BF16, F32, _case, _cuda

pytestmark = pytest.mark.gpu

# The terms' own errors are a few units of 2^-24 each and independent, as the terms are, so their
# sum stays a few units of the result's norm; the additions run at most 128 deep, each with half a
# unit of a partial sum: together below 1e-5 (168 units).  One term more or less in n changes the
# result by about n^-1/2 of its norm, 5e-3 in the longest of these sums.
BOUND = 1e-5


def _form(i):
    return dict(gated=i % 2 == 0, bias=i in (1, 2), per_head=i in (1, 3, 4)), \
        dict(norm="mean" if i in (2, 4) else "rms", act="none" if i in (3, 5) else "silu", eps=1e-3)


# whole vectors in 4, 8, 16 and 32 lanes and in several a lane; pairs of bf16; one by one
SIZES = [(4099, 2, 16), (9001, 3, 40), (601, 33, 64), (6000, 6, 128), (4000, 3, 256), (1500, 2, 1024),
         (700, 2, 1000), (3000, 4, 130), (2000, 2, 258), (1000, 1, 1022), (3000, 5, 17), (2000, 2, 257),
         (1000, 1, 1023)]


@pytest.mark.parametrize("form", range(6))
@pytest.mark.parametrize("io", [BF16, F32])
@pytest.mark.parametrize("T,H,d", SIZES)
def test_sums_over_tokens(T, H, d, io, form):
    make, kw = _form(form)
    x, dy, w, b, z = _case(T, H, d, io, T + d + form, **make)
    got = gdn.group_norm_backward(*_cuda(dy, x, w, b, z), **kw)
    ref = onorm.group_norm_backward(dy, x, w, b, z, **kw)
    for p, r in zip(got[1:3], ref[1:3]):
        if r is None:
            assert p is None
            continue
        p = p.cpu().double().numpy()
        assert np.linalg.norm(p - r) <= BOUND * np.linalg.norm(r)
        # no head and no channel apart from the others
        assert np.abs(p - r).max() <= 10 * BOUND * np.abs(r).max()
    assert gdn.last_device_error() == gdn.GDN_OK

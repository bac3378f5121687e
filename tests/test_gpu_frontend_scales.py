"""gdn_frontend_backward without eps on q and k rows far from unit size: the formula
du = r (dq - q <q, dq>) stays finite where 1 / r^3 or r^3 alone leaves fp32."""
import numpy as np
import pytest
import torch

from linear_attention_12_b200 import gdn
from oracle import frontend_backward as feb
from tests.test_gpu_frontend_backward import UNITS, _case, _half_step, _np64

pytestmark = pytest.mark.gpu


# |u| ~ 1e-14 (r^3 ~ 1e42) and ~ 1e14 (r^3 ~ 1e-42); in between nothing special happens
@pytest.mark.filterwarnings("ignore:overflow encountered in exp")  # (the oracle's unused sigmoid)
@pytest.mark.parametrize("io", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("scale", [1e-14, 1e-7, 1e7, 1e14])
def test_rows_far_from_unit_size(scale, io):
    args = _case([50, 3, 40], 1, 2, io, 71)
    for i in (0, 1):
        args[i] = (args[i].float() * scale).to(io)
    got = gdn.frontend_backward(*[t.cuda() for t in args], act="none", eps=0.0)
    ref = feb.frontend_backward(*args, act="none", eps=0.0)
    for p, q, step in zip(got[:4], ref[:4], [_half_step(io)] * 3 + [2 * UNITS]):
        assert np.isfinite(_np64(p)).all()
        assert np.linalg.norm(_np64(p) - q) <= (step + 2 * UNITS) * np.linalg.norm(q)
    assert gdn.last_device_error() == gdn.GDN_OK

"""GPU tests of linear attention and rotary positions, beside those of test_gpu_linattn: refusals
through the binding."""
import pytest
import torch

import state_space_sequence_cumsum_amd as ssd
from gpu_util import require_gpu

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("given", [False, True])
def test_gradients_of_too_many_heads_are_refused(given):
    """Rows of all heads' dq and dk past the limit: refused, with every output as it was."""
    dev = require_gpu()
    new = lambda *s: torch.ones(s, device=dev, dtype=torch.bfloat16)
    q, v, g = new(1, 64, 1, 256), new(1, 64, 16392, 8), -new(1, 64, 16392)
    outs = {}
    if given:
        outs = dict(dq=3 * new(*q.shape), dk=3 * new(*q.shape), dv=3 * new(*v.shape), dg=3 * new(*g.shape),
                    workspace=torch.empty(1 << 20, dtype=torch.uint8, device=dev))
    with pytest.raises(ssd.SsdError) as e:
        ssd.ssd_linattn_backward(v, q, q, v, g, **outs)
    torch.cuda.synchronize()
    assert e.value.status == 3
    assert all((outs[n] == 3).all() for n in outs if n != "workspace")

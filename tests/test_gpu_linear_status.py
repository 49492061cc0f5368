"""Every linear attention call that takes a workspace leaves a status word that says how it went, whatever the memory held."""
import pytest
import torch

import gated_delta_rule_31_gb300 as gdr
from linear_ref import make
from util import cuda_device, to_dev

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("B,T,Hv", [(2, 40, 4), (1, 2500, 2), (40, 70, 8), (2, 0, 2), (0, 5, 2)])
def test_status_is_set(B, T, Hv, dtype):
    dev = cuda_device()
    d = to_dev(make(B, T, 2, Hv, 64, 64, TYPES[dtype], seed=T), dev)
    args = d["q"], d["k"], d["v"], d["g"], d["h0"]
    ws = torch.empty(64 << 20, dtype=torch.uint8, device=dev)
    states = gdr.linear_fwd(*args, save_states=True)[2]

    def status(call):
        ws.fill_(0xff)
        call()
        return gdr.workspace_status(ws)

    assert status(lambda: gdr.linear_fwd(*args, workspace=ws)) == 0
    assert status(lambda: gdr.linear_fwd(*args, workspace=ws, output_final_state=False)) == 0
    assert status(lambda: gdr.linear_fwd(*args, workspace=ws, save_states=True)) == 0
    assert status(lambda: gdr.linear_bwd(*args, d["do"], d["dht"], workspace=ws)) == 0
    assert status(lambda: gdr.linear_bwd(*args, d["do"], d["dht"], workspace=ws, need_dh0=False)) == 0
    assert status(lambda: gdr.linear_bwd(*args, d["do"], d["dht"], workspace=ws, states=states)) == 0

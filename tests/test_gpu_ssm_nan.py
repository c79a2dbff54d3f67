"""Every NaN that a state may hold comes out as one: all bits set (memory that
was never written, a poisoned pool) and the smallest payloads, of either sign."""
import pytest
import torch

import gated_deltanet_prefill_varlen_amd as gdn
from tests.ssm_util import DEV, Layer

pytestmark = pytest.mark.gpu
BITS = [-1, 0x7FFFFFFF, 0x7F800001, -0x7FFFFF, 0x7FC00000]


@pytest.mark.parametrize("bits", BITS, ids=hex)
def test_step(bits):
    H, G, P, N, B = 2, 1, 32, 64, 3
    y = Layer(H, G, P, N, [B], seed=60, conv=False)
    state = torch.randn(B, H, P, N, device=DEV)
    state.view(torch.int32)[1, 0, 5] = bits
    out = torch.empty(B, H, P, dtype=torch.bfloat16, device=DEV)
    gdn.gdn_ssm_decode(y.shape, 1, y.x, y.dt, y.A, state, out, dt_bias=y.dt_bias, D=y.D)
    want = torch.zeros(B, H, P, dtype=torch.bool, device=DEV)
    want[1, 0, 5] = True
    assert torch.equal(out.isnan(), want) and torch.equal(state.isnan().any(-1), want)


@pytest.mark.parametrize("bits", BITS, ids=hex)
def test_scan(bits):
    y = Layer(2, 1, 32, 64, [40, 70], seed=61, init=True, conv=False)
    y.init.view(torch.int32)[1, 0, 5] = bits
    r = y.run([40 + 33])
    want = torch.zeros(110, 2, 32, dtype=torch.bool, device=DEV)
    want[40:, 0, 5] = True
    assert torch.equal(r["out"][:110].isnan(), want)
    assert torch.equal(r["final"].isnan().any(-1), want[[39, 109]]) and torch.equal(r["kept"].isnan().any(-1), want[[72]])

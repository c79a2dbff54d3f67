"""State space calls at the limits of what they accept: the most groups that a
launch holds, and a pool that keeps its own snapshots."""
import numpy as np
import pytest
import torch

import gated_deltanet_prefill_varlen_amd as gdn
from tests.ssm_util import DEV, Layer

pytestmark = pytest.mark.gpu


def test_most_groups():
    """58,253 groups of one head: the first and the last heads as a layer of their own has them, by the scan and the step."""
    G, P, N, T, k = 58253, 32, 32, 37, 8
    g = torch.Generator(device=DEV).manual_seed(71)
    rnd = lambda *s: torch.randn(*s, generator=g, device=DEV)
    x, dt, A, D = rnd(T, G * 96).bfloat16(), rnd(T, G), -rnd(G).abs(), rnd(G)
    cu = np.array([0, 33, T], np.int32)

    def run(x, dt, A, D):
        n = len(A)
        shape = gdn.make_ssm(n, n, P, N)
        out, final = torch.empty(T, n, P, dtype=torch.bfloat16, device=DEV), torch.empty(2, n, P, N, device=DEV)
        kept, ck = torch.empty(2, n, P, N, device=DEV), np.array([20, 32], np.int32)
        i32 = lambda v: torch.from_numpy(v).to(DEV)
        ws = torch.empty(gdn.gdn_ssm_prefill_workspace(shape, cu), dtype=torch.uint8, device=DEV)
        gdn.gdn_ssm_prefill_packed(shape, i32(cu), cu, x, dt, A, out, D=D, final_state=final, ckpt_positions=i32(ck), ckpt_positions_host=ck,
                                   ckpt_buf=kept, workspace=ws)
        state, step = final.clone(), torch.empty(2, n, P, dtype=torch.bfloat16, device=DEV)
        gdn.gdn_ssm_decode(shape, 1, x[:2], dt[:2], A, state, step, D=D)
        return out, final, kept, state, step

    whole = run(x, dt, A, D)
    for at in (slice(0, k), slice(G - k, G)):
        cols = [x.view(T, 3, G, 32)[:, i, at].reshape(T, k * 32) for i in range(3)]
        part = run(torch.cat(cols, 1).contiguous(), dt[:, at].contiguous(), A[at].contiguous(), D[at].contiguous())
        assert all(torch.equal(a[:, at], b) for a, b in zip(whole, part))


@pytest.mark.parametrize("slots,first", [([3, 0], 4), ([3, 0], 1), ([7, 6], 0)])
def test_snapshots_in_spare_slots(slots, first):
    H, G, P, N, B, pool = 4, 2, 64, 64, 2, 8
    y = Layer(H, G, P, N, [B], seed=72, conv=False)
    s0 = torch.randn(pool, H, P, N, generator=torch.Generator().manual_seed(73)).to(DEV)
    sl = np.array(slots, np.int32)
    slot = torch.from_numpy(sl).to(DEV)

    def run(state, snap):
        out = torch.empty(B, H, P, dtype=torch.bfloat16, device=DEV)
        gdn.gdn_ssm_decode(y.shape, 1, y.x, y.dt, y.A, state, out, dt_bias=y.dt_bias, D=y.D, slot=slot, slot_host=sl, snapshots=snap)
        return out

    a, b, apart = s0.clone(), s0.clone(), torch.empty(B, 1, H, P, N, device=DEV)
    want, got = run(a, apart), run(b, b[first:first + B].view(B, 1, H, P, N))
    a[first:first + B] = apart[:, 0]
    assert torch.equal(want, got) and torch.equal(a, b)

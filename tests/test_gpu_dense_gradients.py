"""The library's gradients of the gated feed-forward block against differences of its 64-bit forward, every
coordinate of every gradient by itself (MI355X only)."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import gradient_bounds as gb
import host_paged_expert_amd as pe
from test_gpu_dense import DEV, _np

pytestmark = pytest.mark.gpu


def _bf16(a):
    return torch.from_numpy(np.asarray(a, np.float32)).to(torch.bfloat16).double().numpy()


@pytest.mark.parametrize("T,H,I", [(5, 24, 16), (1, 16, 8), (19, 16, 8)])
@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_gradients_match_differences_coordinate_by_coordinate(T, H, I, act):
    p = gb.point(T, H, I, act, T + I, _bf16)
    want, tol = gb.differences(*p, act), gb.bounds(*p, act)
    x, w13, w2, dy = (torch.from_numpy(a).to(DEV, torch.bfloat16) for a in p)
    e = lambda *s: torch.zeros(s, dtype=torch.bfloat16, device=DEV)           # noqa: E731
    h, gu, dgu, dx, dw13, dw2 = e(T, I), e(T, 2 * I), e(T, 2 * I), e(T, H), e(2 * I, H), e(H, I)
    pe.glu(x, w13, h, act=act, gu=gu)
    pe.ffn_backward(dy, x, gu, w13, w2, dgu, h, dx=dx, dw13=dw13, dw2=dw2, act=act)
    torch.cuda.synchronize()
    for name, g, w, t in zip(("dx", "dw13", "dw2"), (dx, dw13, dw2), want, tol):
        bad = np.abs(_np(g) - w) > t
        assert not bad.any(), (name, np.argwhere(bad)[0], _np(g)[bad][0], w[bad][0], t[bad][0])

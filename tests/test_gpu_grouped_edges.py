"""Calls at the edges of the expert-grouped operators (MI355X only)."""
import pytest

torch = pytest.importorskip("torch")

import host_paged_expert_amd as pe
from test_gpu_dense import DEV, GUARD

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("weighted", [True, False])
def test_combine_backward_of_tokens_without_rows(weighted):
    """Every id names an expert that is elsewhere: no rows here, tokens all the same."""
    T, k, H = 5, 3, 64
    bf = dict(dtype=torch.bfloat16, device=DEV)
    dout, none = torch.ones((T, H), **bf), torch.empty((0, H), **bf)
    places = torch.full((T, k), -1, dtype=torch.int32, device=DEV)
    w = torch.ones((T, k), device=DEV) if weighted else None
    pe.combine_backward(dout, places, none, topk_w=w)
    dw = torch.full((T, k), GUARD, device=DEV)
    pe.combine_backward(dout, places, none, topk_w=w, y=none, dtopk_w=dw)
    torch.cuda.synchronize()
    assert not dw.any()

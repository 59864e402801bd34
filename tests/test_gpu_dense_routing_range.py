"""Sigmoid routing of rows whose scores come near fp32's smallest numbers (MI355X only)."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import host_paged_expert_amd as pe
from oracle import dense

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.mark.parametrize("E,k", [(8, 3), (128, 8), (300, 40)])
@pytest.mark.parametrize("top", [-20.0, -63.0, -65.0, -87.0, -88.5, -95.0, -102.0])
def test_weights_of_small_scores_are_their_ratios(E, k, top):
    """Renormalised, the weights are the scores' ratios also where the scores themselves, e^-65 to e^-102, are under
    fp32's normal range; the ids are the largest logits'."""
    rng = np.random.default_rng(E)
    lg = (top - np.abs(rng.standard_normal((4, E)))).astype(np.float32)
    lg[:, 0] = top
    ids, w = torch.zeros((4, k), dtype=torch.int32, device=DEV), torch.zeros((4, k), device=DEV)
    pe.route(torch.from_numpy(lg).to(DEV), ids, w, scoring="sigmoid", scale=2.5)
    torch.cuda.synchronize()
    want_ids, want = dense.route(lg, k, "sigmoid", True, 2.5)
    assert np.array_equal(ids.cpu().numpy(), want_ids)
    # exp is good to 2 units in the last place of arguments taken as they are (their difference to the largest is
    # exact or off by 2^-24 of at most 128, 2^-17); a sum of k positive terms, a division, a product
    tol = want * (2.0 ** -17 + (k + 16) * 2.0 ** -24)
    assert (np.abs(w.double().cpu().numpy() - want) <= tol).all()


def test_scores_themselves_down_to_subnormal_numbers():
    lg = np.array([[-80, -87, -88.7, -89, -95, -100]], np.float32)
    ids, w = torch.zeros((1, 6), dtype=torch.int32, device=DEV), torch.zeros((1, 6), device=DEV)
    pe.route(torch.from_numpy(lg).to(DEV), ids, w, scoring="sigmoid", renormalize=False)
    torch.cuda.synchronize()
    want = np.exp(lg.astype(np.float64))             # 1 + e^-80 is 1
    # 4 units in the last place, a subnormal number's being 2^-149
    assert (np.abs(w.double().cpu().numpy() - want) <= want * 2.0 ** -21 + 2.0 ** -147).all()

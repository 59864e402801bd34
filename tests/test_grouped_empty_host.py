"""Calls of the expert-grouped operators in which no token has a row here (as on a process that holds a share of the
experts), on the host: they are nothing to do, not errors."""
import host_paged_expert_amd as pe
from test_grouped_host import _cback, _comb, _gglu, _glin


def test_rows_of_no_token():
    """An empty tensor has no address, so `dy` asked for is NULL here like one that is not."""
    assert _cback(R=0, dy=None, y=None, dtopk_w=None) == pe.PE_OK
    assert _cback(R=0, dy=None, dtopk_w=None) == pe.PE_OK
    for call in (_glin, _gglu):
        assert call(R=0, x=None) == pe.PE_OK
    assert _comb(T=0, R=0, y=None, out=None) == pe.PE_OK

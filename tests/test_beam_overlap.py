"""gdn_beam_select writes a group's scores while others still read theirs: out_scores over scores is
refused but for the call in place (fake device addresses, never dereferenced)."""
import pytest

from gated_delta_rule_44_gb300 import binding as B
from test_beam_slots_refusals import FAKE, beam

FAR = FAKE + (1 << 24)


@pytest.mark.parametrize("K,shift", [(3, 0), (5, 0), (4, 4), (4, -4), (4, 4 * 4), (5, 4 * 7), (3, -4 * 5)])
def test_out_scores_over_scores(K, shift):
    rc, msg = beam(n=2, W=4, K=K, scores=FAR, out_scores=FAR + shift)
    assert rc == B.GDN_ERR_INVALID_ARGUMENT
    assert msg == "beam_select out_scores may be scores only where K = W"


@pytest.mark.parametrize("K,shift", [(4, 0), (4, 32), (3, -24), (5, 32)])
def test_in_place_and_next_to_it(K, shift):
    """Past this check, to the one of the workspace."""
    rc, msg = beam(n=2, W=4, K=K, scores=FAR, out_scores=FAR + shift, workspace_bytes=0)
    assert rc == B.GDN_ERR_INVALID_ARGUMENT and msg.startswith("gdn_beam_select workspace needs")

"""A causal mask that is off by one position changes what the pin of the
attention oracle compares."""
import pytest

from oracle import decode_oracle as do
from tests import test_decode_ops_host as pins


@pytest.mark.parametrize("shift", [-1, 1])
def test_a_causal_mask_off_by_one_is_seen(monkeypatch, shift):
    real = do.paged_attention

    def mistaken(c, q, cu, total, sm_scale, window=0, n_sink=0):
        # every row one position earlier or later: it sees one token less or more
        return real(c, q, cu, [t + shift for t in total], sm_scale, window, n_sink)

    pins.test_oracle_attention_matches_torch()
    monkeypatch.setattr(do, "paged_attention", mistaken)
    with pytest.raises(AssertionError):
        pins.test_oracle_attention_matches_torch()

"""More host-side refusals of the norms of queries and keys with their rotation: calls without rows, sizes of the
workspace."""
import pytest

import megatron_tensor_transformer_tp_gb300 as tp
from tests.test_rotary_host import FAKE, bwd


@pytest.mark.parametrize("over", [dict(dgq=FAKE * 8), dict(dgq=FAKE * 9), dict(dgk=FAKE * 8), dict(dgk=FAKE * 9),
                                  dict(dgq=FAKE * 5), dict(dgk=FAKE * 4)])
def test_gradients_over_gains_refused_without_rows(over):
    """Without rows the gains' gradients are set to zero: at a gain's address that would clear the gain.  (bwd's gains
    lie at 8 and 9 FAKE, their gradients at 4 and 5.)"""
    assert bwd(T=0, b=0, **over) == tp.TP_ERR_INVALID
    assert bwd(T=256, **over) == tp.TP_ERR_INVALID

"""More host-side refusals of the norms of queries and keys with their rotation: calls without rows, sizes of the
workspace."""
import pytest

import megatron_tensor_transformer_tp_gb300 as tp
from tests.test_rotary_host import FAKE, L, bwd, cfg


@pytest.mark.parametrize("over", [dict(dgq=FAKE * 8), dict(dgq=FAKE * 9), dict(dgk=FAKE * 8), dict(dgk=FAKE * 9),
                                  dict(dgq=FAKE * 5), dict(dgk=FAKE * 4)])
def test_gradients_over_gains_refused_without_rows(over):
    """Without rows the gains' gradients are set to zero: at a gain's address that would clear the gain.  (bwd's gains
    lie at 8 and 9 FAKE, their gradients at 4 and 5.)"""
    assert bwd(T=0, b=0, **over) == tp.TP_ERR_INVALID
    assert bwd(T=256, **over) == tp.TP_ERR_INVALID


@pytest.mark.parametrize("bad", [dict(T=2 ** 31), dict(T=2 ** 31 - 1), dict(n_heads=0), dict(n_kv_heads=0), dict(n_heads=-4),
                                 dict(n_kv_heads=3), dict(n_heads=6, n_kv_heads=4), dict(N=0), dict(N=9), dict(N=3), dict(N=-1),
                                 dict(n_heads=2050, n_kv_heads=2050), dict(n_heads=2 ** 31 - 2, n_kv_heads=2), dict(d=-64),
                                 dict(d=512 + 8), dict(d=12)])
def test_no_workspace_for_sizes_that_are_refused(bad):
    """The size is 0 where the call with these sizes is refused, and the same for all that are not."""
    size = lambda **k: L.tp_qk_norm_rotary_workspace_size(cfg(**k))  # noqa: E731
    assert size(**bad) == 0
    assert bwd(**bad) in (tp.TP_ERR_INVALID, tp.TP_ERR_ALIGN)
    assert size() == size(T=2 ** 31 - 512, n_heads=4088, n_kv_heads=8, N=8, b=0, s=0) > 0

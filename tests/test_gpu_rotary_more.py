"""More of the rotation of queries and keys and of their norms: what the call just before has written, positions and
frequencies at their ends."""
import pytest
import torch

import synthetic_inputs as SI
from tests.test_gpu_rotary import NORMS, Case, _tp

pytestmark = pytest.mark.gpu


# ----------------------------------------------------------------------------
# gains that the kernel before writes
# ----------------------------------------------------------------------------
@pytest.mark.parametrize("lens,d,norm", [([40], 64, "rms"), ([3], 512, "layer"), ([900, 700], 128, "rms")])
def test_gains_written_by_the_call_before(lens, d, norm):
    """The optimizer's step of the gains, the forward, the backward, and the next step from the gradients that it left,
    in a row: the same bits as with a wait behind every call and no launch before the last kernel has ended."""
    tp = _tp()
    c = Case(lens, 4, 2, d, 2, norm=norm, seed=60)
    X, dY, w = c.X.cuda(), c.dY.cuda(), c.where()
    hyper = dict(lr=0.05, beta1=0.9, beta2=0.95, eps=1e-8, max_norm=0.0, use_scaler=0, min_scale=1.0, growth_factor=2.0,
                 backoff_factor=0.5, growth_interval=1000, hysteresis=2)

    def chain(wait):
        gains, grads = [g.clone() for g in c.g()], [SI.normal(61, i, (d,), 1.0, "f32").cuda() for i in range(2)]
        groups = [dict(param=p, grad=g, m=torch.zeros_like(p), v=torch.zeros_like(p), weight_decay=0.0)
                  for p, g in zip(gains, grads)]
        state, ows = tp.make_optimizer_state(), torch.empty(tp.tp_adam_step_workspace_size(), dtype=torch.uint8, device="cuda")
        ws, out = c.ws(), [(torch.empty_like(X), torch.empty_like(X)) for _ in range(8)]
        seen = []
        for Y, dX in out:
            for call in (lambda: tp.tp_adam_step(groups, hyper, state, ows),
                         lambda: tp.tp_qk_norm_rotary_fwd(X, c.cfg, c.norm, c.rot, *gains, Y, **w),
                         lambda: tp.tp_adam_step(groups, hyper, state, ows),
                         lambda: tp.tp_qk_norm_rotary_bwd(X, c.cfg, c.norm, c.rot, *gains, dY, dX, *grads, ws, **w)):
                call()
                if wait:
                    torch.cuda.synchronize()
            seen += [Y, dX]
        return seen + gains + grads

    tp.tp_debug_set_pdl(0)
    try:
        want = chain(True)
    finally:
        tp.tp_debug_set_pdl(1)
    assert not torch.equal(want[0], want[2])  # (the gains do move)
    for _ in range(4):
        got = chain(False)
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert tp.tp_get_status() == tp.TP_OK


# ----------------------------------------------------------------------------
# blocks whose number an SM's shared memory limits, not their registers
# ----------------------------------------------------------------------------
@pytest.mark.parametrize("norm", NORMS)
@pytest.mark.parametrize("lens,H,KV,d,inter,dtype", [([9000, 77], 8, 2, 128, False, "bf16"), ([6000], 8, 2, 128, False, "f32"),
                                                     ([5000], 8, 2, 64, False, "f32"), ([4845], 1, 1, 512, True, "bf16"),
                                                     ([6007], 1, 1, 128, True, "f32")])
def test_fewer_blocks_an_sm(lens, H, KV, d, inter, dtype, norm):
    """Wide tables and stages of fp32: fewer blocks on an SM than their registers allow, many steps a block."""
    Case(lens, H, KV, d, 1, None, inter, norm=norm, dtype=dtype, seed=62).check()

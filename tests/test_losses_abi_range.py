"""The range of the losses' temperatures, through the C ABI.  No kernel is launched here."""
from __future__ import annotations

import pytest

from lower_convex_hull_amd import iso
from tests.test_losses_abi import ARG, WS, logp_args, mem, vjp_args  # noqa: F401


def head_args(m, **over):
    a = dict(logits=m(0), dtype=iso.ISO_DT_F32, rows=2, vocab=8, ld=8, target=m(1), temperature=1.0, old=m(2), ref=None, adv=m(3),
             off=None, seqs=1, lo=0.2, hi=0.2, kl=0.0, norm=0.0, loss=m(4), counts=m(5), logp=m(6), grad=m(7), ld_grad=8, scale=1.0,
             ws=m(8), ws_bytes=0, stream=None, flags=0)
    a.update(over)
    return list(a.values())


@pytest.mark.parametrize("temperature", [5e-324, 1e-39, 9.9e-29, 1.01e28, 1e38, 1e308])
def test_temperatures_outside_the_range_are_refused(mem, temperature):  # noqa: F811
    """log2(e)/T or the log-sum times T would leave f32."""
    assert iso.iso_token_logp(*logp_args(mem, temperature=temperature)) == ARG
    assert iso.iso_token_logp_vjp(*vjp_args(mem, temperature=temperature)) == ARG
    assert iso.iso_policy_loss_logits(*head_args(mem, temperature=temperature, ws_bytes=1 << 12)) == ARG


@pytest.mark.parametrize("temperature", [1e-28, 1e-3, 1.0, 1e28])
def test_temperatures_inside_the_range_are_taken(mem, temperature):  # noqa: F811
    """Past the checks of arguments: to that of the workspace, or to a call without rows."""
    assert iso.iso_policy_loss_logits(*head_args(mem, temperature=temperature)) == WS
    assert iso.iso_token_logp(*logp_args(mem, temperature=temperature, rows=0)) == iso.ISO_OK
    assert iso.iso_token_logp_vjp(*vjp_args(mem, temperature=temperature, rows=0)) == iso.ISO_OK

"""Refusals and sizes of the loss entry points, through the C ABI and the
binding.  No kernel is launched here."""
from __future__ import annotations

import ctypes

import pytest

from lower_convex_hull_amd import iso

ARG, WS, OK = iso.ISO_ERR_ARG, iso.ISO_ERR_WORKSPACE, iso.ISO_OK


@pytest.fixture(scope="module")
def mem():
    buf = ctypes.create_string_buffer(1 << 16)
    base = (ctypes.addressof(buf) + 255) // 256 * 256
    place = lambda k=0: base + 4096 * k  # noqa: E731
    place.keep = buf
    return place


def logp_args(m, **over):
    a = dict(logits=m(0), dtype=iso.ISO_DT_F32, rows=2, vocab=8, ld=8, target=m(1), temperature=1.0, logp=m(2),
             lse=m(3), entropy=None, ws=m(4), ws_bytes=1 << 12, stream=None)
    a.update(over)
    return list(a.values())


BAD_LOGP = [dict(dtype=3), dict(dtype=-1), dict(rows=-1), dict(vocab=0), dict(vocab=-4), dict(ld=7), dict(vocab=1 << 31),
            dict(temperature=0.0), dict(temperature=-1.0), dict(temperature=float("nan")), dict(temperature=float("inf")),
            dict(logits=None), dict(target=None), dict(logp=None), dict(lse=None), dict(rows=1 << 31),
            dict(rows=1 << 30, ld=1 << 60)]


@pytest.mark.parametrize("over", BAD_LOGP, ids=str)
def test_token_logp_refuses(mem, over):
    assert iso.iso_token_logp(*logp_args(mem, **over)) == ARG


def test_token_logp_refuses_places(mem):
    assert iso.iso_token_logp(*logp_args(mem, logits=mem(0) + 2)) == ARG  # not aligned to f32
    assert iso.iso_token_logp(*logp_args(mem, target=mem(1) + 2)) == ARG
    assert iso.iso_token_logp(*logp_args(mem, logp=mem(0) + 32)) == ARG  # overlaps the logits
    assert iso.iso_token_logp(*logp_args(mem, lse=mem(2) + 4)) == ARG  # overlaps logp
    assert iso.iso_token_logp(*logp_args(mem, entropy=mem(1))) == ARG  # overlaps target
    assert iso.iso_token_logp(*logp_args(mem, ws=mem(4) + 8)) == ARG
    assert iso.iso_token_logp(*logp_args(mem, rows=0, logits=None, target=None)) == OK


def vjp_args(m, **over):
    a = dict(logits=m(0), dtype=iso.ISO_DT_F32, rows=2, vocab=8, ld=8, target=m(1), temperature=1.0, lse=m(2),
             entropy=None, g_logp=m(3), g_entropy=None, grad=m(4), ld_grad=8, stream=None)
    a.update(over)
    return list(a.values())


@pytest.mark.parametrize("over", [dict(dtype=7), dict(vocab=0), dict(ld=4), dict(ld_grad=7), dict(temperature=0.0),
                                  dict(logits=None), dict(target=None), dict(lse=None), dict(g_logp=None),
                                  dict(grad=None)], ids=str)
def test_vjp_refuses(mem, over):
    assert iso.iso_token_logp_vjp(*vjp_args(mem, **over)) == ARG


def test_vjp_refuses_places(mem):
    assert iso.iso_token_logp_vjp(*vjp_args(mem, g_entropy=mem(5))) == ARG  # without the entropy
    assert iso.iso_token_logp_vjp(*vjp_args(mem, grad=mem(0) + 4)) == ARG  # overlaps the logits, not in their place
    assert iso.iso_token_logp_vjp(*vjp_args(mem, grad=mem(0), ld_grad=9)) == ARG  # in place, another stride
    assert iso.iso_token_logp_vjp(*vjp_args(mem, grad=mem(3))) == ARG
    assert iso.iso_token_logp_vjp(*vjp_args(mem, rows=0)) == OK


def pref_args(m, **over):
    a = dict(logp=m(0), ref=m(1), mask=None, off=m(2), pairs=2, tokens=16, beta=0.1, smooth=0.0, loss=m(3), each=m(4),
             reward=m(5), grad=m(6), scale=1.0, ws=m(7), ws_bytes=1 << 12, stream=None, flags=0)
    a.update(over)
    return list(a.values())


BAD_PREF = [dict(logp=None), dict(loss=None), dict(each=None), dict(reward=None), dict(pairs=-1), dict(tokens=-1),
            dict(tokens=1 << 31), dict(beta=0.0), dict(beta=-1.0), dict(beta=float("nan")), dict(beta=float("inf")),
            dict(smooth=-0.1), dict(smooth=0.6), dict(smooth=float("nan")), dict(smooth=0.1, flags=iso.ISO_PREF_SQUARED),
            dict(flags=4), dict(scale=float("inf")), dict(off=None, tokens=15), dict(off=None, pairs=0, tokens=4)]


@pytest.mark.parametrize("over", BAD_PREF, ids=str)
def test_pref_refuses(mem, over):
    assert iso.iso_pref_loss(*pref_args(mem, **over)) == ARG


def test_pref_refuses_places(mem):
    for over in (dict(grad=mem(0)), dict(grad=mem(1) + 32), dict(loss=mem(4)), dict(reward=mem(2)), dict(logp=mem(0) + 1),
                 dict(off=mem(2) + 2), dict(grad=mem(6) + 2)):
        assert iso.iso_pref_loss(*pref_args(mem, **over)) == ARG
    need = iso.iso_pref_loss_workspace_bytes(16, 2)
    assert need > 0
    assert iso.iso_pref_loss(*pref_args(mem, ws_bytes=need - 1)) == WS
    assert iso.iso_pref_loss(*pref_args(mem, ws=None, ws_bytes=0)) == WS
    assert iso.iso_pref_loss(*pref_args(mem, ws=mem(7) + 16)) == ARG


def policy_args(m, **over):
    a = dict(logp=m(0), old=m(1), ref=m(2), adv=m(3), mask=None, off=m(4), seqs=2, tokens=16, lo=0.2, hi=0.2, kl=0.1,
             norm=0.0, loss=m(5), counts=m(6), grad=m(7), scale=1.0, ws=m(8), ws_bytes=1 << 12, stream=None, flags=0)
    a.update(over)
    return list(a.values())


BAD_POLICY = [dict(logp=None), dict(old=None), dict(adv=None), dict(loss=None), dict(counts=None), dict(seqs=-1),
              dict(tokens=-1), dict(tokens=1 << 31), dict(lo=-0.1), dict(lo=1.5), dict(lo=float("nan")), dict(hi=-0.1),
              dict(hi=float("nan")), dict(kl=float("nan")), dict(ref=None), dict(norm=-1.0), dict(norm=float("inf")),
              dict(scale=float("nan")), dict(flags=4), dict(off=None, tokens=15), dict(off=None, seqs=0)]


@pytest.mark.parametrize("over", BAD_POLICY, ids=str)
def test_policy_refuses(mem, over):
    assert iso.iso_policy_loss(*policy_args(mem, **over)) == ARG


def test_policy_refuses_places(mem):
    for over in (dict(grad=mem(0)), dict(grad=mem(1)), dict(grad=mem(2)), dict(loss=mem(6)), dict(counts=mem(3)),
                 dict(old=mem(1) + 2), dict(adv=mem(3) + 1)):
        assert iso.iso_policy_loss(*policy_args(mem, **over)) == ARG
    need = iso.iso_policy_loss_workspace_bytes(16, 2)
    assert iso.iso_policy_loss(*policy_args(mem, ws_bytes=need - 1)) == WS
    assert iso.iso_policy_loss(*policy_args(mem, ws=None)) == WS
    assert iso.iso_policy_loss(*policy_args(mem, ws=mem(8) + 16)) == ARG


def head_args(m, **over):
    a = dict(logits=m(0), dtype=iso.ISO_DT_F32, rows=4, vocab=8, ld=8, target=m(1), temperature=1.0, old=m(2), ref=m(3),
             adv=m(4), off=m(5), seqs=2, lo=0.2, hi=0.2, kl=0.1, norm=0.0, loss=m(6), counts=m(7), logp=m(8), grad=m(9),
             ld_grad=8, scale=1.0, ws=m(10), ws_bytes=1 << 13, stream=None, flags=0)
    a.update(over)
    return list(a.values())


BAD_HEAD = [dict(dtype=9), dict(vocab=0), dict(ld=7), dict(ld_grad=7), dict(temperature=0.0), dict(logits=None),
            dict(target=None), dict(old=None), dict(adv=None), dict(loss=None), dict(counts=None), dict(logp=None),
            dict(lo=2.0), dict(hi=-1.0), dict(ref=None), dict(norm=-2.0), dict(flags=8), dict(off=None, seqs=3),
            dict(rows=-1)]


@pytest.mark.parametrize("over", BAD_HEAD, ids=str)
def test_policy_logits_refuses(mem, over):
    assert iso.iso_policy_loss_logits(*head_args(mem, **over)) == ARG


def test_policy_logits_refuses_places(mem):
    for over in (dict(grad=mem(0) + 4), dict(grad=mem(0), ld_grad=16), dict(logp=mem(0)), dict(loss=mem(0) + 64),
                 dict(grad=mem(2)), dict(logp=mem(1))):
        assert iso.iso_policy_loss_logits(*head_args(mem, **over)) == ARG
    need = iso.iso_policy_loss_logits_workspace_bytes(4, 8, 2, iso.ISO_DT_F32)
    assert iso.iso_policy_loss_logits(*head_args(mem, ws_bytes=need - 1)) == WS
    assert iso.iso_policy_loss_logits(*head_args(mem, ws=None)) == WS


def test_tokens_without_sequences_are_refused(mem):
    """Offsets of no sequence hold no token."""
    assert iso.iso_pref_loss(*pref_args(mem, pairs=0)) == ARG
    assert iso.iso_policy_loss(*policy_args(mem, seqs=0)) == ARG
    assert iso.iso_policy_loss_logits(*head_args(mem, seqs=0)) == ARG


def test_binding_refuses_cpu_tensors():
    import torch

    x = torch.zeros(2, 8)
    t = torch.zeros(2, dtype=torch.int32)
    for call in (lambda: iso.token_logp(x, t), lambda: iso.token_logp_vjp(x[:, 0], x, t, x[:, 0]),
                 lambda: iso.pref_loss(x, None), lambda: iso.policy_loss(x, x, x[:, 0]),
                 lambda: iso.policy_loss_logits(x, t, x[:, 0], x[0, :1])):
        with pytest.raises(TypeError):
            call()

"""A tensor that a call is given to write has its version raised, so that autograd
knows that what it saved is gone. On the CPU: nothing is launched."""
import types

import pytest
import torch

from grpo_loss_gb300 import _lib as L


@pytest.fixture(autouse=True)
def host_only(monkeypatch):
    names = ("grpo_sample", "grpo_layernorm_fwd", "grpo_layernorm_bwd", "grpo_adamw_step")
    monkeypatch.setattr(L, "lib", lambda: types.SimpleNamespace(**dict.fromkeys(names)))
    monkeypatch.setattr(L, "_call", lambda fn, where, device, stream, *args: None)
    monkeypatch.setattr(L, "_device_of", lambda t, name: t.device)


def results():
    """Every output that a call may be given, by the call that writes it."""
    f, i = torch.zeros, lambda n: torch.zeros(n, dtype=torch.int32)
    x, w, r, ws = f(4, 8), f(8), f(4), f(64)
    return {
        "y": (f(4, 8), lambda t: L.layernorm_fwd(x, w, y=t)),
        "mean": (f(4), lambda t: L.layernorm_fwd(x, w, mean=t)),
        "rstd": (f(4), lambda t: L.layernorm_fwd(x, w, rstd=t)),
        "in place": (f(4, 8), lambda t: L.layernorm_fwd(t, w, y=t)),
        "dx": (f(4, 8), lambda t: L.layernorm_bwd(x, w, x, r, r, dx=t, workspace=ws)),
        "dx is dy": (f(4, 8), lambda t: L.layernorm_bwd(x, w, t, r, r, dx=t, workspace=ws)),
        "dweight": (f(8), lambda t: L.layernorm_bwd(x, w, x, r, r, dweight=t, workspace=ws)),
        "dbias": (f(8), lambda t: L.layernorm_bwd(x, w, x, r, r, dbias=t, workspace=ws)),
        "tokens": (i(4), lambda t: L.sample(x, r, tokens=t)),
        "logp": (f(4), lambda t: L.sample(x, r, logp=t)),
    }


@pytest.mark.parametrize("name", list(results()))
def test_a_given_output_is_known_to_be_written(name):
    t, call = results()[name]
    before = t._version
    call(t)
    assert t._version > before


def test_a_saved_output_is_not_used_again():
    leaf = torch.ones(4, 8, requires_grad=True)
    y, (_, call) = torch.ones(4, 8), results()["y"]
    loss = (leaf * y).sum()                             # saves y
    call(y)
    with pytest.raises(RuntimeError, match="inplace operation"):
        loss.backward()


@pytest.mark.parametrize("name", list(results()))
def test_inference_tensors_are_taken(name):
    """They have no version to raise."""
    with torch.inference_mode():
        t, call = results()[name]
        call(t)


def test_masters_and_parameters_of_a_step(monkeypatch):
    import grpo_loss_gb300 as G
    monkeypatch.setattr(L, "_ptr", lambda t, name: t.data_ptr())
    p, g = torch.zeros(8, dtype=torch.bfloat16), torch.zeros(8)
    opt, out = G.AdamW([p], master=True), G.AdamW([p.clone()], master=True)
    seen = [t._version for o in (opt, out) for t in (o.params[0], o.masters[0])]
    opt.step([g])
    mine = [t._version for o in (opt, out) for t in (o.params[0], o.masters[0])]
    assert [a > b for a, b in zip(mine, seen)] == [True, True, False, False]
    opt.step([g], out=out)
    both = [t._version for o in (opt, out) for t in (o.params[0], o.masters[0])]
    assert [a > b for a, b in zip(both, mine)] == [False, False, True, True]

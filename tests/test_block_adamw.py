"""What ExpertBlock keeps for its AdamW steps between calls (no GPU needed: the
library's calls are replaced by ones that do nothing, the buffers are host tensors)."""

import unittest.mock as mock

import pytest
import torch

import moe_grouped_mlp_amd as mg
from moe_grouped_mlp_amd import binding as B
from moe_grouped_mlp_amd import block as blk_mod

E, H, I, T, K = 2, 128, 128, 16, 2
CALLS = ("moe_permute", "moe_weight_repack_interleave", "moe_adamw", "moe_grad_sumsq", "moe_router_gate", "moe_router_bias_update")


@pytest.fixture
def block():
    with mock.patch.multiple(B, moe_grouped_mlp_workspace_size=lambda *a: 0, moe_grad_workspace_size=lambda n: 64 * n,
                             **{n: lambda *a, **kw: None for n in CALLS}):
        blk = mg.ExpertBlock(E, H, I, T, K, wgrad=True, device="cpu")
        for t in (blk.w1i, blk.w2, blk.dw1, blk.dw2):
            t.zero_()
        yield blk


def _tensors(st):
    return [*st["m"], *st["v"], *(st["m_scale"] or ()), *(st["v_scale"] or ()), *(st["master"] or ()), st["step"]]


def _load(block, value):
    """w1i is repacked by the library, which does nothing here."""
    block.w1i.fill_(value)
    block.load_weights(torch.zeros(E, 2 * I, H, dtype=torch.bfloat16), torch.full((E, H, I), value, dtype=torch.bfloat16))


def _capture(block, **kw):
    with mock.patch.object(blk_mod, "_capturing", lambda t: True):
        block.adamw_step(0.1, **kw)


@pytest.mark.parametrize("state,master", [(mg.STATE_F32, True), (mg.STATE_FP8, False), (mg.STATE_FP8, True)])
def test_load_weights_begins_the_states_anew_in_place(block, state, master):
    kw = dict(state=state, master=master, capturable=True)
    block.adamw_step(0.1, **kw)
    _capture(block, **kw)
    kept = _tensors(block._adamw)
    for t in kept:
        t.fill_(7)
    _load(block, 2.0)
    now = _tensors(block._adamw)
    assert len(now) == len(kept) and all(a is b for a, b in zip(now, kept))
    copies = block._adamw["master"] or []
    assert all((t == 2).all() for t in copies) and len(copies) == 2 * master
    assert not any(t.any() for t in now if not any(t is c for c in copies))
    block.adamw_step(0.1, **kw)
    assert block._adamw["step"].item() == 1 and all(a is b for a, b in zip(_tensors(block._adamw), kept))


def test_states_of_a_graph_stay_when_the_kind_changes(block):
    """Steps of another kind may follow load_weights(); the states that a graph was
    captured with stay, and are begun anew with each load too."""
    one, other = dict(capturable=True), dict(state=mg.STATE_FP8)
    block.adamw_step(0.1, **one)
    _capture(block, **one)
    first = block._adamw
    with pytest.raises(ValueError, match="kind"):
        block.adamw_step(0.1, **other)
    _load(block, 1.0)
    block.adamw_step(0.1, **other)
    assert block._adamw is not first and block.adamw_steps == 1
    for t in _tensors(first):
        t.fill_(7)
    _load(block, 3.0)
    assert all((t == 3).all() for t in first["master"]) and not first["m"][0].any() and not first["step"].any()
    assert (block._adamw["master"][1] == 3).all()
    block.adamw_step(0.1, **one)
    assert block._adamw is first


def test_states_of_no_graph_are_given_back(block):
    block.adamw_step(0.1)
    first = block._adamw
    _load(block, 1.0)
    block.adamw_step(0.1)
    assert block._adamw is first and block.adamw_steps == 1
    _load(block, 1.0)
    block.adamw_step(0.1, state=mg.STATE_FP8)
    assert not block._adamw_captured and block._adamw is not first


@pytest.mark.parametrize("capturable", [False, True])
def test_a_refused_step_is_none(block, capturable):
    """Neither counted nor held to its kind of states."""
    def refuse(**kw):
        raise mg.MoeError("moe_adamw", 1, "no")

    def steps():
        return block._adamw["step"].item() if capturable else block.adamw_steps

    with mock.patch.object(B, "moe_adamw", refuse):
        with pytest.raises(mg.MoeError):
            block.adamw_step(0.1, state=mg.STATE_FP8)
        with pytest.raises(mg.MoeError):
            block.adamw_step(0.1, capturable=capturable)
        assert steps() == 0
    seen = []
    with mock.patch.object(B, "moe_adamw", lambda **kw: seen.append(kw["step_dev"].item() if capturable else kw["step"])):
        block.adamw_step(0.1, capturable=capturable)
        with mock.patch.object(B, "moe_adamw", refuse), pytest.raises(mg.MoeError):
            block.adamw_step(float("nan"), capturable=capturable)
        block.adamw_step(0.1, capturable=capturable)
    assert seen == [1, 2] and steps() == 2


def test_norm_over_other_gradients(block):
    """extra takes part in the norm and nothing else; a sum that is given is taken."""
    more = [torch.zeros(5), torch.zeros(3)]
    with mock.patch.object(B, "moe_grad_sumsq") as total, mock.patch.object(B, "moe_adamw") as step:
        block.adamw_step(0.1, max_norm=2.0, extra=more)
        assert [t is u for t, u in zip(total.call_args.kwargs["tensors"], (block.dw1, block.dw2, *more))] == [True] * 4
        assert len(step.call_args.kwargs["params"]) == 2 and step.call_args.kwargs["sumsq"] is block.grad_sumsq
        total.reset_mock()
        given = torch.ones(1, dtype=torch.float64)
        block.adamw_step(0.1, max_norm=2.0, sumsq=given)
        assert step.call_args.kwargs["sumsq"] is given and not total.called
    for kw in (dict(extra=more), dict(sumsq=given), dict(max_norm=1.0, extra=more, sumsq=given)):
        with pytest.raises(ValueError):
            block.adamw_step(0.1, **kw)
    assert block.adamw_steps == 2


def test_the_norm_is_clip_grads_own(block):
    """adamw_step() leaves it (it held nothing before), and both sum into one buffer."""
    block.adamw_step(0.1, max_norm=1.0)
    assert block.grad_norm is None
    total = block.grad_sumsq
    with mock.patch.object(B, "moe_grad_clip"):
        norm = block.clip_grads(1.0)
    assert norm is block.grad_norm and block.grad_sumsq is total


@pytest.mark.parametrize("kw", [dict(), dict(state=mg.STATE_FP8, master=False), dict(capturable=True)])
def test_states_are_saved_and_loaded_in_place(block, kw):
    for call in (block.adamw_state,):
        with pytest.raises(RuntimeError, match="adamw_step"):
            call()
    block.adamw_step(0.1, **kw)
    block.adamw_step(0.1, **kw)
    for i, t in enumerate(_tensors(block._adamw)[:-1]):
        t.fill_(i + 1)
    saved = {k: [t.clone() for t in v] if isinstance(v, list) else v.clone() if torch.is_tensor(v) else v for k, v in block.adamw_state().items()}
    kept = _tensors(block._adamw)
    _load(block, 1.0)
    block.load_adamw_state(saved)
    now = _tensors(block._adamw)
    assert all(a is b for a, b in zip(now, kept)) and all((t == i + 1).all() for i, t in enumerate(now[:-1]))
    block.adamw_step(0.1, **kw)
    assert (block._adamw["step"].item() if kw.get("capturable") else block.adamw_steps) == 3
    with pytest.raises(ValueError, match="kind"):
        block.load_adamw_state({**saved, "state": 1 - saved["state"]})
    with pytest.raises(ValueError, match="sizes"):
        block.load_adamw_state({**saved, "m": [t[1:] for t in saved["m"]]})


def test_the_blocks_own_states_are_no_checkpoint(block):
    """load_weights() has begun them anew: loading them would go on from zeros with
    the old step's number."""
    block.adamw_step(0.1)
    own = block.adamw_state()
    _load(block, 1.0)
    with pytest.raises(ValueError, match="own"):
        block.load_adamw_state(own)
    assert block.adamw_steps == 0

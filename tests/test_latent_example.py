"""How the serving example hands its states to the two KDA calls (no GPU: the calls are replaced)."""
import torch

from examples import latent_serving as E


def test_only_the_recurrent_call_updates_states_in_place(monkeypatch):
    """include/kda.h allows one buffer as initial and final state for kda_fwd_recurrent, not for kda_fwd."""
    seen = {}

    def stand_in(name):
        def call(q, k, v, *args, initial_state, final_state, **kw):
            seen[name] = initial_state, final_state, initial_state.clone()
            final_state.fill_(7.0)
            return torch.zeros_like(v)
        return call

    for name in ("kda_fwd", "kda_fwd_recurrent"):
        monkeypatch.setattr(E, name, stand_in(name))
    layers = E.Layers(64, 2, torch.device("cpu"), torch.Generator().manual_seed(0))
    for name, tokens in (("kda_fwd", 5), ("kda_fwd_recurrent", 1)):
        states = torch.full((1, 2, 128, 128), 3.0)
        layers.kda(torch.ones(1, tokens, 64, dtype=torch.bfloat16), states)
        initial, final, before = seen[name]
        assert final is states and (before == 3.0).all() and (states == 7.0).all()
        assert (initial.data_ptr() == states.data_ptr()) == (name == "kda_fwd_recurrent")

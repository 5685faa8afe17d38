"""The example that runs sampling, norm, loss and optimizer together."""
import importlib.util
import os

import pytest


def load():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "grpo_iterations.py")
    spec = importlib.util.spec_from_file_location("grpo_iterations", path)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def test_example_imports_without_a_gpu():
    assert load().VOCAB % 8 == 0


@pytest.mark.gpu
@pytest.mark.parametrize("state_bits", [32, 8])
def test_reward_rises_over_the_iterations(state_bits):
    """From 1/8, what the untrained policy draws, to half of the tokens and more."""
    rewards, greedy = load().run(40, seed=0, state_bits=state_bits, quiet=True)
    assert 0.05 < rewards[0] < 0.2
    assert sum(rewards[-5:]) / 5 > 0.5 and greedy > 0.5

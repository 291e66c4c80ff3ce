"""Refusals of the state cache's binding, before any allocation or launch (no GPU needed)."""
import pytest


def test_read_refuses_malformed_arguments_without_an_output():
    import torch
    import selective_state_space_75_amd as m
    codes, exps = torch.zeros(2, 5, dtype=torch.int8), torch.zeros(2, 1, dtype=torch.uint8)
    with pytest.raises(ValueError, match="codes"):
        m.state_cache_read(codes[0], exps)
    with pytest.raises(TypeError, match="codes"):
        m.state_cache_read([1, 2], exps)
    with pytest.raises(TypeError, match="codes"):
        m.state_cache_write(torch.zeros(2, 5), None, exps)
    with pytest.raises(ValueError, match="slots"):
        m.state_cache_read(codes, exps, slots=[0, 1])
    with pytest.raises(ValueError, match="slots"):
        m.state_cache_read(codes, exps, slots=torch.tensor(1, dtype=torch.int32))
    with pytest.raises(ValueError, match="GPU device"):
        m.state_cache_read(codes, exps)

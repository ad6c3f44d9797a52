"""The binding's stream lookup goes through torch's own initialisation of CUDA."""
import pytest
import torch

import kv_cache_block_lowrank_gb300 as hss


class Refused(RuntimeError):
    pass


def test_the_current_stream_asks_torch_to_initialise_cuda(monkeypatch):
    # torch raises here in a forked child of a process that has used CUDA, for instance
    def refuse():
        raise Refused

    monkeypatch.setattr(torch.cuda, "_lazy_init", refuse)
    with pytest.raises(Refused):
        hss._stream(None)


def test_a_given_stream_is_taken_as_it_is(monkeypatch):
    monkeypatch.setattr(torch.cuda, "_lazy_init", None)
    assert hss._stream(0) == 0 and hss._stream(1234) == 1234

    class Stream:
        cuda_stream = 77

    assert hss._stream(Stream()) == 77

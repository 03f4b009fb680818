"""What the decoder asks of a target and what becomes of device status words, on the host: no
GPU needed."""

import pytest

from draft_sampling_lossless_gb300 import decode


class Words:
    """Stands for whatever has a status() of its own."""

    def __init__(self, word=0):
        self.word = word

    def status(self, ws=None):
        return self.word


def decoder(target, step=0):
    d = object.__new__(decode.Decoder)
    d.t, d.step_, d.caches, d.ws = target, Words(step), [Words()], {}
    return d


def test_a_target_without_a_status_of_its_own_is_accepted():
    class Plain:
        def forward(self, tokens, attention):
            return None

    decoder(Plain()).check()
    with pytest.raises(RuntimeError, match="0x10"):
        decoder(Plain(), step=0x10).check()


def test_a_targets_status_is_looked_at():
    decoder(Words()).check()
    with pytest.raises(RuntimeError, match="0x10"):
        decoder(Words(0x10)).check()

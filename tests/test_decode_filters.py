"""The decoder's sampled step verifies with the temperature that its rows were filtered with (CPU)."""
import pytest
import torch


@pytest.fixture(scope="module")
def decoder():
    from speculative_decoding_verification_35_gb300 import _build
    _build.build()
    from speculative_decoding_verification_35_gb300 import decode
    return decode.Decoder(3, 64, device="cpu")


@pytest.mark.parametrize("temperature", [[0.7, 0.8, 0.7], [1.0, 0.0, 0.5], torch.tensor([0.5, 0.25, 0.5]), [0.7, 0.7, 0.70001]])
def test_temperatures_that_differ_are_refused(decoder, temperature):
    with pytest.raises(ValueError, match="one temperature"):
        decoder.filters(temperature)


class Reached(Exception):
    pass


@pytest.mark.parametrize("asked,verified,ok", [(0.7, 0.7, True), ([0.7, 0.0, 0.7], 0.7, True), (0.7, 0.8, False), (0.7, 0.0, False),
                                               (0.0, 0.9, True), ([0.0, 0.0, 1.0], 1.0, True), ([0.0, 0.0, 1.0], 0.0, False)])
def test_a_step_verifies_with_its_filters_temperature(decoder, monkeypatch, asked, verified, ok):
    def stop(*args, **kw):
        raise Reached
    filters = decoder.filters(asked, 5, [0.9, 1.0, 0.8])
    assert [f.temperature.tolist() if f.request is None else f.request.tolist() for f in filters][1:] == [
        [0, 0, 0, 1, 1, 1, 2, 2, 2], [0] * 4 + [1] * 4 + [2] * 4]
    monkeypatch.setattr(type(filters[0]), "sample", stop)
    with pytest.raises(Reached if ok else ValueError):
        decoder.sampled_step(filters, verified)

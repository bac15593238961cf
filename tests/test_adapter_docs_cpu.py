"""What the adapter calls cannot check on their operands stands in their
documentation, in the header and in the binding alike."""
import os

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PKG = os.path.join(ROOT, "w4a8_rotated_quantized_amd")


def _header():
    with open(os.path.join(ROOT, "include", "convrot.h")) as f:
        text = f.read()
    lo = text.index("convrot_lora_forward / convrot_lora_backward - ")
    return " ".join(text[lo:text.index("convrot_act_checkpoint / convrot_act_backward - ")].replace("\n *", " ").split())


@pytest.fixture(scope="module")
def cr():
    pytest.importorskip("torch")
    if not os.path.exists(os.path.join(PKG, "libconvrot.so")):
        pytest.skip("libconvrot.so not built")
    import w4a8_rotated_quantized_amd as m
    return m


def test_codes_of_a_smoothed_input(cr):
    assert "Codes made with `smooth` stand for x * smooth" in _header()
    assert "divided by smooth[k]" in _header()
    assert "smooth stand for x * smooth" in " ".join(cr.convrot_lora_backward.__doc__.split())


def test_infinite_bf16_values():
    text = _header()
    assert "an infinite bf16 value meets a float32 factor (up in out, down in dx, dy in d_up, x in d_down)" in text
    assert "are infinite or NaN" in text


def test_autograd_records_nothing(cr):
    for call, back in ((cr.convrot_lora_forward, "convrot_lora_backward"), (cr.convrot_act_checkpoint, "convrot_act_backward")):
        text = " ".join(call.__doc__.split())
        assert "Not recorded by autograd" in text and back in text

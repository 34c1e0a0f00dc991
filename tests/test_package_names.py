"""The package's names are the binding's, also after the binding's change (CPU)."""
import gated_delta_rule_recurrent_b200 as gdr
from gated_delta_rule_recurrent_b200 import binding


def test_a_name_follows_the_binding(monkeypatch):
    for name in ("decode", "linear_attention_decode", "state_quantize", "last_launch"):
        assert getattr(gdr, name) is getattr(binding, name)  # used once before

        def other():
            return name

        monkeypatch.setattr(binding, name, other)
        assert getattr(gdr, name) is other
        monkeypatch.undo()
        assert getattr(gdr, name) is getattr(binding, name)


def test_all_names_are_there_and_no_others():
    for name in gdr.__all__:
        assert getattr(gdr, name) is getattr(binding, name)
    try:
        gdr.no_such_name
    except AttributeError as e:
        assert "no_such_name" in str(e)
    else:
        raise AssertionError("no AttributeError")

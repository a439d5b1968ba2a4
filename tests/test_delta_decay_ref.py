"""The reference of the decay gradients against reverse-mode differentiation."""
import delta_ref as ref
from delta_decay_ref import decay_gradients


def test_decay_gradients_are_reverse_modes():
    d, gr = ref.make(2, 40, 2, 8, 4, 1, 5, "f32", dt_hi=1.0), ref.make_grads(2, 40, 2, 8, 4, 5, "f32")
    want = ref.grads(d, gr)
    ddt, dA, s = decay_gradients(d, gr)
    assert ref.rel(ddt, want["ddt"]) < 1e-13 and ref.rel(dA, want["dA"]) < 1e-13
    assert (s >= 0).all() and ((ddt / d["A"].double()).abs() <= s * (1 + 1e-12)).all()

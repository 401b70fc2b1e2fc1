"""Rotary plans with axes that turn no pair (no GPU)."""

import pytest

import paged_kv_cache_145_gb300 as pkv


@pytest.mark.parametrize("sections", [[64, 0, 0], [0, 0, 64], [16, 0, 48], [0, 64, 0], [8, 8, 8, 8, 0, 0, 0, 0]])
def test_every_section_is_an_axis(sections):
    """One axis per section, whether it has pairs or not."""
    rot = pkv.RotaryAxes.sections(sections)
    assert rot.num_axes == rot._c.num_axes == len(sections)
    assert list(rot._c.axis[:sum(sections)]) == [a for a, n in enumerate(sections) for _ in range(n)]


def test_axes_of_a_plan_can_be_named():
    rot = pkv.RotaryAxes(8, [1.0, 0.5, 0.25, 0.125], [0, 0, 1, 1], num_axes=3)
    assert rot.num_axes == rot._c.num_axes == 3
    rot = pkv.RotaryAxes(4, [1.0, 0.5], num_axes=2)       # every pair on axis 0
    assert rot.num_axes == 2 and list(rot._c.axis[:2]) == [0, 0]
    assert pkv.RotaryAxes(4, [1.0, 0.5], [1, 0]).num_axes == 2
    assert pkv.RotaryAxes(4, [1.0, 0.5]).num_axes == 1


def test_refusals():
    with pytest.raises(ValueError):
        pkv.RotaryAxes(4, [1.0, 1.0], [0, 2], num_axes=2)  # a pair on an axis that is not there
    with pytest.raises(ValueError):
        pkv.RotaryAxes(4, [1.0, 1.0], num_axes=0)
    with pytest.raises(RuntimeError):
        pkv.RotaryAxes(4, [1.0, 1.0], num_axes=9)
    with pytest.raises(RuntimeError):
        pkv.RotaryAxes.sections([1, 1, 1, 1, 1, 1, 1, 1, 0])

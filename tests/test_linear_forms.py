"""The forms that tests/linear_forms.py names are those that the plans choose (host logic only), so
that its calls on the GPU reach every one of them."""
from __future__ import annotations

from host_forms_util import ask, build
from linear_forms import FEW, TILES, WIDE


def test_forms_are_as_named(tmp_path):
    cases = FEW + TILES + WIDE
    for case, line in zip(cases, ask(build(tmp_path), [c[:5] for c in cases])):
        assert line == case[5], (case, line)


def test_every_form_is_named():
    few = {tuple(int(v) for v in c[5].split()[1:4]) + (c[4],) for c in FEW}
    for nt in (1, 2, 3, 4):
        for gated in (0, 1):
            for r in ((2, 4) if gated else (1, 2, 3, 4)):
                assert (nt, r, 1, gated) in few
        if nt >= 3:                       # waves that share the tokens
            assert (nt, 2, 4, 0) in few and (nt, 2, 4, 1) in few
    blocks = {(b, c[3], c[4]) for c in TILES for b in (int(v) for v in c[5].split()[3:])}
    assert all((b, g, gated) in blocks for b in (1, 3, 4, 5, 6, 7, 8) for g in (32, 64, 128, -1) for gated in (0, 1))
    wide = {(c[3], c[4]) for c in WIDE if c[5].startswith("tiles 1")}
    assert len(wide) == 8
    assert {int(v) for c in WIDE for v in c[5].split()[3:]} == {1, 2, 3, 4}

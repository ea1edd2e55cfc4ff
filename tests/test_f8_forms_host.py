"""Every kernel of f8_linear is reached by a size of its GPU tests, with the loops that only long rows enter."""
import f8_forms as forms


def test_the_tiles_are_those_that_the_rule_knows():
    assert [t[:2] for t in forms.tiles()] == [(64, 32), (64, 64), (64, 128), (128, 128), (128, 256), (256, 256)]


def test_every_form_has_sizes():
    reached = {}
    for size in forms.SIZES + forms.LONG + forms.ODD + [(5, 70, 9)]:
        reached.setdefault(forms.form(*size), []).append(size)
    assert set(reached) == forms.FORMS
    for name in ("tile 64x64", "tile 64x128", "tile 128x128", "tile 128x256", "turns 256x256"):
        blocks = {forms.up(k, 128) for _, _, k in reached[name]}
        assert 1 in blocks and any(b % 2 for b in blocks - {1}) and any(b % 2 == 0 for b in blocks), (name, blocks)
        assert any(k % 128 for _, _, k in reached[name]), name


def test_long_rows_go_round_again():
    strips = set()
    for m, n, k in forms.LONG:
        name = forms.form(m, n, k)
        assert name.startswith("strip") and forms.up(k, 128) > 64 * forms.waves(name), (m, n, k, name)
        strips.add(name)
    assert strips == {f for f in forms.FORMS if f.startswith("strip")}
    assert any(forms.form(*s) == "any" and forms.up(s[2], 128) > 32 for s in forms.ODD)

"""The oracle's capped scores and prefixes against their pins, and planted mistakes that the pins
have to catch."""
import pytest

import oracle
import score_pins

PLANTS = [
    ("cap left out", "s = cap * tanh(s / cap);", "s = s;"),
    ("cap not multiplied back", "s = cap * tanh(s / cap);", "s = tanh(s / cap);"),
    ("cap's derivative left out", "dP[i * N + jj] *= G[i * N + jj];", "dP[i * N + jj] *= 1.0;"),
    ("cap's derivative transposed", "dP[i * N + jj] *= G[i * N + jj];",
     "dP[i * N + jj] *= G[jj * N + i];"),
    ("cap's derivative without the square", "1.0 - tanh(s / cap) * tanh(s / cap)",
     "1.0 - tanh(s / cap)"),
    ("prefix off by one", "if (j < prefix) return 1;", "if (j <= prefix) return 1;"),
    ("prefix of queries", "if (j < prefix) return 1;", "if (i < prefix) return 1;"),
    ("prefix of the first entry for all", "return prefixes ? prefixes[bh / H] : 0;",
     "return prefixes ? prefixes[0] : 0;"),
]


@pytest.mark.parametrize("pin", score_pins.ALL_PINS, ids=lambda p: p.__name__)
def test_pin(orc, pin):
    pin(orc)


@pytest.mark.parametrize("name,old,new", PLANTS, ids=[p[0] for p in PLANTS])
def test_plant_is_caught(tmp_path, name, old, new):
    src = open(oracle.SOURCE).read()
    assert src.count(old) == 1, "plant site must be unique: %r" % old
    bad = tmp_path / "oracle_planted.c"
    bad.write_text(src.replace(old, new))
    orc = oracle.Oracle(oracle.build(str(bad), str(tmp_path / "liboracle_planted.so"),
                                     force=True))
    caught = []
    for pin in score_pins.ALL_PINS:
        try:
            pin(orc)
        except AssertionError:
            caught.append(pin.__name__)
    assert caught, "no pin catches the planted mistake: %s" % name

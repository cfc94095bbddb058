"""The order of the prompt attention's items (CPU): every item goes out once, and the GPU cases
meant for turns without key tiles have such turns."""
import pytest

from prompt_items import empty_turns, in_order, key_tiles, loads, turns

# A pair's second CTA has no key tile in a turn that is not its first: packed prompts of which one
# or several have up to 128 rows; the last two have such turns one after the other.
SHORT_AMONG_LONG = [([100, 8092], 4), ([128, 16000], 2), ([3, 17000, 128], 2), ([60, 30000], 1), ([20, 18220, 18, 21], 1),
                    ([113, 18178, 1, 97], 1)]
SMS = 148


@pytest.mark.parametrize("lens,heads", SHORT_AMONG_LONG + [([100, 2900, 300], 2), ([2048], 16), ([0, 5, 700, 0, 256, 257], 3)])
@pytest.mark.parametrize("sms", [148, 132, 7])
def test_every_item_once(lens, heads, sms):
    pairs, given = turns(lens, heads, sms)
    assert sorted(x for mine in given for x in mine) == sorted(in_order(lens, heads))
    for mine in given:
        for s, q, _ in mine:
            for tile in (0, 1):
                rows = lens[s] - 256 * q - 128 * tile
                both = sum(key_tiles(lens, (s, q, 0), tile, r) for r in (0, 1))
                assert both == (2 * q + 1 + tile if rows > 0 else 0)


@pytest.mark.parametrize("lens,heads", SHORT_AMONG_LONG)
def test_cases_have_turns_without_key_tiles(lens, heads):
    assert turns(lens, heads, SMS)[0] and empty_turns(lens, heads, SMS) > 0


def test_some_case_has_two_in_a_row():
    def in_a_row(lens, heads):
        return any(not loads(lens, a, 1) and not loads(lens, b, 1) for mine in turns(lens, heads, SMS)[1] for a, b in zip(mine, mine[1:]))
    assert any(in_a_row(lens, heads) for lens, heads in SHORT_AMONG_LONG)

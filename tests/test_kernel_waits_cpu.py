"""Copies that a kernel issues ahead of their use are not waited for before it: no wait of the
compiler's for every load where the source counts on some being on their way."""

import pytest

from tests.kernel_asm import kernels


def _main_loop(events):
    return events[events.index("mfma"):]


def test_codes_of_the_next_tile_are_on_their_way():
    # the tile loop's copies of codes end a step: the compiler must not wait for them there
    forms = {n: e for n, e in kernels("attn_paged.hip").items() if n.startswith("attn_kernel") and n.endswith("true>")}
    assert len(forms) == 24
    for name, events in forms.items():
        loop = _main_loop(events)
        assert "copy" in loop
        for a, b in zip(loop, loop[1:]):
            assert not (a in ("copy", "load") and b == "wait"), name


def _waits_before_products(events):
    """Whether a wait for every load stands between a tile's copies and its products."""
    waited = False
    for event in _main_loop(events):
        if event in ("copy", "barrier"):
            waited = False
        elif event == "wait":
            waited = True
        elif event == "mfma" and waited:
            return True
    return False


def test_prompt_tiles_are_on_their_way_under_both_products():
    forms = {n: e for n, e in kernels("attn_prompt.hip").items() if n.startswith("prompt_kernel")}
    assert len(forms) == 6
    for name, events in forms.items():
        loop = _main_loop(events)
        assert "copy" in loop and "transpose" in loop
        assert not _waits_before_products(events), name


def test_counted_waits_count_the_loads_of_codes():
    # a step waits for all but the loads of the tile behind: as many as the compiler made of them
    forms = {n: e for n, e in kernels("attn_paged.hip").items() if n.startswith("attn_kernel") and n.endswith("true>")}
    for name, events in forms.items():
        loop, found = _main_loop(events), 0
        for at, event in enumerate(loop):
            if event != "barrier":
                continue
            back = at - 1
            while loop[back] == "edge":
                back -= 1
            if not loop[back].startswith("wait "):
                continue                     # behind the loop
            left, loads = int(loop[back].split()[1]), 0
            while loop[back] not in ("copy", "load"):
                back -= 1
            while loop[back] in ("copy", "load"):
                loads, back = loads + 1, back - 1
            assert loads == left, (name, loads, left)
            found += 1
        assert found >= 1, name


@pytest.mark.parametrize("source,forms", [("attn_paged.hip", 48), ("attn_prompt.hip", 6)])
def test_no_register_spills_to_memory(source, forms):
    # it would be read back behind the copies on their way
    found = {n: e for n, e in kernels(source).items() if "mfma" in e}
    assert len(found) == forms
    assert not [n for n, e in found.items() if "spill" in e]

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

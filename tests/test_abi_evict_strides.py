"""CPU tests: masses that are updated in place have one row stride, in both entries of the bounded cache."""

import pytest

from tests.test_abi_evict import E_INV, P, _evict, _mass, lib  # noqa: F401


@pytest.mark.parametrize("entry", [_mass, _evict])
@pytest.mark.parametrize("kw", [dict(mo=P[5], mos=300), dict(m=P[6], ms=300), dict(mo=P[5], ms=1 << 20)])
def test_masses_in_place_have_one_stride(lib, entry, kw):  # noqa: F811
    assert entry(lib, **kw) == E_INV, lib.bfp8_last_error_message()
    assert b"one stride" in lib.bfp8_last_error_message()

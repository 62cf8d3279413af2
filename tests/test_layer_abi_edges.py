"""Empty tables and batches at the C ABI of the attention entry points,
decided on the host (no GPU needed)."""
import pytest

from test_layer_abi import decode, lib, prompt  # noqa: F401  (lib: a fixture)

TOO_SMALL = -4  # accepted as far as the workspace, of which these calls give none


@pytest.mark.parametrize("call", [decode, prompt])
def test_a_table_of_no_columns_may_be_null(lib, call):
    assert call(lib, tab=None, most=0, ldt=0) == TOO_SMALL
    assert call(lib, most=0, ldt=0) == TOO_SMALL
    assert call(lib, tab=None, most=1, ldt=1) == -1
    assert call(lib, lens=None, tab=None, most=0, ldt=0) == -1


def test_no_sequences_need_no_lengths(lib):
    assert prompt(lib, B=0, tab=None, lens=None, starts=None, q=None, out=None) == 0
    assert decode(lib, B=0, tab=None, lens=None, q=None, out=None) == 0
    assert prompt(lib, B=0, tab=None, lens=None, most=4, ldt=3) == -1

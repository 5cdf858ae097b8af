"""Host checks of the tree operators' calls that name memory they must not touch (no GPU needed:
each call is refused before anything is launched)."""
import ctypes

import pytest

FAKE = 1 << 20   # an address that a refused call never reads


def view(sd, rows, heads=2, cols=16, hd=16):
    s = hd * cols * heads
    return sd.KvView(FAKE, 2 * s * rows, s * rows, s, hd * cols, sd.F32, 1, rows, heads, hd, cols)


def rotary(sd, B, rows, explicit):
    a = sd.RotaryArgs(cache=view(sd, rows), B=B, T=2, heads_q=2, rot_dim=16, table_len=8)
    for f in ("q", "k", "v", "q_out", "table", "dev_status") + (("positions", "columns") if explicit else ("n_committed", "width")):
        setattr(a, f, FAKE)
    return sd.lib.specdec_rotary_append(ctypes.byref(a), None)


@pytest.mark.parametrize("B,rows", [(2, 1), (5, 1), (3, 2)])
def test_a_verification_pass_needs_a_cache_row_per_batch_row(B, rows):
    """With one cache row the batch rows' nodes would all go to columns W - 1 + t of it."""
    import speculative_decoding_specdec_gb300.specdec as sd
    assert rotary(sd, B, rows, explicit=False) == sd.ERR_INVALID_ARG


def test_what_is_taken_is_not_refused():
    """The same arguments with the rows there, and explicit columns in one cache row, get as far as
    the launch (whose outcome depends on there being a GPU, so it is not made: B = 0)."""
    import speculative_decoding_specdec_gb300.specdec as sd
    for explicit in (False, True):
        assert rotary(sd, 0, 1, explicit) == sd.OK

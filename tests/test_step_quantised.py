"""DecodeStep's calls on a quantised copy, refused on the host where there is none (no GPU needed)."""
import pytest

from self_sparse_speculative_b200.step import DecodeStep


@pytest.mark.parametrize("call", [lambda st: st.quantise(), lambda st: st.draft_quantised(0), lambda st: st.round_quantised()])
def test_calls_without_a_copy_say_so(call):
    st = DecodeStep.__new__(DecodeStep)
    st.kvq = None
    with pytest.raises(ValueError, match="draft_bits"):
        call(st)


@pytest.mark.parametrize("bits", [0, 5, 16, "4"])
def test_other_widths_are_refused(bits):
    with pytest.raises(ValueError, match="draft_bits"):
        DecodeStep(None, draft_bits=bits)

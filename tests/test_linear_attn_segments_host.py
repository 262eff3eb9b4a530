"""The length of linear attention's segments by the sizes of a call."""
import pytest

from selective_ssm_packed_gb300 import binding, build

SMS, MOST = 152, 4096


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()
    binding.lib()


@pytest.mark.parametrize("T,S,Hv", [(32768, 30, 8), (32768, 30, 4), (16384, 25, 12), (9000, 11, 16), (16384, 1, 8), (6000, 1, 32)])
def test_a_bf16_backward_s_segments_are_what_an_sm_has_to_walk_in_a_launch(T, S, Hv):
    """Each of its launches walks one role, a CTA for a segment's head: no more than an SM's part of the tokens of all heads,
    but for the rounding to 256 tokens."""
    seg = binding.linear_attn_segment(T, S, Hv, Hv, 128, 128, binding.VSSM_BF16, True)
    share = T * Hv // SMS
    assert share <= seg <= max(256, share + 255)


@pytest.mark.parametrize("dtype", [binding.VSSM_F32, binding.VSSM_BF16])
@pytest.mark.parametrize("back", [False, True])
def test_segments_are_whole_chunks_between_256_and_4096_tokens(dtype, back):
    for T in (513, 1000, 5000, 40000, 10 ** 6):
        for S in (1, 7, T // 100):
            for Hv in (1, 6, 48, 512):
                seg = binding.linear_attn_segment(T, S, 1, Hv, 96, 72, dtype, back)
                assert 256 <= seg <= MOST and seg % 128 == 0 if dtype == binding.VSSM_BF16 else seg % 64 == 0
    assert binding.linear_attn_segment(500, 1, 1, 2, 64, 64, dtype, back) >= 512


def test_a_bf16_backward_leaves_sequences_whole_that_are_little_longer_than_an_sm_s_part():
    for T, S, Hv, whole in ((32768, 30, 16, True), (32768, 30, 12, False)):
        seg = binding.linear_attn_segment(T, S, Hv, Hv, 128, 64, binding.VSSM_BF16, True)
        assert (seg == MOST) == whole and (4 * T // S <= 1.5 * (T * Hv / SMS)) == whole

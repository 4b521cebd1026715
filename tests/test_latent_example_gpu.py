"""The serving example: planning, KDA, cache, expanded and absorbed attention together."""
import pytest

from examples.latent_serving import serve

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("requests,longest,steps,heads", [(3, 90, 5, 2), (1, 1, 2, 16), (6, 700, 3, 8)])
def test_decoded_tokens_agree_with_whole_sequences(requests, longest, steps, heads):
    """The last decoded tokens' absorbed attention equals the expanded form over whole sequences.
    The two round different intermediates to bf16 (2^-8 each): absorbed queries, absorbed output
    and its values' product on one side, keys, values and output on the other, and the output
    projection on both: rel-RMS below 8 x 2^-8."""
    y, again = serve(requests, longest, steps, heads)
    off = (y.double() - again.double()).norm() / again.double().norm()
    assert off <= 8 * 2.0 ** -8, float(off)

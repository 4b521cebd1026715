"""The serving example with several samples a prompt: fork, shared decoding and release together."""
import pytest

from examples.latent_serving import serve

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("requests,longest,steps,heads,samples", [(3, 90, 5, 2, 4), (2, 1, 2, 16, 3), (2, 700, 3, 8, 2),
                                                                  (4, 3000, 2, 32, 12)])
def test_samples_of_prompts_agree_with_whole_sequences(requests, longest, steps, heads, samples):
    """As test_latent_example_gpu.py, with its bound: absorbed and expanded attention round different
    intermediates to bf16, 2^-8 each, eight of them between the two outputs."""
    y, again = serve(requests, longest, steps, heads, samples=samples)
    off = (y.double() - again.double()).norm() / again.double().norm()
    assert off <= 8 * 2.0 ** -8, float(off)

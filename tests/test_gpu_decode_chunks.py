"""layer_decode where the last gate / up chunk has fewer pairs than the others (the claims
themselves are modelled in test_decode_claims_cpu.py): bit for bit layer_forward."""
import pytest

from test_gpu_decode import Layer, same_as_forward

pytestmark = pytest.mark.gpu


# distinct experts times F / 32 pairs in chunks of three, one or two left over
@pytest.mark.parametrize("T,d,L,F,E,k", [(1, 256, 256, 2560, 20, 16), (1, 2048, 384, 1280, 17, 14), (1, 7168, 3584, 2560, 24, 16),
                                         (2, 256, 128, 2176, 8, 8), (8, 1024, 512, 1024, 41, 8)])
@pytest.mark.parametrize("packed", [False, True])
def test_chunks_that_do_not_divide_the_pairs(T, d, L, F, E, k, packed):
    same_as_forward(Layer(T, d, L, F, E, k, packed=packed))

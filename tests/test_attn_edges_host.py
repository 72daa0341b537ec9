"""Host-side checks of linear attention's C ABI (no GPU, no kernel is launched)
at the ends of its sizes."""
import pytest

import onnx_recurrent_layers_amd as rl
from tests.test_attn_host import FAKE, desc


@pytest.mark.parametrize("layout", [0, 1])
@pytest.mark.parametrize("seq", [0, 1, 16, 3000])
def test_gradient_of_an_empty_batch(layout, seq):
    """No row: success with no launch, whichever kernels the sizes would take, with tensors of no elements (NULL) or not."""
    for dtype in (0, 1, 2):
        h = rl.rnn_attn_create(desc(dtype=dtype, layout=layout, seq=seq, batch=0, heads=4, groups=2, key=64, value=64))
        for names in (("dQ",), ("dK",), ("dV",), ("dG",), ("d_initial_state",), ("dQ", "dK", "dV", "dG", "d_initial_state")):
            g = rl.rnn_attn_gradients()
            for i, n in enumerate(names):
                getattr(g, n).ptr = FAKE + (1 << 16) * (i + 1)
            rl.rnn_attn_encode_backward(h, rl.rnn_attn_operands(), g, FAKE)
        rl.rnn_attn_destroy(h)

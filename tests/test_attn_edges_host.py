"""Host-side checks of linear attention's C ABI (no GPU, no kernel is launched)
at the ends of its sizes."""
import pytest

import onnx_recurrent_layers_amd as rl
from tests.test_attn_host import FAKE, WHO, desc
from tests.test_ssm_host import UNSUPPORTED, filled, refused


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


def created(**kw):
    rl.rnn_attn_destroy(rl.rnn_attn_create(desc(**kw)))


LARGE = "too large for one launch"


def test_limits_of_tokens():
    """A workgroup of 256 threads for 64 values of a head; no launch beside the walk's."""
    token = dict(dtype=2, seq=1, heads=16, groups=16)
    created(**token, batch=16384, key=128, value=128)               # 16 GiB of states
    created(**token, batch=(1 << 19) - 1, key=128, value=128)
    refused(lambda: created(**token, batch=1 << 19, key=128, value=128), UNSUPPORTED, WHO, LARGE)
    created(**token, batch=(1 << 20) - 1, key=256, value=1)
    refused(lambda: created(**token, batch=1 << 20, key=256, value=1), UNSUPPORTED, WHO, LARGE)


def test_limits_of_sequences():
    """512 threads; few rows are walked in pieces, which a launch of a thread a state's element joins."""
    prompt = dict(dtype=2, seq=64, heads=16, groups=16)
    created(**prompt, batch=(1 << 18) - 1, key=128, value=128)
    refused(lambda: created(**prompt, batch=1 << 18, key=128, value=128), UNSUPPORTED, WHO, LARGE)
    created(**prompt, batch=(1 << 19) - 1, key=256, value=1)
    refused(lambda: created(**prompt, batch=1 << 19, key=256, value=1), UNSUPPORTED, WHO, LARGE)


def test_limits_of_pieces(monkeypatch):
    monkeypatch.setenv("RNN_ATTN_PIECE", "64")
    prompt = dict(dtype=2, seq=128, heads=16, groups=16, key=256, value=256)
    created(**prompt, batch=(1 << 12) - 1)
    refused(lambda: created(**prompt, batch=1 << 12), UNSUPPORTED, WHO, LARGE)


@pytest.mark.parametrize("seq,batch", [(1, 1 << 18), (64, 1 << 17)])
def test_limits_of_the_gradient(seq, batch):
    """Four workgroups for 256 keys, one for the forward call's value: refused by the gradient's call alone."""
    h = rl.rnn_attn_create(desc(dtype=2, seq=seq, heads=16, groups=16, batch=batch, key=256, value=1))
    try:
        refused(lambda: rl.rnn_attn_encode_backward(h, filled("attn", "operands"), filled("attn", "gradients"), FAKE << 8), UNSUPPORTED, WHO, LARGE)
    finally:
        rl.rnn_attn_destroy(h)

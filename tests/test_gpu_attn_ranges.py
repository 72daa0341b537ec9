"""Linear attention on the GPU with values of very unlike size side by side:
steps, columns and entries of a state that do not depend on each other do not
take each other's digits.  Bounds: attn_reference.walk, of each output's own
terms; sizes are chosen so that no 16-bit output leaves its type."""
import pytest
import torch

from tests import ssm_reference as ref
from tests import test_gpu_ssm
from tests.test_gpu_attn import attn_case, rounded, values

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def sentinel(monkeypatch):
    """Outputs reach the thousands, where bf16 has every fourth number only and meets the usual -777 (-776) now and then:
    a sentinel above them all, a number of every type."""
    monkeypatch.setattr(test_gpu_ssm, "SENTINEL", -59904.0)


def stored(t, dtype):
    return {n: rounded(x, dtype if n in ("Q", "K", "V", "dY") else "f32") for n, x in t.items()}


@pytest.mark.parametrize("dtype", ref.TYPES)
@pytest.mark.parametrize("k,reverse", [(64, False), (64, True), (200, False)])
def test_a_large_step(dtype, k, reverse):
    """Scores of 64 * 9e8 * scale beside those of 8 * scale: of steps whose value is zero, and that no gradient enters by."""
    b, s, h, v = 2, 130, 2, 40
    t = values(dtype, b, s, h, 1, k, v)
    for at in (12, 77, 125):
        t["Q"][:, at] = t["K"][:, at] = 3e4
        t["V"][:, at] = t["dY"][:, at] = 0
    t["d_final_state"] *= 0.003
    attn_case(dtype, b, s, h, 1, k, v, t=stored(t, dtype), scale=0.003, reverse=reverse)


@pytest.mark.parametrize("dtype", ref.TYPES)
@pytest.mark.parametrize("which", ["values", "keys"])
@pytest.mark.parametrize("k,v", [(32, 48), (48, 200)])
def test_columns_of_unlike_size(dtype, which, k, v):
    """Columns of the values, and keys: columns of the gradients' states."""
    b, s, h = 2, 100, 2
    t = values(dtype, b, s, h, 1, k, v)
    size = torch.tensor([1e4, 1.0, 1e-2, 1e-3], dtype=torch.float64)
    if which == "values":
        t["V"] *= size.repeat(h * v // 4)
        t["initial_state"] *= size.repeat(v // 4)
    else:
        t["K"] *= size.repeat(k // 4)
        t["Q"] *= torch.tensor([1e-3, 1.0, 1e-2, 1.0], dtype=torch.float64).repeat(k // 4)
    t["d_final_state"] *= 0.01
    attn_case(dtype, b, s, h, 1, k, v, t=stored(t, dtype), scale=0.01)


@pytest.mark.parametrize("dtype", ref.TYPES)
def test_a_large_state_that_is_not_asked_for(dtype):
    """One key's 1e10 in two columns, which no query and no gradient meets, beside the ones of the other keys there."""
    b, s, h, k, v = 2, 100, 2, 32, 48
    t = values(dtype, b, s, h, 1, k, v)
    t["initial_state"][..., 3, 5] = t["initial_state"][..., 4, 6] = 1e10
    t["Q"][..., 3:5] = 0
    t["dY"].view(b, s, h, v)[..., 5:7] = 0
    attn_case(dtype, b, s, h, 1, k, v, t=stored(t, dtype))


@pytest.mark.parametrize("dtype", ref.TYPES)
@pytest.mark.parametrize("reverse", [False, True])
def test_values_of_unlike_size_under_keys_of_their_own(dtype, reverse):
    """Steps of 1e4, 1e-3 and 1, each under a key that no step of another size has (33 keys, sizes three by three)."""
    b, s, h, k, v = 2, 130, 2, 33, 24
    t = values(dtype, b, s, h, h, k, v)
    at = torch.arange(s)
    t["K"] = torch.nn.functional.one_hot(at % k, k).double().repeat(b, 1, h)
    t["Q"] = torch.nn.functional.one_hot(7 * at % k, k).double().repeat(b, 1, h)
    t["V"] *= torch.tensor([1e4, 1e-3, 1.0], dtype=torch.float64)[at % 3][:, None]
    t["dY"] *= 0.05
    t["initial_state"] *= 1e-3
    t["d_final_state"] *= 0.05
    attn_case(dtype, b, s, h, h, k, v, t=stored(t, dtype), scale=0.25, reverse=reverse)

"""The feed-forward products where large tiles of 256 x 256 take several rounds of
workgroups, as the largest calls do, at sizes that end inside a tile, against 64
bits with the bounds of test_gpu_feed_forward.py.  (That these sizes are cut so is
pinned by test_feed_forward_cuts_cpu.py.)
"""
import pytest

from tests.test_gpu_feed_forward import TYPES, backward_inputs, check_backward, check_forward, in_8_bits, tensors

pytestmark = pytest.mark.gpu

FORWARD = [(8200, 72, 2056), (4100, 1000, 4104), (700, 136, 33000)]
# dx, dw
BACKWARD = [(4300, 7704, 72), (136, 3912, 4296)]


@pytest.mark.parametrize("rows,hidden,inner", FORWARD)
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_forward(rows, hidden, inner, dtype):
    for act in ("silu", "gelu_tanh"):
        t = tensors(61, rows, hidden, inner, dtype)
        check_forward(t["x"], t["w_gate"], t["w_up"], act)


@pytest.mark.parametrize("rows,hidden,inner", [(r, 16 * -(-h // 16), 16 * -(-i // 16)) for r, h, i in FORWARD])
@pytest.mark.parametrize("out", ["bf16", "fp16"])
def test_forward_in_8_bits(rows, hidden, inner, out):
    t = tensors(62, rows, hidden, inner, "fp32")
    (x, xs), (wg, gs), (wu, us) = (in_8_bits(t[n]) for n in ("x", "w_gate", "w_up"))
    check_forward(x, wg, wu, "silu", (xs, gs, us), TYPES[out])


@pytest.mark.parametrize("rows,hidden,inner", BACKWARD)
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_backward(rows, hidden, inner, dtype):
    check_backward(backward_inputs(63, rows, hidden, inner, dtype), "silu")

"""The convolution refuses outputs over what other threads have yet to read: y over x, dx over
x or the gradient of y."""
import pytest

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,es", [("bf16", 2), ("f32", 4)])
def test_outputs_over_inputs_are_refused(dtype, es):
    import torch
    import bwd_persistent_cta_gb300 as R
    T, B, D = 40, 2, 16
    op = R.CausalConv(B, T, D, 4, dtype=dtype)
    row, n = D * es, T * B * D * es
    m = torch.zeros(64 * n, dtype=torch.uint8, device="cuda")
    p, w, far = m.data_ptr(), m.data_ptr() + 40 * n, m.data_ptr() + 50 * n
    work = m.data_ptr() + 44 * n
    x = p + 16 * n

    def fwd(y, x_row=0):
        return R.rnn_conv_forward(op.handle, R.rnn_conv_in_t(x=x, w=w, x_row=x_row), None, y, None)

    def bwd(dy, dx, x_row=0):
        assert op.backward_workspace_bytes <= 4 * n
        return R.rnn_conv_backward(op.handle, R.rnn_conv_in_t(x=x, w=w, x_row=x_row), None, dy, None, dx, None, None, None, work)

    for y in (x - n, x + n, far):
        assert fwd(y) == R.RNN_OK and bwd(far, y if y != far else p) == R.RNN_OK
    for y in (x, x - n + 16, x + n - 16, x + 16):
        assert fwd(y) == R.RNN_BAD_PARAM and bwd(far, y) == R.RNN_BAD_PARAM, y - x
    for dx in (far, far + 16, far - n + 16):
        assert bwd(far, dx) == R.RNN_BAD_PARAM, dx - far
    # x's rows in a packed projection: memory between two of them is free
    one = R.CausalConv(1, 2, D, 4, dtype=dtype)

    def two(y, x_row):
        return R.rnn_conv_forward(one.handle, R.rnn_conv_in_t(x=x, w=w, x_row=x_row), None, y, None)

    assert two(x + row, 4 * D) == R.RNN_OK               # two rows of y between the two of x
    for y in (x + row - 16, x + 2 * row + 16, x + 3 * row, x + 4 * row, x, x - row):
        assert two(y, 4 * D) == R.RNN_BAD_PARAM, y - x
    assert two(x + 5 * row, 4 * D) == R.RNN_OK and two(x - 2 * row, 4 * D) == R.RNN_OK
    torch.cuda.synchronize()


def test_wrapper():
    import torch
    import bwd_persistent_cta_gb300 as R
    op = R.CausalConv(2, 70, 16, 4)
    x, w = torch.randn(70, 2, 16, device="cuda").bfloat16(), torch.randn(16, 4, device="cuda").bfloat16()
    with pytest.raises(R.RnnError):
        op.forward(x, w, y=x)

"""The formulas that the GPU tests hold the norm's backward to, against differences of those they hold its forward to (no GPU
needed)."""
import pytest

torch = pytest.importorskip("torch")

from test_rmsnorm_gpu import backward_reference, reference  # noqa: E402


@pytest.mark.parametrize("T,H,eps", [(5, 7, 1e-3), (1, 1, 0.5), (3, 16, 1e-6)])
@pytest.mark.parametrize("with_residual", [True, False])
def test_backward_reference_against_differences(T, H, eps, with_residual):
    class Norm(torch.autograd.Function):
        """The sum and the norm of it; the sum's own gradient joins x's and the residual's."""

        @staticmethod
        def forward(ctx, x, w, r):
            h, s, out = reference(x, w, r if with_residual else None, eps)
            ctx.save_for_backward(h, w, s)
            return out, h.clone()

        @staticmethod
        def backward(ctx, dout, d_sum):
            h, w, s = ctx.saved_tensors
            dx, _, dw, _ = backward_reference(dout, h, w, s, d_sum)
            return dx, dw, dx if with_residual else None

    g = torch.Generator().manual_seed(T + H)
    x, w, r = (torch.randn(*shape, generator=g, dtype=torch.float64, requires_grad=True) for shape in ((T, H), (H,), (T, H)))
    assert torch.autograd.gradcheck(Norm.apply, (x, w, r))

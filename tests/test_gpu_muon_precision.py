"""The orthogonalised step's precision for long sums as for short ones, on well spread,
decaying and low-rank spectra.  (Nearly singular matrices of a few rows can be further off
than this bound, whose e32 is one sample of the plain form's roundings.)

test_gpu_muon.py's bound has a term that grows with n, the loss of an MMA that cuts
off its sum over n terms.  The sums run in pieces instead, 128 terms in the large
matrices' products and 32 or 64 in the small ones', which are added up rounded to
nearest.  Of it, with e32 the error of the plain form in 32 bits on the same input:
- 8 e32 as there (22 bits between the products instead of 24, lo lo terms left out,
  twice as many roundings);
- a piece's loss: an MMA takes 8 terms at least (m16n8k8), so a piece has up to eight whose
  cut is of one sign, each 2^-24 of the mean partial sum, and X follows with 4 (as there):
  4 * 8 * 2^-24, whatever n;
- the pieces' additions: n / 64 roundings of 2^-24 at most, of either sign, so their
  root in the mean, again times 4: 4 sqrt(n / 64) 2^-24;
- 2^-18 for one that e32 happens to leave out.
Without the pieces 16 x 7168 is 3.9e-5 off (bound 1.6e-5), and one fp16 term a number
leaves 3e-3."""
import pytest
import torch

import precision_moe_grouped_gb300 as P
import test_gpu_muon as M

pytestmark = pytest.mark.gpu

SHAPES = [(1, 7168), (2, 16, 7168), (7168, 12), (16, 30001), (32, 4096), (30001, 30), (64, 4096), (60, 7168), (64, 20000),
          (33, 2000), (65, 7168), (256, 7168), (7168, 256), (333, 1001), (2, 777, 129), (512, 512), (640, 30000), (1000, 4096),
          (2048, 7168), (8, 1 << 20), (1 << 18, 70)]


def inputs(kind, shape):
    if kind != "positive":
        return M.inputs(kind, shape, 15)
    return M.inputs("noise", shape, 15).abs()      # every sum of X X^T of one sign


@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("kind", ["noise", "strong", "low", "positive"])
def test_error_does_not_grow_with_the_length(cuda_ok, shape, kind):
    grad = inputs(kind, shape)
    p = torch.zeros(shape, device="cuda")
    op = P.Muon([p], [grad], lr=1.0, weight_decay=0.0, momentum=0.0, nesterov=False, update_scale="spectral")
    op.step()
    assert op.device_status() == 0
    x = -p / M.factor("spectral", *shape[-2:])
    ref = M.orthogonal(grad.double(), 5, 1e-7)
    e32 = M.relative(M.orthogonal(grad, 5, 1e-7), ref)
    n = max(shape[-2:])
    bound = 8 * e32 + 4 * (8 + (n / 64) ** 0.5) * 2.0 ** -24 + 2.0 ** -18
    e = M.relative(x, ref)
    print(shape, kind, "error %.2g, 32 bits %.2g, bound %.2g" % (e, e32, bound))
    assert e <= bound

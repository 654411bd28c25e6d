"""The rounding, the 8-bit product and the experts on tensors past 2^32 bytes: the far rows, channels and experts come out as
those of a small call on them alone."""
import pytest
import torch

import int4_group_quantized_w4a16_amd as kaio
from tests.gpu_util import DEV

pytestmark = pytest.mark.gpu
FAR = 2 ** 32


@pytest.fixture(autouse=True)
def memory():
    yield
    torch.cuda.synchronize()
    torch.cuda.empty_cache()


def words(*shape, dtype=torch.int32):
    return torch.empty(shape, dtype=dtype, device=DEV).random_(-2 ** 31, 2 ** 31) if dtype == torch.int32 else \
        torch.randint(-127, 128, shape, dtype=dtype, device=DEV)


def test_rows_to_round():
    m, k = 2 ** 20 + 77, 4112
    assert m * k > FAR
    x = torch.empty((m, k), dtype=torch.bfloat16, device=DEV).normal_()
    q, s = kaio.kaio_quantize_rows(x)
    for at in (0, FAR // k // 2 - 1, FAR // k - 3, m - 9):
        far_q, far_s = kaio.kaio_quantize_rows(x[at:at + 9].clone())
        torch.cuda.synchronize()
        assert torch.equal(q[at:at + 9], far_q) and torch.equal(s[at:at + 9], far_s)
    most = x[-9:].double().abs().amax(1)
    assert torch.equal(q[-9:].double(), torch.round(127 * x[-9:].double() / most[:, None]))


@pytest.mark.parametrize("what,m,n,k", [("rows of x", 2 ** 20 + 77, 40, 4112), ("channels of w", 5, 2 ** 20 + 77, 4112),
                                        ("channels of w", 40, 2 ** 20 + 77, 4112), ("results", 70001, 32003, 64)])
def test_linear(what, m, n, k):
    assert dict([("rows of x", m * k), ("channels of w", n * k), ("results", 2 * m * n)])[what] > FAR
    x, w = words(m, k, dtype=torch.int8), words(n, k, dtype=torch.int8)
    xs, ws = torch.rand(m, device=DEV) * 0.01, torch.rand(n, device=DEV) * 0.01
    y = kaio.kaio_linear_w8a8(x, w, ws, x_scale=xs, activation="silu")
    torch.cuda.synchronize()
    for rows in (slice(0, 5), slice(max(m - 5, 0), m)):
        for cols in (slice(0, 30), slice(n // 2, n // 2 + 3), slice(n - 30, n)):
            small = kaio.kaio_linear_w8a8(x[rows].clone(), w[cols].clone(), ws[cols].clone(), x_scale=xs[rows].clone(), activation="silu")
            z = (x[rows].double() @ w[cols].double().T.contiguous()) * xs[rows].double()[:, None] * ws[cols].double()
            want = z / (1 + torch.exp(-z))
            torch.cuda.synchronize()
            assert torch.equal(y[rows, cols], small)
            assert ((small.double() - want).abs() <= 2.0 ** -11 * want.abs() + 2.0 ** -18 * (1 + z.abs() / 32) * want.abs() +
                    2.0 ** -21 * z.abs() + 2.0 ** -25).all()


def test_experts_of_far_weights():
    e, h, i, t = 512, 4096, 4224, 6
    assert e * h * i // 2 > FAR
    scales = lambda *s: torch.rand(s, device=DEV).mul_(0.015).add_(0.005).half()
    ws = [words(e, h // 8, i), scales(e, h // 128, i), words(e, h // 8, i), scales(e, h // 128, i), words(e, i // 8, h), scales(e, i // 128, h)]
    router, x = torch.zeros((e, h), dtype=torch.float16, device=DEV), torch.randn(t, h, device=DEV).half()
    x[:, 0] = 1
    far = slice(e - 4, e)
    router[far] = torch.randn(4, h, device=DEV).half() / 64
    router[far, 0] = 20                            # the last four experts, whatever the rest of the token says
    y = kaio.kaio_moe_w4a16(x, kaio.KaioExperts(router, *ws), 3)
    few = kaio.kaio_moe_w4a16(x, kaio.KaioExperts(router[far].clone(), *[w[far].clone() for w in ws]), 3)
    torch.cuda.synchronize()
    assert y.isfinite().all() and y.abs().max() > 0
    # (parts of the down product are divided by how many experts there could be: sums in another order, of f32)
    assert ((y.double() - few.double()).abs() <= 2.0 ** -10 * y.double().abs() + 1e-3 * y.double().abs().mean()).all()


def test_experts_of_many_tokens():
    t, e, top, h, i = 2 ** 17, 20, 16, 128, 640
    assert t * top * i * 4 > FAR                   # h between the products, and its workspace
    scales = lambda *s: torch.rand(s, device=DEV).mul_(0.015).add_(0.005).half()
    experts = kaio.KaioExperts(torch.randn(e, h, device=DEV).half() / 8, words(e, h // 8, i), scales(e, 1, i), words(e, h // 8, i), scales(e, 1, i),
                               words(e, i // 8, h), scales(e, i // 128, h))
    assert kaio.lib().kaio_moe_w4a16_workspace_size(experts._ref, t, top) > FAR
    x = torch.randn(t, h, device=DEV).half()
    y = kaio.kaio_moe_w4a16(x, experts, top, residual=x)
    for at in (0, 64 * 300, t // 2, t - 64):
        few = kaio.kaio_moe_w4a16(x[at:at + 64], experts, top, residual=x[at:at + 64])
        torch.cuda.synchronize()
        assert ((y[at:at + 64].double() - few.double()).abs() <= 2.0 ** -10 * few.double().abs() + 1e-3 * few.double().abs().mean()).all()

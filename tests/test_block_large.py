"""The block's calls on matrices whose offsets pass 32 bits: rows and columns at both ends against 64-bit formulas (GPU).
Tolerances as in the calls' own tests."""
import pytest
import torch

import bit_quantization_aware_blockwise_b200 as q
import block_reference as ref
from test_gated_block import check_forward, operands
from test_lowbit_linear import activations, check_linear, product

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


def test_gated_forward_and_backward(cuda_device):
    # 2^32.1 outputs: h 8.7 GB, the gradients' matrix 17 GB
    M, F, K = 270000, 16144, 64
    assert M * F > 1 << 32
    x, wg, wu = operands(M, F, K, seed=50)
    h, kept = q.gated_linear(x, wg, wu, checkpoint=True)
    q.device_status()
    rows = torch.tensor([0, 1, 133000, 133039, 266033, 266034, M - 2, M - 1], device="cuda")
    some = {k: v[rows] for k, v in kept.items()}
    check_forward(x[rows], wg, wu, "silu", h[rows], some)
    grad = q.gated_bwd(h, kept)
    a, b = ref.halves(some)
    want = ref.block_back(h[rows].double(), a, b, "silu")
    size = torch.cat([(h[rows].double() * b).abs() * 2, (h[rows].double() * a).abs()], 1)
    assert ((grad[rows].double() - want).abs() <= 2 ** -8 * want.abs() + 2 ** -16 * size + 1e-30).all()


@pytest.mark.parametrize("kind", ["int8", "packed4"])
def test_weight_grad_of_many_tokens(cuda_device, kind):
    # 2^32.01 saved values, and x_hat 8.6 GB of workspace
    T, N, K = 1050001, 16, 4096
    assert T * K > 1 << 32
    g = torch.Generator(device="cuda").manual_seed(51)
    gy = (torch.randn(T, N, device="cuda", generator=g) * 1e-3).to(BF)
    mask = torch.randint(0, 256, (N, K // 8), device="cuda", generator=g).to(torch.uint8)
    per = 2 if kind == "packed4" else 1
    codes = torch.randint(0, 256, (T, K // per), device="cuda", generator=g, dtype=torch.uint8)
    scales = torch.rand(T, K // 128, device="cuda", generator=g) + 0.5
    got = q.weight_grad(gy, codes, scales, 4 if per == 2 else 8, mask=mask, out_dtype=torch.float32)
    q.device_status()
    total = torch.zeros(N, K, dtype=torch.float64, device="cuda")
    square = torch.zeros_like(total)
    for t in range(0, T, 50000):
        c = codes[t:t + 50000]
        v = ref.midrise4(c, c.shape[0]) if per == 2 else c.view(torch.int8).double() + 0.5
        xh = ref.bf16_input(v, scales[t:t + 50000])
        y = gy[t:t + 50000].double().t()
        total += y @ xh
        square += y.square() @ xh.square()
    m = ref.mask_values(mask, N, K)
    want = ref.transform(m * total, 128)
    block = (m * square).reshape(N, -1, 128).sum(-1).sqrt()
    # each of the T / 16 additions of a segment may cut 2^-23 of a running sum within six times the root of the squares
    acc = (6 * 17 / 16 * T * 2 ** -23) * block + 2 ** -21 * want.reshape(N, -1, 128).norm(dim=-1)
    assert ((got.double() - want).abs() <= acc.repeat_interleave(128, 1) + 2 ** -24 * want.abs()).all()
    # the segments keep it far closer: 32 additions and then the sums of segments and splits, rounded to nearest
    assert (got.double() - want).norm() <= 4e-6 * want.norm()


@pytest.mark.parametrize("M", [1, 16, 40])
def test_lowbit_layers(cuda_device, M):
    # 2^32.3 bytes of codes: rows and scales far behind the first
    N, K = 330000, 32768
    assert N * K // 2 > 1 << 32
    g = torch.Generator(device="cuda").manual_seed(52)
    codes = torch.randint(0, 256, (N, K // 2), device="cuda", generator=g, dtype=torch.uint8)
    scales = (torch.rand(N, K // 128, device="cuda", generator=g) + 0.5) * K ** -0.5 / 4
    x = activations(M, K, seed=53)
    rows = torch.tensor([0, 15, 16, 131071, 131072, 262143, 262144, N - 9, N - 8, N - 1], device="cuda")
    w = ref.scaled(ref.midrise4(codes[rows], len(rows)), scales[rows])
    got = q.lowbit_linear(x, codes, scales)
    check_linear(got[:, rows], x, w, 128)
    h = q.lowbit_gated(x, codes, scales, codes, scales)
    a, ea = product(x, w, 128, "int4")
    v, _ = ref.gate(a, "silu")
    tol = (2 ** -8 + 2 ** -16) * (v * a).abs() + 1.13 * ea * (a.abs() + ea) + v.abs() * ea + 1e-38
    assert ((h[:, rows].double() - v * a).abs() <= tol).all()

"""quest_lowbit_linear and quest_lowbit_gated against 64-bit formulas (GPU).

Tolerances. The transformed input is rounded once: for E2M1 to fp16, off by at most 2^-12 of each value;
for midrise codes to fixed point with the group's largest value A at 32767, off by at most A / 65534. These
K independent roundings, weighted, stay within six times the root of their squares, 6 R with R =
sqrt(sum e^2 w^2), e the bound of each (fixed seeds). The fp32 sums (per group and over groups) and the fp32
transform add less than 2^-17 of sqrt(sum xt^2 w^2). The result's bf16 rounding is 2^-8 of the value. A gated
output adds, through |act'| <= 1.13, the two projections' errors times the other factor.
"""
import pytest
import torch

import bit_quantization_aware_blockwise_b200 as q
import block_reference as ref

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def weight(N, K, grid, rows, seed):
    g = gen(seed)
    codes = torch.randint(0, 256, (N, K // 2), device="cuda", generator=g).to(torch.uint8)
    scales = (torch.rand(N, 1 if rows else K // 128, device="cuda", generator=g) + 0.5) * max(K, 1) ** -0.5 / 4
    v = ref.midrise4(codes, N) if grid == "int4" else ref.e2m1(codes, N)
    return codes, scales, ref.scaled(v, scales)


def activations(M, K, seed):
    x = torch.randn(M, K, device="cuda", generator=gen(seed))
    x[:, :: max(K // 5, 1)] *= 20
    return x.to(BF)


def mode(grid):
    return q.CODES_PACKED if grid == "int4" else q.CODES_FP4_PACKED


def product(x, w, had, grid):
    xt = ref.transform(x.double(), had)
    if grid == "int4":
        e = (xt.reshape(xt.shape[0], -1, 128).abs().amax(-1) / 65534).repeat_interleave(128, 1)
    else:
        e = xt.abs() * 2 ** -12
    w2 = w.square().t()
    return xt @ w.t(), 6 * (e.square() @ w2).sqrt() + 2 ** -17 * (xt.square() @ w2).sqrt() + 1e-38


def check_linear(got, x, w, had, grid="int4"):
    want, err = product(x, w, had, grid)
    assert ((got.double() - want).abs() <= 2 ** -8 * want.abs() + err).all()


@pytest.mark.parametrize("grid", ["int4", "fp4"])
@pytest.mark.parametrize("rows", [False, True])
@pytest.mark.parametrize("M,N,K,had", [(1, 8, 128, 128), (1, 264, 256, 256), (2, 136, 640, 0), (5, 2056, 384, 64),
                                       (8, 40, 2048, 16), (9, 520, 512, 32), (16, 1032, 5632, 128),
                                       (17, 88, 768, 256), (64, 264, 1024, 128)])
def test_matches_formula(cuda_device, M, N, K, had, rows, grid):
    codes, scales, w = weight(N, K, grid, rows, seed=N + K)
    x = activations(M, K, seed=M)
    got = q.lowbit_linear(x, codes, scales, code_mode=mode(grid), had_block=had)
    check_linear(got, x, w, had, grid)


@pytest.mark.parametrize("grid", ["int4", "fp4"])
@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
@pytest.mark.parametrize("M,F,K,had", [(1, 8, 128, 128), (1, 5632, 2048, 128), (3, 136, 256, 256), (16, 520, 640, 0),
                                       (33, 264, 512, 64)])
def test_gated_matches_formula(cuda_device, M, F, K, had, act, grid):
    cg, sg, wg = weight(F, K, grid, False, seed=1)
    cu, su, wu = weight(F, K, grid, False, seed=2)
    x = activations(M, K, seed=M + F)
    got = q.lowbit_gated(x, cg, sg, cu, su, act=act, code_mode=mode(grid), had_block=had)
    a, ea = product(x, wg, had, grid)
    b, eb = product(x, wu, had, grid)
    v, _ = ref.gate(a, act)
    want = v * b
    tol = (2 ** -8 + 2 ** -16) * want.abs() + 1.13 * ea * (b.abs() + eb) + v.abs() * eb + 1e-38
    assert ((got.double() - want).abs() <= tol).all()


@pytest.mark.parametrize("M,N,K", [(1, 24, 32768), (16, 24, 32768), (16, 8192, 22016), (4, 22016, 8192)])
def test_long_rows_and_large_layers(cuda_device, M, N, K):
    codes, scales, w = weight(N, K, "int4", False, seed=3)
    x = activations(M, K, seed=4)
    check_linear(q.lowbit_linear(x, codes, scales), x, w, 128)


def test_quantizer_codes_decode(cuda_device):
    # codes of the library's own quantizer, both grids, per group and per row, against its dequantised weights
    W = (torch.randn(264, 512, device="cuda", generator=gen(5)) * 0.02).to(BF)
    x = activations(6, 512, seed=6)
    for cm, grid in ((q.CODES_PACKED, "int4"), (q.CODES_FP4_PACKED, "fp4")):
        for rg in (128, 512):
            qw = q.quantize_fwd(W, 4, rms_group=rg, code_mode=cm, mask_mode=None, dequant="fp32")
            got = q.lowbit_linear(x, qw["codes"], qw["scales"], code_mode=cm)
            check_linear(got, x, qw["dequant"].double(), 128, grid)


def test_scale_of_the_input(cuda_device):
    # very small and very large tokens side by side, a zero token, a group of zeros
    N, K = 40, 512
    codes, scales, w = weight(N, K, "int4", False, seed=7)
    x = activations(6, K, seed=8).float()
    x[1] *= 2.0 ** -90
    x[2] *= 2.0 ** 80
    x[3] = 0
    x[4, 128:256] = 0
    x = x.to(BF)
    got = q.lowbit_linear(x, codes, scales)
    check_linear(got, x, w, 128)
    assert not got[3].any()


def test_non_finite_tokens_stay_alone(cuda_device):
    N, K = 72, 384
    codes, scales, w = weight(N, K, "int4", False, seed=9)
    x = activations(11, K, seed=10)
    clean = q.lowbit_linear(x, codes, scales)
    x[2, 7] = float("inf")
    x[9, 300] = float("nan")
    got = q.lowbit_linear(x, codes, scales)
    keep = [m for m in range(11) if m not in (2, 9)]
    assert torch.equal(got[keep], clean[keep])
    assert not got[2].isfinite().any() and not got[9].isfinite().any()


def test_pitched_input_and_rows_behind(cuda_device):
    N, K, M = 264, 256, 9
    codes, scales, w = weight(N, K, "fp4", True, seed=11)
    wide = activations(M, K + 72, seed=12)
    x = wide[:, 8:8 + K]
    out = torch.full((M + 16, N), 7.0, dtype=BF, device="cuda")
    q.lowbit_linear(x, codes, scales, code_mode=q.CODES_FP4_PACKED, out=out[:M])
    check_linear(out[:M], x, w, 128, "fp4")
    assert (out[M:] == 7).all()


def test_empty_sizes(cuda_device):
    e = torch.zeros((8, 0), dtype=torch.uint8, device="cuda")
    out = torch.full((3, 8), 7.0, dtype=BF, device="cuda")
    q.lowbit_linear(torch.zeros((3, 0), dtype=BF, device="cuda"), e, torch.zeros((8, 0), device="cuda"), out=out)
    assert not out.any()
    codes, scales, _ = weight(8, 128, "int4", False, seed=13)
    assert q.lowbit_linear(torch.zeros((0, 128), dtype=BF, device="cuda"), codes, scales).shape == (0, 8)


def test_streams_graphs_and_repeats(cuda_device):
    N, K = 1032, 2048
    codes, scales, w = weight(N, K, "int4", False, seed=14)
    x, x2 = activations(4, K, seed=15), activations(4, K, seed=16)
    want, want2 = (q.lowbit_gated(v, codes, scales, codes, scales) for v in (x, x2))
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    outs = [(q.lowbit_gated(x, codes, scales, codes, scales, stream=s1),
             q.lowbit_gated(x2, codes, scales, codes, scales, stream=s2)) for _ in range(8)]
    torch.cuda.synchronize()
    for a, b in outs:
        assert torch.equal(a, want) and torch.equal(b, want2)
    static = x.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = q.lowbit_gated(static, codes, scales, codes, scales)
    static.copy_(x2)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want2)

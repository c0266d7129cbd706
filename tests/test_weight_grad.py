"""quest_weight_grad against 64-bit formulas (GPU).

Tolerances. x_hat is bf16 by definition, so the products are exact and G is an fp32 sum over T
tokens; a tensor-core step adds 16 of them and cuts each of its 17 terms at 2^-23 of the largest, and
the running sum of these zero-mean terms stays within six times R = sqrt(sum gy^2 x^2): off by at most
acc = 6 * 17/16 T 2^-23 R an entry. The transform is orthonormal, so a block's error grows in
no entry beyond the root of the sum of its squares, and its own seven fp32 stages add 2^-21 of the block's
norm. In the 2-norm, where the cuts of different entries do not line up, T / 16 + 17 cuts of 2^-23 with
the same factor six bound the relative error. bf16 outputs: 2^-8 of the value more.
"""
import pytest
import torch

import bit_quantization_aware_blockwise_b200 as q
import block_reference as ref

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def grad_and_mask(T, N, K, seed):
    g = gen(seed)
    gy = (torch.randn(T, N, device="cuda", generator=g) * 1e-3).to(BF)
    mask = torch.randint(0, 256, (N, K // 8), device="cuda", generator=g).to(torch.uint8)
    return gy, mask


def saved(T, K, kind, rows, seed):
    """(codes, scales, the x_hat they stand for, bits, code_mode)."""
    g = gen(seed)
    scales = torch.rand(T, 1 if rows else K // 128, device="cuda", generator=g) + 0.5
    if kind == "packed4":
        codes = torch.randint(0, 256, (T, K // 2), device="cuda", generator=g).to(torch.uint8)
        return codes, scales, ref.bf16_input(ref.midrise4(codes, T), scales), 4, q.CODES_PACKED
    codes = torch.randint(-128, 128, (T, K), device="cuda", generator=g).to(torch.int8)
    if kind == "int8":
        return codes, scales, ref.bf16_input(codes.double() + 0.5, scales), 8, q.CODES_INT8
    return codes, scales, ref.bf16_input(codes.double() / 2, scales), 4, q.CODES_GEMM_OPERAND


def check(got, gy, xh, mask, T):
    want = ref.weight_grad(gy, xh, mask)
    R = (gy.double().square().t() @ xh.square()).sqrt()
    if mask is not None:
        R = R * ref.mask_values(mask, *R.shape)
    block = R.reshape(R.shape[0], -1, 128).square().sum(-1).sqrt()
    acc = (6 * 17 / 16 * T * 2 ** -23) * block + 2 ** -21 * want.reshape(*block.shape, 128).norm(dim=-1)
    acc = acc.repeat_interleave(128, 1)
    half = 2 ** -8 * want.abs() if got.dtype == BF else 2 ** -24 * want.abs()
    assert ((got.double() - want).abs() <= half + acc).all()
    rel = float((got.double() - want).norm() / want.norm().clamp_min(1e-300))
    assert rel <= (2 ** -8 if got.dtype == BF else 0) + 6 * (T / 16 + 17) * 2 ** -23 + 2 ** -21
    return want


@pytest.mark.parametrize("out", [BF, torch.float32])
@pytest.mark.parametrize("kind,rows", [("int8", False), ("int8", True), ("packed4", False), ("packed4", True),
                                       ("operand", True)])
@pytest.mark.parametrize("T,N,K", [(1, 8, 128), (65, 264, 384), (200, 136, 256), (3001, 520, 384)])
def test_matches_formula(cuda_device, T, N, K, kind, rows, out):
    gy, mask = grad_and_mask(T, N, K, seed=T + N)
    codes, scales, xh, bits, mode = saved(T, K, kind, rows, seed=K)
    got = q.weight_grad(gy, codes, scales, bits, code_mode=mode, mask=mask, out_dtype=out)
    q.device_status()
    assert got.dtype == out
    check(got, gy, xh, mask, T)


@pytest.mark.parametrize("kind", ["int8", "packed4"])
def test_many_tiles(cuda_device, kind):
    # more output tiles than CTA pairs: no split, both accumulators of a pair reused
    T, N, K = 150, 2568, 2176
    gy, mask = grad_and_mask(T, N, K, seed=1)
    codes, scales, xh, bits, mode = saved(T, K, kind, False, seed=2)
    assert q.weight_grad_workspace(T, N, K) < 2 * T * K + 256       # no split sums
    for out in (BF, torch.float32):
        check(q.weight_grad(gy, codes, scales, bits, code_mode=mode, mask=mask, out_dtype=out), gy, xh, mask, T)
    q.device_status()


def test_split_tokens(cuda_device):
    # few output tiles: the tokens are cut; results repeat bit for bit, whatever the workspace held
    T, N, K = 8200, 264, 256
    assert q.weight_grad_workspace(T, N, K) > 2 * T * K + N * K * 8  # two splits' sums at least
    gy, mask = grad_and_mask(T, N, K, seed=3)
    codes, scales, xh, bits, mode = saved(T, K, "int8", False, seed=4)
    one = q.weight_grad(gy, codes, scales, bits, code_mode=mode, mask=mask, out_dtype=torch.float32)
    check(one, gy, xh, mask, T)
    need = q.weight_grad_workspace(T, N, K)
    ws = torch.full((need // 4,), float("nan"), device="cuda")
    two = torch.empty_like(one)
    q.weight_grad_raw(gy.data_ptr(), N, codes.data_ptr(), mode, bits, scales.data_ptr(), 128, mask.data_ptr(), T, N, K,
                      128, two.data_ptr(), q.FP32, 0, ws.data_ptr(), need, torch.cuda.current_stream().cuda_stream)
    q.device_status()
    assert torch.equal(one, two)


@pytest.mark.parametrize("kind", ["int8", "packed4"])
def test_repeats_bit_for_bit(cuda_device, kind):
    # long token loops on every SM, back to back: no conversion, copy or sum depends on timing
    T, N, K = 2048, 2048, 2816
    gy, mask = grad_and_mask(T, N, K, seed=18)
    codes, scales, xh, bits, mode = saved(T, K, kind, False, seed=19)
    first = q.weight_grad(gy, codes, scales, bits, code_mode=mode, mask=mask, out_dtype=torch.float32)
    check(first, gy, xh, mask, T)
    bad = torch.zeros((), dtype=torch.int64, device="cuda")
    for _ in range(200):
        again = q.weight_grad(gy, codes, scales, bits, code_mode=mode, mask=mask, out_dtype=torch.float32)
        bad += (again != first).sum()
    q.device_status()
    assert int(bad) == 0


@pytest.mark.parametrize("T", [100, 5000])
def test_accumulates_into_a_master_gradient(cuda_device, T):
    N, K = 136, 384
    gy, mask = grad_and_mask(T, N, K, seed=5)
    codes, scales, xh, bits, mode = saved(T, K, "int8", False, seed=6)
    one = q.weight_grad(gy, codes, scales, bits, code_mode=mode, mask=mask, out_dtype=torch.float32)
    base = torch.randn(N, K, device="cuda", generator=gen(7))
    out = base.clone()
    got = q.weight_grad(gy, codes, scales, bits, code_mode=mode, mask=mask, out=out, accumulate=True)
    q.device_status()
    assert got is out
    assert torch.equal(out, base + one)              # one fp32 addition an entry, rounded to nearest


def test_mask_is_optional_and_extremes(cuda_device):
    T, N, K = 130, 264, 256
    gy, _ = grad_and_mask(T, N, K, seed=8)
    codes, scales, xh, bits, mode = saved(T, K, "packed4", False, seed=9)
    check(q.weight_grad(gy, codes, scales, bits), gy, xh, None, T)
    ones = torch.full((N, K // 8), 255, dtype=torch.uint8, device="cuda")
    assert torch.equal(q.weight_grad(gy, codes, scales, bits, mask=ones), q.weight_grad(gy, codes, scales, bits))
    assert not q.weight_grad(gy, codes, scales, bits, mask=torch.zeros_like(ones)).any()


def test_pitched_gradient_and_canaries(cuda_device):
    # the gate's half of a [T, 2F] gradient matrix; entries around the output stay
    T, F, K = 300, 264, 384
    both, _ = grad_and_mask(T, 2 * F, K, seed=10)
    codes, scales, xh, bits, mode = saved(T, K, "int8", False, seed=11)
    for half in (both[:, :F], both[:, F:]):
        got = q.weight_grad(half, codes, scales, bits, code_mode=mode)
        q.device_status()
        check(got, half, xh, None, T)
    whole = torch.full((F + 300, K), 7.0, device="cuda")
    q.weight_grad(both[:, :F], codes, scales, bits, code_mode=mode, out=whole[:F])
    assert (whole[F:] == 7).all()
    # the two halves in one call: the concatenated weights' gradient
    check(q.weight_grad(both, codes, scales, bits, code_mode=mode), both, xh, None, T)


def test_empty_sums(cuda_device):
    gy = torch.zeros((0, 16), dtype=BF, device="cuda")
    codes = torch.zeros((0, 128), dtype=torch.int8, device="cuda")
    scales = torch.zeros((0, 1), device="cuda")
    for dt in (BF, torch.float32):
        out = torch.full((16, 128), 3.0, dtype=dt, device="cuda")
        q.weight_grad(gy, codes, scales, 8, out=out)
        assert not out.any()
    out = torch.full((16, 128), 3.0, device="cuda")
    q.weight_grad(gy, codes, scales, 8, out=out, accumulate=True)
    assert (out == 3).all()


def test_non_finite_tokens_do_not_leak(cuda_device):
    # an Inf in one column of grad_y reaches that row of the gradient and no other, and zero rows past T add nothing
    T, N, K = 70, 40, 256
    gy, mask = grad_and_mask(T, N, K, seed=12)
    codes, scales, xh, bits, mode = saved(T, K, "int8", False, seed=13)
    clean = q.weight_grad(gy, codes, scales, bits, code_mode=mode)
    gy[5, 9] = float("inf")
    got = q.weight_grad(gy, codes, scales, bits, code_mode=mode)
    keep = torch.arange(N, device="cuda") != 9
    assert torch.equal(got[keep], clean[keep]) and not got[9].isfinite().any()


def test_gradient_against_differences(cuda_device):
    # f(w) = sum(grad_y * (x_hat (m * H w)^T)) is linear in w: its central difference along a direction is exact
    T, N, K = 96, 24, 256
    gy, mask = grad_and_mask(T, N, K, seed=14)
    codes, scales, xh, bits, mode = saved(T, K, "int8", False, seed=15)
    got = q.weight_grad(gy, codes, scales, bits, code_mode=mode, mask=mask, out_dtype=torch.float32).double()
    m = ref.mask_values(mask, N, K)

    def f(w):
        return (gy.double() * (xh @ (m * ref.transform(w, 128)).t())).sum()
    for seed in range(3):
        w = torch.randn(N, K, device="cuda", generator=gen(20 + seed)).double()
        d = torch.randn(N, K, device="cuda", generator=gen(30 + seed)).double()
        num = (f(w + d) - f(w - d)) / 2
        # |<error, d>| <= |error| |d|, with the 2-norm bound above
        tol = (6 * (T / 16 + 17) * 2 ** -23 + 2 ** -21) * got.norm() * d.norm()
        assert (num - (got * d).sum()).abs() <= tol


def test_streams_and_graphs(cuda_device):
    T, N, K = 4100, 264, 256                         # with a workspace
    gy, mask = grad_and_mask(T, N, K, seed=16)
    codes, scales, xh, bits, mode = saved(T, K, "packed4", True, seed=17)
    want = q.weight_grad(gy, codes, scales, bits, mask=mask, out_dtype=torch.float32)
    gy2 = gy.flip(1).contiguous()
    want2 = q.weight_grad(gy2, codes, scales, bits, mask=mask, out_dtype=torch.float32)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    outs = [(q.weight_grad(gy, codes, scales, bits, mask=mask, out_dtype=torch.float32, stream=s1),
             q.weight_grad(gy2, codes, scales, bits, mask=mask, out_dtype=torch.float32, stream=s2)) for _ in range(4)]
    torch.cuda.synchronize()
    for a, b in outs:
        assert torch.equal(a, want) and torch.equal(b, want2)
    static = gy.clone()
    graphs = []
    for _ in range(2):                               # two graphs, each with its own workspace
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = q.weight_grad(static, codes, scales, bits, mask=mask, out_dtype=torch.float32)
        graphs.append((g, out))
    static.copy_(gy2)
    for g, out in graphs:
        g.replay()
    torch.cuda.synchronize()
    for _, out in graphs:
        assert torch.equal(out, want2)
    q.device_status()


@pytest.mark.parametrize("kind", ["int8", "packed4"])
def test_bf16_gradient_over_several_accumulator_segments(cuda_device, kind):
    # uncut tokens, more output tiles than CTA pairs and three segments (4096 + 4096 + 8 tokens): the sums meet in the
    # epilogue's registers, and the accumulators' parity carries from tile to tile
    T, N, K = 8200, 2568, 2176
    assert q.weight_grad_workspace(T, N, K) < 2 * T * K + 256
    gy, mask = grad_and_mask(T, N, K, seed=40)
    codes, scales, xh, bits, mode = saved(T, K, kind, False, seed=41)
    check(q.weight_grad(gy, codes, scales, bits, code_mode=mode, mask=mask), gy, xh, mask, T)
    q.device_status()


@pytest.mark.parametrize("T,N,K,split", [(4096, 2568, 2176, False), (4096, 264, 256, True), (8200, 2568, 2176, False)])
def test_fp32_gradient_keeps_the_precision_of_its_segments(cuda_device, T, N, K, split):
    # A tensor-core addition cuts the running sum toward zero, by half of 2^-23 of it on average, and the sum of
    # zero-mean terms grows as the root of their number, 2/3 of its end on average: 32 additions of 16 tokens a segment
    # give 32 2^-24 2/3 = 1.3e-6 of a segment's sum, and of the whole, whose segments add up like their errors.
    # Without segments 4096 tokens are 256 additions: 1.0e-5 by the same count (4.3e-6 measured)
    assert (q.weight_grad_workspace(T, N, K) >= 2 * T * K + 256) == split
    gy, mask = grad_and_mask(T, N, K, seed=42)
    codes, scales, xh, bits, mode = saved(T, K, "int8", False, seed=43)
    got = q.weight_grad(gy, codes, scales, bits, code_mode=mode, mask=mask, out_dtype=torch.float32)
    q.device_status()
    want = ref.weight_grad(gy, xh, mask)
    assert (got.double() - want).norm() <= 1.5e-6 * want.norm()


@pytest.mark.parametrize("bits", [3, 5, 6, 7])
@pytest.mark.parametrize("rows", [False, True])
def test_packed_codes_of_every_width(cuda_device, bits, rows):
    # the quantizer's own packed codes: 3 bits in 4-bit containers, 5 to 7 in bytes; x_hat is its dequant but for ties
    T, N, K = 200, 136, 384
    gy, mask = grad_and_mask(T, N, K, seed=44)
    X = torch.randn(T, K, device="cuda", generator=gen(45)).to(BF)
    qx = q.quantize_fwd(X, bits, rms_group=K if rows else 128, mask_mode=None, dequant="fp32")
    values = (ref.midrise4(qx["codes"], T) if bits == 3 else qx["codes"].view(torch.int8).view(T, K).double() + 0.5)
    xh = ref.bf16_input(values, qx["scales"])
    assert (xh - qx["dequant"].double()).abs().max() <= 2 ** -8 * qx["dequant"].abs().max()
    got = q.weight_grad(gy, qx["codes"], qx["scales"], bits, mask=mask, K=K, out_dtype=torch.float32)
    q.device_status()
    check(got, gy, xh, mask, T)


@pytest.mark.parametrize("form", ["midrise", "fp4"])
@pytest.mark.parametrize("rows", [False, True])
def test_operand_codes_of_the_quantizer(cuda_device, form, rows):
    # the int8 operand bytes c of the linear layers, x_hat = bf16(c Delta / 2): 2 q + 1, and twice the E2M1 value
    T, N, K = 130, 264, 256
    gy, mask = grad_and_mask(T, N, K, seed=46)
    X = torch.randn(T, K, device="cuda", generator=gen(47)).to(BF)
    mode = q.CODES_GEMM_OPERAND if form == "midrise" else q.CODES_FP4_OPERAND
    qx = q.quantize_fwd(X, 4, rms_group=K if rows else 128, code_mode=mode, mask_mode=None, dequant="fp32")
    c = qx["codes"].view(torch.int8).view(T, K)
    if form == "fp4":
        assert set(c.abs().unique().tolist()) <= {0, 1, 2, 3, 4, 6, 8, 12}
    xh = ref.bf16_input(c.double() / 2, qx["scales"])
    assert (xh - qx["dequant"].double()).abs().max() <= 2 ** -8 * qx["dequant"].abs().max()
    for out in (BF, torch.float32):
        got = q.weight_grad(gy, c, qx["scales"], 4, code_mode=mode, mask=mask, out_dtype=out)
        q.device_status()
        check(got, gy, xh, mask, T)

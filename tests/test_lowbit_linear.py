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
@pytest.mark.parametrize("M,F,K,had", [(1, 8, 128, 128), (1, 5632, 2048, 128), (3, 136, 256, 256), (16, 520, 640, 0), (16, 22016, 8192, 128), (40, 11008, 4096, 256),
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


@pytest.mark.parametrize("grid,had", [("int4", 128), ("fp4", 128), ("int4", 256), ("fp4", 0)])
def test_largest_inputs_do_not_overflow(cuda_device, grid, had):
    # values up to the end of bf16's range, whose plain sums over a block pass fp32's; the results stay inside it
    codes, scales, w = weight(40, 512, grid, False, seed=23)
    x = activations(3, 512, seed=24).float()
    x = (x / x.abs().amax() * 3.3e38).to(BF)
    scales, w = scales * 2.0 ** -8, w * 2.0 ** -8
    got = q.lowbit_linear(x, codes, scales, code_mode=mode(grid), had_block=had)
    assert got.isfinite().all()
    check_linear(got, x, w, had, grid)


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


@pytest.mark.parametrize("M,grid", [(1, "int4"), (4, "int4"), (16, "int4"), (40, "fp4")])
def test_streams_graphs_and_repeats(cuda_device, M, grid):
    # with 16 and 40 tokens x is transformed by a kernel of its own, through a workspace
    N, K = 1032, 2048
    assert (q.lowbit_workspace(M, K) > 0) == (M >= 16)
    codes, scales, w = weight(N, K, grid, False, seed=14)
    x, x2 = activations(M, K, seed=15), activations(M, K, seed=16)

    def call(v, **kw):
        return q.lowbit_gated(v, codes, scales, codes, scales, code_mode=mode(grid), **kw)
    want, want2 = call(x), call(x2)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    outs = [(call(x, stream=s1), call(x2, stream=s2)) for _ in range(8)]
    torch.cuda.synchronize()
    for a, b in outs:
        assert torch.equal(a, want) and torch.equal(b, want2)
    # back to back on one stream, each input written right before its call and the output read right after
    static, acc = x.clone(), torch.zeros_like(want, dtype=torch.float64)
    for i in range(20):
        static.copy_(x if i % 2 else x2)
        acc += call(static).double()
    assert torch.equal(acc, 10 * (want.double() + want2.double()))
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = call(static)
        graphs.append((g, out))
    for v, ref_out in ((x2, want2), (x, want)):
        static.copy_(v)
        for g, _ in graphs:
            g.replay()
        torch.cuda.synchronize()
        for _, out in graphs:
            assert torch.equal(out, ref_out)


def test_weights_written_right_before_the_call(cuda_device):
    # the layer's kernel may start while the one that transforms x runs: codes and scales written by earlier work on the
    # stream must be seen all the same
    M, N, K = 16, 2056, 4096
    codes, scales, w = weight(N, K, "int4", False, seed=17)
    x = activations(M, K, seed=18)
    want = q.lowbit_linear(x, codes, scales)
    cw, sw = torch.empty_like(codes), torch.empty_like(scales)
    for _ in range(20):
        cw.zero_()
        sw.fill_(float("nan"))
        cw.copy_(codes)
        sw.copy_(scales)
        assert torch.equal(q.lowbit_linear(x, cw, sw), want)
    W = (torch.randn(N, K, device="cuda", generator=gen(19)) * 0.02).to(BF)
    first = None
    for _ in range(5):                               # the quantizer's own launch right before
        qw = q.quantize_fwd(W, 4, mask_mode=None)
        got = q.lowbit_linear(x, qw["codes"], qw["scales"])
        first = got if first is None else first
        assert torch.equal(got, first)


@pytest.mark.parametrize("M,N,K,had", [(16, 40, 32768, 128), (9, 24, 32512, 256), (64, 16, 16384, 64)])
def test_gated_longest_rows(cuda_device, M, N, K, had):
    cg, sg, wg = weight(N, K, "int4", False, seed=20)
    cu, su, wu = weight(N, K, "int4", True, seed=21)
    x = activations(M, K, seed=22)
    for grid in ("int4", "fp4"):
        vg = wg if grid == "int4" else ref.scaled(ref.e2m1(cg, N), sg)
        got = q.lowbit_gated(x, cg, sg, cg, sg, code_mode=mode(grid), had_block=had)
        a, ea = product(x, vg, had, grid)
        v, _ = ref.gate(a, "silu")
        want = v * a
        tol = (2 ** -8 + 2 ** -16) * want.abs() + 1.13 * ea * (a.abs() + ea) + v.abs() * ea + 1e-38
        assert ((got.double() - want).abs() <= tol).all()
    with pytest.raises(q.QuestError, match="one form"):
        q.lowbit_gated(x, cg, sg, cu, su, had_block=had)


@pytest.mark.parametrize("rms", [128, 4096])
@pytest.mark.parametrize("M,gated", [(1, False), (16, False), (16, True), (40, False)])
def test_two_weights_in_turn_in_the_same_buffers(cuda_device, M, gated, rms):
    # the quantizer, which lets its dependents start early, writes one of two different weights into the same codes and
    # scales right before each call, with nothing in between: stale codes or scales give the other weight's result
    N, K = 2056, 4096
    g = gen(25)
    W = [(torch.randn(N, K, device="cuda", generator=g) * 0.02).to(BF) for _ in range(2)]
    x = activations(M, K, seed=26)
    want = []
    for w in W:
        qw = q.quantize_fwd(w, 4, rms_group=rms, mask_mode=None, dequant="fp32")
        y, err = product(x, qw["dequant"].double(), 128, "int4")
        if gated:
            v, _ = ref.gate(y, "silu")
            y, err = v * y, 2 ** -16 * (v * y).abs() + 1.13 * err * (y.abs() + err) + v.abs() * err
        want.append((y, 2 ** -8 * y.abs() + err))
    codes = torch.zeros(N * K // 2, dtype=torch.uint8, device="cuda")
    scales = torch.zeros(N, K // rms, device="cuda")
    outs = [torch.zeros((M, N), dtype=BF, device="cuda") for _ in range(60)]
    need = q.lowbit_workspace(M, K)
    assert (need > 0) == (M >= 16)
    ws = torch.empty(max(need, 16), dtype=torch.uint8, device="cuda")
    st = torch.cuda.current_stream().cuda_stream
    torch.cuda.synchronize()
    for i, y in enumerate(outs):
        q.quantize_fwd_raw(W[i % 2].data_ptr(), q.BF16, N, K, K, 4, 128, rms, 1.0, q.CODES_PACKED, codes.data_ptr(),
                           scales.data_ptr(), q.MASK_BITS, None, None, q.BF16, st)
        if gated:
            q.lowbit_gated_raw(x.data_ptr(), K, codes.data_ptr(), scales.data_ptr(), codes.data_ptr(), scales.data_ptr(),
                               q.CODES_PACKED, rms, M, N, K, 128, q.ACT_SILU, y.data_ptr(), ws.data_ptr(), need, st)
        else:
            q.lowbit_linear_raw(x.data_ptr(), K, codes.data_ptr(), q.CODES_PACKED, scales.data_ptr(), rms, M, N, K, 128,
                                y.data_ptr(), ws.data_ptr(), need, st)
    q.device_status()
    for i, y in enumerate(outs):
        value, tol = want[i % 2]
        assert ((y.double() - value).abs() <= tol).all()
        assert torch.equal(y, outs[i % 2])


def product_e2m1(x, w, had):
    """x rounded to fp16 with its group's largest value A in [2^14, 2^15): half a step, 2^-11 of a value (11 bits), or
    2^-25 <= 2^-39 A where fp16 is subnormal. Otherwise as product()."""
    xt = ref.transform(x.double(), had)
    top = xt.reshape(xt.shape[0], -1, 128).abs().amax(-1).repeat_interleave(128, 1)
    e = torch.maximum(xt.abs() * 2 ** -11, top * 2 ** -39)
    w2 = w.square().t()
    return xt @ w.t(), 6 * (e.square() @ w2).sqrt() + 2 ** -17 * (xt.square() @ w2).sqrt() + 1e-38


@pytest.mark.parametrize("M,N,K,had", [(3, 264, 1024, 128), (16, 136, 2048, 256)])
def test_e2m1_input_rounding(cuda_device, M, N, K, had):
    codes, scales, w = weight(N, K, "fp4", False, seed=27)
    x = activations(M, K, seed=28)
    got = q.lowbit_linear(x, codes, scales, code_mode=q.CODES_FP4_PACKED, had_block=had)
    want, err = product_e2m1(x, w, had)
    assert ((got.double() - want).abs() <= 2 ** -8 * want.abs() + err).all()


@pytest.mark.parametrize("M", [2, 16])
def test_e2m1_values_far_below_their_group(cuda_device, M):
    # one value of each group 2^30 to 2^38 above the others and met by a zero weight, so that only the others show: below
    # 2^-28 of the largest they are fp16 subnormals, with 2^-39 of the largest as their bound
    N, K = 72, 512
    codes, scales, _ = weight(N, K, "fp4", False, seed=29)
    codes = codes.reshape(N, -1, 64)
    codes[:, :, 0] &= 0xF0                               # column 0 of each group
    w = ref.scaled(ref.e2m1(codes, N), scales)
    assert not w.reshape(N, -1, 128)[:, :, 0].any()
    g = gen(30)
    x = torch.randn(M, K // 128, 128, device="cuda", generator=g)
    x[:, :, 0] = torch.exp2(torch.randint(30, 39, (M, K // 128), device="cuda", generator=g).float())
    x = x.reshape(M, K).to(BF)
    got = q.lowbit_linear(x, codes.reshape(N, -1), scales, code_mode=q.CODES_FP4_PACKED, had_block=0)
    want, err = product_e2m1(x, w, 0)                    # (the zero weights drop the large values from every sum)
    assert ((got.double() - want).abs() <= 2 ** -8 * want.abs() + err).all()


@pytest.mark.parametrize("M", [1, 9, 40])
def test_three_bit_codes_in_four_bit_containers(cuda_device, M):
    W = (torch.randn(264, 640, device="cuda", generator=gen(31)) * 0.02).to(BF)
    x = activations(M, 640, seed=32)
    for rms in (128, 640):
        qw = q.quantize_fwd(W, 3, rms_group=rms, mask_mode=None, dequant="fp32")
        w = ref.scaled(ref.midrise4(qw["codes"], 264), qw["scales"])
        assert w.abs().max() <= 3.5 * qw["scales"].double().max()      # (in 64 bits, where 3.5 Delta is exact)
        check_linear(q.lowbit_linear(x, qw["codes"], qw["scales"]), x, w, 128)
        a, ea = product(x, w, 128, "int4")
        v, _ = ref.gate(a, "silu")
        got = q.lowbit_gated(x, qw["codes"], qw["scales"], qw["codes"], qw["scales"])
        tol = (2 ** -8 + 2 ** -16) * (v * a).abs() + 1.13 * ea * (a.abs() + ea) + v.abs() * ea + 1e-38
        assert ((got.double() - v * a).abs() <= tol).all()


@pytest.mark.parametrize("grid", ["int4", "fp4"])
@pytest.mark.parametrize("had", [0, 128, 256])
@pytest.mark.parametrize("M", [4, 40])
def test_non_finite_tokens_stay_alone_in_every_form(cuda_device, M, had, grid):
    # untransformed too, where an infinity meets zero weights; transformed by the layer's kernel and by one of its own
    N, K = 72, 1024
    codes, scales, w = weight(N, K, grid, False, seed=33)
    x = activations(M, K, seed=34)

    def both(v):
        return (q.lowbit_linear(v, codes, scales, code_mode=mode(grid), had_block=had),
                q.lowbit_gated(v, codes, scales, codes, scales, code_mode=mode(grid), had_block=had))
    clean = both(x)
    x[1, 7], x[M - 1, 300] = float("-inf"), float("nan")
    keep = [m for m in range(M) if m not in (1, M - 1)]
    for got, was in zip(both(x), clean):
        assert torch.equal(got[keep], was[keep])
    assert not both(x)[0][[1, M - 1]].isfinite().any()

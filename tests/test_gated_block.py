"""quest_gated_linear and quest_gated_bwd against 64-bit formulas (GPU).

Tolerances. Rounding to bf16 is off by at most 2^-8 of the value. A projection is a sum of K
exact products in fp32: its running sum stays within six times R = sqrt(sum x^2 w^2) (a
zero-mean walk; the seeds are fixed), and each of the K additions may cut 2^-23 of it, so it is off by
at most acc = 6 K 2^-23 R. It enters h through |act'| <= 1.13 and |b|, and through |act(a)|. The
sigmoid's exponential and quotient are off by a few 2^-22 of the value, with |z| 2^-23 from the
exponent's argument: 2^-16 covers |z| < 88, beyond which the sigmoid is 0 or 1 in fp32.
"""
import pytest
import torch

import bit_quantization_aware_blockwise_b200 as q
import block_reference as ref

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def operands(M, F, K, seed):
    g = gen(seed)
    x = torch.randn(M, K, device="cuda", generator=g).to(BF)
    w = [(torch.randn(F, K, device="cuda", generator=g) * max(K, 1) ** -0.5).to(BF) for _ in range(2)]
    return x, w[0], w[1]


def check_forward(x, wg, wu, act, h, ckpt):
    K = x.shape[1]
    xd, gd, ud = x.double(), wg.double(), wu.double()
    a, b = xd @ gd.t(), xd @ ud.t()
    ea = 6 * K * 2 ** -23 * (xd.square() @ gd.square().t()).sqrt()
    eb = 6 * K * 2 ** -23 * (xd.square() @ ud.square().t()).sqrt()
    v, _ = ref.gate(a, act)
    want = v * b
    tol = 2 ** -8 * want.abs() + 1.13 * ea * (b.abs() + eb) + v.abs() * eb + 2 ** -16 * want.abs() + 1e-38
    assert ((h.double() - want).abs() <= tol).all()
    if ckpt is None:
        return
    F = wg.shape[0]
    n_groups = (F + 127) // 128
    assert ckpt["codes"].shape == (x.shape[0], 2 * F) and ckpt["scales"].shape == (x.shape[0], 2 * n_groups)
    for got, true, err, s in zip(ref.halves(ckpt), (a, b), (ea, eb), ckpt["scales"].double().split(n_groups, 1)):
        for c in range(n_groups):
            part, e = true[:, 128 * c:128 * c + 128], err[:, 128 * c:128 * c + 128]
            # the step is the largest magnitude over 128 of what the kernel summed, exactly
            assert ((s[:, c] - part.abs().amax(1) / 128).abs() <= e.amax(1) / 128).all()
            off = (got[:, 128 * c:128 * c + 128] - part).abs()
            # half a step, 2^-21 of the quotient (at most 128 steps) at a code's boundary, and the sum's own error
            assert (off <= s[:, c:c + 1] * (0.5 + 128 * 2 ** -21) + e).all()


@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
@pytest.mark.parametrize("M,F,K", [(1, 16, 8), (2, 128, 128), (129, 144, 72), (300, 272, 520), (256, 256, 64),
                                   (513, 1360, 264)])
def test_forward_and_checkpoint(cuda_device, M, F, K, act):
    x, wg, wu = operands(M, F, K, seed=M + F + K)
    h, ckpt = q.gated_linear(x, wg, wu, act=act, checkpoint=True)
    q.device_status()
    check_forward(x, wg, wu, act, h, ckpt)
    # without the checkpoint the output is the same, bit for bit
    assert torch.equal(q.gated_linear(x, wg, wu, act=act).view(torch.int16), h.view(torch.int16))


def test_forward_many_tiles(cuda_device):
    # more tiles than CTA pairs, so that both accumulators of a pair are reused
    x, wg, wu = operands(2560, 2176, 72, seed=3)
    h, ckpt = q.gated_linear(x, wg, wu, checkpoint=True)
    q.device_status()
    check_forward(x, wg, wu, "silu", h, ckpt)


def test_forward_full_layer_sampled(cuda_device):
    # the 1.6B workload's gate and up projections on 16384 tokens; 24 rows recomputed
    x, wg, wu = operands(16384, 5632, 2048, seed=4)
    h, ckpt = q.gated_linear(x, wg, wu, checkpoint=True)
    q.device_status()
    rows = torch.tensor([0, 127, 128, 255, 256, 16383] + list(range(700, 16000, 850)), device="cuda")
    check_forward(x[rows], wg, wu, "silu", h[rows], {k: v[rows] for k, v in ckpt.items()})


def test_checkpoint_codes_of_known_values(cuda_device):
    # x one-hot: the projections are the weights themselves, exact in fp32, so the codes are known
    F, K = 272, 64
    x = torch.eye(K, device="cuda").to(BF)
    g = gen(5)
    wg = (torch.randn(F, K, device="cuda", generator=g) * torch.exp2(torch.randint(-20, 20, (F, 1), device="cuda",
                                                                                  generator=g).float())).to(BF)
    wu = torch.randn(F, K, device="cuda", generator=g).to(BF)
    wu[:128] = 0                                    # a group of zeros: step 0, codes 0
    wu[128:256] = 2.0 ** -110                       # below the floor: kept as zeros
    wg[128:256, 0] = 1.5                            # equal magnitudes: the largest code both ways
    wg[128:192, 0] = -1.5
    h, ckpt = q.gated_linear(x, wg, wu, checkpoint=True)
    q.device_status()
    for half, w in ((0, wg), (1, wu)):
        v = w.double().t()
        for c in range(3):
            part = v[:, 128 * c:128 * c + 128]
            step = ckpt["scales"][:, 3 * half + c].double()
            codes = ckpt["codes"][:, F * half + 128 * c:][:, :part.shape[1]].double()
            big = part.abs().amax(1)
            small = big < 2.0 ** -100
            assert torch.equal(step, torch.where(small, torch.zeros_like(big), big / 128))
            assert (codes[small] == 0).all()
            t = part[~small] / step[~small, None]
            near = (t - t.round()).abs() <= 128 * 2 ** -21
            want = torch.floor(t).clamp(-128, 127)
            ok = codes[~small] == want
            assert (ok | (near & ((codes[~small] - want).abs() <= 1))).all()
    assert (ckpt["codes"][0, 128:192] == -128).all() and (ckpt["codes"][0, 192:256] == 127).all()


def test_non_finite_values_stay_in_their_group(cuda_device):
    x, wg, wu = operands(40, 272, 64, seed=6)
    clean, kept = q.gated_linear(x, wg, wu, checkpoint=True)
    bad = wg.clone()
    bad[130, 3] = float("nan")
    bad[260, 5] = float("inf")
    h, ckpt = q.gated_linear(x, bad, wu, checkpoint=True)
    q.device_status()
    same = torch.ones(272, dtype=torch.bool, device="cuda")
    same[130] = same[260] = False
    assert torch.equal(h[:, same].view(torch.int16), clean[:, same].view(torch.int16))
    assert h[:, 130].isnan().all()
    a, b = ref.halves(ckpt)
    a0, b0 = ref.halves(kept)
    assert torch.equal(a[:, :128], a0[:, :128]) and torch.equal(b, b0)
    assert a[:, 128:256].isnan().all() and not a[:, 256:].isfinite().any()


def test_empty_sizes_and_rows_behind(cuda_device):
    x, wg, wu = operands(4, 48, 0, seed=7)
    h, ckpt = q.gated_linear(x, wg, wu, checkpoint=True)
    assert not h.any() and not ckpt["codes"].any() and not ckpt["scales"].any()
    x, wg, wu = operands(0, 48, 64, seed=7)
    h, ckpt = q.gated_linear(x, wg, wu, checkpoint=True)
    assert h.shape == (0, 48)
    assert q.gated_bwd(h, ckpt).shape == (0, 96)
    # rows behind the last token stay as they were
    M, F, K = 130, 144, 64
    x, wg, wu = operands(M, F, K, seed=8)
    hb = torch.full((M + 140, F), 7.0, dtype=BF, device="cuda")
    cb = torch.full((M + 140, 2 * F), 77, dtype=torch.int8, device="cuda")
    sb = torch.full((M + 140, 4), 7.0, device="cuda")
    st = torch.cuda.current_stream().cuda_stream
    q.gated_linear_raw(x.data_ptr(), wg.data_ptr(), wu.data_ptr(), M, F, K, q.ACT_SILU, hb.data_ptr(), cb.data_ptr(),
                       sb.data_ptr(), st)
    gb = torch.full((M + 140, 2 * F), 7.0, dtype=BF, device="cuda")
    q.gated_bwd_raw(hb.data_ptr(), cb.data_ptr(), sb.data_ptr(), M, F, q.ACT_SILU, gb.data_ptr(), None, st)
    q.device_status()
    check_forward(x, wg, wu, "silu", hb[:M], {"codes": cb[:M], "scales": sb[:M]})
    assert (hb[M:] == 7).all() and (cb[M:] == 77).all() and (sb[M:] == 7).all() and (gb[M:] == 7).all()


def checkpoint(M, F, seed, spread=1.0):
    g = gen(seed)
    n = 2 * ((F + 127) // 128)
    return {"codes": torch.randint(-128, 128, (M, 2 * F), device="cuda", generator=g).to(torch.int8),
            "scales": torch.rand(M, n, device="cuda", generator=g) * (spread / 32)}


@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
@pytest.mark.parametrize("M,F", [(1, 16), (3, 128), (33, 144), (257, 1360), (1024, 5632)])
def test_backward(cuda_device, M, F, act):
    ckpt = checkpoint(M, F, seed=M + F, spread=8.0 if M == 33 else 1.0)
    gh = (torch.randn(M, F, device="cuda", generator=gen(9)) * 1e-3).to(BF)
    grad, h = q.gated_bwd(gh, ckpt, act=act, recompute_h=True)
    a, b = ref.halves(ckpt)
    want = ref.block_back(gh.double(), a, b, act)
    v, dv = ref.gate(a, act)
    # the slope's two terms may cancel: their magnitudes bound what rounding adds
    s = torch.where(a != 0, v / a, torch.full_like(a, 0.5))
    size = torch.cat([(gh.double() * b).abs() * (s + (dv - s).abs()), (gh.double() * v).abs()], 1)
    # the fp32 quotient 1 / (1 + exp(-z)) is 0 where it would be below 2^-126 (its divisor above 2^126), so s may
    # be off by 2^-126, which the slope multiplies by 1 + |a z'| = 1 + |a| |z'|
    flush = 2.0 ** -126
    zp = torch.ones_like(a) if act == "silu" else 1.5957691216 * (1 + 0.134145 * a ** 2)
    under = flush * torch.cat([(gh.double() * b).abs() * (1 + (a * zp).abs()), (gh.double() * a).abs()], 1)
    assert ((grad.double() - want).abs() <= 2 ** -8 * want.abs() + 2 ** -16 * size + under + 1e-38).all()
    assert ((h.double() - v * b).abs() <= (2 ** -8 + 2 ** -16) * (v * b).abs() + flush * (a * b).abs() + 1e-38).all()
    assert torch.equal(q.gated_bwd(gh, ckpt, act=act).view(torch.int16), grad.view(torch.int16))


@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
def test_backward_against_differences(cuda_device, act):
    # the loss sum(grad_h * act(a) b) at the restored a, b, by central differences in 64 bits
    ckpt = checkpoint(16, 160, seed=11)
    gh = (torch.randn(16, 160, device="cuda", generator=gen(12)) * 1e-2).to(BF)
    grad = q.gated_bwd(gh, ckpt, act=act).double()
    a, b = ref.halves(ckpt)
    d = 1e-5                                         # truncation d^2 |act'''| / 6 < 1e-10
    num_a = gh.double() * b * (ref.gate(a + d, act)[0] - ref.gate(a - d, act)[0]) / (2 * d)
    num_b = gh.double() * ref.gate(a, act)[0]
    want = torch.cat([num_a, num_b], 1)
    size = torch.cat([(gh.double() * b).abs() * 2, num_b.abs()], 1)
    assert ((grad - want).abs() <= 2 ** -8 * want.abs() + 2 ** -16 * size + 1e-9).all()


def test_backward_extremes(cuda_device):
    # saturated gates (the sigmoid 0 or 1, z' overflowing) and zero steps give finite gradients
    F = 256
    ckpt = {"codes": torch.tensor([[-128, 127, 0, -1] * (F // 2)], device="cuda").to(torch.int8),
            "scales": torch.tensor([[1e18, 0.0, 1.0, 0.0]], device="cuda")}
    gh = torch.full((1, F), 1.0, dtype=BF, device="cuda")
    for act in ("silu", "gelu_tanh"):
        grad = q.gated_bwd(gh, ckpt, act=act)
        a, b = ref.halves(ckpt)
        assert grad.isfinite().all()
        want = torch.cat([b * (a > 0), torch.where(a > 0, a, torch.zeros_like(a))], 1)
        want[:, 128:256] = b[:, 128:] * 0.5          # a = 0: slope 1/2
        want[:, F + 128:] = 0
        assert ((grad.double() - want).abs() <= 2 ** -8 * want.abs()).all()


def test_streams_graphs_and_repeats(cuda_device):
    M, F, K = 384, 272, 136
    x, wg, wu = operands(M, F, K, seed=13)
    h, ckpt = q.gated_linear(x, wg, wu, checkpoint=True)
    grad = q.gated_bwd(h, ckpt)
    torch.cuda.synchronize()
    # two calls at once, each on a stream of its own, give the same bits as one after the other
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    x2 = x.flip(0).contiguous()
    torch.cuda.synchronize()
    outs = []
    for _ in range(3):
        outs.append((q.gated_linear(x, wg, wu, checkpoint=True, stream=s1),
                     q.gated_linear(x2, wg, wu, checkpoint=True, stream=s2)))
    torch.cuda.synchronize()
    for (h1, c1), (h2, c2) in outs:
        assert torch.equal(h1, h) and torch.equal(c1["codes"], ckpt["codes"])
        assert torch.equal(h2, h.flip(0)) and torch.equal(c2["scales"], ckpt["scales"].flip(0))
    # captured forward and backward, replayed on other inputs
    xs = x.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        hg, cg = q.gated_linear(xs, wg, wu, checkpoint=True)
        gg = q.gated_bwd(hg, cg)
    xs.copy_(x2)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(hg, h.flip(0)) and torch.equal(gg, grad.flip(0))
    xs.copy_(x)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(hg, h) and torch.equal(gg, grad)
    q.device_status()


@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
def test_forward_with_steep_negative_gates(cuda_device, act):
    # gates down to where the sigmoid leaves fp32's normal range: exp's error there is about 104 units in the last place
    # (2^-16), and a quotient below 2^-126 is 0. x is one-hot and up is 1, so the projections are exact
    F, K = 256, 64
    wg = torch.zeros(F, K, device="cuda")
    top = 95.0 if act == "silu" else 11.0                # z = -(95, and 1.6 (11 + 0.0447 1331) = 113)
    wg[:, 0] = -torch.linspace(1.0, top, F, device="cuda")
    wu = torch.zeros(F, K, device="cuda")
    wu[:, 0] = 1
    x = torch.zeros(2, K, device="cuda")
    x[:, 0] = 1
    x, wg, wu = x.to(BF), wg.to(BF), wu.to(BF)
    h = q.gated_linear(x, wg, wu, act=act)
    q.device_status()
    a = wg[:, 0].double()
    want = ref.gate(a, act)[0]
    # GELU's own exponent z is a product of fp32 roundings, 2 2^-23 of |z|, which exp turns into as much of the value
    z = 0.0 if act == "silu" else 113 * 2 * 2 ** -23
    tol = (2 ** -8 + 2 ** -16 + z) * want.abs() + 2.0 ** -126 * a.abs() + 2.0 ** -133
    assert ((h[0].double() - want).abs() <= tol).all() and torch.equal(h[0], h[1])

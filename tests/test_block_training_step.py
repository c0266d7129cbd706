"""The block's calls as a training step and a decoding step run them: the library's own
intermediates feed the next call, and each result is held to the 64-bit formula of those intermediates."""
import pytest
import torch

import bit_quantization_aware_blockwise_b200 as q
import block_reference as ref

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


@pytest.mark.parametrize("bits", [4, 8])
def test_training_step(cuda_device, bits):
    T, K, F = 384, 512, 272
    g = gen(1)
    X = torch.randn(T, K, device="cuda", generator=g).to(BF)
    Wg, Wu = [(torch.randn(F, K, device="cuda", generator=g) * K ** -0.5).to(BF) for _ in range(2)]
    gh = (torch.randn(T, F, device="cuda", generator=g) * 1e-2).to(BF)

    # forward: quantize both operands, the block keeps its projections in 8 bits and its input as codes
    qx = q.quantize_fwd(X, bits, dequant="bf16")
    qg, qu = [q.quantize_fwd(W, 4, dequant="bf16") for W in (Wg, Wu)]
    h, kept = q.gated_linear(qx["dequant"], qg["dequant"], qu["dequant"], checkpoint=True)
    # backward: the projections' gradients, then the input's and both weights' in one call each
    grad_ab = q.gated_bwd(gh, kept)
    w_t = torch.cat([q.transpose_bf16(w["dequant"]) for w in (qg, qu)], 1)               # [K, 2F]
    masks = torch.cat([w["mask"].view(F, -1) for w in (qg, qu)])                         # [2F, K / 8]
    grad_x = q.trust_bwd_linear(grad_ab, w_t, qx["mask"])
    grad_w = q.weight_grad(grad_ab, qx["codes"], qx["scales"], bits, mask=masks, K=K, out_dtype=torch.float32)
    q.device_status()

    # The codes stand for the operand the forward multiplied. The quantizer's dequant adds (1/2 - 2^(b-1)) Delta, itself
    # rounded, to q_b Delta in fp32: off by 2^-24 2^(b-1) Delta, which is 2^-16 of the smallest value Delta / 2 at b = 8,
    # so the two bf16 roundings differ by one step at most, where the value lies that close to a tie.
    codes = ref.midrise4(qx["codes"], T) if bits == 4 else qx["codes"].view(torch.int8).view(T, K).double() + 0.5
    xh = ref.bf16_input(codes, qx["scales"])
    assert ((xh - qx["dequant"].double()).abs() <= 2 ** -7 * xh.abs()).all()
    xf = qx["dequant"].double()
    a, b = xf @ qg["dequant"].double().t(), xf @ qu["dequant"].double().t()
    ra, rb = ref.halves(kept)
    for got, want in ((ra, a), (rb, b)):
        peak = torch.stack([c.abs().amax(1) for c in want.split(128, 1)], 1)
        step = peak.repeat_interleave(128, 1)[:, :F] / 128
        # half a step, and fp32 sums of K = 512 terms (off by at most 512 * 2^-23 of a magnitude below 4 peaks)
        assert ((got - want).abs() <= step * 0.51 + 4 * 512 * 2 ** -23 * peak.amax(1, keepdim=True)).all()
    assert (h.double() - ref.gate(a, "silu")[0] * b).norm() <= 2 ** -8 * h.double().norm()
    want_ab = ref.block_back(gh.double(), ra, rb, "silu")
    assert (grad_ab.double() - want_ab).norm() <= 2 ** -8 * want_ab.norm()
    m = ref.mask_values(qx["mask"], T, K)
    want_x = ref.transform(m * (grad_ab.double() @ torch.cat([qg["dequant"], qu["dequant"]]).double()), 128)
    assert (grad_x.double() - want_x).norm() <= (2 ** -8 + 2 ** -13) * want_x.norm()
    want_w = ref.weight_grad(grad_ab, xh, masks)
    assert (grad_w.double() - want_w).norm() <= (6 * (T / 16 + 17) * 2 ** -23 + 2 ** -21) * want_w.norm()

    # a second micro-batch adds its gradient to the first
    total = q.weight_grad(grad_ab, qx["codes"], qx["scales"], bits, mask=masks, K=K, out=grad_w.clone(), accumulate=True)
    assert torch.equal(total, 2 * grad_w)


def test_checkpoint_changes_the_gradient_by_its_rounding_only(cuda_device):
    # against the gradients of the unrounded projections: an 8-bit step is 1/128 of a group's largest value, about 3
    # standard deviations, so a and b are off by up to 3 / 256 (rms 3 / 128 / sqrt(12) = 0.7 %) of one. d grad / d a and
    # d grad / d b are of the gradient's own size: 2 % of its norm covers both, and bf16's 2^-8
    T, F, K = 512, 512, 256
    g = gen(2)
    x, wg, wu = [(torch.randn(n, K, device="cuda", generator=g) * s).to(BF) for n, s in ((T, 1.0), (F, K ** -0.5), (F, K ** -0.5))]
    gh = torch.randn(T, F, device="cuda", generator=g).to(BF)
    _, kept = q.gated_linear(x, wg, wu, checkpoint=True)
    got = q.gated_bwd(gh, kept).double()
    a, b = x.double() @ wg.double().t(), x.double() @ wu.double().t()
    want = ref.block_back(gh.double(), a, b, "silu")
    assert (got - want).norm() <= (0.02 + 2 ** -8) * want.norm()


@pytest.mark.parametrize("code_mode", [q.CODES_PACKED, q.CODES_FP4_PACKED])
def test_decoding_step(cuda_device, code_mode):
    # the block for one token after a prefill of the same weights: the last token's h agrees
    K, F = 512, 1360
    g = gen(3)
    X = torch.randn(40, K, device="cuda", generator=g).to(BF)
    W = [(torch.randn(F, K, device="cuda", generator=g) * K ** -0.5).to(BF) for _ in range(2)]
    Wd = (torch.randn(K, F, device="cuda", generator=g) * F ** -0.5).to(BF)[:, :1024].contiguous()
    qg, qu = [q.quantize_fwd(w, 4, code_mode=code_mode, mask_mode=None, dequant="fp32") for w in W]
    qd = q.quantize_fwd(Wd, 4, rms_group=1024, code_mode=code_mode, mask_mode=None, dequant="fp32")
    x = X[-1:]
    h = q.lowbit_gated(x, qg["codes"], qg["scales"], qu["codes"], qu["scales"], code_mode=code_mode)
    y = q.lowbit_linear(h[:, :1024], qd["codes"], qd["scales"], code_mode=code_mode)
    xt = ref.transform(x.double(), 128)
    want = ref.gate(xt @ qg["dequant"].double().t(), "silu")[0] * (xt @ qu["dequant"].double().t())
    assert (h.double() - want).norm() <= 2 ** -8 * want.norm()
    want_y = ref.transform(h[:, :1024].double(), 128) @ qd["dequant"].double().t()
    assert (y.double() - want_y).norm() <= 2 ** -8 * want_y.norm()
    # prefill: the input in bf16 in the Hadamard domain (rounded to 2^-9 rms of each value), the weights in bf16
    xh = ref.transform(X.double(), 128).to(BF)
    hp = q.gated_linear(xh, qg["dequant"].to(BF), qu["dequant"].to(BF))
    assert (hp[-1:].double() - want).norm() <= 4 * 2 ** -8 * want.norm()

"""The gated block's calls refuse bad arguments on the host, before any CUDA call: these
run without a GPU, and the pointers are never dereferenced."""
import pytest
import torch

import bit_quantization_aware_blockwise_b200 as q

P = [(i + 1) << 32 for i in range(10)]   # aligned addresses, far apart, never touched
EINVAL, EUNSUPPORTED, ECUDA = 1, 2, 3


def gated_linear(x=P[0], wg=P[1], wu=P[2], M=4, F=32, K=64, act=0, h=P[3], codes=P[4], scales=P[5]):
    return q.load_library().quest_gated_linear(x, wg, wu, M, F, K, act, h, codes, scales, None)


def gated_bwd(gh=P[0], codes=P[1], scales=P[2], M=4, F=32, act=0, grad=P[3], h=P[4]):
    return q.load_library().quest_gated_bwd(gh, codes, scales, M, F, act, grad, h, None)


def weight_grad(gy=P[0], ld=32, codes=P[1], mode=0, bits=8, scales=P[2], rms=128, mask=P[3], T=4, N=32, K=256, had=128,
                out=P[4], dt=0, acc=0, ws=P[5], ws_bytes=1 << 24):
    return q.load_library().quest_weight_grad(gy, ld, codes, mode, bits, scales, rms, mask, T, N, K, had, out, dt, acc,
                                              ws, ws_bytes, None)


def lowbit_linear(x=P[0], ld=256, codes=P[1], mode=0, scales=P[2], rms=128, M=4, N=32, K=256, had=128, y=P[3],
                  ws=P[6], ws_bytes=1 << 24):
    return q.load_library().quest_lowbit_linear(x, ld, codes, mode, scales, rms, M, N, K, had, y, ws, ws_bytes, None)


def lowbit_gated(x=P[0], ld=256, cg=P[1], sg=P[2], cu=P[3], su=P[4], mode=0, rms=128, M=4, F=32, K=256, had=128, act=0,
                 h=P[5], ws=P[6], ws_bytes=1 << 24):
    return q.load_library().quest_lowbit_gated(x, ld, cg, sg, cu, su, mode, rms, M, F, K, had, act, h, ws, ws_bytes, None)


REFUSED = [
    (gated_linear, EINVAL, [dict(M=-1), dict(F=-16), dict(K=-8), dict(F=24), dict(K=12), dict(act=2), dict(x=None),
                            dict(wg=None), dict(wu=None), dict(h=None), dict(codes=None), dict(scales=None),
                            dict(x=P[0] + 8), dict(wu=P[2] + 2), dict(h=P[3] + 8), dict(codes=P[4] + 8),
                            dict(scales=P[5] + 2), dict(M=1 << 31), dict(F=1 << 30), dict(h=P[0] + 64),
                            dict(codes=P[1] + 16), dict(scales=P[3] + 4), dict(h=P[2])]),
    (gated_bwd, EINVAL, [dict(M=-1), dict(F=8), dict(act=-1), dict(gh=None), dict(codes=None), dict(scales=None),
                         dict(grad=None), dict(gh=P[0] + 2), dict(codes=P[1] + 8), dict(scales=P[2] + 1),
                         dict(grad=P[3] + 8), dict(h=P[4] + 4), dict(grad=P[0]), dict(h=P[0] + 16), dict(h=P[3] + 32),
                         dict(M=1 << 31)]),
    (weight_grad, EINVAL, [dict(T=-1), dict(N=-8), dict(K=-128), dict(N=12), dict(K=200), dict(ld=24), dict(ld=36), dict(ld=1 << 40),
                           dict(bits=0), dict(bits=9), dict(mode=6), dict(had=100), dict(rms=64), dict(dt=2),
                           dict(acc=1), dict(acc=2, dt=1), dict(gy=None), dict(codes=None), dict(scales=None),
                           dict(out=None), dict(gy=P[0] + 8), dict(codes=P[1] + 4), dict(scales=P[2] + 2),
                           dict(mask=P[3] + 8), dict(out=P[4] + 4), dict(out=P[1] + 128), dict(out=P[3]),
                           dict(T=1 << 31), dict(ws=None), dict(ws_bytes=2047), dict(ws=P[5] + 8), dict(ws=P[0]),
                           dict(ws=P[4] + 64)]),
    (weight_grad, EUNSUPPORTED, [dict(mode=3, bits=4), dict(mode=4, bits=4), dict(bits=2), dict(bits=1), dict(had=64)]),
    (lowbit_linear, EINVAL, [dict(M=-1), dict(N=12), dict(K=192), dict(K=384, ld=384, had=256), dict(ld=128),
                             dict(ld=260), dict(ld=1 << 40), dict(had=100), dict(had=-1), dict(rms=64), dict(mode=9), dict(x=None),
                             dict(codes=None), dict(scales=None), dict(y=None), dict(x=P[0] + 8), dict(codes=P[1] + 8),
                             dict(scales=P[2] + 2), dict(y=P[3] + 2), dict(y=P[0]), dict(y=P[1] + 16),
                             dict(y=P[2]), dict(N=1 << 31)]),
    (lowbit_linear, EINVAL, [dict(M=64, K=4096, ld=4096, **kw) for kw in (
        dict(ws=None), dict(ws_bytes=1000), dict(ws=P[6] + 8), dict(ws=P[0]), dict(ws=P[1]), dict(ws=P[3]))]),
    (lowbit_linear, EUNSUPPORTED, [dict(M=65), dict(K=32896, ld=32896), dict(mode=1), dict(mode=2), dict(mode=5)]),
    (lowbit_gated, EINVAL, [dict(cu=None), dict(su=None), dict(cu=P[3] + 4), dict(su=P[4] + 2), dict(act=7),
                            dict(h=P[3]), dict(F=4), dict(h=None)]),
    (lowbit_gated, EUNSUPPORTED, [dict(M=65)]),
]


@pytest.mark.parametrize("call,status,kw", [(c, s, kw) for c, s, kws in REFUSED for kw in kws])
def test_refuses(call, status, kw):
    assert call(**kw) == status
    assert q.load_library().quest_last_error_message()


def test_nothing_to_do_needs_no_pointers():
    assert gated_linear(M=0, x=None, wg=None, wu=None, h=None, codes=None, scales=None) == 0
    assert gated_linear(F=0, x=None, wg=None, wu=None, h=None, codes=None, scales=None) == 0
    assert gated_bwd(M=0, gh=None, codes=None, scales=None, grad=None, h=None) == 0
    assert weight_grad(N=0, gy=None, codes=None, scales=None, mask=None, out=None) == 0
    assert weight_grad(K=0, rms=0, gy=None, codes=None, scales=None, mask=None, out=None) == 0
    # the empty sum added to a gradient leaves it
    assert weight_grad(T=0, gy=None, codes=None, scales=None, mask=None, dt=1, acc=1) == 0
    assert lowbit_linear(M=0, x=None, codes=None, scales=None, y=None) == 0
    assert lowbit_gated(F=0, x=None, cg=None, sg=None, cu=None, su=None, h=None) == 0


@pytest.mark.parametrize("call", [gated_linear, gated_bwd, weight_grad, lowbit_linear, lowbit_gated])
def test_injected_launch_failure(call):
    lib = q.load_library()
    assert lib.quest_debug_inject_fault(q.FAULT_LAUNCH) == 0
    assert call() == ECUDA
    assert b"injected" in lib.quest_last_error_message()


def test_workspace_query():
    assert q.weight_grad_workspace(-1, 8, 128) == 0
    assert q.weight_grad_workspace(64, 12, 128) == 0
    assert q.weight_grad_workspace(0, 8, 128) == 0
    assert q.lowbit_workspace(1, 2048) == 0 and q.lowbit_workspace(65, 2048) == 0
    assert q.lowbit_workspace(16, 8192) >= 16 * 8192 * 2


def test_wrappers_refuse_host_tensors():
    x = torch.zeros((4, 128), dtype=torch.bfloat16)
    w = torch.zeros((16, 128), dtype=torch.bfloat16)
    codes, scales = torch.zeros((16, 64), dtype=torch.uint8), torch.zeros((16, 1))
    for call in (lambda: q.gated_linear(x, w, w), lambda: q.gated_bwd(x, {"codes": codes, "scales": scales}),
                 lambda: q.weight_grad(x, codes, scales, 4), lambda: q.lowbit_linear(x, codes, scales),
                 lambda: q.lowbit_gated(x, codes, scales, codes, scales)):
        with pytest.raises(q.QuestError, match="CUDA tensor"):
            call()


BIG = (1 << 31) - 128   # a multiple of 128


@pytest.mark.parametrize("call,kw,what", [
    (weight_grad, dict(T=BIG, N=8, ld=8, K=BIG), "T * K"),
    (weight_grad, dict(T=1 << 30, N=8, ld=8, K=1 << 15), "T * K"),
    (weight_grad, dict(T=BIG, N=8, ld=BIG, K=128), "T * ld_gy"),
    (weight_grad, dict(T=4, N=1 << 30, ld=1 << 30, K=1 << 30), "N * K"),
    (gated_linear, dict(M=BIG, F=16, K=BIG), "M * K"),
    (gated_linear, dict(M=1, F=1 << 29, K=BIG), "F * K"),
    (gated_bwd, dict(M=BIG, F=1 << 29), "M * F"),
])
def test_sizes_whose_products_pass_64_bits_are_refused(call, kw, what):
    # before any byte count is formed from them (and, with the largest workspace a caller can claim, before any launch)
    if call is weight_grad:
        kw = dict(kw, ws_bytes=(1 << 64) - 1)
    assert call(**kw) == EINVAL
    assert what in q.load_library().quest_last_error_message().decode()


def test_workspace_query_of_impossible_sizes():
    assert q.weight_grad_workspace(BIG, 8, BIG) == 0
    assert q.weight_grad_workspace(8, BIG, BIG) == 0
    assert q.weight_grad_workspace(1 << 29, 8, 1 << 14) >= 1 << 44


def host_weight_grad(monkeypatch, T=4, N=16, width=256, **kw):
    """weight_grad on host tensors, up to its library call (which is recorded, not made)."""
    made = []
    monkeypatch.setattr(q._binding, "_require_cuda", lambda t, name: None)
    monkeypatch.setattr(q._binding, "_at", lambda device, stream: q._binding._HERE_ALREADY)
    monkeypatch.setattr(q._binding, "_stream_handle", lambda stream, device: 0)
    monkeypatch.setattr(q._binding, "weight_grad_raw", lambda *a, **k: made.append(a))
    args = dict(codes=torch.zeros((T, width), dtype=torch.int8), scales=torch.ones((T, width // 128)), bits=8)
    args.update(kw)
    q.weight_grad(torch.zeros((T, N), dtype=torch.bfloat16), args.pop("codes"), args.pop("scales"), args.pop("bits"), **args)
    assert len(made) == 1


def test_weight_grad_takes_mask_bits_only(monkeypatch):
    host_weight_grad(monkeypatch, mask=torch.zeros((16, 32), dtype=torch.uint8))
    host_weight_grad(monkeypatch, mask=torch.zeros((16, 8), dtype=torch.int32))
    host_weight_grad(monkeypatch, mask=torch.zeros(16 * 32, dtype=torch.uint8))
    # the quantizer's other mask form, one byte a value, holds the bytes of eight masks of bits
    for mask in (torch.ones((16, 256), dtype=torch.uint8), torch.ones(17 * 32, dtype=torch.uint8),
                 torch.ones(15 * 32, dtype=torch.uint8)):
        with pytest.raises(q.QuestError, match="mask"):
            host_weight_grad(monkeypatch, mask=mask)


def test_weight_grad_codes_rows(monkeypatch):
    host_weight_grad(monkeypatch, codes=torch.zeros(4 * 256, dtype=torch.int8), K=256)
    host_weight_grad(monkeypatch, codes=torch.zeros(9 * 256, dtype=torch.int8), K=256)      # rows behind the last token
    host_weight_grad(monkeypatch, codes=torch.zeros((4, 128), dtype=torch.uint8), bits=4, K=256)
    for codes, kw in ((torch.zeros((4, 384), dtype=torch.int8), dict(K=256)),               # longer rows than K
                      (torch.zeros((5, 256), dtype=torch.int8), dict(K=256)),               # another token count
                      (torch.zeros((4, 256), dtype=torch.uint8), dict(K=256, bits=4)),      # not packed
                      (torch.zeros(3 * 256, dtype=torch.int8), dict(K=256))):
        with pytest.raises(q.QuestError, match="codes"):
            host_weight_grad(monkeypatch, codes=codes, **kw)


def test_steps_of_another_row_count(monkeypatch):
    for scales in (torch.ones((4, 2)), torch.ones((4, 1)), torch.ones(4)):
        host_weight_grad(monkeypatch, scales=scales)
    # as many numbers as tokens, but two groups for each of two tokens
    for scales in (torch.ones((2, 2)), torch.ones((1, 4)), torch.ones((3, 2)), torch.ones(())):
        with pytest.raises(q.QuestError, match="scales"):
            host_weight_grad(monkeypatch, scales=scales)


def test_low_bit_steps_without_rows(monkeypatch):
    monkeypatch.setattr(q._binding, "_require_cuda", lambda t, name: None)
    x, codes, s = torch.zeros((1, 128), dtype=torch.bfloat16), torch.zeros(64, dtype=torch.uint8), torch.ones(())
    for call in (lambda: q.lowbit_linear(x, codes, s), lambda: q.lowbit_gated(x, codes, s, codes, s)):
        with pytest.raises(q.QuestError, match="scales"):
            call()

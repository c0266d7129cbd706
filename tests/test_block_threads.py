"""The block's calls from several host threads at once, each on a stream of its own (GPU): the same bits as alone."""
import threading

import pytest
import torch

import bit_quantization_aware_blockwise_b200 as q

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


def job(i):
    g = torch.Generator(device="cuda").manual_seed(60 + i)
    T, F, K, M = 200 + 64 * i, 272, 256 + 128 * i, 1 + 12 * i
    x = torch.randn(T, K, device="cuda", generator=g).to(BF)
    w = [(torch.randn(F, K, device="cuda", generator=g) * K ** -0.5).to(BF) for _ in range(2)]
    qx = q.quantize_fwd(x, 8, dequant="bf16")
    qw = [q.quantize_fwd(v, 4, mask_mode=None) for v in w]
    act = "silu" if i % 2 else "gelu_tanh"

    def run(stream=None):
        h, kept = q.gated_linear(qx["dequant"], w[0], w[1], act=act, checkpoint=True, stream=stream)
        gab = q.gated_bwd(h, kept, act=act, stream=stream)
        gw = q.weight_grad(gab, qx["codes"], qx["scales"], 8, K=K, out_dtype=torch.float32, stream=stream)
        y = q.lowbit_linear(x[:M], qw[0]["codes"], qw[0]["scales"], stream=stream)
        z = q.lowbit_gated(x[:M], qw[0]["codes"], qw[0]["scales"], qw[1]["codes"], qw[1]["scales"], act=act, stream=stream)
        return h, kept["codes"], kept["scales"], gab, gw, y, z
    return run


def test_calls_from_several_threads(cuda_device):
    jobs = [job(i) for i in range(5)]
    want = [run() for run in jobs]
    streams = [torch.cuda.Stream() for _ in jobs]
    torch.cuda.synchronize()
    got, failed = [[] for _ in jobs], []
    start = threading.Barrier(len(jobs))

    def work(i):
        try:
            start.wait(30)
            for _ in range(20):
                got[i].append(jobs[i](streams[i]))
            # a refused call's message is the thread's own
            with pytest.raises(q.QuestError, match="act"):
                q.gated_linear(got[i][0][0], got[i][0][0], got[i][0][0], act="relu", stream=streams[i])
        except BaseException as e:   # noqa: BLE001  (reported by the test's own thread)
            failed.append(e)
    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(jobs))]
    for t in threads:
        t.start()
    for t in threads:
        t.join(120)
    torch.cuda.synchronize()
    q.device_status()
    assert not failed
    for alone, runs in zip(want, got):
        assert len(runs) == 20
        for r in runs:
            assert all(torch.equal(a, b) for a, b in zip(alone, r))

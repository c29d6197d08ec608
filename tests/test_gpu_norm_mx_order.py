"""The norm, the balance loss and the 4-bit products among other work: operands that the
launch before writes, and several host threads at once on one stream and on their own.
(The products start while the launch before them drains, and read the weights early.)"""
import threading

import pytest
import torch

import newton_schulz_bucket_gb300 as muon

pytestmark = pytest.mark.gpu


def _randn(*shape, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(*shape, generator=g, device="cuda").bfloat16()


@pytest.mark.parametrize("rows", [1, 5, 16, 17, 40, 64, 70, 300])
def test_operands_written_just_before(rows):
    held = [muon.mx_quantize(_randn(1024, 700, seed=i)) for i in range(2)]
    xs = [_randn(rows, 1024, seed=2 + i) for i in range(2)]
    want = {(i, j): muon.mx_linear(xs[j], *held[i]) for i in range(2) for j in range(2)}
    v, s, x = held[0][0].clone(), held[0][1].clone(), xs[0].clone()
    torch.cuda.synchronize()
    out = []
    for it in range(48):
        i, j = it // 3 % 2, it // 5 % 2
        v.copy_(held[i][0])
        s.copy_(held[i][1])
        x.copy_(xs[j])
        out.append((i, j, muon.mx_linear(x, v, s)))
    assert all(torch.equal(y, want[i, j]) for i, j, y in out)
    muon.check_ops_error()


@pytest.mark.parametrize("rows", [9, 200, 2000])
def test_expert_weights_and_offsets_written_just_before(rows):
    held = [muon.mx_quantize(_randn(6, 512, 300, seed=i)) for i in range(2)]
    offs = [torch.tensor(o, dtype=torch.int32, device="cuda")
            for o in ([0, rows // 3, rows // 3, rows // 2, rows, rows, rows], [0, 0, 1, 2, 3, rows - 1, rows])]
    x = _randn(rows, 512, seed=3)
    want = {(i, j): muon.mx_expert_linear(x, offs[j], *held[i]) for i in range(2) for j in range(2)}
    v, s, off = held[0][0].clone(), held[0][1].clone(), offs[0].clone()
    torch.cuda.synchronize()
    out = []
    for it in range(48):
        i, j = it // 3 % 2, it // 5 % 2
        off.copy_(offs[j])
        v.copy_(held[i][0])
        s.copy_(held[i][1])
        out.append((i, j, muon.mx_expert_linear(x, off, v, s)))
    assert all(torch.equal(y, want[i, j]) for i, j, y in out)
    muon.check_ops_error()


def test_threads_on_one_stream_and_on_their_own():
    wrong = []

    def work(k):
        stream = torch.cuda.Stream() if k % 2 else torch.cuda.default_stream()
        with torch.cuda.stream(stream):
            x = _randn(300, 1024, seed=k)
            values, scales = muon.mx_quantize(_randn(4, 1024, 520, seed=k))
            off = torch.tensor([0, 20, 100, 100, 300], dtype=torch.int32, device="cuda")
            logits = _randn(3000, 100, seed=k)
            idx, _ = muon.gate(logits, 4)
            first = None
            for it in range(60):
                n = muon.layer_norm(x, keep_stats=True)
                now = (*n, *muon.layer_norm_backward(x, x, n[1], n[2], bias=True), *muon.balance_loss(logits, idx),
                       muon.mx_expert_linear(x, off, values, scales))
                first = first or now
                if it % 6 == 5 and not all(torch.equal(p, q) for p, q in zip(first, now)):
                    wrong.append((k, it))
        stream.synchronize()

    threads = [threading.Thread(target=work, args=(k,)) for k in range(6)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong
    muon.check_ops_error()

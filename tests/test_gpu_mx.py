"""Microscaled 4-bit weights and their products on the GPU: the packed bytes exactly
the oracle's, the products against fp64 products of the same rounded numbers,
element by element (tolerances as for linear: 4-bit products and their scales are
exact, the sum is fp32)."""
import math

import numpy as np
import pytest
import torch

import newton_schulz_bucket_gb300 as muon
from oracle import layers_ref as ref

from layers_tol import check_forward, to64

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def _randn(shape, dtype, seed, std=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(*shape, generator=g, device="cuda") * std).to(dtype)


def _rounded(x):
    """The numbers that the rows of x stand for in 4 bits, as fp64 on the host."""
    return torch.from_numpy(ref.mx_round(to64(x))[0])


def _held(values, scales, n):
    return torch.from_numpy(ref.mx_held(values.cpu().numpy(), scales.cpu().numpy(), n))


def _check_quantize(w):
    values, scales = muon.mx_quantize(w)
    q, s = ref.mx_round(np.swapaxes(to64(w), -1, -2))
    n = w.shape[-2]
    assert np.array_equal(scales.cpu().numpy(), s)
    blocks = s.shape[-1]
    assert values.shape == (*s.shape[:-1], 16 * blocks)
    whole = ref.mx_held(values.cpu().numpy(), s, 32 * blocks)
    assert np.array_equal(np.isnan(whole[..., :n]), np.isnan(q))
    assert np.array_equal(np.nan_to_num(whole[..., :n]), np.nan_to_num(q))
    assert not np.nan_to_num(whole[..., n:]).any()
    for dt in (torch.float32, w.dtype):
        back = muon.mx_dequantize(values, scales, n, dtype=dt)
        assert back.shape == w.shape and back.dtype == dt
        want = torch.from_numpy(np.swapaxes(q, -1, -2).copy()).to(dt)  # (rounded once: fp16 has a smaller range)
        assert torch.equal(torch.nan_to_num(back.cpu()), torch.nan_to_num(want))
        assert torch.equal(torch.isnan(back.cpu()), torch.isnan(want))
    return values, scales


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("out_in", [False, True])
@pytest.mark.parametrize("shape", [(1, 1), (31, 3), (32, 64), (33, 65), (100, 7), (256, 64), (300, 130), (512, 20), (777, 33),
                                   (2, 40, 50), (3, 288, 70), (5, 65, 129)], ids=lambda s: "x".join(map(str, s)))
def test_quantize(shape, dtype, out_in):
    *lead, n, m = shape
    if out_in:
        w = _randn((*lead, m, n), DT[dtype], n + m).transpose(-1, -2)
    else:
        w = _randn((*lead, n, m), DT[dtype], n + m)
    _check_quantize(w)


def test_quantize_strides_and_slices():
    big = _randn((4, 200, 136), torch.bfloat16, 1)
    for w in (big[1:3, 8:168, 8:72], big[:, 3:100, 5:60], big[::2, :64, :64], big[2, :, 1:2], big[0, 7:8, :],
              big.transpose(-1, -2)[:, 8:72, 8:168], big.transpose(-1, -2)[1, 5:60, 3:100]):
        values, scales = _check_quantize(w)
        again = muon.mx_quantize(w.contiguous())
        assert torch.equal(values, again[0]) and torch.equal(scales, again[1])


@pytest.mark.parametrize("out_in", [False, True])
@pytest.mark.parametrize("dtype", list(DT))
def test_quantize_every_border(dtype, out_in):
    """Each middle between neighbours, the numbers next to it on both sides, in both
    signs and many scales, the largest and smallest ones, zeros."""
    dt = DT[dtype]
    middles = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, 7.0, 7.9], device="cuda")
    eps = torch.finfo(dt).eps
    at = torch.cat((middles, middles * (1 + eps), middles * (1 - eps / 2), torch.tensor([4.0, 0.0], device="cuda")))
    scale = 2.0 ** torch.arange(-14 if dtype == "fp16" else -120, 12 if dtype == "fp16" else 120, 1, device="cuda").float()
    w = (at[None, :] * scale[:, None]).to(dt)
    w = torch.cat((w, -w))
    ends = torch.zeros(4, 32, device="cuda")
    ends[0, 0], ends[1, 5], ends[2, 31] = torch.finfo(dt).max, torch.finfo(dt).tiny, torch.finfo(dt).smallest_normal / 8
    ends[3] = -0.0
    w = torch.cat((w, ends.to(dt))).contiguous()  # rows are blocks
    _check_quantize(w.t() if out_in else w.t().contiguous())


@pytest.mark.parametrize("out_in", [False, True])
@pytest.mark.parametrize("dtype", list(DT))
def test_quantize_non_finite_blocks(dtype, out_in):
    w = _randn((6, 96), DT[dtype], 3)
    w[1, 40], w[2, 0], w[4, 95], w[5, 33] = math.inf, math.nan, -math.inf, math.nan
    values, scales = _check_quantize(w.t() if out_in else w.t().contiguous())
    assert (scales.cpu() == 255).nonzero().tolist() == [[1, 1], [2, 0], [4, 2], [5, 1]]


# one matrix: up to 64 rows in clusters that share the sum (16 to 64 columns), then pairs with tiles of 64, 128 and 192
# tokens; sums of part of a block, an odd number of 128 steps, part of a stage of 256
LINEAR = [(1, 32, 1), (1, 64, 128), (1, 1000, 129), (3, 512, 300), (16, 777, 129), (17, 1024, 256), (40, 2048, 100),
          (64, 300, 500), (64, 4096, 260), (65, 64, 128), (100, 33, 7), (129, 256, 256), (190, 384, 300), (200, 777, 129),
          (300, 1024, 512), (1000, 130, 1000), (2, 12345, 40), (70, 9000, 70), (33, 320, 9800), (64, 96, 12300), (7, 96, 12300)]


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("case", LINEAR, ids=lambda c: "x".join(map(str, c)))
def test_linear(case, dtype):
    rows, n_in, n_out = case
    dt = DT[dtype]
    x = _randn((rows, n_in), dt, 1)
    values, scales = muon.mx_quantize(_randn((n_in, n_out), torch.float32, 2, n_in ** -0.5))
    X, W = _rounded(x), _held(values, scales, n_in).T
    b, r = _randn((n_out,), dt, 3), _randn((rows, n_out), dt, 4)
    check_forward(muon.mx_linear(x, values, scales), None, X, W, None, "none", None)
    kind = ("relu", "silu", "gelu", "gelu_tanh")[sum(case) % 4]
    check_forward(muon.mx_linear(x, values, scales, bias=b, activation=kind, residual=r), None, X, W, b, kind, r)
    muon.check_ops_error()


def test_linear_fills_the_gpu_with_every_tile():
    """As many tiles as the GPU takes at a time and more, of 192, 128 and 64 tokens."""
    for rows, n_in, n_out in ((1500, 256, 2560), (900, 320, 2560), (400, 256, 2560), (192, 1024, 20000)):
        x = _randn((rows, n_in), torch.bfloat16, rows)
        values, scales = muon.mx_quantize(_randn((n_in, n_out), torch.float32, 2, n_in ** -0.5))
        check_forward(muon.mx_linear(x, values, scales), None, _rounded(x), _held(values, scales, n_in).T, None, "none", None)
    muon.check_ops_error()


def _experts(rows, experts, n_in, n_out, dtype, offsets, kind, bias=True, residual=True):
    dt = DT[dtype]
    x = _randn((rows, n_in), dt, rows)
    values, scales = muon.mx_quantize(_randn((experts, n_in, n_out), torch.float32, 2, n_in ** -0.5))
    off = torch.tensor(offsets, dtype=torch.int32, device="cuda")
    b = _randn((experts, n_out), dt, 3) if bias else None
    r = _randn((rows, n_out), dt, 4) if residual else None
    y = muon.mx_expert_linear(x, off, values, scales, bias=b, activation=kind, residual=r)
    muon.check_ops_error()
    X, W = _rounded(x), _held(values, scales, n_in).transpose(-1, -2)
    lo, hi = offsets[0], offsets[-1]
    if lo:  # the check wants rows from the first range on
        assert not y[:lo].any()
        y, X, r, offsets = y[lo:], X[lo:], None if r is None else r[lo:], [o - lo for o in offsets]
    live = offsets[-1]
    assert not y[live:].any()
    check_forward(y[:live], None, X[:live], W, b, kind, None if r is None else r[:live], offsets)


def _cut(rows, experts, seed, empty=0.2):
    rng = np.random.default_rng(seed)
    share = rng.exponential(size=experts) * (rng.random(experts) >= empty)
    ends = np.floor(rows * np.cumsum(share) / max(share.sum(), 1e-9)).astype(int)
    ends[-1] = rows
    return [0, *(int(e) for e in ends)]


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("case", [(1, 3, 64, 40), (9, 16, 96, 70), (64, 8, 300, 129), (200, 4, 512, 256), (700, 3, 160, 300),
                                  (1000, 64, 130, 260), (1500, 5, 256, 256), (40, 200, 64, 32)],
                         ids=lambda c: "x".join(map(str, c)))
def test_experts(case, dtype):
    rows, experts, n_in, n_out = case
    kind = ("none", "silu", "gelu", "relu")[sum(case) % 4]
    _experts(rows, experts, n_in, n_out, dtype, _cut(rows, experts, sum(case)), kind)


def test_experts_of_any_number_of_rows():
    """Ranges that end anywhere in a tile of each size, and rows of no expert on both sides."""
    for sizes in ([1, 31, 32, 33, 63, 64, 65], [127, 128, 129, 0, 160], [191, 192, 193, 1], [383, 385, 100, 0, 0, 577]):
        ends = np.cumsum([5, *sizes]).tolist()
        _experts(ends[-1] + 7, len(sizes), 288, 264, "bf16", ends, "silu")
    _experts(300, 4, 256, 256, "fp16", [0, 0, 0, 0, 0], "none", residual=False)
    _experts(300, 4, 256, 256, "fp16", [0, 300, 300, 300, 300], "none")
    _experts(300, 4, 256, 256, "fp16", [0, 0, 0, 0, 300], "none")


def test_experts_with_offsets_outside_the_rows():
    """Clamped: they lead nowhere else."""
    x = _randn((100, 128), torch.bfloat16, 1)
    values, scales = muon.mx_quantize(_randn((3, 128, 64), torch.float32, 2, 0.1))
    bad = torch.tensor([-7, 40, 90, 1000], dtype=torch.int32, device="cuda")
    good = torch.tensor([0, 40, 90, 100], dtype=torch.int32, device="cuda")
    assert torch.equal(muon.mx_expert_linear(x, bad, values, scales), muon.mx_expert_linear(x, good, values, scales))
    falling = torch.tensor([0, 80, 30, 100], dtype=torch.int32, device="cuda")
    assert muon.mx_expert_linear(x, falling, values, scales).shape == (100, 64)
    muon.check_ops_error()


def test_rows_do_not_depend_on_their_batch():
    for n_in in (1024, 1000):
        x = _randn((600, n_in), torch.bfloat16, 1)
        values, scales = muon.mx_quantize(_randn((n_in, 520), torch.float32, 2, n_in ** -0.5))
        y = muon.mx_linear(x, values, scales)
        for rows in (65, 130, 300):  # other tiles, the same order of the sum
            assert torch.equal(muon.mx_linear(x[:rows], values, scales), y[:rows])
        for _ in range(3):
            assert torch.equal(muon.mx_linear(x, values, scales), y)


def test_strides_alignment_and_slices_of_packed_weights():
    wide = _randn((70, 1100), torch.bfloat16, 1)
    values, scales = muon.mx_quantize(_randn((4, 1024, 72), torch.float32, 2, 0.03))
    for rows in (5, 70):
        for shift in (0, 1, 8, 76):
            x = wide[:rows, shift:shift + 1024]
            for e in (0, 3):
                y = muon.mx_linear(x, values[e], scales[e], residual=wide[:rows, 3:75])
                want = muon.mx_linear(x.contiguous(), values[e].clone(), scales[e].clone(),
                                      residual=wide[:rows, 3:75].contiguous())
                assert torch.equal(y, want)
    odd_v, odd_s = muon.mx_quantize(_randn((3, 100, 33), torch.float32, 2, 0.1))
    x = _randn((70, 100), torch.float16, 4)
    for e in range(3):  # scales of the later ones start anywhere
        check_forward(muon.mx_linear(x, odd_v[e], odd_s[e]), None, _rounded(x), _held(odd_v[e], odd_s[e], 100).T, None,
                      "none", None)


def test_non_finite_operands_reach_their_own_results_only():
    for rows in (20, 300):
        x = _randn((rows, 512), torch.bfloat16, 1)
        values, scales = muon.mx_quantize(_randn((512, 300), torch.float32, 2, 0.05))
        clean = muon.mx_linear(x, values, scales)
        bad = x.clone()
        bad[7, 100], bad[11, 511] = math.nan, math.inf
        y = muon.mx_linear(bad, values, scales)
        keep = torch.ones(rows, dtype=torch.bool)
        keep[[7, 11]] = False
        assert torch.equal(y[keep], clean[keep]) and torch.isnan(y[[7, 11]]).all()
        s2 = scales.clone()
        s2[33, 15] = 255
        y = muon.mx_linear(x, values, s2)
        cols = torch.ones(300, dtype=torch.bool)
        cols[33] = False
        assert torch.equal(y[:, cols], clean[:, cols]) and torch.isnan(y[:, 33]).all()


def test_the_range_of_scales():
    """Products of scales far apart: what the fp32 sum holds of them."""
    x = torch.zeros(3, 64, device="cuda")
    x[0, :32], x[0, 32:], x[1], x[2] = 2.0 ** 60, 2.0 ** -60, 2.0 ** -70, 1.0
    w = torch.zeros(64, 2, device="cuda")
    w[:32, 0], w[32:, 0], w[:, 1] = 2.0 ** -60, 2.0 ** 60, 2.0 ** 50
    values, scales = muon.mx_quantize(w)
    for rows in (3, 99):
        xs = torch.cat((x, torch.zeros(rows - 3, 64, device="cuda")))
        y = muon.mx_linear(xs, values, scales)
        want = (_rounded(xs) @ _held(values, scales, 64).T).float()
        assert torch.equal(y.cpu(), want)


def test_no_rows_streams_and_changing_offsets_in_a_graph():
    experts, n_in, n_out, tokens, top_k = 16, 288, 96, 300, 2
    x = _randn((tokens, n_in), torch.bfloat16, 1)
    values, scales = muon.mx_quantize(_randn((experts, n_in, n_out), torch.float32, 2, n_in ** -0.5))
    assert muon.mx_linear(x[:0], values[0], scales[0]).shape == (0, n_out)
    zero = torch.zeros(experts + 1, dtype=torch.int32, device="cuda")
    assert muon.mx_expert_linear(x[:0], zero, values, scales).shape == (0, n_out)
    want = muon.mx_linear(x, values[0], scales[0])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = muon.mx_linear(x, values[0], scales[0], stream=s)
    s.synchronize()
    assert torch.equal(got, want)
    g = torch.Generator(device="cuda").manual_seed(5)
    idx = torch.zeros(tokens, top_k, dtype=torch.int32, device="cuda")

    def run():
        xs, slot, offsets = muon.dispatch(x, idx, experts)
        return xs, offsets, muon.mx_expert_linear(xs, offsets, values, scales), muon.mx_linear(xs, values[1], scales[1])

    run()
    torch.cuda.synchronize()
    graph, other = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = run()
    with torch.cuda.graph(other, pool=graph.pool()):  # scratch shared with the first one
        held2 = run()
    for i in range(12):
        idx.copy_((int(torch.randint(16, (1,), generator=None)) + torch.randint(-1, 5, idx.shape, generator=g, device="cuda"))
                  % (experts + 1) - 1)
        for gr, h in ((graph, held), (other, held2)):
            gr.replay()
            now = [t.clone() for t in h]
            fresh = run()
            assert all(torch.equal(p, q) for p, q in zip(now, fresh)), i
    muon.check_ops_error()


def test_two_streams_at_once():
    x = [_randn((200, 512), torch.bfloat16, i) for i in range(2)]
    values, scales = muon.mx_quantize(_randn((512, 512), torch.float32, 2, 0.05))
    want = [muon.mx_linear(t, values, scales) for t in x]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for _ in range(20):
        for i in range(2):
            got[i].append(muon.mx_linear(x[i], values, scales, stream=streams[i]))
    torch.cuda.synchronize()
    assert all(torch.equal(t, want[i]) for i in range(2) for t in got[i])
    muon.check_ops_error()


def test_refusals():
    x = _randn((4, 64), torch.bfloat16, 1)
    w = _randn((64, 8), torch.bfloat16, 2)
    values, scales = muon.mx_quantize(w)
    v3, s3 = values[None], scales[None]
    off = torch.tensor([0, 4], dtype=torch.int32, device="cuda")
    for f in (lambda: muon.mx_quantize(w[0]), lambda: muon.mx_quantize(w.double()), lambda: muon.mx_quantize(w[:, ::2]),
              lambda: muon.mx_quantize(w[:0]), lambda: muon.mx_dequantize(values, scales, 65),
              lambda: muon.mx_dequantize(values, scales, 64, dtype=torch.int32), lambda: muon.mx_dequantize(values, scales[:4], 64),
              lambda: muon.mx_linear(x[:, :32], values, scales), lambda: muon.mx_linear(x, values.int(), scales),
              lambda: muon.mx_linear(x, values, scales[:, :1]), lambda: muon.mx_linear(x, v3, s3),
              lambda: muon.mx_linear(x, values.t(), scales), lambda: muon.mx_linear(x, values, scales, activation="tanh"),
              lambda: muon.mx_linear(x, values, scales, bias=w[0].float()),
              lambda: muon.mx_linear(x, values, scales, residual=x), lambda: muon.mx_expert_linear(x, off, values, scales),
              lambda: muon.mx_expert_linear(x, None, v3, s3), lambda: muon.mx_expert_linear(x, off.long(), v3, s3),
              lambda: muon.mx_expert_linear(x, off, v3[:0], s3[:0]), lambda: muon.mx_expert_linear(x, off, v3, s3, bias=w[0])):
        with pytest.raises(ValueError):
            f()
    shifted = torch.empty(values.numel() + 8, dtype=torch.uint8, device="cuda")[8:].view(values.shape).copy_(values)
    with pytest.raises(muon.MuonError):  # packed numbers start on 16 bytes
        muon.mx_linear(x, shifted, scales)
